// A layer over prompts (lora_sgmv_layer): base weight and adapter term in one tensor-memory
// accumulator, then bias, activation, gate product and residual, y written once:
//
//     z[t, n] = sum_j x[t, j] W[n, j] + sum_k v[t, k] B_i[n, k],   v = s_i x A_i^T (bf16 hi + lo)
//     y[t, n] = act(z[t, n] + bias[n]) * mul[t, n] + residual[t, n]
//
// Bound by the tensor cores (2 T h o flop).  A persistent pair of CTAs (cta_group::2) works on
// 256-token by 256-column tiles: each CTA loads its 128 rows of x and its 128 rows of W, so a k-block
// costs an SM 32 KiB of shared memory traffic for 128 x 256 x 64 products where a single CTA's
// 128 x 256 tile costs 48 KiB.
//
// Row tiles are cut at multiples of 256, wherever the segments lie, so short and ragged segments
// waste no rows of the base product.  A tile then adds, for each segment that meets it, two more
// k-blocks (v's hi and lo parts against that adapter's B_i, rank zero-filled to 64) with the MMA's
// output-lane mask, which leaves the rows of other segments as they are; rows outside the segment
// may hold anything in v.
//
// Warp roles in each CTA: warp 0 loads by TMA into a ring of (x, W) half tiles, counted on the even
// CTA's barriers; warp 1 of the even CTA issues the MMAs into two 256-column accumulators used in
// turn; warps 2..9 drain an accumulator (one output row and 128 columns a thread) while the next tile
// accumulates.  No TMA multicast.  Every wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "layer_epilogue.cuh"
#include "lora_common.cuh"
#include "lora_internal.h"
#include "tcgen05.cuh"

namespace lora {
namespace {

constexpr int kGM = 256;                      // tokens per tile, 128 in each CTA
constexpr int kGN = 256;                      // output columns per tile
constexpr int kGK = 64;                       // k-block: 64 bf16 = one 128-byte swizzled row
constexpr int kGHalf = 128 * 128;             // bytes of a 128-row half of x or W
constexpr int kGStage = 2 * kGHalf;
constexpr int kGStages = 6;
constexpr int kGEpiWarps = 8;
constexpr int kGThreads = (2 + kGEpiWarps) * 32;
constexpr int kGRankPad = 64;                 // the intermediate's columns

struct LayerGemmParams {
    CUtensorMap tm_x;             // x [T, h], box 64 x 128
    CUtensorMap tm_w;             // W [o, h], box 64 x 128
    CUtensorMap tm_vhi, tm_vlo;   // [T, 64], box 64 x 128
    const uint8_t *tm_B;          // per adapter: B_i [o, r], box 64 x 128
    const int32_t *seg_ptr, *seg_adapter, *num_segs;
    int32_t max_segs, T, h, o, n;
    int32_t early;                // launched right behind the shrink (see the kernel)
    uint16_t *y;                  // at column y_offset
    int64_t ldy;
    EpiParams epi;
    uint32_t *status;
    uint64_t wait_ns;
};

struct __align__(8) LayerGemmCtl {
    uint64_t full[kGStages], empty[kGStages];
    uint64_t accfull[2], accempty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
};

// The segments that meet rows [row0, row1), in order.  Bounds are clamped to [0, T] and made
// non-decreasing (running maximum), so a malformed table gives every row at most one segment;
// segments with a bad adapter are passed over.  Warp-collective; 32 table entries at a time.
struct SegmentScan {
    int row0, row1, q0, prev_end, S;
    uint32_t hits;
    int start, end, adapter;   // this lane's entry

    __device__ __forceinline__ void begin(const LayerGemmParams &p, int r0, int r1)
    {
        row0 = r0;
        row1 = min(r1, p.T);
        q0 = -32;
        prev_end = 0;
        S = p.max_segs > 0 ? max(0, min(*p.num_segs, p.max_segs)) : 0;
        hits = 0;
    }
    __device__ bool next(const LayerGemmParams &p, int *lo, int *hi, int *a)
    {
        const int lane = threadIdx.x & 31;
        while (hits == 0) {
            q0 += 32;
            if (q0 >= S || prev_end >= row1) return false;
            const int q = q0 + lane;
            int b = 0;
            start = end = 0;
            adapter = -1;
            if (q < S) {
                b = min(p.T, max(0, p.seg_ptr[q]));
                end = min(p.T, max(0, p.seg_ptr[q + 1]));
                adapter = p.seg_adapter[q];
            }
            int m = max(max(b, end), prev_end);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, m, d);
                if (lane >= d) m = max(m, o);
            }
            int before = __shfl_up_sync(0xffffffffu, m, 1);
            if (lane == 0) before = prev_end;
            start = max(b, before);
            const bool hit = q < S && adapter >= 0 && adapter < p.n && max(start, row0) < min(end, row1);
            hits = __ballot_sync(0xffffffffu, hit);
            prev_end = __shfl_sync(0xffffffffu, m, 31);
        }
        const int src = __ffs(hits) - 1;
        hits &= hits - 1;
        *lo = max(row0, __shfl_sync(0xffffffffu, start, src)) - row0;
        *hi = min(row1, __shfl_sync(0xffffffffu, end, src)) - row0;
        *a = __shfl_sync(0xffffffffu, adapter, src);
        return true;
    }
};

// Latch a bad table entry (one warp): bounds out of order or outside [0, T], an unknown adapter.
__device__ void report_bad_segments(const LayerGemmParams &p)
{
    const int S = p.max_segs > 0 ? max(0, min(*p.num_segs, p.max_segs)) : 0;
    bool bad = p.max_segs > 0 && (*p.num_segs < 0 || *p.num_segs > p.max_segs);
    for (int q = threadIdx.x & 31; q < S; q += 32) {
        const int b = p.seg_ptr[q], e = p.seg_ptr[q + 1], a = p.seg_adapter[q];
        bad |= b < 0 || e < b || e > p.T || a < 0 || a >= p.n;
    }
    if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) atomicOr(p.status, LORA_STATUS_BAD_SEGMENT);
}

// Bits of the tile rows outside [lo, hi), 32 a word.
__device__ __forceinline__ void rows_off(int lo, int hi, uint32_t (&off)[8])
{
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const int a = min(32, max(0, lo - 32 * w)), b = min(32, max(0, hi - 32 * w));
        const uint32_t below_b = b >= 32 ? 0xffffffffu : (1u << b) - 1, below_a = a >= 32 ? 0xffffffffu : (1u << a) - 1;
        off[w] = ~(below_b & ~below_a);
    }
}

__global__ void __launch_bounds__(kGThreads, 1) layer_gemm_kernel(const __grid_constant__ LayerGemmParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LayerGemmCtl &ctl = *reinterpret_cast<LayerGemmCtl *>(ring + kGStages * kGStage);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int crank = (int)cluster_ctarank();   // 0: the even CTA, which issues
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int MT = (p.T + kGM - 1) / kGM, NT = (p.o + kGN - 1) / kGN;
    const int nkb = (p.h + kGK - 1) / kGK;
    const int total = MT * NT;

    if (tid == 0) {
        for (int i = 0; i < kGStages; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), 1);
            mbar_init(smem_u32(&ctl.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl.accfull[i]), 1);
            mbar_init(smem_u32(&ctl.accempty[i]), 2 * kGEpiWarps);
        }
        mbar_init(smem_u32(&ctl.mma_done), 1);
        fence_mbar_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl.tmem_base), 512);   // two 256-column accumulators
        tmem_relinquish_pair();
    }
    // Programmatic launch: the shrink before this kernel lets it start only after its own wait on
    // everything earlier, so x, mul, residual and the segment table are final here; only the
    // intermediate is not, and the producer waits for it before its first adapter k-block.  Without
    // that shrink every thread waits here.
    if (!p.early) pdl_wait();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    pdl_launch_dependents();   // after the allocation, so that no dependent's CTA takes tensor memory first
    const uint32_t tmem = ctl.tmem_base;

    // Tiles t = pair, + npairs, ...: row tile fastest, so the pairs working at one time share a few W
    // column tiles (read from DRAM once, then from L2) and all of x.
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int kbi = 0;
        bool ok = true, waited = !p.early;
        // one k-block: this CTA's half of the A side and of the B side
        auto load = [&](const void *ta, int ca, const void *tb, int cb, int row, int col) {
            const int s = kbi % kGStages, m = kbi / kGStages;
            if (m >= 1 &&
                !__all_sync(0xffffffffu, mbar_wait(smem_u32(&ctl.empty[s]), (m - 1) & 1, p.status, p.wait_ns)))
                return false;
            if (lane == 0) {
                uint8_t *st = ring + s * kGStage;
                if (crank == 0) mbar_arrive_expect_tx(smem_u32(&ctl.full[s]), 2 * kGStage);
                const uint32_t fb = pair_leader(smem_u32(&ctl.full[s]));
                tma_load_2d_pair(smem_u32(st), ta, ca, row, fb);
                tma_load_2d_pair(smem_u32(st + kGHalf), tb, cb, col, fb);
            }
            __syncwarp();
            ++kbi;
            return true;
        };
        for (int t = pair; t < total && ok; t += npairs) {
            const int tile_row = (t % MT) * kGM, row = tile_row + crank * 128, col = (t / MT) * kGN + crank * 128;
            for (int kb = 0; kb < nkb && ok; ++kb) ok = load(&p.tm_x, kb * kGK, &p.tm_w, kb * kGK, row, col);
            SegmentScan sc;
            sc.begin(p, tile_row, tile_row + kGM);
            int lo, hi, a;
            while (ok && sc.next(p, &lo, &hi, &a)) {
                if (!waited) {
                    pdl_wait();
                    waited = true;
                }
                const void *tb = p.tm_B + (size_t)a * 128;
                ok = load(&p.tm_vhi, 0, tb, 0, row, col) && load(&p.tm_vlo, 0, tb, 0, row, col);
            }
        }
        if (!waited) pdl_wait();   // this grid never completes before the shrink
        // drain: the copies of the last stages have landed in both CTAs before either leaves (earlier
        // ones were consumed before their stage was loaded again)
        if (crank == 0) {
            if (lane == 0)
                for (int i = max(0, kbi - kGStages); i < kbi; ++i)
                    mbar_wait(smem_u32(&ctl.full[i % kGStages]), (i / kGStages) & 1, p.status, p.wait_ns);
        } else if (!ok) {
            __nanosleep(1000000);   // a wait ran out: let this CTA's own copies land
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (even CTA)
        const uint32_t idesc = idesc_bf16(kGM, kGN);
        int kbi = 0, li = 0;
        bool ok = true;
        for (int t = pair; crank == 0 && t < total && ok; t += npairs, ++li) {
            const int tile_row = (t % MT) * kGM;
            const int ab = li & 1;
            if (li >= 2 && !__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&ctl.accempty[ab]), ((li >> 1) - 1) & 1,
                                                                      p.status, p.wait_ns))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + (uint32_t)(ab * kGN);
            auto ready = [&]() {
                const bool got = __all_sync(0xffffffffu, mbar_wait(smem_u32(&ctl.full[kbi % kGStages]),
                                                                   (kbi / kGStages) & 1, p.status, p.wait_ns));
                tc_fence_after();
                return got;
            };
            for (int kb = 0; kb < nkb; ++kb, ++kbi) {
                if (!ready()) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint8_t *st = ring + (kbi % kGStages) * kGStage;
                    const uint64_t ad = sw128_desc(smem_u32(st)), bd = sw128_desc(smem_u32(st + kGHalf));
#pragma unroll
                    for (int k = 0; k < kGK / 16; ++k)
                        umma_bf16_pair(acc, ad + 2 * k, bd + 2 * k, idesc, (kb | k) != 0 ? 1u : 0u);
                    umma_commit_pair(smem_u32(&ctl.empty[kbi % kGStages]));
                }
                __syncwarp();
            }
            SegmentScan sc;
            sc.begin(p, tile_row, tile_row + kGM);
            int lo, hi, a;
            while (ok && sc.next(p, &lo, &hi, &a)) {
                uint32_t off[8];
                rows_off(lo, hi, off);
                for (int part = 0; part < 2; ++part, ++kbi) {
                    if (!ready()) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        const uint8_t *st = ring + (kbi % kGStages) * kGStage;
                        const uint64_t ad = sw128_desc(smem_u32(st)), bd = sw128_desc(smem_u32(st + kGHalf));
#pragma unroll
                        for (int k = 0; k < kGK / 16; ++k) umma_bf16_pair_rows(acc, ad + 2 * k, bd + 2 * k, idesc, off);
                        umma_commit_pair(smem_u32(&ctl.empty[kbi % kGStages]));
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (lane == 0) umma_commit_pair(smem_u32(&ctl.accfull[ab]));
            __syncwarp();
        }
        if (crank == 0 && lane == 0) umma_commit_pair(smem_u32(&ctl.mma_done));   // after every MMA, in both CTAs
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        if (blockIdx.x == 0 && warp == 2) report_bad_segments(p);
        const int q = warp & 3;                        // TMEM lane quarter of this warp
        const int c_first = ((warp - 2) >> 2) * (kGN / 2);
        int li = 0;
        for (int t = pair; t < total; t += npairs, ++li) {
            const int ab = li & 1;
            const int64_t row = (int64_t)(t % MT) * kGM + crank * 128 + q * 32 + lane;
            const int col0 = (t / MT) * kGN;
            // every epilogue warp leaves together if any lane ran out of time
            const bool okw = mbar_wait(smem_u32(&ctl.accfull[ab]), (li >> 1) & 1, p.status, p.wait_ns);
            if (!named_bar_and(2, kGEpiWarps * 32, okw)) break;
            tc_fence_after();
            const bool row_ok = row < p.T;
#pragma unroll 1
            for (int c = c_first; c < c_first + kGN / 2; c += 32) {
                float z[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ab * kGN + c), z);
                const int n0 = col0 + c, ncol = min(32, p.o - n0);
                if (!row_ok || ncol <= 0) continue;
                if (p.epi.bias) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e * 8 < ncol) {
                            const uint4 b = *reinterpret_cast<const uint4 *>(p.epi.bias + n0 + e * 8);
                            const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                z[e * 8 + 2 * i] += bf16_lo(w[i]);
                                z[e * 8 + 2 * i + 1] += bf16_hi(w[i]);
                            }
                        }
                }
                activate(z, p.epi.act);
                if (p.epi.mul) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(p.epi.mul + row * p.epi.ldmul + n0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e * 8 < ncol) {
                            const uint4 b = src[e];
                            const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                z[e * 8 + 2 * i] *= bf16_lo(w[i]);
                                z[e * 8 + 2 * i + 1] *= bf16_hi(w[i]);
                            }
                        }
                }
                if (p.epi.res) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(p.epi.res + row * p.epi.ldres + n0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e * 8 < ncol) {
                            const uint4 b = src[e];
                            const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                z[e * 8 + 2 * i] += bf16_lo(w[i]);
                                z[e * 8 + 2 * i + 1] += bf16_hi(w[i]);
                            }
                        }
                }
                uint4 *dst = reinterpret_cast<uint4 *>(p.y + row * p.ldy + n0);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e * 8 < ncol)
                        dst[e] = make_uint4(pack_bf16x2(z[e * 8], z[e * 8 + 1]), pack_bf16x2(z[e * 8 + 2], z[e * 8 + 3]),
                                            pack_bf16x2(z[e * 8 + 4], z[e * 8 + 5]), pack_bf16x2(z[e * 8 + 6], z[e * 8 + 7]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(smem_u32(&ctl.accempty[ab]), 0);
        }
    }
    // Both CTAs: all roles are done, and the last MMA (which reads and writes both) has completed.
    __syncthreads();
    if (warp == 1 && lane == 0) mbar_wait(smem_u32(&ctl.mma_done), 0, p.status, p.wait_ns);
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

constexpr int kGSmem = kGStages * kGStage + (int)sizeof(LayerGemmCtl) + 1024;
static_assert(kGSmem <= 227 * 1024, "layer GEMM shared memory");

}  // namespace

int launch_layer_gemm(const lora_table *t, const lora_segments *seg, const void *x, int64_t ldx, const void *W,
                      int64_t ldw, const lora_epilogue *epi, void *y, int64_t ldy, int32_t y_off, const void *v,
                      bool after_shrink, cudaStream_t s)
{
    LayerGemmParams p;
    std::memset(&p, 0, sizeof p);
    const uint16_t *v_hi = static_cast<const uint16_t *>(v);
    const uint16_t *v_lo = v_hi + (int64_t)seg->T * kGRankPad;
    int rc;
    if ((rc = encode_sw128(&p.tm_x, x, (uint64_t)t->h, (uint64_t)seg->T, (uint64_t)ldx, 128)) != LORA_OK ||
        (rc = encode_sw128(&p.tm_w, W, (uint64_t)t->h, (uint64_t)t->o, (uint64_t)ldw, 128)) != LORA_OK ||
        (rc = encode_sw128(&p.tm_vhi, v_hi, kGRankPad, (uint64_t)seg->T, kGRankPad, 128)) != LORA_OK ||
        (rc = encode_sw128(&p.tm_vlo, v_lo, kGRankPad, (uint64_t)seg->T, kGRankPad, 128)) != LORA_OK)
        return rc;
    p.tm_B = static_cast<const uint8_t *>(t->d_tmaps_pfB);
    p.seg_ptr = seg->seg_ptr;
    p.seg_adapter = seg->seg_adapter;
    p.num_segs = seg->num_segs;
    p.max_segs = seg->max_segs;
    p.T = seg->T;
    p.h = t->h;
    p.o = t->o;
    p.n = t->n;
    p.early = (after_shrink && options().pdl) ? 1 : 0;
    p.y = static_cast<uint16_t *>(y) + y_off;
    p.ldy = ldy;
    p.epi = epi_params(epi);
    p.status = t->d_status;
    p.wait_ns = wait_limit_ns();

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return LORA_ERR_CUDA;
    static std::once_flag once[64];
    static cudaError_t attr_rc[64];
    static int n_sms[64];
    std::call_once(once[dev], [&] {
        attr_rc[dev] = cudaFuncSetAttribute(layer_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
        cudaDeviceGetAttribute(&n_sms[dev], cudaDevAttrMultiProcessorCount, dev);
    });
    if (attr_rc[dev] != cudaSuccess || n_sms[dev] < 2) return LORA_ERR_CUDA;
    const int64_t tiles = (int64_t)((seg->T + kGM - 1) / kGM) * ((t->o + kGN - 1) / kGN);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(n_sms[dev] / 2, tiles)));
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = kGSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int na = 0;
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 2;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
    if (options().pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    if (cudaLaunchKernelEx(&cfg, layer_gemm_kernel, p) != cudaSuccess) return LORA_ERR_CUDA;
    note_launch(kKernLayerGemm);
    return LORA_OK;
}

}  // namespace lora
