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
// CTA's barriers; warp 1 of the even CTA issues the MMAs into two accumulators used in turn; warps 2..9
// drain an accumulator while the next tile accumulates, 32 rows by 64 columns at a time: mul and residual
// come by TMA into the warp's own shared-memory tiles (a tile's first piece while its products are still
// running), the result goes into the tile in place and out by a TMA store, so no output row is touched by
// strided 16-byte accesses.  No TMA multicast.  Every wait is bounded.
//
// 4096 tokens, 4096 -> 14336, rank 64, silu and mul: 302 us for one launch from rest (1.61 PFLOP/s, tensor cores 86 %
// active), 379 to 415 in a loop, under the power cap.  1531 ragged tokens, 4096 -> 1024: 20.5 us with the shrink.
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
constexpr int kGK = 64;                       // k-block: 64 bf16 = one 128-byte swizzled row
constexpr int kGMaxStages = 6;
constexpr int kGPiece = 32 * 128;             // bytes of an epilogue piece: 32 rows of 64 columns
constexpr int kGEpiWarps = 8;
constexpr int kGThreads = (2 + kGEpiWarps) * 32;
constexpr int kGRankPad = 64;                 // the intermediate's columns

struct LayerGemmParams {
    CUtensorMap tm_x;             // x [T, h], box 64 x 128
    CUtensorMap tm_w;             // W [o, h], box 64 x half a tile's columns
    CUtensorMap tm_vhi, tm_vlo;   // [T, 64], box 64 x 128
    CUtensorMap tm_y, tm_mul, tm_res;   // [T, o], box 64 x 32
    const uint8_t *tm_B;          // per adapter: B_i [o, r], box 64 x half a tile's columns
    const int32_t *seg_ptr, *seg_adapter, *num_segs;
    int32_t max_segs, T, h, o, n;
    int32_t early;                // launched right behind the shrink (see the kernel)
    EpiParams epi;
    uint32_t *status;
    uint64_t wait_ns;
    int32_t inject;               // test-only: a tile's first k-block is armed but never loaded
};

struct __align__(8) LayerGemmCtl {
    uint64_t full[kGMaxStages], empty[kGMaxStages];
    uint64_t accfull[2], accempty[2];
    uint64_t piece[kGEpiWarps];   // an epilogue warp's mul and residual have landed
    // of a stage: whether the tile's sum ends with it, and for an adapter's k-blocks the tile rows [lo, hi)
    // that they are added to
    int16_t lo[kGMaxStages], hi[kGMaxStages];
    int32_t last[kGMaxStages];
    uint64_t mma_done;
    uint32_t tmem_base;
};

// The segments that meet rows [row0, row1), in order.  Bounds are clamped to [0, T] and made
// non-decreasing (running maximum), so a malformed table gives every row at most one segment;
// segments with a bad adapter are passed over.  Warp-collective; 32 table entries at a time, of which
// the first 32 are read once per kernel and stay in registers.
struct SegmentScan {
    int S;
    int b0, e0, a0;            // this lane's entry of the first window
    int row0, row1, q0, prev_end;
    uint32_t hits;
    int start, end, adapter;   // this lane's entry of the window at hand

    __device__ __forceinline__ void entry(const LayerGemmParams &p, int q, int *b, int *e, int *a) const
    {
        *b = *e = 0;
        *a = -1;
        if (q < S) {
            *b = min(p.T, max(0, p.seg_ptr[q]));
            *e = min(p.T, max(0, p.seg_ptr[q + 1]));
            *a = p.seg_adapter[q];
        }
    }
    __device__ __forceinline__ void init(const LayerGemmParams &p)
    {
        S = p.max_segs > 0 ? max(0, min(*p.num_segs, p.max_segs)) : 0;
        entry(p, threadIdx.x & 31, &b0, &e0, &a0);
    }
    __device__ __forceinline__ void begin(const LayerGemmParams &p, int r0, int r1)
    {
        row0 = r0;
        row1 = min(r1, p.T);
        q0 = -32;
        prev_end = 0;
        hits = 0;
    }
    __device__ bool next(const LayerGemmParams &p, int *lo, int *hi, int *a)
    {
        const int lane = threadIdx.x & 31;
        while (hits == 0) {
            q0 += 32;
            if (q0 >= S || prev_end >= row1) return false;
            int b = b0;
            end = e0;
            adapter = a0;
            if (q0 > 0) entry(p, q0 + lane, &b, &end, &adapter);
            int m = max(max(b, end), prev_end);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, m, d);
                if (lane >= d) m = max(m, o);
            }
            int before = __shfl_up_sync(0xffffffffu, m, 1);
            if (lane == 0) before = prev_end;
            start = max(b, before);
            const bool hit = adapter >= 0 && adapter < p.n && max(start, row0) < min(end, row1);
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

// v[i] <- v[i] op the 32 bf16 values at 16-byte pieces c0..c0+3 of this lane's row of a swizzled tile
template <bool MUL>
__device__ __forceinline__ void combine(const uint8_t *tile, int row, int c0, float (&v)[32])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint4 b = *reinterpret_cast<const uint4 *>(tile + sw128_off(row, c0 + e));
        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float &lo = v[e * 8 + 2 * i], &hi = v[e * 8 + 2 * i + 1];
            lo = MUL ? lo * bf16_lo(w[i]) : lo + bf16_lo(w[i]);
            hi = MUL ? hi * bf16_hi(w[i]) : hi + bf16_hi(w[i]);
        }
    }
}

// k-blocks of 64 in a stage: a narrow tile's products take half the time, so each wait and each commit has to
// serve two of them (one: 200 ns a k-block where the tensor cores need 135).
constexpr int k_blocks(int bn) { return bn == 256 ? 1 : 2; }

// BN: output columns per tile, 256, or 128 where those fill the SMs better.
template <int BN, int STAGES>
__global__ void __launch_bounds__(kGThreads, 1) layer_gemm_kernel(const __grid_constant__ LayerGemmParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int crank = (int)cluster_ctarank();   // 0: the even CTA, which issues
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int MT = (p.T + kGM - 1) / kGM, NT = (p.o + BN - 1) / BN;
    const int nkb = (p.h + kGK - 1) / kGK;
    const int total = MT * NT;
    constexpr int kA = 128 * 128, kB = BN / 2 * 128, kSub = kA + kB;   // bytes of the A and B side of a k-block
    constexpr int KB = k_blocks(BN), kStage = KB * kSub;               // k-blocks and bytes of a stage
    const int nst = (nkb + KB - 1) / KB;                               // stages of a tile's base product
    const int nops = (p.epi.mul != nullptr) + (p.epi.res != nullptr), tiles = nops > 1 ? 2 : 1;
    uint8_t *pieces = ring + (STAGES * kStage + 1023) / 1024 * 1024;   // `tiles` for each epilogue warp
    LayerGemmCtl &ctl = *reinterpret_cast<LayerGemmCtl *>(pieces + kGEpiWarps * tiles * kGPiece);

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), 1);
            mbar_init(smem_u32(&ctl.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl.accfull[i]), 1);
            mbar_init(smem_u32(&ctl.accempty[i]), 2 * kGEpiWarps);
        }
        for (int i = 0; i < kGEpiWarps; ++i) mbar_init(smem_u32(&ctl.piece[i]), 1);
        mbar_init(smem_u32(&ctl.mma_done), 1);
        fence_mbar_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl.tmem_base), 2 * BN);   // two accumulators
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
        // The whole warp runs the loops and one lane issues (see the issuer).
        const uint32_t empty0 = smem_u32(&ctl.empty[0]), full0 = smem_u32(&ctl.full[0]), lead0 = pair_leader(full0);
        const uint32_t ring0 = smem_u32(ring);
        const bool one = elect_one();
        int s = 0, used = 0;
        uint32_t phase = 1;   // the first pass finds every stage free
        bool ok = true, waited = !p.early;
        auto free_stage = [&]() {
            return __all_sync(0xffffffffu, mbar_wait_hot(empty0 + s * 8, phase, p.status, p.wait_ns)) != 0;
        };
        // arms the stage and moves on; a k-block's two loads: this CTA's half of the A side and of the B side
        auto arm = [&]() {
            if (crank == 0 && one) mbar_arrive_expect_tx(full0 + s * 8, 2 * kStage);
        };
        auto load = [&](int u, const void *ta, int ca, const void *tb, int cb, int row, int col) {
            const uint32_t at = ring0 + s * kStage + u * kSub;
            if (one) {
                tma_load_2d_pair(at, ta, ca, row, lead0 + s * 8);
                tma_load_2d_pair(at + kA, tb, cb, col, lead0 + s * 8);
            }
        };
        auto next_stage = [&]() {
            if (used < STAGES) ++used;
            if (++s == STAGES) {
                s = 0;
                phase ^= 1;
            }
        };
        SegmentScan sc;
        sc.init(p);
        for (int t = pair; t < total && ok; t += npairs) {
            const int tile_row = (t % MT) * kGM, row = tile_row + crank * 128, col = (t / MT) * BN + crank * (BN / 2);
            int lo, hi, a;
            sc.begin(p, tile_row, tile_row + kGM);
            bool more = sc.next(p, &lo, &hi, &a);
            for (int st = 0; st < nst; ++st) {
                ok = free_stage();
                if (!ok) break;
                if (st + 1 == nst && one) ctl.last[s] = !more;
                arm();
                if (!(p.inject && st == 0))
#pragma unroll
                    for (int u = 0; u < KB; ++u)   // columns past h are zero-filled
                        load(u, &p.tm_x, (st * KB + u) * kGK, &p.tm_w, (st * KB + u) * kGK, row, col);
                next_stage();
            }
            while (ok && more) {
                if (!waited) {
                    pdl_wait();
                    waited = true;
                }
                const int lo1 = lo, hi1 = hi;
                const void *tb = p.tm_B + (size_t)a * 128;
                more = sc.next(p, &lo, &hi, &a);
                for (int part = 0; part < 2; part += KB) {   // hi, lo
                    ok = free_stage();
                    if (!ok) break;
                    if (one) {
                        ctl.lo[s] = (int16_t)lo1;
                        ctl.hi[s] = (int16_t)hi1;
                        ctl.last[s] = part + KB == 2 && !more;
                    }
                    arm();
#pragma unroll
                    for (int u = 0; u < KB; ++u) load(u, part + u ? &p.tm_vlo : &p.tm_vhi, 0, tb, 0, row, col);
                    next_stage();
                }
            }
        }
        if (!waited) pdl_wait();   // this grid never completes before the shrink
        // drain: the copies of the last stages have landed in both CTAs before either leaves (earlier
        // ones were consumed before their stage was loaded again)
        if (crank == 0) {
            for (int i = 0; i < used; ++i) {   // newest first
                if (--s < 0) {
                    s = STAGES - 1;
                    phase ^= 1;
                }
                mbar_wait(full0 + s * 8, phase ^ 1, p.status, p.wait_ns);
            }
        } else if (!ok) {
            __nanosleep(1000000);   // a wait ran out: let this CTA's own copies land
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (even CTA)
        // The whole warp runs the loop and one lane issues: the instruction takes its operands from uniform
        // registers, and a loop inside one lane spent 75 cycles an instruction on moving them there.
        if (crank == 0) {
            const uint32_t idesc = idesc_bf16(kGM, BN);
            const uint64_t ad0 = sw128_desc(smem_u32(ring)), bd0 = sw128_desc(smem_u32(ring) + kA);
            const uint32_t full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
            const bool one = elect_one();
            int s = 0, li = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = pair; t < total && ok; t += npairs, ++li) {
                const int ab = li & 1;
                if (li >= 2 && !__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&ctl.accempty[ab]), ((li >> 1) - 1) & 1,
                                                                          p.status, p.wait_ns)))
                    break;
                tc_fence_after();
                const uint32_t acc = tmem + (uint32_t)(ab * BN);
                // nst stages of the base product, then as many of adapters as the producer says
                bool last = false;
                for (int st = 0; !last; ++st) {
                    ok = __all_sync(0xffffffffu, mbar_wait_hot(full0 + s * 8, phase, p.status, p.wait_ns));
                    if (!ok) break;
                    // read before the commit below gives the stage, and with it its record, back to the producer
                    if (st + 1 >= nst) last = __all_sync(0xffffffffu, ctl.last[s] != 0);
                    tc_fence_after();
                    const uint64_t ad = ad0 + (uint64_t)(s * (kStage >> 4)), bd = bd0 + (uint64_t)(s * (kStage >> 4));
                    if (st < nst) {
                        if (one) {
#pragma unroll
                            for (int u = 0; u < KB; ++u)
#pragma unroll
                                for (int k = 0; k < kGK / 16; ++k)
                                    umma_bf16_pair(acc, ad + u * (kSub >> 4) + 2 * k, bd + u * (kSub >> 4) + 2 * k, idesc,
                                                   (st | u | k) ? 1u : 0u);
                            umma_commit_pair(empty0 + s * 8);
                        }
                    } else {
                        uint32_t off[8];
                        rows_off(ctl.lo[s], ctl.hi[s], off);
                        if (one) {
#pragma unroll
                            for (int u = 0; u < KB; ++u)
#pragma unroll
                                for (int k = 0; k < kGK / 16; ++k)
                                    umma_bf16_pair_rows(acc, ad + u * (kSub >> 4) + 2 * k, bd + u * (kSub >> 4) + 2 * k, idesc,
                                                        off);
                            umma_commit_pair(empty0 + s * 8);
                        }
                    }
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (ok && one) umma_commit_pair(smem_u32(&ctl.accfull[ab]));
            }
            if (one) umma_commit_pair(smem_u32(&ctl.mma_done));   // after every MMA, in both CTAs
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        if (blockIdx.x == 0 && warp == 2) report_bad_segments(p);
        const int q = warp & 3;                        // TMEM lane quarter of this warp
        const int wi = warp - 2, c_first = (wi >> 2) * (BN / 2);
        constexpr int kPieces = BN / 2 / 64;           // 64-column pieces of this warp per tile
        uint8_t *buf = pieces + wi * tiles * kGPiece;   // mul, else residual; then the result
        uint8_t *const second = buf + kGPiece;         // residual beside mul
        const uint32_t bar = smem_u32(&ctl.piece[wi]);
        const uint64_t once = policy_evict_first();   // x and W are what L2 is for
        auto fetch = [&](int t, int c) {               // operands of piece c of tile t
            if (nops == 0 || t >= total || lane != 0) return;
            const int row = (t % MT) * kGM + crank * 128 + q * 32, col = (t / MT) * BN + c_first + c * 64;
            mbar_arrive_expect_tx(bar, (uint32_t)(nops * kGPiece));
            if (p.epi.mul) tma_load_2d_hint(smem_u32(buf), &p.tm_mul, col, row, bar, once);
            if (p.epi.res) tma_load_2d_hint(smem_u32(nops == 2 ? second : buf), &p.tm_res, col, row, bar, once);
        };
        int li = 0, k = 0;
        bool okw = true;
        fetch(pair, 0);
        for (int t = pair; t < total && okw; t += npairs, ++li) {
            const int ab = li & 1;
            const int row0 = (t % MT) * kGM + crank * 128 + q * 32, col0 = (t / MT) * BN + c_first;
            okw = mbar_wait(smem_u32(&ctl.accfull[ab]), (li >> 1) & 1, p.status, p.wait_ns);
            okw = __all_sync(0xffffffffu, okw);
            if (!okw) break;
            tc_fence_after();
            for (int c = 0; c < kPieces; ++c, ++k) {
                if (nops && !__all_sync(0xffffffffu, mbar_wait(bar, k & 1, p.status, p.wait_ns))) {
                    okw = false;
                    break;
                }
                if (nops == 0) {   // the piece before has been read by its store
                    if (lane == 0) bulk_wait_group_read0();
                    __syncwarp();
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float z[32];
                    tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ab * BN + c_first + c * 64 + hh * 32), z);
                    if (p.epi.bias) {
                        const int n0 = col0 + c * 64 + hh * 32;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n0 + e * 8 < p.o) {
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
                    if (p.epi.mul) combine<true>(buf, lane, hh * 4, z);
                    if (p.epi.res) combine<false>(nops == 2 ? second : buf, lane, hh * 4, z);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4 *>(buf + sw128_off(lane, hh * 4 + e)) =
                            make_uint4(pack_bf16x2(z[e * 8], z[e * 8 + 1]), pack_bf16x2(z[e * 8 + 2], z[e * 8 + 3]),
                                       pack_bf16x2(z[e * 8 + 4], z[e * 8 + 5]), pack_bf16x2(z[e * 8 + 6], z[e * 8 + 7]));
                }
                if (c + 1 == kPieces) {   // the accumulator is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(smem_u32(&ctl.accempty[ab]), 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && row0 < p.T && col0 + c * 64 < p.o) {
                    tma_store_2d_hint(&p.tm_y, smem_u32(buf), col0 + c * 64, row0, once);   // rows and columns outside are dropped
                    bulk_commit_group();
                    if (nops) bulk_wait_group_read0();
                }
                __syncwarp();
                fetch(c + 1 < kPieces ? t : t + npairs, c + 1 < kPieces ? c + 1 : 0);
            }
        }
        if (lane == 0) {
            bulk_wait_group0();
            // a wait that ran out: the operands under way land before shared memory is given up
            if (!okw && nops) mbar_wait(bar, k & 1, p.status, p.wait_ns);
        }
        __syncwarp();
    }
    // Both CTAs: all roles are done, and the last MMA (which reads and writes both) has completed.
    __syncthreads();
    if (warp == 1 && lane == 0) mbar_wait(smem_u32(&ctl.mma_done), 0, p.status, p.wait_ns);
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 2 * BN);
}

// Shared memory: a ring of STAGES stages, the epilogue's tiles (two for each warp where it takes both mul
// and residual), the control block.
constexpr int gemm_smem(int bn, int stages, int tiles)
{
    return stages * k_blocks(bn) * (128 * 128 + bn / 2 * 128) + kGEpiWarps * tiles * kGPiece + (int)sizeof(LayerGemmCtl) + 2048;
}
// The deepest rings that fit beside one and beside two tiles.
constexpr int gemm_stages(int bn, int tiles) { return bn == 256 ? (tiles == 2 ? 5 : 6) : (tiles == 2 ? 3 : 4); }
static_assert(gemm_smem(256, 6, 1) <= 227 * 1024 && gemm_smem(256, 5, 2) <= 227 * 1024, "shared memory");
static_assert(gemm_smem(128, 4, 1) <= 227 * 1024 && gemm_smem(128, 3, 2) <= 227 * 1024, "shared memory");
// no other pair or cluster that takes tensor memory fits beside a CTA (kColumnSmem in layer_shape.h says why)
static_assert(gemm_smem(256, 5, 2) >= 200 * 1024 && gemm_smem(128, 3, 2) >= 200 * 1024, "alone on its SM");

template <int BN, int TILES>
int launch_tiles(const LayerGemmParams &p, int64_t pairs, int dev, cudaStream_t s)
{
    constexpr int kStages = gemm_stages(BN, TILES), kSmem = gemm_smem(BN, kStages, TILES);
    static std::once_flag once[64];
    static cudaError_t attr_rc[64];
    std::call_once(once[dev], [&] {
        attr_rc[dev] =
            cudaFuncSetAttribute(layer_gemm_kernel<BN, kStages>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (attr_rc[dev] != cudaSuccess) return LORA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = kSmem;
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
    if (cudaLaunchKernelEx(&cfg, layer_gemm_kernel<BN, kStages>, p) != cudaSuccess) return LORA_ERR_CUDA;
    note_launch(kKernLayerGemm);
    return LORA_OK;
}

}  // namespace

int launch_layer_gemm(const lora_table *t, const lora_segments *seg, const void *x, int64_t ldx, const void *W,
                      int64_t ldw, const lora_epilogue *epi, void *y, int64_t ldy, int32_t y_off, const void *v,
                      bool after_shrink, cudaStream_t s)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return LORA_ERR_CUDA;
    static std::once_flag once[64];
    static int n_sms[64];
    std::call_once(once[dev], [&] { cudaDeviceGetAttribute(&n_sms[dev], cudaDevAttrMultiProcessorCount, dev); });
    if (n_sms[dev] < 2) return LORA_ERR_CUDA;
    const int64_t pairs = n_sms[dev] / 2;
    auto tiles_of = [&](int bn_) { return (int64_t)((seg->T + kGM - 1) / kGM) * ((t->o + bn_ - 1) / bn_); };
    auto rounds = [&](int bn_) { return (tiles_of(bn_) + pairs - 1) / pairs; };
    // Narrow tiles where they end sooner: a round of them takes about 0.65 of a round of wide ones (half the
    // products, three quarters of the loads).
    const int bn = rounds(128) * 65 < rounds(256) * 100 ? 128 : 256;
    LayerGemmParams p;
    std::memset(&p, 0, sizeof p);
    const uint16_t *v_hi = static_cast<const uint16_t *>(v);
    const uint16_t *v_lo = v_hi + (int64_t)seg->T * kGRankPad;
    int rc;
    if ((rc = encode_sw128(&p.tm_x, x, (uint64_t)t->h, (uint64_t)seg->T, (uint64_t)ldx, 128)) != LORA_OK ||
        (rc = encode_sw128(&p.tm_w, W, (uint64_t)t->h, (uint64_t)t->o, (uint64_t)ldw, (uint32_t)bn / 2)) != LORA_OK ||
        (rc = encode_sw128(&p.tm_y, static_cast<uint16_t *>(y) + y_off, (uint64_t)t->o, (uint64_t)seg->T, (uint64_t)ldy, 32)) !=
            LORA_OK)
        return rc;
    if (v && ((rc = encode_sw128(&p.tm_vhi, v_hi, kGRankPad, (uint64_t)seg->T, kGRankPad, 128)) != LORA_OK ||
              (rc = encode_sw128(&p.tm_vlo, v_lo, kGRankPad, (uint64_t)seg->T, kGRankPad, 128)) != LORA_OK))
        return rc;
    if (epi->mul && (rc = encode_sw128(&p.tm_mul, epi->mul, (uint64_t)t->o, (uint64_t)seg->T, (uint64_t)epi->ldmul, 32)) != LORA_OK)
        return rc;
    if (epi->residual &&
        (rc = encode_sw128(&p.tm_res, epi->residual, (uint64_t)t->o, (uint64_t)seg->T, (uint64_t)epi->ldres, 32)) != LORA_OK)
        return rc;
    if (v) p.tm_B = static_cast<const uint8_t *>(t->d_tmaps_pfB) + (bn == 256 ? 0 : (size_t)t->n * 128);
    p.seg_ptr = seg->seg_ptr;
    p.seg_adapter = seg->seg_adapter;
    p.num_segs = seg->num_segs;
    p.max_segs = seg->max_segs;
    p.T = seg->T;
    p.h = t->h;
    p.o = t->o;
    p.n = t->n;
    p.early = (after_shrink && options().pdl) ? 1 : 0;
    p.epi = epi_params(epi);
    p.status = t->d_status;
    p.wait_ns = wait_limit_ns();
    p.inject = (int32_t)(options().inject_stall & 16);

    const int64_t run = std::min<int64_t>(pairs, tiles_of(bn));
    if (epi->mul && epi->residual) return bn == 256 ? launch_tiles<256, 2>(p, run, dev, s) : launch_tiles<128, 2>(p, run, dev, s);
    return bn == 256 ? launch_tiles<256, 1>(p, run, dev, s) : launch_tiles<128, 1>(p, run, dev, s);
}

}  // namespace lora
