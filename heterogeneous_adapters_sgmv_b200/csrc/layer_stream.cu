// A layer for a decode batch (lora_bgmv_layer): base weight, adapter term, bias, activation, gate
// product and residual, each token with its own adapter:
//
//     z[t, n] = sum_j x[t, j] W[n, j] + s_i sum_k B_i[n, k] (x[t] . A_i[k]) + bias[n]
//     y[t, n] = act(z[t, n]) * mul[t, n] + residual[t, n]
//
// Two launches.  layer_shrink_kernel forms v[t, k] = s_i x[t] . A_i[k] in fp32.  The pass over W,
// layer_stream_kernel, is bound by the bytes of W for the batches it is made for (2 h o bytes
// against 2 T h o flop: below ~250 tokens the tensor cores wait for memory), so it is built to keep
// weight loads in flight: W takes the MMA's M side (128 rows of W a tile) and the tokens its N side
// (16 to 256), so that no tensor-core row is spent on absent tokens, and the k axis of a tile is
// split over the CTAs of a cluster where there are fewer tiles than SMs.  The CTAs' partial sums meet
// through distributed shared memory and are added in CTA order (no atomics: bit-identical from run
// to run).  The adapter term is added by the epilogue threads in fp32: a thread holds one output
// column, so it reads its own row of B_i, and the token's v is the same for the whole warp.
//
// Warp roles: warp 0 fills a ring of (W, x) k-blocks by TMA; warp 1 issues tcgen05.mma; warps 2..9
// drain the accumulator (two per lane quarter), exchange it and finish the outputs.  Weight loads of
// the first stages are issued before the grid-dependency wait: W is never written by a call in flight.
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

// ------------------------------------------------------------------------------- shrink

constexpr int kShrinkWarps = 8;

struct LayerShrinkParams {
    const AdapterDesc *desc;
    const int32_t *ids;
    const uint16_t *x;
    int64_t ldx;
    float *v;
    int32_t ldv, n, h, split;   // split: warps that share one row of A_i (1, 2, 4 or 8)
    uint32_t *status;
};

// Block (rank-row group, token).  A group of `split` warps forms one v[t, k]: 16-byte loads of x[t]
// and A_i[k], fp32 sums folded by shuffles, then over the group's warps in their order.
__global__ void __launch_bounds__(kShrinkWarps * 32) layer_shrink_kernel(const __grid_constant__ LayerShrinkParams p)
{
    __shared__ float part[kShrinkWarps];
    // the wait comes first: launch_dependents then tells the pass over W that x and the epilogue's
    // operands are final, and that only v is still to come
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int a = p.ids[t];
    if (a < 0 || a >= p.n) {
        if (a != -1 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, LORA_STATUS_BAD_ID);
        return;
    }
    const int rank = p.desc[a].rank;
    const int rows = kShrinkWarps / p.split;
    const int k = blockIdx.x * rows + warp / p.split, sub = warp % p.split;
    if (blockIdx.x * rows >= rank) return;   // the whole block
    float s0 = 0.f, s1 = 0.f;
    if (k < rank) {
        const uint4 *xa = reinterpret_cast<const uint4 *>(p.x + t * p.ldx);
        const uint4 *wa = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.desc[a].A) + (int64_t)k * p.h);
        const int hv = p.h / 8;
#pragma unroll 4
        for (int j = sub * 32 + lane; j < hv; j += p.split * 32) {
            const uint4 u = xa[j], w = wa[j];
            const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s0 = fmaf(bf16_lo(uu[i]), bf16_lo(ww[i]), s0);
                s1 = fmaf(bf16_hi(uu[i]), bf16_hi(ww[i]), s1);
            }
        }
    }
    float s = s0 + s1;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (p.split > 1) {
        if (lane == 0) part[warp] = s;
        __syncthreads();
        if (sub == 0)
            for (int i = 1; i < p.split; ++i) s += part[warp + i];
    }
    if (lane == 0 && sub == 0 && k < rank) p.v[t * p.ldv + k] = s * p.desc[a].scale;
}

// ------------------------------------------------------------------------------- pass over W

constexpr int kLM = 128;                      // rows of W per tile (MMA M)
constexpr int kLK = 64;                       // k-block: one 128-byte swizzled row of bf16
constexpr int kLWBytes = kLM * 128;
constexpr int kLMaxN = 256;                   // tokens per tile (MMA N)
constexpr int kLMaxStages = 8;
constexpr int kLEpiWarps = 8;
constexpr int kLThreads = (2 + kLEpiWarps) * 32;

struct LayerStreamParams {
    CUtensorMap tm_x;             // x [T, h], box 64 x N
    CUtensorMap tm_w;             // W [o, h], box 64 x 128
    const AdapterDesc *desc;
    const int32_t *ids;           // null: no adapters
    const float *v;               // [T, ldv] scaled intermediate
    int32_t ldv, n;
    int32_t T, h, o;
    int32_t N, NT, stages;        // tokens per tile, token tiles, ring depth
    int32_t early;                // launched right behind the shrink (see above)
    uint16_t *y;                  // at column y_offset
    int64_t ldy;
    EpiParams epi;
    uint32_t *status;
    uint64_t wait_ns;
};

struct __align__(16) LayerStreamCtl {
    uint64_t full[kLMaxStages], empty[kLMaxStages];
    uint64_t done;
    uint32_t tmem_base;
    int32_t pad;
    const void *B[kLMaxN];        // per token of this CTA's share: its B_i,
    int32_t rank[kLMaxN];         // and rank (0: no adapter, -1: bad id)
};

// Distributed-shared-memory address of `local` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_cluster(uint32_t local, uint32_t rank)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    return remote;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// sum_k B_i[n, k] v[t, k] of one output; `row` is the row of B_i.
__device__ __forceinline__ float expand_row(const uint16_t *row, const float *v, int rank)
{
    float s0 = 0.f, s1 = 0.f;
    if ((rank & 7) == 0) {   // the row is 16-byte aligned
#pragma unroll 2
        for (int k = 0; k < rank; k += 8) {
            const uint4 b = *reinterpret_cast<const uint4 *>(row + k);
            const float4 p = *reinterpret_cast<const float4 *>(v + k), q = *reinterpret_cast<const float4 *>(v + k + 4);
            s0 = fmaf(bf16_lo(b.x), p.x, s0);
            s1 = fmaf(bf16_hi(b.x), p.y, s1);
            s0 = fmaf(bf16_lo(b.y), p.z, s0);
            s1 = fmaf(bf16_hi(b.y), p.w, s1);
            s0 = fmaf(bf16_lo(b.z), q.x, s0);
            s1 = fmaf(bf16_hi(b.z), q.y, s1);
            s0 = fmaf(bf16_lo(b.w), q.z, s0);
            s1 = fmaf(bf16_hi(b.w), q.w, s1);
        }
    } else {
        for (int k = 0; k < rank; ++k) s0 = fmaf(bf16_f(row[k]), v[k], s0);
    }
    return s0 + s1;
}

template <int S>   // CTAs per cluster that split the k axis
__global__ void __launch_bounds__(kLThreads, 2) layer_stream_kernel(const __grid_constant__ LayerStreamParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stage_bytes = kLWBytes + p.N * 128;
    LayerStreamCtl &ctl = *reinterpret_cast<LayerStreamCtl *>(ring + p.stages * stage_bytes);
    float *part = reinterpret_cast<float *>(ring);   // [N][128] fp32 once the ring is done with

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int crank = S > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / S;
    const int mt = tile / p.NT, tt = tile % p.NT;   // token tiles of one W tile side by side: W once from HBM
    const int row0 = mt * kLM, t0 = tt * p.N;
    const int nkb_all = (p.h + kLK - 1) / kLK;
    const int kb0 = (int)((int64_t)crank * nkb_all / S), nkb = (int)((int64_t)(crank + 1) * nkb_all / S) - kb0;
    uint32_t ncols = 32;
    while ((int)ncols < p.N) ncols *= 2;

    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), 1);
            mbar_init(smem_u32(&ctl.empty[i]), 1);
        }
        mbar_init(smem_u32(&ctl.done), 1);
        fence_mbar_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl.tmem_base), ncols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // After the allocation: a dependent kernel's CTA on this SM cannot take the tensor memory that
    // this one is still waiting for.
    pdl_launch_dependents();
    const uint32_t tmem = ctl.tmem_base;
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int pre = min(nkb, p.stages);
        if (lane == 0) {
            for (int kb = 0; kb < pre; ++kb) {
                const uint32_t fb = smem_u32(&ctl.full[kb]);
                mbar_arrive_expect_tx(fb, (uint32_t)stage_bytes);
                tma_load_2d(smem_u32(ring + kb * stage_bytes), &p.tm_w, (kb0 + kb) * kLK, row0, fb);
            }
            if (!p.early) pdl_wait();
            for (int kb = 0; kb < pre; ++kb)
                tma_load_2d(smem_u32(ring + kb * stage_bytes + kLWBytes), &p.tm_x, (kb0 + kb) * kLK, t0,
                            smem_u32(&ctl.full[kb]));
        }
        __syncwarp();
        int kb = pre;
        for (; kb < nkb; ++kb) {
            const int s = kb % p.stages, m = kb / p.stages;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&ctl.empty[s]), (m - 1) & 1, p.status, p.wait_ns))) break;
            if (lane == 0) {
                const uint32_t fb = smem_u32(&ctl.full[s]);
                mbar_arrive_expect_tx(fb, (uint32_t)stage_bytes);
                tma_load_2d(smem_u32(ring + s * stage_bytes), &p.tm_w, (kb0 + kb) * kLK, row0, fb);
                tma_load_2d(smem_u32(ring + s * stage_bytes + kLWBytes), &p.tm_x, (kb0 + kb) * kLK, t0, fb);
            }
            __syncwarp();
        }
        // drain: the copies of the last stages armed have landed before the ring is reused
        if (lane == 0)
            for (int i = max(0, kb - p.stages); i < kb; ++i)
                mbar_wait(smem_u32(&ctl.full[i % p.stages]), (i / p.stages) & 1, p.status, p.wait_ns);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16(kLM, p.N);
            for (int kb = 0; kb < nkb; ++kb) {
                const int s = kb % p.stages, m = kb / p.stages;
                if (!mbar_wait(smem_u32(&ctl.full[s]), m & 1, p.status, p.wait_ns)) break;
                tc_fence_after();
                const uint64_t wd = sw128_desc(smem_u32(ring + s * stage_bytes));
                const uint64_t xd = sw128_desc(smem_u32(ring + s * stage_bytes + kLWBytes));
#pragma unroll
                for (int k = 0; k < kLK / 16; ++k) umma_bf16(tmem, wd + 2 * k, xd + 2 * k, idesc, (kb | k) != 0 ? 1u : 0u);
                umma_commit(smem_u32(&ctl.empty[s]));
            }
            umma_commit(smem_u32(&ctl.done));   // every MMA issued so far
        }
        __syncwarp();
    }
    // This CTA's share of the tile's tokens, and their adapters.
    const int nv = min(p.N, p.T - t0);
    const int share = (nv + S - 1) / S;
    const int ta = min(nv, crank * share), tb = min(nv, ta + share);
    if (warp >= 2) {
        if (!p.early) pdl_wait();   // ids may come from the kernel before
        for (int i = tid - 64; i < tb - ta; i += kLEpiWarps * 32) {
            int r = 0;
            const void *B = nullptr;
            if (p.ids) {
                const int a = p.ids[t0 + ta + i];
                if (a >= 0 && a < p.n) {
                    r = p.desc[a].rank;
                    B = p.desc[a].B;
                } else if (a != -1) {
                    r = -1;
                }
            }
            ctl.rank[i] = r;
            ctl.B[i] = B;
        }
    }
    // Every thread learns whether the accumulator is complete; a wait that ran out anywhere in the
    // CTA makes all of it skip the warp-collective loads (the cluster barriers are still met).
    ok = mbar_wait(smem_u32(&ctl.done), 0, p.status, p.wait_ns);
    ok = __syncthreads_and(ok) != 0;
    tc_fence_after();
    if (warp >= 2 && ok) {
        // the partial sum, token by token, into the ring: lane = row of W
        const int q = warp & 3, half = (warp - 2) >> 2;
        for (int c = half * 16; c < p.N; c += 32) {
            float f[16];
            tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * kLM + q * 32 + lane] = f[i];
        }
    }
    tc_fence_before();
    if (S > 1) cluster_sync_all();
    else __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, ncols);
    if (warp >= 2) {
        if (p.early) pdl_wait();   // v
        const int e = tid - 64;
        const int m = e & (kLM - 1), n = row0 + m;
        const bool live = ok && n < p.o;
        const float bias = (live && p.epi.bias) ? bf16_f(p.epi.bias[n]) : 0.f;
        uint32_t peer[S];
#pragma unroll
        for (int c = 0; c < S; ++c) peer[c] = S > 1 ? map_cluster(smem_u32(part), c) : smem_u32(part);
        for (int i = e / kLM; i < tb - ta; i += kLEpiWarps * 32 / kLM) {
            const int r = ctl.rank[i];
            if (!live || r < 0) continue;
            const int64_t t = t0 + ta + i;
            float z[1] = {bias};
#pragma unroll
            for (int c = 0; c < S; ++c) z[0] += ld_cluster(peer[c] + (uint32_t)((ta + i) * kLM + m) * 4);
            if (r > 0)
                z[0] += expand_row(static_cast<const uint16_t *>(ctl.B[i]) + (int64_t)n * r, p.v + t * p.ldv, r);
            activate(z, p.epi.act);
            if (p.epi.mul) z[0] *= bf16_f(p.epi.mul[t * p.epi.ldmul + n]);
            if (p.epi.res) z[0] += bf16_f(p.epi.res[t * p.epi.ldres + n]);
            p.y[t * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(z[0]));
        }
    }
    if (S > 1) cluster_sync_all();   // no CTA leaves while a peer still reads its partial sums
}

struct StreamShape {
    int N, NT, S, stages, smem;
};

// Tokens per tile: all of them up to 256 (rounded up to the MMA's 16), else equal tiles of at most
// 256.  Clusters: as many CTAs splitting k as fill two CTAs per SM, up to 8.  Ring: half an SM's
// shared memory, or all of it where a stage with its x tile leaves room for fewer than three stages
// in half.
StreamShape stream_shape(int T, int h, int o, int n_sms)
{
    StreamShape sh;
    sh.NT = (T + kLMaxN - 1) / kLMaxN;
    const int per = (T + sh.NT - 1) / sh.NT;
    sh.N = (per + 15) & ~15;
    const int stage = kLWBytes + sh.N * 128;
    const int ctl = (int)sizeof(LayerStreamCtl) + 1024;
    const int half = 113 * 1024 - ctl, whole = 226 * 1024 - ctl;
    const bool two = half / stage >= 3;
    sh.stages = std::min(kLMaxStages, (two ? half : whole) / stage);
    const int64_t tiles = (int64_t)((o + kLM - 1) / kLM) * sh.NT;
    const int64_t slots = (int64_t)n_sms * (two ? 2 : 1);
    const int nkb = (h + kLK - 1) / kLK;
    sh.S = 1;
    while (sh.S < 8 && tiles * sh.S * 2 <= slots && sh.S * 2 <= nkb) sh.S *= 2;
    sh.smem = sh.stages * stage + ctl;
    return sh;
}

template <int S>
int launch_stream(const LayerStreamParams &p, const StreamShape &sh, cudaStream_t s, int dev)
{
    static std::once_flag once[64];
    static cudaError_t attr_rc[64];
    std::call_once(once[dev], [&] {
        attr_rc[dev] = cudaFuncSetAttribute(layer_stream_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
    });
    if (attr_rc[dev] != cudaSuccess) return LORA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)((p.o + kLM - 1) / kLM) * p.NT * S));
    cfg.blockDim = dim3(kLThreads);
    cfg.dynamicSmemBytes = (size_t)sh.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (S > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = S;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (options().pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    if (cudaLaunchKernelEx(&cfg, layer_stream_kernel<S>, p) != cudaSuccess) return LORA_ERR_CUDA;
    note_launch(kKernLayerStream);
    return LORA_OK;
}

int device_sms(int *dev, int *n_sms)
{
    static std::once_flag once[64];
    static int sms[64];
    if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= 64) return LORA_ERR_CUDA;
    const int d = *dev;
    std::call_once(once[d], [&] { cudaDeviceGetAttribute(&sms[d], cudaDevAttrMultiProcessorCount, d); });
    *n_sms = sms[d];
    return *n_sms > 0 ? LORA_OK : LORA_ERR_CUDA;
}

}  // namespace

int launch_layer_shrink(const lora_table *t, const int32_t *ids, int32_t T, const void *x, int64_t ldx, float *v,
                        int32_t ldv, cudaStream_t s)
{
    int dev = 0, n_sms = 0;
    if (device_sms(&dev, &n_sms) != LORA_OK) return LORA_ERR_CUDA;
    LayerShrinkParams p;
    p.desc = t->d_desc;
    p.x = static_cast<const uint16_t *>(x);
    p.ldx = ldx;
    p.ldv = ldv;
    p.n = t->n;
    p.h = t->h;
    p.status = t->d_status;
    // Warps per row of A_i: several while there are fewer rows than warps to keep the SMs busy
    // (and a row long enough to share).
    p.split = 1;
    while (p.split < kShrinkWarps && (int64_t)T * t->max_rank * p.split < 16ll * n_sms && t->h >= 256 * 2 * p.split)
        p.split *= 2;
    const int rows = kShrinkWarps / p.split;
    for (int64_t t0 = 0; t0 < T; t0 += 65535) {   // gridDim.y
        p.ids = ids + t0;
        p.x = static_cast<const uint16_t *>(x) + t0 * ldx;
        p.v = v + t0 * ldv;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((t->max_rank + rows - 1) / rows), (unsigned)std::min<int64_t>(65535, T - t0));
        cfg.blockDim = dim3(kShrinkWarps * 32);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        if (options().pdl) {
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.numAttrs = 1;
        }
        cfg.attrs = attr;
        if (cudaLaunchKernelEx(&cfg, layer_shrink_kernel, p) != cudaSuccess) return LORA_ERR_CUDA;
        note_launch(kKernLayerShrink);
    }
    return LORA_OK;
}

int launch_layer_stream(const lora_table *t, const int32_t *ids, int32_t T, const void *x, int64_t ldx, const void *W,
                        int64_t ldw, const lora_epilogue *epi, void *y, int64_t ldy, int32_t y_off, const float *v,
                        int32_t ldv, cudaStream_t s)
{
    int dev = 0, n_sms = 0, rc;
    if (device_sms(&dev, &n_sms) != LORA_OK) return LORA_ERR_CUDA;
    const StreamShape sh = stream_shape(T, t->h, t->o, n_sms);
    LayerStreamParams p;
    std::memset(&p, 0, sizeof p);
    if ((rc = encode_sw128(&p.tm_x, x, (uint64_t)t->h, (uint64_t)T, (uint64_t)ldx, (uint32_t)sh.N)) != LORA_OK ||
        (rc = encode_sw128(&p.tm_w, W, (uint64_t)t->h, (uint64_t)t->o, (uint64_t)ldw, kLM)) != LORA_OK)
        return rc;
    p.desc = t->d_desc;
    p.ids = ids;
    p.v = v;
    p.ldv = ldv;
    p.n = t->n;
    p.T = T;
    p.h = t->h;
    p.o = t->o;
    p.N = sh.N;
    p.NT = sh.NT;
    p.stages = sh.stages;
    p.early = (ids && options().pdl) ? 1 : 0;
    p.y = static_cast<uint16_t *>(y) + y_off;
    p.ldy = ldy;
    p.epi = epi_params(epi);
    p.status = t->d_status;
    p.wait_ns = wait_limit_ns();
    switch (sh.S) {
    case 8: return launch_stream<8>(p, sh, s, dev);
    case 4: return launch_stream<4>(p, sh, s, dev);
    case 2: return launch_stream<2>(p, sh, s, dev);
    default: return launch_stream<1>(p, sh, s, dev);
    }
}

}  // namespace lora
