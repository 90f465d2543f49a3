// The norms around a block, with each token's own weights (lora_norm_before, lora_norm_after):
//
//     before:  h = N(x)
//     after:   u = N(z),  r = res_scale * residual + branch_scale * gate * u,  h = N_next(r)
//
// N is a root-mean-square or a layer norm over the d values of a row; gain, shift and gate come
// from the row of the token's adapter, from one row for all, or (the gate) from the token.
//
// Bound by HBM: every operand is read once and every result written once, and between the two a
// row stays in registers as fp32, spread over the threads of one block (so a sum over the row is a
// shuffle and one exchange through shared memory).  The variance of a layer norm is taken from the
// centred values in a second sum over the registers, not from the difference of two large sums.
// h is computed from the unrounded r, so that a fused call adds no rounding of its own.
#include <algorithm>

#include "lora_common.cuh"
#include "lora_internal.h"

namespace lora {
namespace {

template <typename E> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4 &w, float *f)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(u[i]);
            f[2 * i + 1] = bf16_hi(u[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <> struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void unpack(const uint4 &w, float *f)
    {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// Sum over the block's NT threads, the same value in every thread.  `slot` must differ between
// consecutive calls (two are used in turn), so that one barrier per sum is enough.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float (*part)[32], int slot)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if constexpr (NT > 32) {
        constexpr int kWarps = NT / 32;
        if ((threadIdx.x & 31) == 0) part[slot][threadIdx.x >> 5] = v;
        __syncthreads();
        v = part[slot][threadIdx.x & (kWarps - 1)];
#pragma unroll
        for (int d = kWarps / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    }
    return v;
}

// Thread i holds vectors i, i + NT, ... of the row (V of them at most); values past the row are 0.
template <typename E, int NT, int V>
struct Row {
    static constexpr int kN = Vec<E>::kN;
    float f[V][kN];

    __device__ __forceinline__ void load(const void *base, int64_t off, int nvec)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const E *>(base) + off);
        uint4 w[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = threadIdx.x + j * NT;
            w[j] = c < nvec ? p[c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) Vec<E>::unpack(w[j], f[j]);
    }
    __device__ __forceinline__ void store(void *base, int64_t off, int nvec) const
    {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<E *>(base) + off);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = threadIdx.x + j * NT;
            if (c < nvec) p[c] = Vec<E>::pack(f[j]);
        }
    }
    // f <- N(f) with the weights of row `wrow`
    __device__ __forceinline__ void normalise(const lora_norm &nm, int64_t wrow, int d, int nvec, float (*part)[32])
    {
        const float inv_d = 1.f / (float)d;
        if (nm.kind == LORA_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < kN; ++i) s += f[j][i];
            const float mean = block_sum<NT>(s, part, 0) * inv_d;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (threadIdx.x + j * NT < nvec)
#pragma unroll
                    for (int i = 0; i < kN; ++i) f[j][i] -= mean;
        }
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < kN; ++i) q = fmaf(f[j][i], f[j][i], q);
        const float inv = rsqrtf(block_sum<NT>(q, part, 1) * inv_d + nm.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = threadIdx.x + j * NT;
            if (c >= nvec) continue;
            float g[kN], b[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                g[i] = 1.f;
                b[i] = 0.f;
            }
            if (nm.gain) Vec<E>::unpack(reinterpret_cast<const uint4 *>(static_cast<const E *>(nm.gain) + wrow * nm.ld)[c], g);
            if (nm.shift)
                Vec<E>::unpack(reinterpret_cast<const uint4 *>(static_cast<const E *>(nm.shift) + wrow * nm.ld)[c], b);
#pragma unroll
            for (int i = 0; i < kN; ++i) f[j][i] = fmaf(f[j][i] * inv, g[i], b[i]);
        }
    }
};

template <typename E, int NT, int V, bool AFTER>
__global__ void __launch_bounds__(NT) block_norm_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float part[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int nvec = p.d / Vec<E>::kN;
    Row<E, NT, V> x;
    x.load(p.x, t * p.ldx, nvec);
    int id = -1;
    if (p.ids) {
        id = p.ids[t];
        if (id < -1 || id >= p.n) {   // the whole block leaves: the row stays as it was
            if (threadIdx.x == 0) atomicOr(p.status, LORA_STATUS_BAD_ID);
            return;
        }
    }
    const int64_t wrow = id + 1;
    if constexpr (!AFTER) {
        x.normalise(p.norm, wrow, p.d, nvec, part);
        x.store(p.h, t * p.ldh, nvec);
    } else {
        Row<E, NT, V> s;
        if (p.res.residual) {
            s.load(p.res.residual, t * p.res.ldres, nvec);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < Vec<E>::kN; ++i) s.f[j][i] = 0.f;
        }
        if (p.norm.kind) x.normalise(p.norm, wrow, p.d, nvec, part);
        if (p.res.gate_kind != LORA_GATE_NONE) {
            Row<E, NT, V> g;
            g.load(p.res.gate, (p.res.gate_kind == LORA_GATE_TOKEN ? t : wrow) * p.res.ldgate, nvec);
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < Vec<E>::kN; ++i) x.f[j][i] *= g.f[j][i];
        }
        const float a = p.res.residual ? p.res.res_scale : 0.f, c = p.res.branch_scale;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < Vec<E>::kN; ++i) x.f[j][i] = fmaf(a, s.f[j][i], c * x.f[j][i]);
        if (p.r) x.store(p.r, t * p.ldr, nvec);
        if (p.h) {
            // the first norm's sums are read by every thread before the second norm's are written
            if (NT > 32 && p.norm.kind) __syncthreads();
            x.normalise(p.next, wrow, p.d, nvec, part);
            x.store(p.h, t * p.ldh, nvec);
        }
    }
}

template <typename E, int NT, int V>
int launch_one(const NormParams &p, bool after, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.T);
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (options().pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    cfg.attrs = attr;
    const cudaError_t e = after ? cudaLaunchKernelEx(&cfg, block_norm_kernel<E, NT, V, true>, p)
                                : cudaLaunchKernelEx(&cfg, block_norm_kernel<E, NT, V, false>, p);
    if (e != cudaSuccess) return LORA_ERR_CUDA;
    note_launch(kKernBlockNorm);
    return LORA_OK;
}

template <typename E>
int launch_typed(const NormParams &p, bool after, cudaStream_t s)
{
    const int nvec = p.d / Vec<E>::kN;
    if (nvec <= 32) return launch_one<E, 32, 1>(p, after, s);
    if (nvec <= 128) return launch_one<E, 128, 1>(p, after, s);
    if (nvec <= 256) return launch_one<E, 256, 1>(p, after, s);
    if (nvec <= 512) return launch_one<E, 256, 2>(p, after, s);
    if (nvec <= 1024) return launch_one<E, 512, 2>(p, after, s);
    if (nvec <= 2048) return launch_one<E, 512, 4>(p, after, s);
    if constexpr (LORA_MAX_NORM_WIDTH > 2048 * Vec<E>::kN) return launch_one<E, 1024, 4>(p, after, s);
    return LORA_ERR_UNSUPPORTED;
}
static_assert(LORA_MAX_NORM_WIDTH <= 1024 * 4 * Vec<float>::kN && LORA_MAX_NORM_WIDTH <= 2048 * Vec<__nv_bfloat16>::kN,
              "the widest block holds the widest row");

}  // namespace

int launch_block_norm(const NormParams &p, bool after, int dtype, cudaStream_t s)
{
    return dtype == LORA_BF16 ? launch_typed<__nv_bfloat16>(p, after, s) : launch_typed<float>(p, after, s);
}

}  // namespace lora
