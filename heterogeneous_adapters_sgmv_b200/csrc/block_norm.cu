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
// shuffle and one exchange through shared memory; the weights are read before the sums, which they do not
// depend on).  Where there are many rows the blocks are persistent (ring_norm_kernel): a warp of its own brings the
// operands of the rows to come, the weights of each row's adapter among them, into a ring in shared memory by bulk
// copies, and weights that serve all rows once, so that neither a global load's latency nor the issue of the copies
// lies between a row's sums.  4096 rows of 4096 bf16: before 14.8 us, after (with the next norm) 31.3, 69 and 82 %
// of the copy bandwidth; a block a row takes 18.0 and 43.9.
// The variance of a layer norm is taken from the centred values in a second sum over the registers, not from the
// difference of two large sums.  h is computed from the unrounded r, so that a fused call adds no rounding of its
// own.
#include <algorithm>
#include <mutex>

#include "lora_common.cuh"
#include "lora_internal.h"
#include "tcgen05.cuh"

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

// Sum over the block's first NT threads, the same value in every thread.  `slot` must differ between
// consecutive calls (two are used in turn), so that one barrier per sum is enough.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float (*part)[32], int slot)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if constexpr (NT > 32) {
        constexpr int kWarps = NT / 32;
        if ((threadIdx.x & 31) == 0) part[slot][threadIdx.x >> 5] = v;
        named_bar_sync(1, NT);
        v = part[slot][threadIdx.x & (kWarps - 1)];
#pragma unroll
        for (int d = kWarps / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    }
    return v;
}

// Thread i holds vectors i, i + NT, ... of a row, V of them at most.
template <typename E, int NT, int V>
struct Packed {
    uint4 w[V];

    __device__ __forceinline__ void load(const void *base, int64_t off, int nvec)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const E *>(base) + off);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = threadIdx.x + j * NT;
            w[j] = c < nvec ? p[c] : make_uint4(0, 0, 0, 0);
        }
    }
};

// The gain and shift of a norm for one row.
template <typename E, int NT, int V>
struct Weights {
    Packed<E, NT, V> g, b;

    __device__ __forceinline__ void load(const lora_norm &nm, int64_t wrow, int nvec)
    {
        if (nm.gain) g.load(nm.gain, wrow * nm.ld, nvec);
        if (nm.shift) b.load(nm.shift, wrow * nm.ld, nvec);
    }
};

template <typename E, int NT, int V>
struct Row {
    static constexpr int kN = Vec<E>::kN;
    float f[V][kN];   // values past the row are 0

    __device__ __forceinline__ void set(const Packed<E, NT, V> &p)
    {
#pragma unroll
        for (int j = 0; j < V; ++j) Vec<E>::unpack(p.w[j], f[j]);
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
    // f <- N(f)
    __device__ __forceinline__ void normalise(const lora_norm &nm, const Weights<E, NT, V> &wt, int d, int nvec,
                                              float (*part)[32])
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
            if (threadIdx.x + j * NT >= nvec) continue;
            float g[kN], b[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                g[i] = 1.f;
                b[i] = 0.f;
            }
            if (nm.gain) Vec<E>::unpack(wt.g.w[j], g);
            if (nm.shift) Vec<E>::unpack(wt.b.w[j], b);
#pragma unroll
            for (int i = 0; i < kN; ++i) f[j][i] = fmaf(f[j][i] * inv, g[i], b[i]);
        }
    }
};

// u * gate * branch_scale + res_scale * residual
template <typename E>
__device__ __forceinline__ void join(const lora_residual &rs, float (&f)[Vec<E>::kN], const uint4 &gate, const uint4 &res)
{
    float o[Vec<E>::kN];
    if (rs.gate_kind != LORA_GATE_NONE) {
        Vec<E>::unpack(gate, o);
#pragma unroll
        for (int i = 0; i < Vec<E>::kN; ++i) f[i] *= o[i];
    }
#pragma unroll
    for (int i = 0; i < Vec<E>::kN; ++i) f[i] *= rs.branch_scale;
    if (rs.residual) {
        Vec<E>::unpack(res, o);
#pragma unroll
        for (int i = 0; i < Vec<E>::kN; ++i) f[i] = fmaf(rs.res_scale, o[i], f[i]);
    }
}

// One row a block.
template <typename E, int NT, int V, bool AFTER>
__global__ void __launch_bounds__(NT) block_norm_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float part[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int nvec = p.d / Vec<E>::kN;
    Packed<E, NT, V> x, res, gate;
    x.load(p.x, t * p.ldx, nvec);
    if constexpr (AFTER) {
        if (p.res.residual) res.load(p.res.residual, t * p.res.ldres, nvec);
        if (p.res.gate_kind == LORA_GATE_TOKEN) gate.load(p.res.gate, t * p.res.ldgate, nvec);
    }
    int id = -1;
    if (p.ids) {
        id = p.ids[t];
        if (id < -1 || id >= p.n) {   // the whole block leaves: the row stays as it was
            if (threadIdx.x == 0) atomicOr(p.status, LORA_STATUS_BAD_ID);
            return;
        }
    }
    const int64_t wrow = (int64_t)id + 1;
    Weights<E, NT, V> w1, w2;
    if (p.norm.kind) w1.load(p.norm, wrow, nvec);
    if constexpr (AFTER) {
        if (p.res.gate_kind == LORA_GATE_ADAPTER) gate.load(p.res.gate, wrow * p.res.ldgate, nvec);
        if (p.h) w2.load(p.next, wrow, nvec);
    }
    Row<E, NT, V> f;
    f.set(x);
    if (p.norm.kind) f.normalise(p.norm, w1, p.d, nvec, part);
    if constexpr (!AFTER) {
        f.store(p.h, t * p.ldh, nvec);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) join<E>(p.res, f.f[j], gate.w[j], res.w[j]);
        if (p.r) f.store(p.r, t * p.ldr, nvec);
        if (p.h) {
            if (NT > 32 && p.norm.kind) __syncthreads();   // the first norm's sums are read by all
            f.normalise(p.next, w2, p.d, nvec, part);
            f.store(p.h, t * p.ldh, nvec);
        }
    }
}

// ------------------------------------------------------------------------------- persistent blocks

// The seven operands a row may have, in the order in which they lie in a stage (or in the block's area for
// what serves all rows).
enum NormOperand { kOpX, kOpRes, kOpGate, kOpGain1, kOpShift1, kOpGain2, kOpShift2, kOps };
constexpr int kNormStages = 4;
// Blocks per SM: what 64 registers a thread allow, or 80 for the larger kernel; 56 where 64 would leave one
// large block alone (8192 wide: 16.2 against 17.9 us).
template <int NT, int V, bool AFTER>
constexpr int kRingBlocks = 65536 / (AFTER ? 80 : NT >= 512 && V <= 2 ? 56 : 64) / (NT + 32);

struct RingShape {
    int32_t row_bytes, stages, stage_bytes;
    int32_t fixed_bytes;          // of the operands that serve all rows, at the start of shared memory
    int32_t at[kOps];             // offset of each operand in its stage or area, -1: absent
    int32_t per_row;              // bit: the operand changes from row to row
    uint64_t wait_ns;
    int32_t inject;               // test-only: rows are armed but never loaded
};

// Row `t` of operand `op` for a token with adapter row `w`.
template <typename E>
__device__ __forceinline__ const void *norm_source(const NormParams &p, int op, int64_t t, int64_t w)
{
    const void *b;
    int64_t row;
    switch (op) {
    case kOpX: b = p.x, row = t * p.ldx; break;
    case kOpRes: b = p.res.residual, row = t * p.res.ldres; break;
    case kOpGate: b = p.res.gate, row = (p.res.gate_kind == LORA_GATE_TOKEN ? t : w) * p.res.ldgate; break;
    case kOpGain1: b = p.norm.gain, row = w * p.norm.ld; break;
    case kOpShift1: b = p.norm.shift, row = w * p.norm.ld; break;
    case kOpGain2: b = p.next.gain, row = w * p.next.ld; break;
    default: b = p.next.shift, row = w * p.next.ld; break;
    }
    return static_cast<const E *>(b) + row;
}

// NT threads work on rows; the warp behind them fetches.
template <typename E, int NT, int V, bool AFTER>
__global__ void __launch_bounds__(NT + 32, kRingBlocks<NT, V, AFTER>)
ring_norm_kernel(const __grid_constant__ NormParams p, const __grid_constant__ RingShape sh)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float part[2][32];
    __shared__ uint64_t full[kNormStages], empty[kNormStages], fixed;
    __shared__ int32_t row_id[kNormStages];
    uint8_t *ring = smem + sh.fixed_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < sh.stages; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        mbar_init(smem_u32(&fixed), 1);
        fence_mbar_init_cluster();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const int nvec = p.d / Vec<E>::kN;
    int s = 0;
    uint32_t phase = 0;
    if (threadIdx.x >= NT) {
        // ------------------------------------------------------------ fetch
        const int lane = threadIdx.x & 31;
        const bool one = elect_one();
        if (one) {
            mbar_arrive_expect_tx(smem_u32(&fixed), (uint32_t)sh.fixed_bytes);
#pragma unroll
            for (int op = 0; op < kOps; ++op)
                if (sh.at[op] >= 0 && !((sh.per_row >> op) & 1))
                    bulk_g2s(smem_u32(smem) + (uint32_t)sh.at[op], norm_source<E>(p, op, 0, 0), (uint32_t)sh.row_bytes,
                             smem_u32(&fixed));
        }
        int ids = -1, i = 0;   // ids: lane l holds that of the l-th of the next 32 rows
        for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, ++i) {
            if (p.ids && (i & 31) == 0) {
                const int64_t mine = t + (int64_t)lane * gridDim.x;
                ids = mine < p.T ? p.ids[mine] : -1;
            }
            const int id = __shfl_sync(0xffffffffu, ids, i & 31);
            if (!__all_sync(0xffffffffu, mbar_wait_hot(smem_u32(&empty[s]), phase ^ 1, p.status, sh.wait_ns))) break;
            if (one) {
                const bool bad = id < -1 || id >= p.n;   // nothing is read for it: the row stays as it was
                const uint32_t bar = smem_u32(&full[s]);
                row_id[s] = bad ? -2 : id;
                mbar_arrive_expect_tx(bar, bad ? 0u : (uint32_t)sh.stage_bytes);
                if (!bad && !sh.inject)
#pragma unroll
                    for (int op = 0; op < kOps; ++op)
                        if ((sh.per_row >> op) & 1)
                            bulk_g2s(smem_u32(ring) + (uint32_t)(s * sh.stage_bytes + sh.at[op]),
                                     norm_source<E>(p, op, t, (int64_t)id + 1), (uint32_t)sh.row_bytes, bar);
            }
            __syncwarp();
            if (++s == sh.stages) {
                s = 0;
                phase ^= 1;
            }
        }
        // the copies under way have landed before the block ends
        for (int k = 0; k < min(i, sh.stages); ++k) {
            if (--s < 0) {
                s = sh.stages - 1;
                phase ^= 1;
            }
            mbar_wait(smem_u32(&full[s]), phase, p.status, sh.wait_ns);
        }
        mbar_wait(smem_u32(&fixed), 0, p.status, sh.wait_ns);
        return;
    }
    // ------------------------------------------------------------ rows
    bool ok = mbar_wait(smem_u32(&fixed), 0, p.status, sh.wait_ns);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        ok = mbar_wait(smem_u32(&full[s]), phase, p.status, sh.wait_ns) && ok;
        auto operand = [&](int op) {
            return reinterpret_cast<const uint4 *>(((sh.per_row >> op) & 1 ? ring + s * sh.stage_bytes : smem) + sh.at[op]);
        };
        auto weights = [&](const lora_norm &nm, int gain, Weights<E, NT, V> &w) {
            if (nm.gain) w.g.load(operand(gain), 0, nvec);
            if (nm.shift) w.b.load(operand(gain + 1), 0, nvec);
        };
        const bool bad = row_id[s] == -2;
        if (bad && ok) {
            if (threadIdx.x == 0) atomicOr(p.status, LORA_STATUS_BAD_ID);
        } else if (ok) {
            Packed<E, NT, V> in;
            Row<E, NT, V> f;
            Weights<E, NT, V> w;
            in.load(operand(kOpX), 0, nvec);
            f.set(in);
            if (p.norm.kind) {
                weights(p.norm, kOpGain1, w);
                f.normalise(p.norm, w, p.d, nvec, part);
            }
            if constexpr (!AFTER) {
                f.store(p.h, t * p.ldh, nvec);
            } else {
                Packed<E, NT, V> gate;
                if (p.res.residual) in.load(operand(kOpRes), 0, nvec);
                if (p.res.gate_kind != LORA_GATE_NONE) gate.load(operand(kOpGate), 0, nvec);
#pragma unroll
                for (int j = 0; j < V; ++j) join<E>(p.res, f.f[j], gate.w[j], in.w[j]);
                if (p.r) f.store(p.r, t * p.ldr, nvec);
                if (p.h) {
                    if (NT > 32 && p.norm.kind) named_bar_sync(1, NT);   // the first norm's sums are read by all
                    weights(p.next, kOpGain2, w);
                    f.normalise(p.next, w, p.d, nvec, part);
                    f.store(p.h, t * p.ldh, nvec);
                }
            }
        }
        // The stage and the sums have been read by all.  A wait that ran out in any thread ends them all.
        if (!named_bar_and(2, NT, ok)) return;
        if (threadIdx.x == 0) mbar_arrive(smem_u32(&empty[s]));
        if (++s == sh.stages) {
            s = 0;
            phase ^= 1;
        }
    }
}

cudaLaunchConfig_t norm_config(int64_t grid, int block, size_t smem, cudaStream_t s, cudaLaunchAttribute *attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    if (options().pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    return cfg;
}

// Launches the persistent kernel, or returns LORA_ERR_UNSUPPORTED where two stages do not fit.
template <typename E, int NT, int V, bool AFTER>
int launch_ring(const NormParams &p, int dev, int sms, cudaStream_t s)
{
    auto kern = ring_norm_kernel<E, NT, V, AFTER>;
    constexpr int kShared = 227 * 1024;
    RingShape sh = {};
    sh.row_bytes = p.d * (int)sizeof(E);
    sh.wait_ns = wait_limit_ns();
    sh.inject = (int32_t)(options().inject_stall & 32);
    const bool gate = AFTER && p.res.gate_kind != LORA_GATE_NONE;
    const bool present[kOps] = {true,
                                AFTER && p.res.residual,
                                gate,
                                p.norm.kind && p.norm.gain,
                                p.norm.kind && p.norm.shift,
                                AFTER && p.next.kind && p.next.gain,
                                AFTER && p.next.kind && p.next.shift};
    const bool rows[kOps] = {true,
                             true,
                             p.res.gate_kind == LORA_GATE_TOKEN || (p.ids && p.res.ldgate),
                             p.ids && p.norm.ld,
                             p.ids && p.norm.ld,
                             p.ids && p.next.ld,
                             p.ids && p.next.ld};
    for (int op = 0; op < kOps; ++op) {
        int32_t &bytes = rows[op] ? sh.stage_bytes : sh.fixed_bytes;
        sh.at[op] = present[op] ? bytes : -1;
        if (!present[op]) continue;
        bytes += sh.row_bytes;
        if (rows[op]) sh.per_row |= 1 << op;
    }
    // As many blocks as registers allow, as long as each has a ring of at least two stages.
    int blocks = kRingBlocks<NT, V, AFTER>;
    auto depth = [&](int n) { return (kShared / n - 2048 - sh.fixed_bytes) / sh.stage_bytes; };
    while (blocks > 1 && depth(blocks) < 2) --blocks;
    sh.stages = std::min(kNormStages, depth(blocks));
    if (sh.stages < 2) return LORA_ERR_UNSUPPORTED;
    static std::once_flag once[64];
    static cudaError_t attr_rc[64];
    std::call_once(once[dev], [&] {
        attr_rc[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared - 1024);
    });
    if (attr_rc[dev] != cudaSuccess) return LORA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = norm_config(std::min<int64_t>(p.T, (int64_t)blocks * sms), NT + 32,
                                               (size_t)(sh.fixed_bytes + sh.stages * sh.stage_bytes), s, attr);
    if (cudaLaunchKernelEx(&cfg, kern, p, sh) != cudaSuccess) return LORA_ERR_CUDA;
    note_launch(kKernRingNorm);
    return LORA_OK;
}

template <typename E, int NT, int V, bool AFTER>
int launch_kernel(const NormParams &p, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = norm_config(p.T, NT, 0, s, attr);
    if (cudaLaunchKernelEx(&cfg, block_norm_kernel<E, NT, V, AFTER>, p) != cudaSuccess) return LORA_ERR_CUDA;
    note_launch(kKernBlockNorm);
    return LORA_OK;
}

// Rows per SM from which a ring pays, measured 4096 wide in bf16 only and taken for all widths and types (a block a
// row against the ring): before a block, which has
// one operand, 8 rows an SM 6.1 and 6.5 us, 12 rows 9.35 and 8.4; after it, 1 row 3.0 and 3.5 us, 4 rows 8.8 and
// 8.4, 8 rows 15.5 and 12.6.
constexpr int ring_rows_per_sm(bool after) { return after ? 4 : 12; }

// NT threads with V vectors each for a row: NT1, V1 where a block takes one row (latency counts, so many
// threads), NT2, V2 for persistent blocks (rows side by side count, so few; but not more than two vectors a
// thread while rows are short enough, whose registers spill otherwise; 0: none).
template <typename E, int NT1, int V1, int NT2, int V2>
int launch_one(const NormParams &p, bool after, int dev, int sms, cudaStream_t s)
{
    if constexpr (NT2 > 0)
        if (p.T >= ring_rows_per_sm(after) * sms) {
            const int rc =
                after ? launch_ring<E, NT2, V2, true>(p, dev, sms, s) : launch_ring<E, NT2, V2, false>(p, dev, sms, s);
            if (rc != LORA_ERR_UNSUPPORTED) return rc;
        }
    return after ? launch_kernel<E, NT1, V1, true>(p, s) : launch_kernel<E, NT1, V1, false>(p, s);
}

template <typename E>
int launch_typed(const NormParams &p, bool after, cudaStream_t s)
{
    const int nvec = p.d / Vec<E>::kN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return LORA_ERR_CUDA;
    static std::once_flag once[64];
    static int sms[64];
    std::call_once(once[dev], [&] { cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev); });
    if (sms[dev] < 1) return LORA_ERR_CUDA;
    if (nvec <= 32) return launch_one<E, 32, 1, 32, 1>(p, after, dev, sms[dev], s);
    if (nvec <= 128) return launch_one<E, 128, 1, 64, 2>(p, after, dev, sms[dev], s);
    if (nvec <= 256) return launch_one<E, 256, 1, 128, 2>(p, after, dev, sms[dev], s);
    if (nvec <= 512) return launch_one<E, 256, 2, 256, 2>(p, after, dev, sms[dev], s);
    if (nvec <= 1024) return launch_one<E, 512, 2, 512, 2>(p, after, dev, sms[dev], s);
    if (nvec <= 2048) return launch_one<E, 512, 4, 512, 4>(p, after, dev, sms[dev], s);
    if constexpr (LORA_MAX_NORM_WIDTH > 2048 * Vec<E>::kN) return launch_one<E, 1024, 4, 0, 0>(p, after, dev, sms[dev], s);
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
