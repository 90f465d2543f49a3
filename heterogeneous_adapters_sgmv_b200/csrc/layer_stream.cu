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
// split over the CTAs of a cluster where there are fewer tiles than SMs.  Each CTA finishes a share of the
// tokens; the others send it their partial sums (st.async into its shared memory), which are added in a
// fixed order (no atomics: bit-identical from run
// to run).  The adapter term is formed by the epilogue warps in fp32 while W streams: a thread holds one
// output column, so it reads its own row of B_i, and the token's v is the same for the whole warp; the
// terms wait in tensor memory, in the columns behind the accumulator.
//
// Warp roles: warp 0 fills a ring of (W, x) k-blocks by TMA; warp 1 issues tcgen05.mma; the others
// drain the accumulator (one, two or four per lane quarter), exchange it and finish the outputs.  Behind the shrink
// the pass over W starts before the grid-dependency wait, which only the adapter terms need.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "layer_epilogue.cuh"
#include "layer_shape.h"
#include "lora_common.cuh"
#include "lora_internal.h"
#include "tcgen05.cuh"

namespace lora {
namespace {

// ------------------------------------------------------------------------------- shrink

constexpr int kShrinkWarps = 8;
constexpr int kShrinkThreads = kShrinkWarps * 32;     // also the tokens that a cluster plans at a time
constexpr int kShrinkRows = 16;                       // rank rows of a unit (mma M)
constexpr int kShrinkTokens = 8;                      // tokens of a unit (mma N)
constexpr int kShrinkK = 32;                          // k elements of one warp step
constexpr int kVParts = 4;                            // parts of the k axis, at most

struct LayerShrinkParams {
    const AdapterDesc *desc;
    const int32_t *ids;
    const uint16_t *x;
    int64_t ldx;
    float *v;                      // [parts][T, ldv]
    int32_t ldv, n, h, T, parts;   // parts: pieces of the k axis, summed by the reader of v
    uint32_t *status;
};

// D += A . B, 16 x 8 x 16.  The sum over k may be taken in any order, so the fragments are not laid out
// by ldmatrix from shared memory but loaded from global memory as they lie: a lane's 16 bytes of row
// (lane / 4) at k = 8 (lane % 4) are the k elements it holds in two of these products, the same ones in
// A and in B.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Token of the nth (0 to 7) set bit of the window's mask; -1 when there are not that many.
__device__ __forceinline__ int nth_member(const uint32_t *members, int nth, int w0)
{
    uint32_t word = 0;
    int base = -1;
#pragma unroll
    for (int i = 0; i < kShrinkWarps; ++i) {
        const uint32_t m = members[i];
        const int c = __popc(m);
        if (base < 0 && nth < c) {
            word = m;
            base = w0 + 32 * i;
        }
        if (base < 0) nth -= c;
    }
    if (base < 0) return -1;
#pragma unroll
    for (int k = 0; k < kShrinkTokens - 1; ++k)
        if (k < nth) word &= word - 1;
    return base + __ffs(word) - 1;
}

// Asks L2 for the rows of A_i of the batch's first 256 tokens: a few blocks share each token (the first of
// those with its adapter).
__device__ __forceinline__ void shrink_hints(const LayerShrinkParams &p)
{
    const volatile int32_t *ids = p.ids;
    const int tid = threadIdx.x, tokens = min(p.T, kShrinkThreads);
    const int blocks = max(1, (int)gridDim.x / tokens), t = blockIdx.x / blocks;
    const int mine = tid < tokens ? ids[tid] : -1, a = t < tokens ? ids[t] : -1;
    if (__syncthreads_or(tid < t && mine == a) || a < 0 || a >= p.n) return;
    const AdapterDesc d = p.desc[a];
    const int64_t bytes = (int64_t)d.rank * p.h * 2;
    for (int64_t at = ((int64_t)(blockIdx.x % blocks) * kShrinkThreads + tid) * 128; at < bytes;
         at += (int64_t)blocks * kShrinkThreads * 128)
        prefetch_l2(static_cast<const uint8_t *>(d.A) + at);
}

// A unit of work is up to 8 tokens of one adapter (found among 256 consecutive tokens) times 16 of its
// rank rows times one part of the k axis, so a row of A_i is read once for 8 tokens and x once for 16
// rows.  The reads bound it; the products (2 T r h flop, a few percent of the pass over W) go to the
// warp-level tensor-core instruction, whose operands need no shared memory here, so that all of the
// kernel's warps do nothing but keep loads in flight.  The parts of the k axis are sized for about four
// steps a warp and go to memory one by one (the pass over W adds them up as it reads them): in a small
// batch the time is a chain of dependent loads, and every step or barrier more is felt (one token: ids,
// descriptor, A_i and x, store).
__global__ void __launch_bounds__(kShrinkThreads, 2) layer_shrink_kernel(const __grid_constant__ LayerShrinkParams p)
{
    __shared__ __align__(16) int32_t ids[kShrinkThreads];
    __shared__ AdapterDesc desc[kShrinkThreads];
    __shared__ int32_t first_unit[kShrinkThreads];
    __shared__ int32_t warp_units[kShrinkWarps];
    __shared__ uint32_t members[kShrinkWarps];
    __shared__ float part[kShrinkWarps][kShrinkRows * kShrinkTokens];
    // While the kernel before ends, the weights that this batch will ask for go to L2.  The ids may not be
    // final yet: what is read here serves as a hint and for nothing else (a range check makes any value safe).
    shrink_hints(p);
    // then the wait, and only behind it launch_dependents, which tells the pass over W that x and the
    // epilogue's operands are final and that only v is still to come
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int steps = (p.h + kShrinkK - 1) / kShrinkK;
    const int row = lane >> 2, kl = (lane & 3) * 8;
    int64_t item = blockIdx.x;   // counts the items of all windows
    int64_t skipped = 0;
    for (int w0 = 0; w0 < p.T; w0 += kShrinkThreads) {
        // ---- the window's units, one token a thread
        const int a = w0 + tid < p.T ? p.ids[w0 + tid] : -1;
        const bool good = a >= 0 && a < p.n;
        if (a != -1 && !good && blockIdx.x == 0) atomicOr(p.status, LORA_STATUS_BAD_ID);
        AdapterDesc mine = {};
        if (good) mine = p.desc[a];
        ids[tid] = a;
        __syncthreads();
        // earlier tokens with the same adapter: of the warps before, then of this warp
        int before = 0;
        if (w0 + warp * 32 < p.T)
#pragma unroll 8
            for (int s = 0; s < warp * 32; s += 4) {
                const int4 o = *reinterpret_cast<const int4 *>(ids + s);
                before += (o.x == a) + (o.y == a) + (o.z == a) + (o.w == a);
            }
        before += __popc(__match_any_sync(0xffffffffu, a) & ((1u << lane) - 1));
        const int units = good && before % kShrinkTokens == 0 ? (mine.rank + kShrinkRows - 1) / kShrinkRows : 0;
        desc[tid] = mine;
        int incl = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) warp_units[warp] = incl;
        __syncthreads();
        int first = incl - units, total = 0;
#pragma unroll
        for (int i = 0; i < kShrinkWarps; ++i) {
            if (i < warp) first += warp_units[i];
            total += warp_units[i];
        }
        first_unit[tid] = first;
        // ---- every gridDim.x-th item
        for (; item - skipped < (int64_t)total * p.parts; item += gridDim.x) {
            const int at_item = (int)(item - skipped), u = at_item / p.parts, ks = at_item - u * p.parts;
            const int lo = __syncthreads_count(first <= u) - 1;   // the token that leads the unit
            const int ad = ids[lo], k0 = (u - first_unit[lo]) * kShrinkRows;
            const uint32_t vote = __ballot_sync(0xffffffffu, tid >= lo && a == ad);
            if (lane == 0) members[warp] = vote;
            const int rank = desc[lo].rank;
            const uint16_t *A = static_cast<const uint16_t *>(desc[lo].A);
            __syncthreads();
            const int tok = nth_member(members, row, w0);   // this lane's token column
            const uint16_t *a0 = k0 + row < rank ? A + (int64_t)(k0 + row) * p.h + kl : nullptr;
            const uint16_t *a1 = k0 + row + 8 < rank ? A + (int64_t)(k0 + row + 8) * p.h + kl : nullptr;
            const uint16_t *xr = tok >= 0 ? p.x + tok * p.ldx + kl : nullptr;
            const int per = (steps + p.parts - 1) / p.parts, s1 = min(steps, (ks + 1) * per);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int j = ks * per + warp; j < s1; j += kShrinkWarps) {
                const int k = j * kShrinkK;
                const bool in = k + kl < p.h;   // h is a multiple of 8
                const uint4 zero = make_uint4(0, 0, 0, 0);
                const uint4 wa = in && a0 ? *reinterpret_cast<const uint4 *>(a0 + k) : zero;
                const uint4 wb = in && a1 ? *reinterpret_cast<const uint4 *>(a1 + k) : zero;
                const uint4 xv = in && xr ? *reinterpret_cast<const uint4 *>(xr + k) : zero;
                mma_16x8x16(acc, wa.x, wb.x, wa.y, wb.y, xv.x, xv.y);
                mma_16x8x16(acc, wa.z, wb.z, wa.w, wb.w, xv.z, xv.w);
            }
            // lane's outputs: rows lane / 4 and + 8, tokens 2 (lane % 4) and + 1
            float *out = part[warp] + row * kShrinkTokens + (lane & 3) * 2;
            out[0] = acc[0];
            out[1] = acc[1];
            out[8 * kShrinkTokens] = acc[2];
            out[8 * kShrinkTokens + 1] = acc[3];
            __syncthreads();
            if (tid < kShrinkRows * kShrinkTokens) {
                const int r = tid / kShrinkTokens, at = nth_member(members, tid % kShrinkTokens, w0);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kShrinkWarps; ++i) sum += part[i][tid];
                if (at >= 0 && k0 + r < rank) p.v[((int64_t)ks * p.T + at) * p.ldv + k0 + r] = sum * desc[lo].scale;
            }
        }
        skipped += (int64_t)total * p.parts;
        __syncthreads();   // the plan is read by all before the next window's is written
    }
}

// ------------------------------------------------------------------------------- pass over W

struct LayerStreamParams {
    CUtensorMap tm_x;             // x [T, h], box 64 x N
    CUtensorMap tm_w;             // W [o, h], box 64 x 128
    const AdapterDesc *desc;
    const int32_t *ids;           // null: no adapters
    const float *v;               // [v_parts][T, ldv]: the scaled intermediate is their sum
    int32_t v_parts;
    int32_t ldv, n;
    int32_t T, h, o;
    int32_t N, NT, stages;        // tokens per tile, token tiles, ring depth
    int32_t share, ncols;         // tokens of a tile that one CTA of a cluster finishes, TMEM columns
    int32_t recv;                 // offset in shared memory of the peers' partial sums
    int32_t alias;                // they land in the ring
    int32_t early;                // launched right behind the shrink (see above)
    uint16_t *y;                  // at column y_offset
    int64_t ldy;
    EpiParams epi;
    uint32_t *status;
    uint64_t wait_ns;
    int32_t inject;               // test-only: the first k-block is armed but never loaded
};

// One token's term for a rank of 8 LR.  The warp's 32 rows of B are one block, read in LR contiguous pieces of 512
// bytes: 16 bytes a lane, always the same 8 elements of a row (lane % LR), of row e (32 / LR) + lane / LR in piece e
// (a lane a row takes 32 sectors a load, and there is next to no L1 beside this much shared memory).  The sums over a
// row's LR lanes are formed while the rows are dealt out, so that lane = row again.
template <int LR>
__device__ __forceinline__ float expand_block(const void *B, int64_t n, int rows, const float *v)
{
    const int lane = threadIdx.x & 31;
    const uint16_t *src = static_cast<const uint16_t *>(B) + (n - lane) * (8 * LR) + lane * 8;
    const float4 p = *reinterpret_cast<const float4 *>(v + lane % LR * 8);
    const float4 q = *reinterpret_cast<const float4 *>(v + lane % LR * 8 + 4);
    float s[LR];
#pragma unroll
    for (int e = 0; e < LR; ++e) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (e * (32 / LR) + lane / LR < rows) w = *reinterpret_cast<const uint4 *>(src + e * 256);
        float s0 = bf16_lo(w.x) * p.x, s1 = bf16_hi(w.x) * p.y;
        s0 = fmaf(bf16_lo(w.y), p.z, s0);
        s1 = fmaf(bf16_hi(w.y), p.w, s1);
        s0 = fmaf(bf16_lo(w.z), q.x, s0);
        s1 = fmaf(bf16_hi(w.z), q.y, s1);
        s0 = fmaf(bf16_lo(w.w), q.z, s0);
        s1 = fmaf(bf16_hi(w.w), q.w, s1);
        s[e] = s0 + s1;
    }
#pragma unroll
    for (int g = LR / 2; g > 0; g /= 2)
#pragma unroll
        for (int e = 0; e < g; ++e) {
            const bool up = lane & g;
            const float give = up ? s[e] : s[e + g];
            s[e] = (up ? s[e + g] : s[e]) + __shfl_xor_sync(0xffffffffu, give, g);
        }
    return __shfl_sync(0xffffffffu, s[0], lane % (32 / LR) * LR + lane / (32 / LR));
}

// The adapter terms of one thread's output column n, a batch of tokens at a time:
//   d[j] = sum_k B_j[n, k] v_j[k].
// Rows of a rank that is a multiple of 8 are 16-byte aligned and read NP pieces of 8 a step, the step's
// loads together (under a saturated memory system a load takes 2 to 4 us) and the first step's before v is
// there.
// ANY: the table may hold other ranks.  Rows of a rank that is no multiple of 8 are read by the aligned pieces that
// they lie in (the matrix starts on 16 bytes and, o being a multiple of 8, ends there, so no piece leaves it), and
// what belongs to their neighbours is passed over (4096 -> 14336, 64 tokens of rank 60: 461 us element by element,
// 117 so; of rank 12: 65.7 and 46.2).  Ranks of 64 and 128 go by expand_block (92.5 -> 76.1 and 170.5 -> 107.4 us).  A
// kernel of its own, since the registers that this takes cost the others (rank 16: 31.6 us without, 41.9 with).
template <int NP, bool ANY>
struct ExpandRows {
    static constexpr int NB = kLBatch;
    const int32_t *rank;        // per token; <= 0: none
    const void *const *B;
    int64_t n;
    bool col_ok;
    int rows;                   // rows of W in this warp
    int end;                    // tokens of this thread: the batches end here
    uint4 b[NB][NP];            // the step at hand

    // ranks whose rows are read 16 bytes a lane, a lane a row
    static __device__ __forceinline__ bool in_steps(int r)
    {
        return r > 0 && (!ANY || ((r & 7) == 0 && r != 64 && r != 128));
    }
    __device__ __forceinline__ int even(int i) const
    {
        const int r = i < end && col_ok ? rank[i] : 0;
        return in_steps(r) ? r : 0;
    }
    __device__ __forceinline__ void load(int i, int k)
    {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int r = even(i + j);
            const uint16_t *row = r ? static_cast<const uint16_t *>(B[i + j]) + n * r + k : nullptr;
#pragma unroll
            for (int e = 0; e < NP; ++e)
                if (k + 8 * e < r) b[j][e] = *reinterpret_cast<const uint4 *>(row + 8 * e);
        }
    }
    __device__ __forceinline__ int steps(int i) const   // the batch's pieces end here; the same in all lanes
    {
        int most = 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int r = i + j < end ? rank[i + j] : 0;
            if (in_steps(r)) most = max(most, r);
        }
        return most;
    }
    // the batch at i, whose first step is loaded; loads the first step of the next
    __device__ __forceinline__ void run(int i, const float *v, int ldv, float (&d)[NB])
    {
        const int most = steps(i);
        for (int k = 0; k < most; k += 8 * NP) {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int r = even(i + j);
#pragma unroll
                for (int e = 0; e < NP; ++e)
                    if (k + 8 * e < r) {
                        const float4 p = *reinterpret_cast<const float4 *>(v + j * ldv + k + 8 * e);
                        const float4 q = *reinterpret_cast<const float4 *>(v + j * ldv + k + 8 * e + 4);
                        float s0 = d[j], s1 = bf16_hi(b[j][e].x) * p.y;
                        s0 = fmaf(bf16_lo(b[j][e].x), p.x, s0);
                        s0 = fmaf(bf16_lo(b[j][e].y), p.z, s0);
                        s1 = fmaf(bf16_hi(b[j][e].y), p.w, s1);
                        s0 = fmaf(bf16_lo(b[j][e].z), q.x, s0);
                        s1 = fmaf(bf16_hi(b[j][e].z), q.y, s1);
                        s0 = fmaf(bf16_lo(b[j][e].w), q.z, s0);
                        s1 = fmaf(bf16_hi(b[j][e].w), q.w, s1);
                        d[j] = s0 + s1;
                    }
            }
            if (k + 8 * NP < most) load(i, k + 8 * NP);
        }
        if constexpr (ANY) others(i, v, ldv, d);
        load(i + NB, 0);
    }
    // what is not in_steps of the batch at i
    __device__ __forceinline__ void others(int i, const float *v, int ldv, float (&d)[NB]) const
    {
#pragma unroll 1
        for (int j = 0; j < NB; ++j) {
            const int r = i + j < end && rows > 0 ? rank[i + j] : 0;
            if (r != 64 && r != 128) continue;
            const float t = r == 64 ? expand_block<8>(B[i + j], n, rows, v + j * ldv)
                                    : expand_block<16>(B[i + j], n, rows, v + j * ldv);
#pragma unroll
            for (int u = 0; u < NB; ++u) d[u] += u == j ? t : 0.f;
        }
        // a row starts `off` elements into an aligned piece
        int odd[NB], off[NB], longest = 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int r = i + j < end && col_ok ? rank[i + j] : 0;
            odd[j] = r > 0 && (r & 7) ? r : 0;
            off[j] = (int)(n * odd[j]) & 7;
            longest = max(longest, off[j] + odd[j]);
        }
        for (int k = 0; k < longest; k += 8) {
            uint4 w[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (k < off[j] + odd[j])
                    w[j] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(B[i + j]) + n * odd[j] -
                                                            off[j] + k);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                const int at = k - off[j];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if ((uint32_t)(at + q) < (uint32_t)odd[j])
                        d[j] = fmaf(q & 1 ? bf16_hi(u[q / 2]) : bf16_lo(u[q / 2]), v[j * ldv + at + q], d[j]);
            }
        }
    }
};

// S CTAs of a cluster split the k axis; E epilogue warps (see stream_shape); CTAS to an SM.
template <int S, int E, int CTAS, bool ANY>
__global__ void __launch_bounds__(E * 32 + 64, CTAS) layer_stream_kernel(const __grid_constant__ LayerStreamParams p)
{
    // 16-byte pieces of B_i's rows in registers, for each token of a batch: four where there are registers for
    // them (8 warps on 4096 columns, 256 tokens, ranks to 64: 81 against 95 us with two)
    constexpr int NP = E == 4 || (E == 8 && CTAS == 1) ? 4 : 2;
    constexpr int H = E / 4;   // epilogue warps per TMEM lane quarter, each with its part of the tokens
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stage_bytes = kLWBytes + p.N * 128;
    LayerStreamCtl &ctl = *reinterpret_cast<LayerStreamCtl *>(ring + p.stages * stage_bytes);
    uint8_t *v_buf = reinterpret_cast<uint8_t *>(&ctl + 1);
    const void **tok_B = reinterpret_cast<const void **>(v_buf + H * v_bytes(E));
    int32_t *tok_rank = reinterpret_cast<int32_t *>(tok_B + p.share);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int crank = S > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / S;
    const int mt = tile / p.NT, tt = tile % p.NT;   // token tiles of one W tile side by side: W once from HBM
    const int row0 = mt * kLM, t0 = tt * p.N;
    const int nkb_all = (p.h + kLK - 1) / kLK;
    const int kb0 = (int)((int64_t)crank * nkb_all / S), nkb = (int)((int64_t)(crank + 1) * nkb_all / S) - kb0;
    // this CTA finishes tokens [ta, tb) of the tile
    const int nv = min(p.N, p.T - t0);
    const int ta = min(nv, crank * p.share), tb = min(nv, ta + p.share);

    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), 1);
            mbar_init(smem_u32(&ctl.empty[i]), 1);
        }
        mbar_init(smem_u32(&ctl.done), 1);
        mbar_init(smem_u32(&ctl.recv), 1);
        fence_mbar_init_cluster();
        // the partial sums of the other CTAs: 16 bytes per row of W and four tokens
        if (S > 1) mbar_arrive_expect_tx(smem_u32(&ctl.recv), (uint32_t)((S - 1) * ((tb - ta + 3) / 4) * kLM * 16));
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl.tmem_base), (uint32_t)p.ncols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // After the allocation: a dependent kernel's CTA on this SM cannot take the tensor memory that
    // this one is still waiting for.
    pdl_launch_dependents();
    // The first cluster barrier says that a CTA may be sent partial sums: its barriers are set up, and
    // where the sums land in the ring, its products are complete.
    if (S > 1 && !p.alias) cluster_arrive_release();
    const uint32_t tmem = ctl.tmem_base;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // The whole warp runs the loop and one lane issues: the copy and MMA instructions take their operands
        // from uniform registers, which a loop inside one lane has to move them to one by one.
        const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
        const bool one = elect_one();
        const int pre = min(nkb, p.stages);
        // Behind the shrink, whose CTAs have all waited for what came earlier, x and W are final.  Without it
        // nothing is, W included (a kernel right before this one may have written it), and what W holds now is
        // only asked into L2, where a later write changes it.
        if (!p.early) {
            if (one)
                for (int kb = 0; kb < pre; ++kb) tma_prefetch_2d(&p.tm_w, (kb0 + kb) * kLK, row0);
            pdl_wait();
        }
        if (one)
            for (int kb = 0; kb < pre; ++kb) {
                mbar_arrive_expect_tx(full0 + kb * 8, (uint32_t)stage_bytes);
                if (p.inject && kb == 0) continue;
                tma_load_2d(ring0 + kb * stage_bytes, &p.tm_w, (kb0 + kb) * kLK, row0, full0 + kb * 8);
                tma_load_2d(ring0 + kb * stage_bytes + kLWBytes, &p.tm_x, (kb0 + kb) * kLK, t0, full0 + kb * 8);
            }
        int kb = pre, s = pre == p.stages ? 0 : pre;
        uint32_t phase = 0;
        for (; kb < nkb; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_hot(empty0 + s * 8, phase, p.status, p.wait_ns))) break;
            if (one) {
                mbar_arrive_expect_tx(full0 + s * 8, (uint32_t)stage_bytes);
                tma_load_2d(ring0 + s * stage_bytes, &p.tm_w, (kb0 + kb) * kLK, row0, full0 + s * 8);
                tma_load_2d(ring0 + s * stage_bytes + kLWBytes, &p.tm_x, (kb0 + kb) * kLK, t0, full0 + s * 8);
            }
            if (++s == p.stages) {
                s = 0;
                phase ^= 1;
            }
        }
        // drain: the copies of the last stages armed have landed before the ring is given up
        for (int i = max(0, kb - p.stages); i < kb; ++i)
            mbar_wait(full0 + i % p.stages * 8, (i / p.stages) & 1, p.status, p.wait_ns);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_bf16(kLM, p.N);
        const uint32_t full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
        const uint64_t wd0 = sw128_desc(smem_u32(ring)), xd0 = sw128_desc(smem_u32(ring) + kLWBytes);
        const bool one = elect_one();
        int s = 0;
        uint32_t phase = 0;
        for (int kb = 0; kb < nkb; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_hot(full0 + s * 8, phase, p.status, p.wait_ns))) break;
            tc_fence_after();
            const uint64_t wd = wd0 + (uint64_t)(s * (stage_bytes >> 4)), xd = xd0 + (uint64_t)(s * (stage_bytes >> 4));
            if (one) {
#pragma unroll
                for (int k = 0; k < kLK / 16; ++k) umma_bf16(tmem, wd + 2 * k, xd + 2 * k, idesc, (kb | k) != 0 ? 1u : 0u);
                umma_commit(empty0 + s * 8);
            }
            if (++s == p.stages) {
                s = 0;
                phase ^= 1;
            }
        }
        if (one) umma_commit(smem_u32(&ctl.done));   // every MMA issued so far
        mbar_wait(smem_u32(&ctl.done), 0, p.status, p.wait_ns);
        __syncwarp();
    }
    if (warp < 2) {
        if (S > 1) {
            if (p.alias) cluster_arrive_release();
            cluster_wait_acquire();
            cluster_arrive_release();
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // lane = row of W; this thread's tokens are [i0, i1) of the share
        const int q = warp & 3, part = (warp - 2) >> 2, et = tid - 64;
        const int m = q * 32 + lane, n = row0 + m;
        const bool col_ok = n < p.o;
        const int hs = (p.share / H + kLBatch - 1) / kLBatch * kLBatch;
        const int i0 = part * hs, i1 = min(tb - ta, i0 + hs);
        const uint32_t tmem_row = tmem + ((uint32_t)(q * 32) << 16);
        const int64_t tok0 = t0 + ta;
        if (!p.early) pdl_wait();   // ids may come from the kernel before
        for (int i = et; i < tb - ta; i += E * 32) {
            int r = 0;
            const void *B = nullptr;
            if (p.ids) {
                const int a = p.ids[tok0 + i];
                if (a >= 0 && a < p.n) {
                    r = p.desc[a].rank;
                    B = p.desc[a].B;
                } else if (a != -1) {
                    r = -1;
                }
            }
            tok_rank[i] = r;
            tok_B[i] = B;
        }
        const float bias = (col_ok && p.epi.bias) ? bf16_f(p.epi.bias[n]) : 0.f;
        named_bar_sync(1, E * 32);
        // what the steps below read goes to L2 while there is nothing else to do
        const int rows_left = min(32, p.o - (n - lane));   // rows of this warp inside W
        for (int i = i0; i < i1 && rows_left > 0; ++i) {
            const int r = tok_rank[i];
            const uint8_t *b = static_cast<const uint8_t *>(tok_B[i]) + (int64_t)(n - lane) * r * 2;
            for (int off = lane * 128; off < rows_left * r * 2; off += 32 * 128) prefetch_l2(b + off);
            if (lane == 0) {
                if (p.epi.mul) prefetch_l2(p.epi.mul + (tok0 + i) * p.epi.ldmul + n);
                if (p.epi.res) prefetch_l2(p.epi.res + (tok0 + i) * p.epi.ldres + n);
            }
        }
        // While W streams: bias and adapter term of every output, kept in tensor memory behind the
        // accumulator.
        ExpandRows<NP, ANY> ex;
        ex.rank = tok_rank;
        ex.B = tok_B;
        ex.n = n;
        ex.col_ok = col_ok;
        ex.rows = rows_left;
        ex.end = i1;
        ex.load(i0, 0);
        float *vs = reinterpret_cast<float *>(v_buf + part * v_bytes(E));
        const int at_once = p.ids ? v_bytes(E) / 4 / p.ldv / kLBatch * kLBatch : p.N;
        if (p.early) pdl_wait();   // v
        for (int c = i0; c < i1; c += at_once) {
            const int ce = min(i1, c + at_once);
            if (p.ids) {
                if (c > i0) named_bar_sync(2 + part, 128);   // the last tokens' v is done with
                const float4 *src = reinterpret_cast<const float4 *>(p.v + (tok0 + c) * p.ldv);
                for (int e = et & 127; e < (ce - c) * p.ldv / 4; e += 128) {
                    float4 f[kVParts];
#pragma unroll
                    for (int k = 0; k < kVParts; ++k)
                        if (k < p.v_parts) f[k] = src[e + (int64_t)k * p.T * (p.ldv / 4)];
#pragma unroll
                    for (int k = 1; k < kVParts; ++k)
                        if (k < p.v_parts) {
                            f[0].x += f[k].x;
                            f[0].y += f[k].y;
                            f[0].z += f[k].z;
                            f[0].w += f[k].w;
                        }
                    reinterpret_cast<float4 *>(vs)[e] = f[0];
                }
                named_bar_sync(2 + part, 128);
            }
            for (int i = c; i < ce; i += kLBatch) {
                float d[kLBatch] = {bias, bias, bias, bias};
                ex.run(i, vs + (i - c) * p.ldv, p.ldv, d);
                __syncwarp();
                tmem_st4(tmem_row + (uint32_t)(p.N + i), d[0], d[1], d[2], d[3]);
            }
        }
        // mul and residual of two batches, read ahead of their use
        uint16_t mu[2][kLBatch], re[2][kLBatch];
        auto operands = [&](int i, uint16_t (&m4)[kLBatch], uint16_t (&r4)[kLBatch]) {
#pragma unroll
            for (int j = 0; j < kLBatch; ++j) {
                const bool in = i + j < i1 && col_ok;
                m4[j] = in && p.epi.mul ? p.epi.mul[(tok0 + i + j) * p.epi.ldmul + n] : (uint16_t)0;
                r4[j] = in && p.epi.res ? p.epi.res[(tok0 + i + j) * p.epi.ldres + n] : (uint16_t)0;
            }
        };
#pragma unroll
        for (int u = 0; u < 2; ++u) operands(i0 + u * kLBatch, mu[u], re[u]);
        // a wait that ran out makes the warp skip the rest, but not the cluster's barriers
        bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&ctl.done), 0, p.status, p.wait_ns));
        tc_fence_after();
        const uint8_t *recv = ring + p.recv;
        const int groups = p.share / 4;   // slots of four tokens per source
        if (S > 1) {
            if (p.alias) cluster_arrive_release();
            cluster_wait_acquire();
            // partial sums of the tokens that other CTAs finish, four tokens of a row at a time
            for (int c = part * 16; ok && c < nv; c += 16 * H) {
                float f[16];
                tmem_ld16(tmem_row + (uint32_t)c, f);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int tok = c + 4 * g, to = tok / p.share;
                    if (tok >= nv || to == crank) continue;
                    const int slot = (crank - to - 1 + S) % S;
                    const uint32_t at = smem_u32(recv) + (uint32_t)(((slot * groups + (tok - to * p.share) / 4) * kLM + m) * 16);
                    st_async_v4(at, smem_u32(&ctl.recv), (uint32_t)to,
                                make_float4(f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]));
                }
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&ctl.recv), 0, p.status, p.wait_ns)) && ok;
            cluster_arrive_release();   // nothing more comes to this CTA
        }
        for (int i2 = i0; ok && i2 < i1; i2 += 2 * kLBatch) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = i2 + u * kLBatch;
                if (i >= i1) break;
                float z[kLBatch], f[kLBatch];
                tmem_ld4(tmem_row + (uint32_t)(p.N + i), z);
                tmem_ld4(tmem_row + (uint32_t)(ta + i), f);
                float4 o[S > 1 ? S - 1 : 1];
#pragma unroll
                for (int c = 0; c < S - 1; ++c)
                    o[c] = *reinterpret_cast<const float4 *>(recv + ((c * groups + i / 4) * kLM + m) * 16);
#pragma unroll
                for (int j = 0; j < kLBatch; ++j) z[j] += f[j];
#pragma unroll
                for (int c = 0; c < S - 1; ++c) {
                    z[0] += o[c].x;
                    z[1] += o[c].y;
                    z[2] += o[c].z;
                    z[3] += o[c].w;
                }
                activate(z, p.epi.act);
#pragma unroll
                for (int j = 0; j < kLBatch; ++j) {
                    if (p.epi.mul) z[j] *= bf16_f(mu[u][j]);
                    if (p.epi.res) z[j] += bf16_f(re[u][j]);
                    if (i + j < i1 && col_ok && tok_rank[i + j] >= 0)
                        p.y[(tok0 + i + j) * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(z[j]));
                }
                operands(i + 2 * kLBatch, mu[u], re[u]);
                __syncwarp();
            }
        }
        tc_fence_before();
    }
    if (S > 1) cluster_wait_acquire();   // no CTA leaves while it may still be sent something
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, (uint32_t)p.ncols);
}

template <int S, int E, int CTAS, bool ANY>
int launch_stream(const LayerStreamParams &p, const StreamShape &sh, cudaStream_t s, int dev)
{
    auto kern = layer_stream_kernel<S, E, CTAS, ANY>;
    static std::once_flag once[64];
    static cudaError_t attr_rc[64];
    std::call_once(once[dev], [&] {
        attr_rc[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (attr_rc[dev] != cudaSuccess) return LORA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)((p.o + kLM - 1) / kLM) * p.NT * S));
    cfg.blockDim = dim3((2 + E) * 32);
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
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return LORA_ERR_CUDA;
    note_launch(kKernLayerStream);
    return LORA_OK;
}

template <int S>
int clusters_at_once()
{
    auto kern = layer_stream_kernel<S, 8, 1, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(10 * 32);
    cfg.dynamicSmemBytes = 210 * 1024;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = S;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess)
        return 0;   // no clusters
    return n;
}

const ClusterFit &cluster_fit(int dev, int n_sms)
{
    static std::once_flag once[64];
    static ClusterFit fit[64];
    std::call_once(once[dev], [&] {
        fit[dev] = {{n_sms, clusters_at_once<2>(), clusters_at_once<4>(), clusters_at_once<8>()}};
    });
    return fit[dev];
}

template <int E, int CTAS, bool ANY>
int launch_stream_width(const LayerStreamParams &p, const StreamShape &sh, cudaStream_t s, int dev)
{
    switch (sh.S) {
    case 8: return launch_stream<8, E, CTAS, ANY>(p, sh, s, dev);
    case 4: return launch_stream<4, E, CTAS, ANY>(p, sh, s, dev);
    case 2: return launch_stream<2, E, CTAS, ANY>(p, sh, s, dev);
    default: return launch_stream<1, E, CTAS, ANY>(p, sh, s, dev);
    }
}

template <bool ANY>
int launch_stream_shape(const LayerStreamParams &p, const StreamShape &sh, cudaStream_t s, int dev)
{
    if (sh.E == 16) return launch_stream_width<16, 1, ANY>(p, sh, s, dev);
    if (sh.E == 8)
        return sh.ctas == 2 ? launch_stream_width<8, 2, ANY>(p, sh, s, dev) : launch_stream_width<8, 1, ANY>(p, sh, s, dev);
    return sh.ctas == 2 ? launch_stream_width<4, 2, ANY>(p, sh, s, dev) : launch_stream_width<4, 1, ANY>(p, sh, s, dev);
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

int layer_v_parts(int32_t T, int32_t h)
{
    if (T > kLayerPartTokens) return 1;   // enough units without
    return std::min(kVParts, std::max(1, h / (kShrinkK * kShrinkWarps * 4)));
}

// Batches above kLayerPartTokens need fewer rows a token; a workspace made for one serves the smaller ones too.
int64_t layer_v_rows(int32_t T, int32_t h)
{
    const int32_t in_parts = std::min(T, kLayerPartTokens);
    return std::max<int64_t>(T, (int64_t)layer_v_parts(in_parts, h) * in_parts);
}

int launch_layer_shrink(const lora_table *t, const int32_t *ids, int32_t T, const void *x, int64_t ldx, float *v,
                        int32_t ldv, cudaStream_t s)
{
    int dev = 0, n_sms = 0;
    if (device_sms(&dev, &n_sms) != LORA_OK) return LORA_ERR_CUDA;
    // With the same split of the SM's shared memory as the pass over W, whose CTAs can then join this kernel's on an
    // SM where registers allow (4 epilogue warps, or two CTAs to an SM) instead of waiting for the SM to empty.
    static std::once_flag once[64];
    std::call_once(once[dev], [] {
        cudaFuncSetAttribute(layer_shrink_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    });
    LayerShrinkParams p;
    p.desc = t->d_desc;
    p.ldx = ldx;
    p.ldv = ldv;
    p.n = t->n;
    p.h = t->h;
    p.status = t->d_status;
    p.T = T;
    p.ids = ids;
    p.x = static_cast<const uint16_t *>(x);
    p.v = v;
    p.parts = layer_v_parts(T, t->h);
    const int64_t items = (int64_t)T * ((t->max_rank + kShrinkRows - 1) / kShrinkRows) * p.parts;   // at most
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, 2 * n_sms));
    cfg.blockDim = dim3(kShrinkThreads);
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
    return LORA_OK;
}

int launch_layer_stream(const lora_table *t, const int32_t *ids, int32_t T, const void *x, int64_t ldx, const void *W,
                        int64_t ldw, const lora_epilogue *epi, void *y, int64_t ldy, int32_t y_off, const float *v,
                        int32_t ldv, cudaStream_t s)
{
    int dev = 0, n_sms = 0, rc;
    if (device_sms(&dev, &n_sms) != LORA_OK) return LORA_ERR_CUDA;
    const StreamShape sh = stream_shape(T, t->h, t->o, n_sms, cluster_fit(dev, n_sms), ids != nullptr);
    LayerStreamParams p;
    std::memset(&p, 0, sizeof p);
    if ((rc = encode_sw128(&p.tm_x, x, (uint64_t)t->h, (uint64_t)T, (uint64_t)ldx, (uint32_t)sh.N)) != LORA_OK ||
        (rc = encode_sw128(&p.tm_w, W, (uint64_t)t->h, (uint64_t)t->o, (uint64_t)ldw, kLM)) != LORA_OK)
        return rc;
    p.desc = t->d_desc;
    p.ids = ids;
    p.v = v;
    p.v_parts = layer_v_parts(T, t->h);
    p.ldv = ldv;
    p.n = t->n;
    p.T = T;
    p.h = t->h;
    p.o = t->o;
    p.N = sh.N;
    p.NT = sh.NT;
    p.stages = sh.stages;
    p.share = sh.share;
    p.ncols = sh.ncols;
    p.recv = sh.recv;
    p.alias = sh.alias;
    p.early = (ids && options().pdl) ? 1 : 0;
    p.y = static_cast<uint16_t *>(y) + y_off;
    p.ldy = ldy;
    p.epi = epi_params(epi);
    p.status = t->d_status;
    p.wait_ns = wait_limit_ns();
    p.inject = (int32_t)(options().inject_stall & 8);
    // the table's ranks: all multiples of 8, none above 64 and some below (a table of 64 alone is better off with
    // its block reads, 92.5 -> 76.1 us; one of 8 to 64 is not, 51.2 -> 58.2; 4096 -> 14336, 64 tokens)
    const bool plain = !ids || (t->ranks_of_8 && t->max_rank <= 64 && t->min_rank < 64);
    return plain ? launch_stream_shape<false>(p, sh, s, dev) : launch_stream_shape<true>(p, sh, s, dev);
}

}  // namespace lora
