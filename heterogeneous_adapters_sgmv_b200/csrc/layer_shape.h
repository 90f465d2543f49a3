// How a call of lora_bgmv_layer's pass over W is cut into tiles, clusters and shared memory
// (layer_stream.cu).  Host code without CUDA, so that it can be looked over without a GPU.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "lora_sgmv.h"

namespace lora {
namespace {

constexpr int kLM = 128;                      // rows of W per tile (MMA M)
constexpr int kLK = 64;                       // k-block: one 128-byte swizzled row of bf16
constexpr int kLWBytes = kLM * 128;
constexpr int kLMaxN = 256;                   // tokens per tile (MMA N)
constexpr int kLMaxStages = 8;

struct alignas(16) LayerStreamCtl {
    uint64_t full[kLMaxStages], empty[kLMaxStages];
    uint64_t done, recv;
    uint32_t tmem_base, pad[3];
    // behind it: v of the tokens at hand (v_bytes for each four epilogue warps), then per token of the
    // share its B_i and its rank (0: no adapter, -1: bad id)
};

constexpr int kLBatch = 4;                    // tokens an epilogue thread works on at a time
// Bytes of v that four epilogue warps hold at a time: at least a batch of tokens.
constexpr int v_bytes(int epi_warps) { return epi_warps == 4 ? 2048 : epi_warps == 8 ? 8192 : 4096; }
static_assert(v_bytes(4) / (LORA_MAX_RANK * 4) >= kLBatch, "a batch of tokens fits");

// Least shared memory of a CTA in a cluster, a column of tensor memory (64 at least).  Such a CTA holds its tensor
// memory until its peers have sent their sums, and they may still be waiting for theirs: if the CTAs that fit an SM
// could ask for more than its 512 columns, two clusters (of one launch, or of two streams) could each hold what the
// other waits for, for good.  An SM has 228 KB, of which a CTA takes 1 KB beside its own: what fits it then has at most
// 571 columns, in steps of 64, so 512.  The other clusters that take tensor memory take more (the long segments' shrink
// 97 KB for 64 columns; lora_sgmv_layer's pairs fill an SM), and what runs without a cluster ends by itself.
constexpr int kColumnSmem = 408;

struct StreamShape {
    int N, NT, S, E, ctas, stages, share, ncols, recv, alias, smem;
};

// Clusters that the device runs at once, with one CTA to an SM; a GPC's odd SMs hold none, so these are fewer
// than the SMs give (of 148 SMs: 74, 33 and 15).
struct ClusterFit {
    int of[4];   // of 1, 2, 4 and 8 CTAs
    int at_once(int S, int ctas) const
    {
        const int w = S / ctas;   // two CTAs to an SM: half the SMs
        return of[w == 8 ? 3 : w == 4 ? 2 : w == 2 ? 1 : 0];
    }
};

// Tokens per tile: all of them up to 256 (rounded up to the MMA's 16), else equal tiles of at most 256.  Tiles of
// at most 128, each of at least 96, where twice as many would still find an SM each: the epilogue's work per token
// is then the longer part (4096 columns, 256 tokens: 1024 rows 23.8 -> 20.1 us, 4608 rows 43.3 -> 30.3; but
// 14336 -> 4096, 136 tokens 52.4 -> 59.3, and 5120 rows, 192 tokens 35.2 -> 36.7, which the bounds leave out).
// Clusters: up to 8 CTAs split k, as many as run at once (4096 -> 2048, 64 tokens: 16 clusters of 8 take two
// rounds, 19.3 us, 16 of 4 one, 13.8), without adapters two to an SM (4096 -> 4096, one token:
// 8.3 us with 8, 9.3 with 4), with adapters no more than make four CTAs for five SMs (64 tokens: 17.5 us with 4,
// 18.9 with 8; 14336 outputs: 32.0 with 2, 36.4 with 1), since every CTA more waits for v and for its peers.
// CTAs per SM: two where half an SM's shared memory holds three stages and half of its tensor memory the
// accumulator with the adapter terms behind it, else one, as where there is no second CTA to put beside it.
// Epilogue warps: 16 where the SM has one CTA and more than 64 tokens, since their loads wait on memory most of
// the time (4096 -> 14336, 256 tokens: 98.9 us with 8, 72.2 with 16; 64 tokens, 14336 -> 4096: 34.6 and 37.3).
// One CTA alone of 4 epilogue warps leaves 16 KB so that a CTA of the shrink (256 threads of 118 registers) fits
// beside it (not beside the kernel for other ranks, of 254 registers a thread); with more warps registers do not
// allow it, and the ring takes all (4096 -> 14336, 256 tokens: 67.6 -> 66.5 us; 512
// tokens: 126.6 -> 124.7; 128 tokens: 41.9 -> 41.5).
StreamShape stream_shape(int T, int h, int o, int n_sms, const ClusterFit &fit, bool adapters)
{
    StreamShape sh;
    const int row_tiles = (o + kLM - 1) / kLM;
    const int halves = (T + kLMaxN / 2 - 1) / (kLMaxN / 2);
    const bool narrow = T >= halves * 96 && T > kLMaxN / 2 && (int64_t)row_tiles * halves * 2 <= n_sms;
    sh.NT = narrow ? halves : (T + kLMaxN - 1) / kLMaxN;
    const int per = (T + sh.NT - 1) / sh.NT;
    sh.N = (per + 15) & ~15;
    const int stage = kLWBytes + sh.N * 128;
    const int64_t tiles = (int64_t)row_tiles * sh.NT;
    const int nkb = (h + kLK - 1) / kLK;
    for (int ctas = 2;; --ctas) {
        sh.E = sh.N <= 32 ? 4 : ctas == 2 || sh.N <= 64 ? 8 : 16;
        sh.ctas = ctas;
        const int H = sh.E / 4;
        sh.S = 1;
        while (sh.S < 8 && tiles <= fit.at_once(2 * sh.S, ctas) && sh.S * 2 <= nkb &&
               !(adapters && tiles * sh.S * 5 >= 4ll * n_sms))
            sh.S *= 2;
        // S shares cover a whole tile (N, which is more than `per` when there are several)
        sh.share = ((std::min(sh.N, T) + sh.S - 1) / sh.S + kLBatch - 1) / kLBatch * kLBatch;
        const int hs = (sh.share / H + kLBatch - 1) / kLBatch * kLBatch;
        sh.ncols = 32;
        while (sh.ncols < sh.N + H * hs) sh.ncols *= 2;
        const int ctl = 1024 + (int)sizeof(LayerStreamCtl) + H * v_bytes(sh.E) + sh.share * 12;
        const int recv = (sh.S - 1) * sh.share * kLM * 4;
        const int room = (ctas == 1 ? (sh.E == 4 ? 210 : 226) : 227 / ctas - 1) * 1024 - ctl;
        // the peers' partial sums beside the ring where that leaves it three stages, else in it
        sh.alias = (room - recv) / stage < 3;
        sh.stages = std::min(kLMaxStages, (room - (sh.alias ? 0 : recv)) / stage);
        if (sh.alias && sh.stages * stage < recv) sh.stages = 0;
        if (ctas > 1 && (sh.stages < 3 || sh.ncols > 512 / ctas || tiles * sh.S <= n_sms)) continue;
        sh.stages = std::max(sh.alias ? (recv + stage - 1) / stage : 1, std::min(sh.stages, (nkb + sh.S - 1) / sh.S));
        sh.recv = sh.alias ? 0 : (sh.stages * stage + ctl - 1024 + 15) & ~15;
        sh.smem = sh.stages * stage + ctl + (sh.alias ? 0 : recv + 16);
        if (sh.S > 1) sh.smem = std::max(sh.smem, std::max(64, sh.ncols) * kColumnSmem);
        return sh;
    }
}

}  // namespace
}  // namespace lora
