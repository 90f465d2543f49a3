// What follows a layer's product (lora_epilogue), shared by the layer kernels: the activations and
// the operand pointers as the kernels take them.
#pragma once

#include "lora_common.cuh"

namespace lora {
namespace {

struct EpiParams {
    const uint16_t *bias, *mul, *res;   // bf16, or null
    int64_t ldmul, ldres;
    int32_t act;
};

EpiParams epi_params(const lora_epilogue *e)
{
    EpiParams p;
    p.bias = static_cast<const uint16_t *>(e->bias);
    p.mul = static_cast<const uint16_t *>(e->mul);
    p.res = static_cast<const uint16_t *>(e->residual);
    p.ldmul = e->ldmul;
    p.ldres = e->ldres;
    p.act = e->act;
    return p;
}

__device__ __forceinline__ float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// The results are rounded to bf16 (2^-8 of the value), so the fast exponential and division are exact enough: 2 +
// 1.17 |u| and 2 steps of 2^-23 by their documentation, about 2^-18 at |u| = 20 and 2^-16 at the far end, which is
// |u| = 87.3 (from where 1 + exp(-u) passes 2^126 the quotient is 0, and the result, below |z| 2^-126, with it).
// The tanh form is the same function as z times the logistic function of 2u, which keeps its relative accuracy where
// 1 + tanh(u) cancels; the normal distribution function likewise keeps it in the lower tail.
__device__ __forceinline__ float logistic(float u) { return __fdividef(1.f, 1.f + __expf(-u)); }

template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act)
{
    switch (act) {
    case LORA_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];   // keeps NaN
        break;
    case LORA_ACT_GELU:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= normcdff(z[i]);
        break;
    case LORA_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= logistic(1.5957691216057308f * fmaf(0.044715f * z[i] * z[i], z[i], z[i]));
        break;
    case LORA_ACT_SILU:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= logistic(z[i]);
        break;
    default: break;
    }
}

}  // namespace
}  // namespace lora
