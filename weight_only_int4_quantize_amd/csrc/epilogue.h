// The linear layer's epilogue, y = act(v + bias) * mul + residual on the fp32
// sum v of an output element, rounded once to fp16 (awq_gemm_fused). Every
// linear kernel has a second instance that applies it where it stores; the
// plain instances are unchanged.
//
// The operands are loaded as raw bits ahead of their use, by the thread that
// stores the element (so residual or mul may be y itself). A sigmoid is
// 1 / (1 + 2^(-x log2 e)) with the hardware's exponential and reciprocal,
// within 2^-19 relative for |x| < 16, against the output's 2^-11.
#pragma once

#include "awq_internal.h"

namespace awq {

struct NoEpilogue {};

// the operands of one output element, as stored (0 where there is none)
struct EpilogueBits {
    uint16_t bias, mul, residual;
};

__device__ inline float epilogue_sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}
__device__ inline float epilogue_act(float v, int act) {
    switch (act) {
        case AWQ_ACT_RELU: return fmaxf(v, 0.f);
        case AWQ_ACT_SILU: return v * epilogue_sigmoid(v);
        // 0.5 (1 + erf(v / sqrt 2)) by the complement: exact to the last bits
        // where the sum would cancel
        case AWQ_ACT_GELU: return 0.5f * v * erfcf(-0.70710678f * v);
        // 0.5 (1 + tanh u) = sigmoid(2 u)
        case AWQ_ACT_GELU_TANH: return v * epilogue_sigmoid(1.59576912f * (v + 0.044715f * v * v * v));
        default: return v;
    }
}
__device__ inline float epilogue_f(uint16_t b) { return static_cast<float>(__builtin_bit_cast(half_t, b)); }
__device__ inline half_t epilogue_apply(const Epilogue& e, float v, const EpilogueBits& b) {
    v = epilogue_act(v + epilogue_f(b.bias), e.act);
    if (e.mul != nullptr) v *= epilogue_f(b.mul);
    return static_cast<half_t>(v + epilogue_f(b.residual));
}

// The operands of element (m, n), n < N: plain loads under uniform branches.
__device__ inline EpilogueBits epilogue_load(const Epilogue& e, int64_t m, int64_t n) {
    EpilogueBits b{0, 0, 0};
    if (e.bias != nullptr) b.bias = __builtin_bit_cast(uint16_t, e.bias[n]);
    if (e.mul != nullptr) b.mul = __builtin_bit_cast(uint16_t, e.mul[m * e.mul_stride + n]);
    if (e.residual != nullptr) b.residual = __builtin_bit_cast(uint16_t, e.residual[m * e.residual_stride + n]);
    return b;
}

}  // namespace awq
