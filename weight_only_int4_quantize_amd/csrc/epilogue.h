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
// (a register each: two halves in one would make loads wait for each other)
struct EpilogueBits {
    uint32_t bias, mul, residual;
};

__device__ inline float epilogue_sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}
// Phi(v) = 0.5 (1 + erf(v / sqrt 2)), by its tail H(a) = 0.5 erfc(a / sqrt 2),
// a = |v|: H(a) e^(a^2 / 2) is smooth in t = 1 / (1 + 0.36 a), and the
// coefficients are a weighted least-squares fit of it for a up to 14 (relative
// error 9e-7; with the fp32 steps below 2^-18 for v > -6). The library's erfc
// is several times the code, of which the kernels hold many copies.
__device__ inline float epilogue_phi(float v) {
    const float a = fabsf(v);
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.36f * a);
    float p = 0.04706965759396553f;
    p = p * t - 0.1798105090856552f;
    p = p * t + 0.18101643025875092f;
    p = p * t + 0.026506338268518448f;
    p = p * t + 0.13973495364189148f;
    p = p * t + 0.14176958799362183f;
    p = p * t + 0.14371325075626373f;
    const float h = p * t * __builtin_amdgcn_exp2f(-0.72134752f * a * a);
    return v < 0.f ? h : 1.0f - h;
}
// v[0 .. N) in place; the choice of the activation is outside the elements
template <int N>
__device__ inline void epilogue_act(float (&v)[N], int act) {
    switch (act) {
        case AWQ_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];    // a NaN stays
            break;
        case AWQ_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= epilogue_sigmoid(v[i]);
            break;
        case AWQ_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= epilogue_phi(v[i]);
            break;
        // 0.5 (1 + tanh u) = sigmoid(2 u)
        case AWQ_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] *= epilogue_sigmoid(1.59576912f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
            break;
        default: break;
    }
}
__device__ inline float epilogue_f(uint32_t b) {
    return static_cast<float>(__builtin_bit_cast(half_t, static_cast<uint16_t>(b)));
}
__device__ inline uint32_t epilogue_bits(const half_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
// v[0 .. N) to the outputs, in place
template <int N>
__device__ inline void epilogue_apply(const Epilogue& e, float (&v)[N], const EpilogueBits (&b)[N], half_t (&y)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += epilogue_f(b[i].bias);
    epilogue_act(v, e.act);
    if (e.mul != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= epilogue_f(b[i].mul);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = static_cast<half_t>(v[i] + epilogue_f(b[i].residual));
}
__device__ inline half_t epilogue_apply(const Epilogue& e, float v, const EpilogueBits& b) {
    float vv[1] = {v};
    const EpilogueBits bb[1] = {b};
    half_t y[1];
    epilogue_apply(e, vv, bb, y);
    return y[0];
}

// The operands of element (m, n), n < N: plain loads under uniform branches.
__device__ inline EpilogueBits epilogue_load(const Epilogue& e, int64_t m, int64_t n) {
    EpilogueBits b{0, 0, 0};
    if (e.bias != nullptr) b.bias = epilogue_bits(e.bias + n);
    if (e.mul != nullptr) b.mul = epilogue_bits(e.mul + m * e.mul_stride + n);
    if (e.residual != nullptr) b.residual = epilogue_bits(e.residual + m * e.residual_stride + n);
    return b;
}

// The same for eight neighbouring elements of a row, (m, n) .. (m, n + 7),
// by 16-byte accesses: only where e.vectors (N and the strides whole eights,
// every address a multiple of 16).
struct EpilogueRun {
    half8_t mul, residual;
};
__device__ inline EpilogueRun epilogue_load8(const Epilogue& e, int64_t m, int64_t n, int M, int N) {
    EpilogueRun r{};
    if (m >= M || n >= N) return r;
    if (e.mul != nullptr) r.mul = *reinterpret_cast<const half8_t*>(e.mul + m * e.mul_stride + n);
    if (e.residual != nullptr)
        r.residual = *reinterpret_cast<const half8_t*>(e.residual + m * e.residual_stride + n);
    return r;
}
__device__ inline void epilogue_store8(const Epilogue& e, float (&v)[8], const half8_t& bias, const EpilogueRun& r,
                                       half_t* y, int64_t m, int64_t n, int M, int N) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += static_cast<float>(bias[j]);
    epilogue_act(v, e.act);
    if (e.mul != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= static_cast<float>(r.mul[j]);
    }
    half8_t h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = static_cast<half_t>(v[j] + static_cast<float>(r.residual[j]));
    if (m < M && n < N) *reinterpret_cast<half8_t*>(y + m * N + n) = h;
}

}  // namespace awq
