// Activations shared by the gated feed-forward layer and the block norms:
// value and derivative in fp32.
#pragma once

#include "common.hpp"

#include <type_traits>

namespace convmi {

enum Act { kActNone = 0, kActSigmoid, kActSilu, kActGelu, kActGeluTanh, kActRelu, kActTanh, kActs };

struct ActPair {
    float v, d;  // act(t), act'(t)
};

// The hardware's base-2 exponential and reciprocal (one unit in the last place
// each) instead of the library's: an epilogue holds tens of activations a lane,
// and the library's forms (range reduction, exact division, both branches of
// erf) cost three to eight times the instructions.  exp(t) as 2^(t log2 e)
// carries an error of about |t| 2^-24 relative, no more than t's own last place
// moves it.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_hw(float t) { return __builtin_amdgcn_exp2f(t); }
__device__ __forceinline__ float rcp_hw(float t) { return __builtin_amdgcn_rcpf(t); }

// 1 / (1 + exp(-t)).  The exponential overflows to infinity for t below -88,
// where the quotient is 0 as it should be.
__device__ __forceinline__ float sigmoid_f(float t) { return rcp_hw(1.0f + exp2_hw(-kLog2e * t)); }

// tanh(t): 1 - 2 / (exp(2t) + 1), and where that cancels an odd polynomial
// (fitted for the relative error: 9e-8 below 0.6).
__device__ __forceinline__ float tanh_f(float t)
{
    const float z = t * t;
    const float near = t + t * z * (-0.33332597f + z * (0.13313115f + z * (-0.052211695f + z * 0.015612447f)));
    const float far = 1.0f - 2.0f * rcp_hw(exp2_hw((2.0f * kLog2e) * t) + 1.0f);
    return fabsf(t) < 0.6f ? near : far;
}

// The normal distribution function.  The tail
// Phi(-|t|) is exp(-t^2 / 2) times a polynomial in s = 1 / (1 + P|t|) without
// a constant term, fitted for its relative error (1.3e-7 up to 13.5, past which
// the tail is below the smallest fp32 value), so small values of t Phi(t) are
// good too; the larger side is one minus it.
struct Normal {
    float p, m, e;  // Phi(t), |t| Phi(-|t|), exp(-t^2 / 2)
};
__device__ __forceinline__ Normal normal_f(float t)
{
    const float e = exp2_hw((-0.5f * kLog2e) * t * t);
    const float m = __builtin_fminf(fabsf(t), 64.0f);  // the tail is 0 long before
    const float s = rcp_hw(__builtin_fmaf(0.3f, m, 1.0f));
    float q = 0.035931705f;
    q = __builtin_fmaf(q, s, -0.158275877f);
    q = __builtin_fmaf(q, s, 0.208206396f);
    q = __builtin_fmaf(q, s, -0.055393656f);
    q = __builtin_fmaf(q, s, 0.129469100f);
    q = __builtin_fmaf(q, s, 0.099637523f);
    q = __builtin_fmaf(q, s, 0.120798354f);
    q = __builtin_fmaf(q, s, 0.119626390f);
    const float tail = q * s * e;
    return {t < 0.f ? tail : 1.0f - tail, tail * m, e};
}

// x / 2 (1 + tanh(w)) is x times the logistic function of 2 w.
constexpr float kTanhScale = 0.79788456080286536f, kTanhCube = 0.044715f;
__device__ __forceinline__ float gelu_tanh_p(float t) { return sigmoid_f(2.0f * kTanhScale * (t + kTanhCube * t * t * t)); }

template <int K>
__device__ __forceinline__ float act_value(float t)
{
    if constexpr (K == kActSigmoid) return sigmoid_f(t);
    else if constexpr (K == kActSilu) return t * sigmoid_f(t);
    else if constexpr (K == kActGelu) return __builtin_fmaxf(t, 0.f) - normal_f(t).m;  // t Phi(t) on either side
    else if constexpr (K == kActGeluTanh) return t * gelu_tanh_p(t);
    else if constexpr (K == kActRelu) return t <= 0.f ? 0.f : t;  // NaN stays NaN
    else if constexpr (K == kActTanh) return tanh_f(t);
    else return t;
}

template <int K>
__device__ __forceinline__ ActPair act_pair(float t)
{
    if constexpr (K == kActSigmoid) {
        const float p = sigmoid_f(t);
        return {p, p * (1.0f - p)};
    } else if constexpr (K == kActSilu) {
        const float p = sigmoid_f(t);
        return {t * p, p * (1.0f + t * (1.0f - p))};
    } else if constexpr (K == kActGelu) {
        const Normal n = normal_f(t);
        return {__builtin_fmaxf(t, 0.f) - n.m, n.p + t * 0.39894228040143268f * n.e};
    } else if constexpr (K == kActGeluTanh) {
        // p (1 - p) is 0 from |t| = 11 on; there the square's overflow must not meet it.
        const float p = gelu_tanh_p(t), z = __builtin_fminf(t * t, 1e4f);
        return {t * p, p + t * p * (1.0f - p) * (2.0f * kTanhScale) * (1.0f + 3.0f * kTanhCube * z)};
    } else if constexpr (K == kActRelu) {
        return {t <= 0.f ? 0.f : t, t > 0.f ? 1.0f : 0.0f};
    } else if constexpr (K == kActTanh) {
        const float h = tanh_f(t);
        return {h, 1.0f - h * h};
    } else {
        return {t, 1.0f};
    }
}

// Calls f with the activation as a compile-time constant.  One choice for many
// elements: the code of one activation then runs straight through, where a
// choice for each element jumps through all of them and its code outgrows the
// instruction cache (a 256 x 128 gated tile with that took 36 us).
template <typename F>
__device__ __forceinline__ void with_act(int kind, F f)
{
    switch (kind) {
    case kActSigmoid: f(std::integral_constant<int, kActSigmoid>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActTanh: f(std::integral_constant<int, kActTanh>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
    }
}
__device__ __forceinline__ float act_value(int kind, float t)
{
    float v = 0.f;
    with_act(kind, [&](auto k) __attribute__((always_inline)) { v = act_value<k()>(t); });
    return v;
}
__device__ __forceinline__ ActPair act_pair(int kind, float t)
{
    ActPair p{};
    with_act(kind, [&](auto k) __attribute__((always_inline)) { p = act_pair<k()>(t); });
    return p;
}

}  // namespace convmi
