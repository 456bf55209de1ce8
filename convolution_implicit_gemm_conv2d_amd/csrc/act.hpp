// Activations shared by the gated feed-forward layer and the block norms:
// value and derivative in fp32.
#pragma once

#include "common.hpp"

namespace convmi {

enum Act { kActNone = 0, kActSigmoid, kActSilu, kActGelu, kActGeluTanh, kActRelu, kActTanh, kActs };

struct ActPair {
    float v, d;  // act(t), act'(t)
};

// 1 / (1 + exp(-t)).  exp overflows to infinity for t below -88, where the
// quotient is 0 as it should be.
__device__ __forceinline__ float sigmoid_f(float t) { return 1.0f / (1.0f + expf(-t)); }

__device__ __forceinline__ float act_value(int kind, float t)
{
    switch (kind) {
    case kActSigmoid: return sigmoid_f(t);
    case kActSilu: return t * sigmoid_f(t);
    case kActGelu: return 0.5f * t * (1.0f + erff(t * 0.70710678118654752f));
    case kActGeluTanh: {
        const float k = 0.79788456080286536f;
        return 0.5f * t * (1.0f + tanhf(k * (t + 0.044715f * t * t * t)));
    }
    case kActRelu: return t <= 0.f ? 0.f : t;  // NaN stays NaN
    case kActTanh: return tanhf(t);
    default: return t;
    }
}

__device__ __forceinline__ ActPair act_pair(int kind, float t)
{
    switch (kind) {
    case kActSigmoid: {
        const float p = sigmoid_f(t);
        return {p, p * (1.0f - p)};
    }
    case kActSilu: {
        const float p = sigmoid_f(t);
        return {t * p, p * (1.0f + t * (1.0f - p))};
    }
    case kActGelu: {
        const float p = 0.5f * (1.0f + erff(t * 0.70710678118654752f));
        return {t * p, p + t * 0.39894228040143268f * expf(-0.5f * t * t)};
    }
    case kActGeluTanh: {
        const float k = 0.79788456080286536f, c = 0.044715f;
        const float h = tanhf(k * (t + c * t * t * t));
        return {0.5f * t * (1.0f + h), 0.5f * (1.0f + h) + 0.5f * t * (1.0f - h * h) * k * (1.0f + 3.0f * c * t * t)};
    }
    case kActRelu: return {t <= 0.f ? 0.f : t, t > 0.f ? 1.0f : 0.0f};
    case kActTanh: {
        const float h = tanhf(t);
        return {h, 1.0f - h * h};
    }
    default: return {t, 1.0f};
    }
}

}  // namespace convmi
