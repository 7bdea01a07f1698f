// Device side of a product's epilogue (internal.hpp, Epilogue).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.hpp"
#include "internal.hpp"
#include "tsl_block.h"

namespace tsl {

// The epilogues of a launch's items in its kernel arguments; nothing at all
// (an empty base) in the plain build.
template <int N> struct EpTable {
    Epilogue e[N];
    __device__ __forceinline__ const Epilogue &ep(int i) const { return e[i]; }
    void set_ep(int i, const Epilogue *p) {
        if (p)
            e[i] = *p;
    }
};
struct NoEpTable {
    __device__ __forceinline__ Epilogue ep(int) const { return Epilogue{}; }
    void set_ep(int, const Epilogue *) {}
};
template <int N> using Epilogues = std::conditional_t<kEpilogue, EpTable<N>, NoEpTable>;

__device__ __forceinline__ float ep_get(const void *p, bool bf, int64_t i) {
    return bf ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16)
              : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void ep_put(void *p, bool bf, int64_t i, float v) {
    if (bf) {
        __bf16 h = (__bf16)v;
        static_cast<uint16_t *>(p)[i] = __builtin_bit_cast(uint16_t, h);
    } else {
        static_cast<float *>(p)[i] = v;
    }
}

// The activations.  silu(v) = v s(v) and the tanh form of gelu,
// v (1 + tanh a) / 2 = v s(2 a) with a = sqrt(2/pi) (v + 0.044715 v^3), are
// both v times the logistic function s(t) = 1 / (1 + 2^(-t log2 e)) of an odd
// cubic t = v (c0 + c1 v^2): one exponential and one reciprocal (each within
// an ulp), no cancellation.  The error-function form, v (1 + erf(v / sqrt 2))
// / 2 = v erfc(-v / sqrt 2) / 2, keeps its relative accuracy for large
// negative v the same way.
__device__ __forceinline__ float logistic(float t) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * t));
}
constexpr float kGeluC0 = 1.59576912f;              // 2 sqrt(2/pi)
constexpr float kGeluC1 = 1.59576912f * 0.044715f;

__device__ __forceinline__ float act_value(float v, int act) {
    switch (act) {
    case TSL_ACT_RELU: return v < 0.f ? 0.f : v; // NaN stays NaN
    case TSL_ACT_SILU: return v * logistic(v);
    case TSL_ACT_GELU: return 0.5f * v * erfcf(-0.707106781f * v);
    case TSL_ACT_GELU_TANH: return v * logistic(v * __builtin_fmaf(kGeluC1 * v, v, kGeluC0));
    default: return v;
    }
}

// An activation and its slope.  With s = s(t): (v s)' = s + v s (1 - s) t'.
// The cubic's arguments are clamped where s is 0 or 1 to the last bit, so
// that t' stays finite.
__device__ __forceinline__ void act_both(float v, int act, float &a, float &d) {
    switch (act) {
    case TSL_ACT_RELU:
        a = v < 0.f ? 0.f : v;
        d = v > 0.f ? 1.f : 0.f;
        break;
    case TSL_ACT_SILU: {
        const float s = logistic(v);
        a = v * s;
        d = __builtin_fmaf(a, 1.f - s, s);
        break;
    }
    case TSL_ACT_GELU: {
        const float p = 0.5f * erfcf(-0.707106781f * v);
        a = v * p;
        d = __builtin_fmaf(v, 0.398942280f * __builtin_amdgcn_exp2f(-0.721347520f * v * v), p);
        break;
    }
    case TSL_ACT_GELU_TANH: {
        const float c = v > 64.f ? 64.f : (v < -64.f ? -64.f : v);
        const float s = logistic(c * __builtin_fmaf(kGeluC1 * c, c, kGeluC0));
        a = v * s;
        d = __builtin_fmaf(c * s * (1.f - s), __builtin_fmaf(3.f * kGeluC1 * c, c, kGeluC0), s);
        break;
    }
    default:
        a = v;
        d = 1.f;
    }
}

// v with its bias, kept in pre, through the activation, plus the residual.
__device__ __forceinline__ float ep_apply(const Epilogue &e, float v, int64_t m, int64_t n) {
    if (e.bias)
        v += ep_get(e.bias, e.flags & kEpBiasBf16, n);
    if (e.pre)
        ep_put(e.pre, e.flags & kEpPreBf16, m * e.ldp + n, v);
    v = act_value(v, e.act);
    if (e.res)
        v += ep_get(e.res, e.flags & kEpResBf16, m * e.ldr + n);
    return v;
}

// The gate: act(g) * u.
__device__ __forceinline__ float ep_gate(const Epilogue &e, float g, float u, int64_t m, int64_t n) {
    if (e.pre)
        ep_put(e.pre, e.flags & kEpPreBf16, m * e.ldp + n, g);
    if (e.pre2)
        ep_put(e.pre2, e.flags & kEpPreBf16, m * e.ldp + n, u);
    return act_value(g, e.act) * u;
}

} // namespace tsl
