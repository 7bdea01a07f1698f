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
    // by value: a reference would make the compiler copy the whole kernel
    // argument to private memory
    __device__ __forceinline__ Epilogue ep(int i) const { return e[i]; }
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

// The activations as function objects: with_act picks one before a store
// loop, so that the loop holds only its own code.
struct ActLine { // none, relu: not below lo
    float lo;
    __device__ __forceinline__ float operator()(float v) const { return v < lo ? lo : v; }
};
struct ActSilu {
    __device__ __forceinline__ float operator()(float v) const { return act_value(v, TSL_ACT_SILU); }
};
struct ActGelu {
    __device__ __forceinline__ float operator()(float v) const { return act_value(v, TSL_ACT_GELU); }
};
struct ActGeluTanh {
    __device__ __forceinline__ float operator()(float v) const {
        return act_value(v, TSL_ACT_GELU_TANH);
    }
};
template <class F> __device__ __forceinline__ void with_act(int act, F f) {
    if (act == TSL_ACT_SILU)
        f(ActSilu{});
    else if (act == TSL_ACT_GELU)
        f(ActGelu{});
    else if (act == TSL_ACT_GELU_TANH)
        f(ActGeluTanh{});
    else
        f(ActLine{act == TSL_ACT_RELU ? 0.f : -__builtin_inff()});
}

// The epilogue of a 32x32-tile GEMM wave: MT x NT accumulator tiles, register
// r of lane l holding row row0 + 32 i + 8 (r / 4) + r % 4 (row0 includes
// 4 (l / 32)), column col0 + 32 j (col0 includes l % 32) of a matrix of M x
// Ns.  value(i, j, r) is the product's binary32 result.  One base address per
// lane and operand; every access is that base plus a compile-time row step
// times the (uniform) row stride.  The residuals of a tile row are all loaded
// before its first store, which the compiler could not move them across (Y
// may be the residual).  DUAL: tiles 2 p and 2 p + 1 hold a gate's column and
// its up column, both col0 + 32 p.
template <int MT, int NT, bool DUAL, class V>
__device__ __forceinline__ void ep_store(const Epilogue e, void *Y, bool ybf, int64_t ldy,
                                         int64_t row0, int64_t col0, int64_t M, int64_t Ns, V value) {
    constexpr int NP = DUAL ? NT / 2 : NT;
    const bool rbf = e.flags & kEpResBf16, pbf = e.flags & kEpPreBf16;
    const int ysz = ybf ? 2 : 4, rsz = rbf ? 2 : 4, psz = pbf ? 2 : 4;
    const int64_t ystep = ldy * ysz, rstep = e.ldr * rsz, pstep = e.ldp * psz;
    char *const yb = static_cast<char *>(Y) + (row0 * ldy + col0) * ysz;
    const char *const rb = static_cast<const char *>(e.res) + (row0 * e.ldr + col0) * rsz;
    char *const pb = static_cast<char *>(e.pre) + (row0 * e.ldp + col0) * psz;
    char *const pb2 = static_cast<char *>(e.pre2) + (row0 * e.ldp + col0) * psz;
    const int64_t rows = M - row0; // of this lane
    bool ok[NP];
    float bias[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        ok[j] = col0 + 32 * j < Ns;
        bias[j] = !DUAL && e.bias && ok[j] ? ep_get(e.bias, e.flags & kEpBiasBf16, col0 + 32 * j) : 0.f;
    }
    with_act(e.act, [&](auto A) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float res[16][NP];
            if (!DUAL && e.res) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int rr = 32 * i + 8 * (r >> 2) + (r & 3);
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        res[r][j] = rr < rows && ok[j] ? ep_get(rb + rr * rstep, rbf, 32 * j) : 0.f;
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int rr = 32 * i + 8 * (r >> 2) + (r & 3);
                float v[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    v[j] = value(i, j, r);
                if (rr >= rows)
                    continue;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    if (!ok[j])
                        continue;
                    float y;
                    if constexpr (DUAL) {
                        if (e.pre) {
                            ep_put(pb + rr * pstep, pbf, 32 * j, v[2 * j]);
                            ep_put(pb2 + rr * pstep, pbf, 32 * j, v[2 * j + 1]);
                        }
                        y = A(v[2 * j]) * v[2 * j + 1];
                    } else {
                        y = v[j] + bias[j];
                        if (e.pre)
                            ep_put(pb + rr * pstep, pbf, 32 * j, y);
                        y = A(y);
                        if (e.res)
                            y += res[r][j];
                    }
                    ep_put(yb + rr * ystep, ybf, 32 * j, y);
                }
            }
        }
    });
}

// Binary32 partials of a dual product's k-split: the first weight's at p0,
// the second's at p1, each [M][Ns] (rows and columns as in ep_store).
template <int MT, int NT, class V>
__device__ __forceinline__ void dual_partials(float *p0, float *p1, int64_t row0, int64_t col0,
                                              int64_t M, int64_t Ns, V value) {
    p0 += row0 * Ns + col0;
    p1 += row0 * Ns + col0;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int rr = 32 * i + 8 * (r >> 2) + (r & 3);
            float v[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                v[j] = value(i, j, r);
            if (row0 + rr >= M)
                continue;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (col0 + 32 * (j >> 1) < Ns)
                    (j & 1 ? p1 : p0)[rr * Ns + 32 * (j >> 1)] = v[j];
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
__device__ __forceinline__ float ep_apply(const Epilogue e, float v, int64_t m, int64_t n) {
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
__device__ __forceinline__ float ep_gate(const Epilogue e, float g, float u, int64_t m, int64_t n) {
    if (e.pre)
        ep_put(e.pre, e.flags & kEpPreBf16, m * e.ldp + n, g);
    if (e.pre2)
        ep_put(e.pre2, e.flags & kEpPreBf16, m * e.ldp + n, u);
    return act_value(g, e.act) * u;
}

} // namespace tsl
