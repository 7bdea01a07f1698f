// Root-mean-square norm of the residual stream after a row-parallel product
// (mlxcel manual "Tensor parallelism", "Row Parallel": the rank partials of
// o_proj / down_proj are summed; the norm before the next column-parallel
// products reads that sum), and its backward pass:
//     r = residual + ((P_0 + P_1) + ...)
//     y_j = r_j rstd w_j,  rstd = (mean_j r_j^2 + eps)^(-1/2)
// and, with t = dy w and xh = x rstd,
//     dx = rstd (t - xh mean(t xh)) + dres,   dw_j = sum_m dy_mj xh_mj.
// Both are bound by the bytes of one pass: a row stays in the registers of
// the TPR threads that own it (NV runs of 8 columns each) from its only read
// to its only write, so every input is read once and every output written
// once.  A row's threads are one wave up to 512 columns (four rows share a
// workgroup), a workgroup of four waves up to 8192 and of sixteen up to
// 32768.  All sums are binary32.
#include "device.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace tsl {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v += __shfl_xor(v, o, 64);
    return v;
}

// Sum over the TPR threads of a row: the same value in each of them, added
// in a fixed order.  `red` holds one slot per wave; a barrier frees it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < NW; ++w)
            v += red[w];
    }
    return v;
}

// The larger magnitude, a NaN before every number: magnitudes order as
// their bit patterns.
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float *red) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v = umax(v, (uint32_t)__shfl_xor((int)v, o, 64));
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = __uint_as_float(v);
        __syncthreads();
        v = __float_as_uint(red[0]);
#pragma unroll
        for (int w = 1; w < NW; ++w)
            v = umax(v, __float_as_uint(red[w]));
    }
    return v;
}

constexpr float kE4M3Max = 448.f;

// 8 values times 1 / scale as e4m3 (nearest, ties to even; gfx950 converts
// a pair per instruction).  Every |v| is at most the scale times 448 up to
// rounding, and clamped to it; a scale of zero has only zeros.
__device__ __forceinline__ u32x2 quant8(f32x8 v, float scale) {
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    u32x2 w = {0, 0};
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // a scale below 2^-128 has an infinite reciprocal: divide instead
        float x = __builtin_isinf(inv) ? v[i] / scale : v[i] * inv;
        if (scale != scale || __builtin_isinf(scale))
            x = __builtin_nanf("");
        q[i] = x > kE4M3Max ? kE4M3Max : (x < -kE4M3Max ? -kE4M3Max : x);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int p = 0;
        p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], p, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], p, true);
        w[h] = (uint32_t)p;
    }
    return w;
}

// ---- forward ----------------------------------------------------------------
template <int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_kernel(NormArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1; // rows per workgroup
    __shared__ float red[TPR / 64];
    const int t = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (m >= a.M)
        return; // whole waves only (RPB > 1), before any barrier of wider rows
    const int64_t n = a.n;
    f32x8 r[NV];
    const int64_t prow = m * a.ld_part * (a.p_bf16 ? 2 : 4);
#pragma unroll
    for (int v = 0; v < NV; ++v)
        r[v] = load8<VEC>(static_cast<const char *>(a.parts[0]) + prow, a.p_bf16,
                          ((int64_t)v * TPR + t) * 8, n);
    for (int q = 1; q < a.n_parts; ++q) {
        const char *p = static_cast<const char *>(a.parts[q]) + prow;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const f32x8 w = load8<VEC>(p, a.p_bf16, ((int64_t)v * TPR + t) * 8, n);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[v][i] += w[i];
        }
    }
    if (a.residual) {
        const char *p = static_cast<const char *>(a.residual) + m * a.ldr * (a.r_bf16 ? 2 : 4);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const f32x8 w = load8<VEC>(p, a.r_bf16, ((int64_t)v * TPR + t) * 8, n);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[v][i] += w[i];
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = __builtin_fmaf(r[v][i], r[v][i], ss);
    if (a.sum_out) {
        char *p = static_cast<char *>(a.sum_out) + m * a.ld_sum * (a.r_bf16 ? 2 : 4);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store8<VEC>(p, a.r_bf16, ((int64_t)v * TPR + t) * 8, n, r[v]);
    }
    ss = row_sum<TPR>(ss, red);
    const float rstd = 1.f / __builtin_sqrtf(ss / (float)n + a.eps);
    if (a.rstd && t == 0)
        a.rstd[m] = rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[v][i] *= rstd;
        if (a.weight) {
            const f32x8 w = load8<VEC>(a.weight, a.w_bf16, ((int64_t)v * TPR + t) * 8, n);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[v][i] *= w[i];
        }
    }
    if (a.y_type != TSL_E4M3) {
        char *y = static_cast<char *>(a.Y) + m * a.ldy * (a.y_type == TSL_BF16 ? 2 : 4);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store8<VEC>(y, a.y_type == TSL_BF16, ((int64_t)v * TPR + t) * 8, n, r[v]);
        return;
    }
    // e4m3: the largest magnitude of each group of columns (the threads of a
    // group are neighbours: 8 columns each) or of the row
    uint32_t mx[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        mx[v] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mx[v] = umax(mx[v], __float_as_uint(r[v][i]) & 0x7FFFFFFFu);
    }
    if (a.group == 0) {
        uint32_t all = mx[0];
#pragma unroll
        for (int v = 1; v < NV; ++v)
            all = umax(all, mx[v]);
        all = row_max<TPR>(all, red);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            mx[v] = all;
    } else {
        for (int o = 1; o < a.group / 8; o <<= 1)
#pragma unroll
            for (int v = 0; v < NV; ++v)
                mx[v] = umax(mx[v], (uint32_t)__shfl_xor((int)mx[v], o, 64));
    }
    uint8_t *y = static_cast<uint8_t *>(a.Y) + m * a.ldy;
    const int64_t groups = a.group ? (n + a.group - 1) / a.group : 1;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t col = ((int64_t)v * TPR + t) * 8;
        if (col >= n)
            continue;
        const float scale = __uint_as_float(mx[v]) / kE4M3Max;
        if (a.group ? col % a.group == 0 : col == 0)
            a.scales[m * groups + (a.group ? col / a.group : 0)] = scale;
        const u32x2 w = quant8(r[v], scale);
        if (VEC && col + 8 <= n) {
            *reinterpret_cast<u32x2 *>(y + col) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < n)
                    y[col + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
        }
    }
}

// ---- backward ----------------------------------------------------------------
// Row groups walk the rows with the grid's stride; each thread keeps the
// weight gradient of its own columns over its rows and leaves it in the
// workspace, [row groups][n rounded up to 8], which column_sum_kernel adds in
// order.
template <int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_grad_kernel(NormGradArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    __shared__ float red[TPR / 64];
    const int t = threadIdx.x % TPR;
    const int64_t g = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; // row group
    if (g >= a.row_groups)
        return; // whole waves only (RPB > 1), before any barrier of wider rows
    const int64_t n = a.n;
    f32x8 w[NV], dw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        w[v] = f32x8{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        if (a.weight)
            w[v] = load8<VEC>(a.weight, a.w_bf16, ((int64_t)v * TPR + t) * 8, n);
        dw[v] = f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    }
    for (int64_t m = g; m < a.M; m += a.row_groups) {
        const char *xp = static_cast<const char *>(a.X) + m * a.ldx * (a.x_bf16 ? 2 : 4);
        const char *yp = static_cast<const char *>(a.dY) + m * a.lddy * (a.dy_bf16 ? 2 : 4);
        f32x8 x[NV], dy[NV], dr[NV];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            x[v] = load8<VEC>(xp, a.x_bf16, ((int64_t)v * TPR + t) * 8, n);
            dy[v] = load8<VEC>(yp, a.dy_bf16, ((int64_t)v * TPR + t) * 8, n);
        }
        if (a.dres) {
            const char *rp = static_cast<const char *>(a.dres) + m * a.ld_dres * (a.dx_bf16 ? 2 : 4);
#pragma unroll
            for (int v = 0; v < NV; ++v)
                dr[v] = load8<VEC>(rp, a.dx_bf16, ((int64_t)v * TPR + t) * 8, n);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1 = __builtin_fmaf(x[v][i], x[v][i], s1);
                s2 = __builtin_fmaf(dy[v][i] * w[v][i], x[v][i], s2);
            }
        float rstd;
        if (a.rstd) {
            rstd = a.rstd[m];
        } else {
            s1 = row_sum<TPR>(s1, red);
            rstd = 1.f / __builtin_sqrtf(s1 / (float)n + a.eps);
        }
        s2 = row_sum<TPR>(s2, red);
        const float c = s2 * rstd / (float)n; // mean of t xh
        char *op = a.dX ? static_cast<char *>(a.dX) + m * a.lddx * (a.dx_bf16 ? 2 : 4) : nullptr;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            f32x8 o;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = x[v][i] * rstd;
                o[i] = rstd * (dy[v][i] * w[v][i] - xh * c);
                dw[v][i] = __builtin_fmaf(dy[v][i], xh, dw[v][i]);
                if (a.dres)
                    o[i] += dr[v][i];
            }
            if (op)
                store8<VEC>(op, a.dx_bf16, ((int64_t)v * TPR + t) * 8, n, o);
        }
    }
    if (!a.part)
        return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        store8<true>(a.part + g * ((n + 7) / 8 * 8), false, ((int64_t)v * TPR + t) * 8, n, dw[v]);
}

// dW[j] (+)= sum over the row groups' partials, 16 columns per workgroup:
// 16 threads per column take every 16th partial, then add up in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float *__restrict__ part, int64_t groups,
                                                      int64_t n, float *__restrict__ dW,
                                                      int accumulate) {
    __shared__ float red[16][17];
    const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
    const int64_t j = (int64_t)blockIdx.x * 16 + c;
    const int64_t ld = (n + 7) / 8 * 8;
    float s = 0.f;
    if (j < n)
        for (int64_t g = q; g < groups; g += 16)
            s += part[g * ld + j];
    red[q][c] = s;
    __syncthreads();
    if (q != 0 || j >= n)
        return;
#pragma unroll
    for (int i = 1; i < 16; ++i)
        s += red[i][c];
    dW[j] = accumulate ? dW[j] + s : s;
}

// (threads per row, runs of 8 per thread) for a width
#define TSL_NORM_SHAPES(X)                                                                         \
    X(64, 1, 512) X(256, 1, 2048) X(256, 2, 4096) X(256, 4, 8192) X(1024, 2, 16384) X(1024, 4, 32768)

inline int rows_per_group(int64_t n) { return n <= 512 ? 4 : 1; }

} // namespace

hipError_t launch_norm(const NormArgs &a, bool vec, hipStream_t stream) {
    const int64_t rpb = rows_per_group(a.n);
    const dim3 grid((unsigned)((a.M + rpb - 1) / rpb));
#define TSL_CASE(TPR_, NV_, MAX_)                                                                  \
    if (a.n <= MAX_) {                                                                             \
        const dim3 block(TPR_ < 256 ? 256 : TPR_);                                                 \
        if (vec)                                                                                   \
            hipLaunchKernelGGL((norm_kernel<TPR_, NV_, true>), grid, block, 0, stream, a);         \
        else                                                                                       \
            hipLaunchKernelGGL((norm_kernel<TPR_, NV_, false>), grid, block, 0, stream, a);        \
        return hipGetLastError();                                                                  \
    }
    TSL_NORM_SHAPES(TSL_CASE)
#undef TSL_CASE
    return hipErrorInvalidValue;
}

// Row groups of a backward launch: enough workgroups to fill the chip, few
// enough that their weight-gradient partials stay small beside the rows.
int64_t norm_grad_groups(int64_t M, int64_t n) {
    const int64_t most = (n <= 4096 ? 1024 : 512) * rows_per_group(n);
    return M < most ? M : most;
}

hipError_t launch_column_sum(const float *part, int64_t groups, int64_t n, float *out,
                             int accumulate, hipStream_t stream) {
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, stream, part,
                       groups, n, out, accumulate);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs &a, bool vec, float *dW, int accumulate,
                            hipStream_t stream) {
    if (a.M > 0) {
        const int64_t rpb = rows_per_group(a.n);
        const dim3 grid((unsigned)((a.row_groups + rpb - 1) / rpb));
        hipError_t e = hipErrorInvalidValue;
#define TSL_CASE(TPR_, NV_, MAX_)                                                                  \
    if (e == hipErrorInvalidValue && a.n <= MAX_) {                                                \
        const dim3 block(TPR_ < 256 ? 256 : TPR_);                                                 \
        if (vec)                                                                                   \
            hipLaunchKernelGGL((norm_grad_kernel<TPR_, NV_, true>), grid, block, 0, stream, a);    \
        else                                                                                       \
            hipLaunchKernelGGL((norm_grad_kernel<TPR_, NV_, false>), grid, block, 0, stream, a);   \
        e = hipGetLastError();                                                                     \
        if (e != hipSuccess)                                                                       \
            return e;                                                                              \
    }
        TSL_NORM_SHAPES(TSL_CASE)
#undef TSL_CASE
        if (e != hipSuccess)
            return e;
    }
    return dW ? launch_column_sum(a.part, a.M > 0 ? a.row_groups : 0, a.n, dW, accumulate, stream)
              : hipSuccess;
}

} // namespace tsl
