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
// workgroup), a workgroup of four waves up to 8192 (backward, three operands
// a row: up to 4096, eight waves up to 8192) and of sixteen up to 32768 -- where
// the backward pass does not fit: see norm_grad_kernel.  All sums are binary32.
// Measured, forward, four partials and a residual to e4m3, 2048 x 5120: 52 us,
// 221 MB, 4.2 TB/s, where a copy reaches 4.9; 2048 x 16384, one bf16 part, 59 us,
// 4.0 TB/s.
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

// 8 values over their scale as e4m3 (nearest, ties to even; gfx950 converts a
// pair per instruction).  The quotient is a division: a product with the rounded
// reciprocal falls on the other side of a tie now and then (2 codes of 13
// million), and the pass is bound by memory either way (2048 x 5120, four
// partials: 51.2 us with the reciprocal, 51.7 divided; one bf16 part 23.0 and
// 23.6).  Every |v| is at most the scale times 448 up to the scale's rounding,
// and clamped to it.  A scale of zero (the largest |v| over 448 rounds to zero)
// has only zeros.
__device__ __forceinline__ u32x2 quant8(f32x8 v, float scale) {
    const float d = scale == 0.f ? 1.f : scale; // |v| < 2^-140 there: codes of zero
    const bool bad = !__builtin_isfinite(scale);
    u32x2 w = {0, 0};
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = bad ? __builtin_nanf("") : v[i] / d;
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
// Row groups (a wave up to 512 columns, else a workgroup) walk the rows with
// the grid's stride; each thread keeps the weight gradient of its own columns
// over its rows.  A workgroup leaves one partial row in the workspace (of its
// four waves' sums, added in order, where a row is a wave), which
// column_sum_kernel adds in order.  Aligned bf16 rows (RAW) are loaded one
// row ahead, as they lie: a row's loads are in flight over the reduction of
// the row before (8192 x 4096, 268 MB: 110 -> 61 us with
// the sums, 4.4 TB/s; 1024 x 8192 20.7 us, 3.2 TB/s).  Above 8192 columns a
// thread's 16 or 32 columns of a row and of the weight gradient pass the 128
// registers that sixteen waves leave it: 100 to 110 of them spill up to 16384
// columns, 236 to 258 up to 32768, and the pass is bound by that traffic (1024 x
// 16384 74 us, 1.8 TB/s; 1024 x 32768 219 us, 1.2 TB/s).

// The runs of 8 of a row, still in bf16.
template <int NV>
struct RawRow {
    u32x4 v[NV];
};
template <int TPR, int NV>
__device__ __forceinline__ void raw_load(RawRow<NV> &r, const void *row, int t, int64_t n) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t col = ((int64_t)v * TPR + t) * 8;
        const uint16_t *p = static_cast<const uint16_t *>(row) + col;
        u32x4 w = {0, 0, 0, 0};
        if (col + 8 <= n) {
            w = *reinterpret_cast<const u32x4 *>(p);
        } else if (col < n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t l0 = col + 2 * e < n ? p[2 * e] : 0u;
                const uint32_t h0 = col + 2 * e + 1 < n ? p[2 * e + 1] : 0u;
                w[e] = l0 | (h0 << 16);
            }
        }
        r.v[v] = w;
    }
}
__device__ __forceinline__ f32x8 widen(u32x4 w) {
    f32x8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
    return v;
}

template <int TPR, int NV, bool VEC, bool RAW>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_grad_kernel(NormGradArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    constexpr int NW = TPR / 64;
    __shared__ float red[2][2][NW];
    __shared__ float join[RPB > 1 ? RPB * 512 : 1];
    const int t = threadIdx.x % TPR;
    const int64_t g = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; // row group
    const int64_t n = a.n;
    // The weight stays in registers except at the widest rows, which read it
    // again (from the cache) where they use it, and dres late, so that fewer of
    // the 1024 threads' registers spill.
    constexpr bool WIDE = TPR > 512;
    f32x8 w[WIDE ? 1 : NV], dw[NV];
    auto weight = [&](int v) __attribute__((always_inline)) {
        if constexpr (WIDE) {
            if (!a.weight)
                return f32x8{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            return load8<VEC>(a.weight, a.w_bf16, ((int64_t)v * TPR + t) * 8, n);
        } else {
            return w[v];
        }
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if constexpr (!WIDE) {
            w[v] = f32x8{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            if (a.weight)
                w[v] = load8<VEC>(a.weight, a.w_bf16, ((int64_t)v * TPR + t) * 8, n);
        }
        dw[v] = f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    }
    RawRow<RAW ? NV : 1> rx, ry, rr; // the next row, RAW only
    auto fetch = [&](int64_t m) __attribute__((always_inline)) {
        if constexpr (RAW) {
            raw_load<TPR, NV>(rx, static_cast<const uint16_t *>(a.X) + m * a.ldx, t, n);
            raw_load<TPR, NV>(ry, static_cast<const uint16_t *>(a.dY) + m * a.lddy, t, n);
            if (a.dres)
                raw_load<TPR, NV>(rr, static_cast<const uint16_t *>(a.dres) + m * a.ld_dres, t, n);
        }
    };
    int odd = 0;
    if (g < a.M && g < a.row_groups)
        fetch(g);
    for (int64_t m = g; m < a.M && g < a.row_groups; m += a.row_groups, odd ^= 1) {
        f32x8 x[NV], dy[NV], dr[WIDE ? 1 : NV];
        const char *rp = static_cast<const char *>(a.dres) + m * a.ld_dres * (a.dx_bf16 ? 2 : 4);
        if constexpr (RAW) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                x[v] = widen(rx.v[v]);
                dy[v] = widen(ry.v[v]);
                if (a.dres)
                    dr[WIDE ? 0 : v] = widen(rr.v[v]);
            }
            if (m + a.row_groups < a.M)
                fetch(m + a.row_groups);
        } else {
            const char *xp = static_cast<const char *>(a.X) + m * a.ldx * (a.x_bf16 ? 2 : 4);
            const char *yp = static_cast<const char *>(a.dY) + m * a.lddy * (a.dy_bf16 ? 2 : 4);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                x[v] = load8<VEC>(xp, a.x_bf16, ((int64_t)v * TPR + t) * 8, n);
                dy[v] = load8<VEC>(yp, a.dy_bf16, ((int64_t)v * TPR + t) * 8, n);
            }
            if (!WIDE && a.dres) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    dr[WIDE ? 0 : v] = load8<VEC>(rp, a.dx_bf16, ((int64_t)v * TPR + t) * 8, n);
            }
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const f32x8 wv = weight(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1 = __builtin_fmaf(x[v][i], x[v][i], s1);
                s2 = __builtin_fmaf(dy[v][i] * wv[i], x[v][i], s2);
            }
        }
        // both sums over the row, in one exchange (rows take turns at two
        // buffers, so that one barrier a row is enough)
        s2 = wave_sum(s2);
        if (!a.rstd)
            s1 = wave_sum(s1);
        if constexpr (NW > 1) {
            if ((threadIdx.x & 63) == 0) {
                red[odd][0][threadIdx.x >> 6] = s1;
                red[odd][1][threadIdx.x >> 6] = s2;
            }
            __syncthreads();
            s1 = red[odd][0][0];
            s2 = red[odd][1][0];
#pragma unroll
            for (int q = 1; q < NW; ++q) {
                s1 += red[odd][0][q];
                s2 += red[odd][1][q];
            }
        }
        const float rstd = a.rstd ? a.rstd[m] : 1.f / __builtin_sqrtf(s1 / (float)n + a.eps);
        const float c = s2 * rstd / (float)n; // mean of t xh
        char *op = a.dX ? static_cast<char *>(a.dX) + m * a.lddx * (a.dx_bf16 ? 2 : 4) : nullptr;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            f32x8 o;
            const f32x8 wv = weight(v);
            if (WIDE && a.dres)
                dr[0] = load8<VEC>(rp, a.dx_bf16, ((int64_t)v * TPR + t) * 8, n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = x[v][i] * rstd;
                o[i] = rstd * (dy[v][i] * wv[i] - xh * c);
                dw[v][i] = __builtin_fmaf(dy[v][i], xh, dw[v][i]);
                if (a.dres)
                    o[i] += dr[WIDE ? 0 : v][i];
            }
            if (op)
                store8<VEC>(op, a.dx_bf16, ((int64_t)v * TPR + t) * 8, n, o);
        }
    }
    if (!a.part)
        return;
    float *const out = a.part + (int64_t)blockIdx.x * ((n + 7) / 8 * 8);
    if constexpr (RPB > 1) { // the waves' sums in order (a wave without rows has zeros)
        const int q = threadIdx.x / TPR;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            join[q * 512 + t * 8 + i] = dw[0][i];
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += 256) {
            float s = join[j];
#pragma unroll
            for (int k = 1; k < RPB; ++k)
                s += join[k * 512 + j];
            out[j] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store8<true>(out, false, ((int64_t)v * TPR + t) * 8, n, dw[v]);
    }
}

// out[j] (+)= sum over the partial rows, 16 columns per workgroup: 16 threads
// per column take every 16th partial (eight loads in flight), then add up in
// order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float *__restrict__ part, int64_t groups,
                                                      int64_t n, float *__restrict__ dW,
                                                      int accumulate) {
    __shared__ float red[16][17];
    const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
    const int64_t j = (int64_t)blockIdx.x * 16 + c;
    const int64_t ld = (n + 7) / 8 * 8;
    float s = 0.f;
    if (j < n) {
        int64_t g = q;
        for (; g + 7 * 16 < groups; g += 8 * 16) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = part[(g + 16 * i) * ld + j];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s += v[i];
        }
        for (; g < groups; g += 16)
            s += part[g * ld + j];
    }
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

// ... of the backward pass, whose rows hold three operands at once
#define TSL_NORM_GRAD_SHAPES(X)                                                                    \
    X(64, 1, 512) X(256, 1, 2048) X(256, 2, 4096) X(512, 2, 8192) X(1024, 2, 16384) X(1024, 4, 32768)

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

// Row groups of a backward launch: enough workgroups to fill the chip, and at
// least four rows each once there are 256 workgroups, so that their partial
// weight gradients stay small beside the rows.
static int64_t grad_row_groups(int64_t M, int64_t n) {
    const int64_t rpb = rows_per_group(n), most = (n <= 4096 ? 1024 : 512) * rpb;
    const int64_t want = (M + 3) / 4 > 256 * rpb ? (M + 3) / 4 : 256 * rpb;
    const int64_t groups = want < most ? want : most;
    return M < groups ? M : groups;
}

int64_t norm_grad_partials(int64_t M, int64_t n) {
    const int64_t rpb = rows_per_group(n);
    return (grad_row_groups(M, n) + rpb - 1) / rpb;
}

hipError_t launch_column_sum(const float *part, int64_t groups, int64_t n, float *out,
                             int accumulate, hipStream_t stream) {
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, stream, part,
                       groups, n, out, accumulate);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs &args, bool vec, float *dW, int accumulate,
                            hipStream_t stream) {
    NormGradArgs a = args;
    a.row_groups = grad_row_groups(a.M, a.n);
    const int64_t parts = norm_grad_partials(a.M, a.n);
    const bool raw = vec && a.x_bf16 && a.dy_bf16 && a.dx_bf16;
    if (a.M > 0) {
        const dim3 grid((unsigned)parts);
        hipError_t e = hipErrorInvalidValue;
#define TSL_CASE(TPR_, NV_, MAX_)                                                                  \
    if (e == hipErrorInvalidValue && a.n <= MAX_) {                                                \
        const dim3 block(TPR_ < 256 ? 256 : TPR_);                                                 \
        if (raw && TPR_ <= 512)                                                                    \
            hipLaunchKernelGGL((norm_grad_kernel<TPR_, NV_, true, (TPR_ <= 512)>), grid, block, 0, \
                               stream, a);                                                         \
        else if (vec)                                                                              \
            hipLaunchKernelGGL((norm_grad_kernel<TPR_, NV_, true, false>), grid, block, 0, stream, \
                               a);                                                                 \
        else                                                                                       \
            hipLaunchKernelGGL((norm_grad_kernel<TPR_, NV_, false, false>), grid, block, 0,        \
                               stream, a);                                                         \
        e = hipGetLastError();                                                                     \
        if (e != hipSuccess)                                                                       \
            return e;                                                                              \
    }
        TSL_NORM_GRAD_SHAPES(TSL_CASE)
#undef TSL_CASE
        if (e != hipSuccess)
            return e;
    }
    return dW ? launch_column_sum(a.part, parts, a.n, dW, accumulate, stream) : hipSuccess;
}

} // namespace tsl
