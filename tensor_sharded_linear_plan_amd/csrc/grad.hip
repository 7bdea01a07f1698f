// The operands of a shard product's backward pass.  With dZ the gradient at
// the product's output, dX = dZ W^T and dW = X^T dZ are two more products of
// the forward's own GEMM: dX over the packed transposed weight with dZ as its
// rows, dW over the token rows with X^T as rows and dZ as the weight (or dZ^T
// as rows and X as the weight, for a gradient stored [N][K]).  This pass makes
// what they read, each input read once:
//   - dZ itself where an activation lies between (dY act'(Z)), or the gated
//     block's pair dG = dH u act'(g), dU = dH act(g), in binary32, rounded
//     once to the operands' type;
//   - the transposed copies, through LDS: a workgroup takes 64 x 64 elements,
//     a thread two neighbouring rows of 8 columns, whose values go to LDS as
//     row pairs, 33 words a column (conflict free), and leave it as 16-byte
//     runs along the token rows, whole 1 KB tiles of the packed layout;
//   - the column sums of the unrounded dZ (the bias gradient), one partial per
//     64 rows.
// With few entries (split) what the rounding of dZ left is an operand of its
// own, rows and k-range doubled, so that its error does not show.
// Bound by bytes: gated, 3 values read and 4 written per element (4096 rows,
// 3584 columns, with the copy of X of 4096: 272 MB in 54 us, 5.0 TB/s).
#include "device.hpp"
#include "epilogue.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace tsl {
namespace {

constexpr int kTile = 64;

struct GradJobs {
    int32_t n, pad_;
    GradJob j[kGradJobs];
};

template <typename T> struct Elem;
template <> struct Elem<uint16_t> {
    static constexpr bool bf = true;
    static constexpr int WPP = 1;  // words of a row pair
    static constexpr int LDW = 33; // words of a column in LDS: 32 row pairs and one more
};
template <> struct Elem<float> {
    static constexpr bool bf = false;
    static constexpr int WPP = 2;
    static constexpr int LDW = 65;
};

// One transposed copy of the tile's values v (rows 2 r, 2 r + 1 of the
// thread's 8 columns, zero outside the matrix) at rows m0 on of the copy's Mt.
template <typename T>
__device__ __forceinline__ void transpose_tile(const GradJob &g, void *out, const f32x8 (&v)[2],
                                               uint32_t *lds, int64_t m0, int64_t Mt, int64_t n0) {
    using E = Elem<T>;
    const int cc = threadIdx.x & 7, r = threadIdx.x >> 3;
    __syncthreads(); // the tile's last readers are done
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t *p = lds + (8 * cc + i) * E::LDW + r * E::WPP;
        if constexpr (E::bf) {
            p[0] = pack_bf16(v[0][i], v[1][i]);
        } else {
            p[0] = __float_as_uint(v[0][i]);
            p[1] = __float_as_uint(v[1][i]);
        }
    }
    __syncthreads();
    constexpr int PER = 16 / sizeof(T);      // rows of a 16-byte run
    constexpr int RUNS = kTile / PER;        // runs of a column of the tile
    const int64_t cols = g.packed ? (g.N + 15) / 16 * 16 : g.N;
#pragma unroll
    for (int q = 0; q < kTile * RUNS / 256; ++q) {
        const int id = q * 256 + threadIdx.x;
        // runs in the destination's order: packed, 16 columns of 4 runs make a
        // 1 KB tile; else the runs of a column follow one another
        int n, c;
        if (g.packed) {
            const int tile = id >> 6, l = id & 63;
            n = (tile & 3) * 16 + (l & 15);
            c = (tile >> 2) * 4 + (l >> 4);
        } else {
            n = id / RUNS;
            c = id % RUNS;
        }
        if (n0 + n >= cols)
            continue;
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = lds[n * E::LDW + c * 4 + i];
        const int64_t cg = m0 / PER + c, col = n0 + n;
        const int64_t at = g.packed ? ((col >> 4) * (Mt / PER / 4) + (cg >> 2)) * 64 +
                                          (cg & 3) * 16 + (col & 15)
                                    : col * (Mt / PER) + cg;
        static_cast<u32x4 *>(out)[at] = w;
    }
}

// What rounding to bf16 left of 8 values (exact; nothing of one that is, or
// rounds to, an infinity or a NaN).
__device__ __forceinline__ f32x8 left_of(f32x8 v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float h = (float)(__bf16)v[i];
        v[i] = __builtin_isfinite(h) ? v[i] - h : 0.f;
    }
    return v;
}

template <typename T>
__global__ void __launch_bounds__(256) grad_rows_kernel(GradJobs jobs) {
    using E = Elem<T>;
    __shared__ uint32_t lds[kTile * E::LDW];
    __shared__ float red[4][kTile];
    const int job = jobs.n > 1 && (int)blockIdx.x >= jobs.j[1].start ? 1 : 0;
    const GradJob &g = jobs.j[job];
    const int b = blockIdx.x - g.start;
    const int64_t mb = b / g.nblk, m0 = mb * kTile, n0 = (int64_t)(b % g.nblk) * kTile;
    const int cc = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int64_t col = n0 + 8 * cc, N = g.N;
    f32x8 z[2], y[2] = {}; // dZ (gated: dG, dU) of rows m0 + 2 r and the next
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t m = m0 + 2 * r + q;
        const int64_t lim = m < g.M ? N : 0; // columns read
        auto rowof = [&](const void *p, int64_t ld) { return static_cast<const T *>(p) + m * ld; };
        z[q] = load8<true>(rowof(g.a, g.lda), E::bf, col, lim);
        if (g.kind == kGradCopy)
            continue;
        const f32x8 v = load8<true>(rowof(g.b, g.ldb), E::bf, col, lim);
        if (g.kind == kGradAct) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a, d;
                act_both(v[i], g.act, a, d);
                z[q][i] *= d;
            }
        } else {
            const f32x8 u = load8<true>(rowof(g.c, g.ldc), E::bf, col, lim);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a, d;
                act_both(v[i], g.act, a, d);
                y[q][i] = z[q][i] * a;
                z[q][i] = z[q][i] * u[i] * d;
            }
        }
        // a column past N holds act'(0) times zero: still zero
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t m = m0 + 2 * r + q;
        if (m < g.M && g.row[0])
            store8<true>(static_cast<T *>(g.row[0]) + m * g.ld_row, E::bf, col, g.ld_row, z[q]);
        if (m < g.M && g.row[1])
            store8<true>(static_cast<T *>(g.row[1]) + m * g.ld_row, E::bf, col, g.ld_row, y[q]);
    }
    if (g.part) { // the wave's 16 rows, then the four waves in order
        f32x8 s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = z[0][i] + z[1][i];
#pragma unroll
            for (int o = 8; o <= 32; o <<= 1)
                s[i] += __shfl_xor(s[i], o, 64);
        }
        if ((threadIdx.x & 63) < 8)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                red[threadIdx.x >> 6][8 * cc + i] = s[i];
        __syncthreads();
        const int64_t n = n0 + threadIdx.x;
        if (threadIdx.x < kTile && n < N) {
            const int t = threadIdx.x;
            float *const p = g.part + mb * ((N + 7) / 8 * 8) + n;
            const float v = ((red[0][t] + red[1][t]) + red[2][t]) + red[3][t];
            *p = g.add ? *p + v : v;
        }
    }
    const int64_t Mp = (g.M + 63) / 64 * 64, Mt = g.split ? 2 * Mp : Mp;
    if (g.tr[0])
        transpose_tile<T>(g, g.tr[0], z, lds, m0, Mt, n0);
    if (g.tr[1])
        transpose_tile<T>(g, g.tr[1], y, lds, m0, Mt, n0);
    if (!E::bf || !g.split)
        return;
    if (g.kind != kGradCopy) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            z[q] = left_of(z[q]);
            y[q] = left_of(y[q]);
            const int64_t m = m0 + 2 * r + q;
            if (m < g.M && g.row_lo[0])
                store8<true>(static_cast<T *>(g.row_lo[0]) + m * g.ld_row, E::bf, col, g.ld_row, z[q]);
            if (m < g.M && g.row_lo[1])
                store8<true>(static_cast<T *>(g.row_lo[1]) + m * g.ld_row, E::bf, col, g.ld_row, y[q]);
        }
    }
    if (g.tr[0])
        transpose_tile<T>(g, g.tr[0], z, lds, Mp + m0, Mt, n0);
    if (g.tr[1])
        transpose_tile<T>(g, g.tr[1], y, lds, Mp + m0, Mt, n0);
}

template <typename T>
__global__ void __launch_bounds__(256) zero_rows_kernel(T *__restrict__ out, int64_t rows,
                                                        int64_t cols, int64_t ld) {
    for (int64_t m = blockIdx.x; m < rows; m += gridDim.x)
        for (int64_t j = threadIdx.x; j < cols; j += 256)
            out[m * ld + j] = T(0);
}

} // namespace

hipError_t launch_zero_rows(void *out, int64_t rows, int64_t cols, int64_t ld, bool bf16,
                            hipStream_t stream) {
    const dim3 grid((unsigned)(rows < 65536 ? rows : 65536));
    if (bf16)
        hipLaunchKernelGGL(zero_rows_kernel<uint16_t>, grid, dim3(256), 0, stream,
                           static_cast<uint16_t *>(out), rows, cols, ld);
    else
        hipLaunchKernelGGL(zero_rows_kernel<float>, grid, dim3(256), 0, stream,
                           static_cast<float *>(out), rows, cols, ld);
    return hipGetLastError();
}

// 64 x 64 blocks of a job: its rows up to Mp, its columns up to what any of
// its results holds.
int64_t grad_blocks(const GradJob &j) { return (j.M + 63) / 64 * ((j.N + 63) / 64); }

hipError_t launch_grad_rows(GradJob *jobs, int n, bool bf16, hipStream_t stream) {
    GradJobs g{};
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i) {
        if (grad_blocks(jobs[i]) == 0)
            continue;
        GradJob &j = g.j[g.n++];
        j = jobs[i];
        j.nblk = (int32_t)((j.N + 63) / 64);
        j.start = (int32_t)blocks;
        blocks += grad_blocks(j);
    }
    if (blocks == 0)
        return hipSuccess;
    if (bf16)
        hipLaunchKernelGGL(grad_rows_kernel<uint16_t>, dim3((unsigned)blocks), dim3(256), 0, stream,
                           g);
    else
        hipLaunchKernelGGL(grad_rows_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, stream, g);
    return hipGetLastError();
}

} // namespace tsl
