// Rotary positions of the query and key heads (between the q/k column shards
// and attention): columns (x1, x2) of pair p turn by t = position freq[p],
//     y1 = x1 cos t - x2 sin t,   y2 = x2 cos t + x1 sin t;
// the backward pass is the turn by -t.  Bound by the bytes of one pass, each
// value read once and written once (8192 rows of 72 heads of 128, out of memory:
// 65.5 us, 4.6 TB/s).  A workgroup takes a few token rows: its
// threads form the rows' cosines and sines once, into LDS, and every head of
// every item reads them from there.
//
// The angle is a binary64 product (a position times a binary32 frequency is
// exact to 2^-53), divided by 2 pi and reduced to half a turn there; only
// then is it rounded to binary32: a position of 10^6 has an angle of 10^6,
// whose binary32 would be off by 0.03.
#include "attn.hpp"
#include "rows.hpp"

namespace tsl {
namespace {

constexpr int kThreads = 256;
constexpr int kTableMax = 256; // (token, pair) entries of a workgroup

// Columns col .. col + 7 of one head, turned as pairs where they are rotated (of
// halves only columns passed through come here).
__device__ __forceinline__ f32x8 turned(const void *x, bool bf, int col, int head_dim, int rot,
                                        const float2 *cs) {
    f32x8 v = load8<true>(x, bf, col, head_dim);
    if (col >= rot)
        return v;
    f32x8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 w = cs[col / 2 + i];
        y[2 * i] = v[2 * i] * w.x - v[2 * i + 1] * w.y;
        y[2 * i + 1] = v[2 * i + 1] * w.x + v[2 * i] * w.y;
    }
    return y;
}

// The (cos, sin) of `tokens` rows from m0 on: entry (i, p) at i * half + p.
__device__ __forceinline__ void fill_table(const RotateArgs &a, int64_t m0, int tokens, float2 *cs) {
    const int half = a.rot_dim / 2;
    for (int e = threadIdx.x; e < tokens * half; e += kThreads) {
        const int i = e / half, p = e % half;
        const int axis = (a.axis[p >> 4] >> (2 * (p & 15))) & 3;
        const int32_t pos = a.positions[axis * a.ld_pos + m0 + i];
        const double turns = (double)pos * (double)a.freq[p] * 0.15915494309189533577;
        const float u = (float)(turns - rint(turns));
        float s, c;
        sincospif(2.f * u, &s, &c);
        cs[e] = make_float2(c, a.inverse ? -s : s);
    }
}

// Vector form: every row and head of every item 16-byte aligned, rot_dim / 2 a
// multiple of 8 (halves) or rot_dim one (pairs).  A thread turns one run of 8
// columns (pairs) or both runs of 8 pairs (halves).
__global__ void __launch_bounds__(kThreads) rotate_kernel(RotateArgs a, int tokens, int heads_each) {
    __shared__ float2 cs[kTableMax];
    const int64_t m0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)(a.M - m0 < tokens ? a.M - m0 : tokens);
    fill_table(a, m0, n, cs);
    __syncthreads();
    const int half = a.rot_dim / 2;
    // runs of a head: halves have half / 8 pairs of runs, then the columns
    // passed through; pairs simply its runs of 8
    const int runs = a.pairs ? a.head_dim / 8 : half / 8 + (a.head_dim - a.rot_dim) / 8;
    const int h0 = blockIdx.y * heads_each;
    const int heads = a.heads - h0 < heads_each ? a.heads - h0 : heads_each;
    for (int e = threadIdx.x; e < n * heads * runs; e += kThreads) {
        const int run = e % runs, q = e / runs;
        int h = h0 + q % heads, k = 0;
        const int i = q / heads;
        while (h >= a.item[k].n_heads)
            h -= a.item[k++].n_heads;
        const RotateArgs::Item &it = a.item[k];
        const float2 *turn = cs + i * half; // of the row
        const char *x = static_cast<const char *>(it.X) +
                        ((m0 + i) * it.ldx + h * it.x_head) * (it.x_bf16 ? 2 : 4);
        char *y = static_cast<char *>(it.Y) +
                  ((m0 + i) * it.ldy + h * it.y_head) * (it.y_bf16 ? 2 : 4);
        if (!a.pairs && run < half / 8) {
            const int col = run * 8;
            const f32x8 p = load8<true>(x, it.x_bf16, col, a.head_dim);
            const f32x8 r = load8<true>(x, it.x_bf16, col + half, a.head_dim);
            f32x8 u, v;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 w = turn[col + j];
                u[j] = p[j] * w.x - r[j] * w.y;
                v[j] = r[j] * w.x + p[j] * w.y;
            }
            store8<true>(y, it.y_bf16, col, a.head_dim, u);
            store8<true>(y, it.y_bf16, col + half, a.head_dim, v);
        } else {
            const int col = a.pairs ? run * 8 : a.rot_dim + (run - half / 8) * 8;
            store8<true>(y, it.y_bf16, col, a.head_dim,
                         turned(x, it.x_bf16, col, a.head_dim, a.rot_dim, turn));
        }
    }
}

// Any alignment and width: a thread turns one pair, or passes one column on.
__global__ void __launch_bounds__(kThreads) rotate_any_kernel(RotateArgs a, int tokens,
                                                              int heads_each) {
    __shared__ float2 cs[kTableMax];
    const int64_t m0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)(a.M - m0 < tokens ? a.M - m0 : tokens);
    fill_table(a, m0, n, cs);
    __syncthreads();
    const int half = a.rot_dim / 2;
    const int work = half + a.head_dim - a.rot_dim;
    const int h0 = blockIdx.y * heads_each;
    const int heads = a.heads - h0 < heads_each ? a.heads - h0 : heads_each;
    for (int e = threadIdx.x; e < n * heads * work; e += kThreads) {
        const int p = e % work, q = e / work;
        int h = h0 + q % heads, k = 0;
        const int i = q / heads;
        while (h >= a.item[k].n_heads)
            h -= a.item[k++].n_heads;
        const RotateArgs::Item &it = a.item[k];
        const int64_t xo = (m0 + i) * it.ldx + h * it.x_head, yo = (m0 + i) * it.ldy + h * it.y_head;
        auto get = [&](int col) {
            return it.x_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(it.X)[xo + col] << 16)
                             : static_cast<const float *>(it.X)[xo + col];
        };
        auto put = [&](int col, float v) {
            if (it.y_bf16)
                static_cast<uint16_t *>(it.Y)[yo + col] = (uint16_t)pack_bf16(v, 0.f);
            else
                static_cast<float *>(it.Y)[yo + col] = v;
        };
        if (p < half) {
            const int c1 = a.pairs ? 2 * p : p, c2 = a.pairs ? 2 * p + 1 : p + half;
            const float x1 = get(c1), x2 = get(c2);
            const float2 w = cs[i * half + p];
            put(c1, x1 * w.x - x2 * w.y);
            put(c2, x2 * w.x + x1 * w.y);
        } else {
            const int col = a.rot_dim + p - half;
            put(col, get(col));
        }
    }
}

} // namespace

hipError_t launch_rotate(const RotateArgs &a, hipStream_t stream) {
    const int half = a.rot_dim / 2;
    // rows of a workgroup: 8192 rows of 72 heads of 128 take 54.6 us with 4 (in
    // cache; 57.5 with 2, 61.6 with 1, 80.7 with 8), but fewer rows than make 512
    // workgroups are spread thinner (1531 of 40 heads of 64 in binary32: 8.2 us with
    // 2, 8.9 with 4)
    int tokens = kTableMax / half;
    tokens = tokens < 1 ? 1 : (tokens > 4 ? 4 : tokens);
    while (tokens > 1 && (a.M + tokens - 1) / tokens < 512)
        tokens /= 2;
    // and with fewer yet the heads are divided over workgroups too, whose tables
    // repeat (16 to 250 rows of 32 heads 7.4 us, undivided 8.0)
    const int64_t groups = (a.M + tokens - 1) / tokens;
    int parts = (int)(512 / groups);
    parts = parts < 1 ? 1 : (parts > (a.heads + 3) / 4 ? (a.heads + 3) / 4 : parts);
    const int each = (a.heads + parts - 1) / parts;
    const dim3 grid((unsigned)groups, (unsigned)((a.heads + each - 1) / each));
    if (a.wide)
        hipLaunchKernelGGL(rotate_kernel, grid, dim3(kThreads), 0, stream, a, tokens, each);
    else
        hipLaunchKernelGGL(rotate_any_kernel, grid, dim3(kThreads), 0, stream, a, tokens, each);
    return hipGetLastError();
}

} // namespace tsl
