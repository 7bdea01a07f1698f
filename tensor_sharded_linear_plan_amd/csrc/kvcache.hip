// Keys and values into and out of the paged 4-bit cache (layout: tsl_attn.h,
// tsl_cache).  A run x of 64 columns of a head of a token becomes
//     b = bf16(min x),  s = bf16((max x - b) / 15),  c = round((x - b) / s).
// Bound by bytes: 2 or 4 read and 0.5625 written a value (append), the
// reverse (read).  One workgroup takes one record (32 tokens of one head), so
// the words that tokens share have one writer.  7370 tokens of 8 heads of 128:
// read to binary32 15.5 us, 4.5 TB/s; append from bf16 17.8 us, 2.2 TB/s, bound by
// vector instructions (25 a value, of which 9 are the code's).
#include "attn.hpp"
#include "rows.hpp"

namespace tsl {
namespace {

constexpr int kThreads = 256;

// The record, and the tokens of it that the call's rows are (lo .. hi - 1),
// of one workgroup; row is that of token 0 (it may lie before the rows).
struct Span {
    char *rec;
    int lo, hi;
    int64_t row;
    int head;
    int row0, before; // the sequence's first row; rows before position 0 (of the first workgroup)
};
template <int D>
__device__ __forceinline__ Span span_of(const MoveArgs &a) {
    // neighbouring workgroups take the heads of the same rows
    Span w;
    const int blk_i = quotient(blockIdx.x, a.by_heads), s = blockIdx.y;
    w.head = blockIdx.x - blk_i * a.c.n_kv_heads;
    const SeqRows q = seq_rows(a.c, s);
    const int n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
    const int start = q.ctx - q.n; // position of row 0
    w.row0 = q.row0;
    w.before = blk_i > 0 || start >= 0 ? 0 : (n < -start ? n : -start);
    const int first = start > 0 ? start : 0;
    const int64_t end = (int64_t)start + n;
    const int blk = (first >> 5) + blk_i;
    const int64_t t0 = (int64_t)blk * kBlock;
    w.lo = t0 < first ? (int)(first - t0) : 0;
    w.hi = end - t0 < kBlock ? (int)(end - t0 > 0 ? end - t0 : 0) : kBlock;
    w.row = q.row0 + t0 - start;
    w.rec = w.hi > w.lo ? record_of(a.c, s, w.head, blk, record_bytes(D)) : nullptr;
    return w;
}

// Index of 32-bit word n of a lane in a record's codes.
__device__ __forceinline__ int word_at(int n, int lane) { return (n >> 2) * 256 + lane * 4 + (n & 3); }
// Place of a token in the 32 scales (or biases) of a record.
__device__ __forceinline__ int scale_at(int t) {
    return ((t & 15) >> 2) * 8 + (t >> 4) * 4 + (t & 3);
}
__device__ __forceinline__ int nibble_at(int i) { return 4 * ((i >> 1) + 4 * (i & 1)); }

// f over the 8 lanes of a lane's group: neighbours, pairs, and quads mirrored.
template <class F> __device__ __forceinline__ float over8(float v, F f) {
    v = f(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true)));
    v = f(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true)));
    v = f(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, true)));
    return v;
}

// Codes of 8 columns of a run whose other columns the 8 lanes of this lane's group
// hold, 4 bits each at `place`; scale_bias is the run's.  The quotients are
// binary64 (a product, its remainder, the remainder's share: exact where the
// quotient is half way between two codes, which is what rounding needs); in
// binary32 the exact decision takes three times the instructions (append of 7370
// tokens of 8 heads of 128: 25 us that way, 18 us so).
template <class F> __device__ __forceinline__ uint32_t quantise(f32x8 x, uint32_t *scale_bias, F place) {
    float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad = fmaf(x[i], 0.f, bad); // NaN where a value is not finite
    }
    lo = over8(lo, [](float u, float v) { return fminf(u, v); });
    hi = over8(hi, [](float u, float v) { return fmaxf(u, v); });
    bad = over8(bad, [](float u, float v) { return u + v; });
    const uint32_t bb = pack_pair(lo, 0.f);
    const float bias = bf16_lo(bb);
    const uint32_t sb = pack_pair((hi - bias) / 15.f, 0.f);
    const float scale = bf16_lo(sb);
    const bool whole = bad == 0.f && __builtin_isfinite(scale) && __builtin_isfinite(bias);
    *scale_bias = whole ? sb | bb << 16 : 0x7FC07FC0u;
    if (!whole || scale == 0.f)
        return 0;
    const double s = scale, inv = 1.0 / s, b = bias;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double d = (double)x[i] - b;
        double q = d * inv;
        q = fma(fma(-q, s, d), inv, q);
        int c = (int)rint(q);
        c = c < 0 ? 0 : (c > 15 ? 15 : c);
        codes |= (uint32_t)c << place(i);
    }
    return codes;
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(MoveArgs a) {
    constexpr int LPT = D / 8;                // lanes of a token, 8 columns each
    constexpr int TPP = kThreads / LPT;       // tokens a pass
    constexpr int PASSES = kBlock / TPP, W = D / 32;
    __shared__ __attribute__((aligned(16))) uint32_t kc[4 * D]; // K codes as they are stored
    __shared__ uint32_t vc[kBlock][D / 8 + 1];                  // V codes of a token, 4 bits a column
    __shared__ uint16_t sc[D / 64 * 128];
    const Span w = span_of<D>(a);
    if (w.hi <= w.lo)
        return;
    const int cl = threadIdx.x % LPT, t0 = threadIdx.x / LPT;
    const int e = a.bf16 ? 2 : 4;
    f32x8 xk[PASSES], xv[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int t = t0 + p * TPP;
        if (t >= w.lo && t < w.hi) { // (a token's lanes are in or out together)
            const int64_t row = w.row + t;
            xk[p] = load8<true>(static_cast<const char *>(a.K) + (row * a.ldk + w.head * a.k_head) * e, a.bf16,
                                cl * 8, D);
            xv[p] = load8<true>(static_cast<const char *>(a.V) + (row * a.ldv + w.head * a.v_head) * e, a.bf16,
                                cl * 8, D);
        }
    }
    if (!w.rec) // (asked for here: the page is on its way with the rows)
        return;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int t = t0 + p * TPP;
        if (t >= w.lo && t < w.hi) {
            uint32_t k2, v2;
            kc[word_at((t >> 4) * W + cl / 4, (cl & 3) * 16 + (t & 15))] = quantise(xk[p], &k2, nibble_at);
            vc[t][cl] = quantise(xv[p], &v2, [](int i) { return 4 * i; });
            if (cl % 8 == 0) {
                uint16_t *g = sc + (cl / 8) * 128 + scale_at(t);
                g[0] = (uint16_t)k2;
                g[32] = (uint16_t)(k2 >> 16);
                g[64] = (uint16_t)v2;
                g[96] = (uint16_t)(v2 >> 16);
            }
        }
    }
    __syncthreads();
    uint32_t *kw = reinterpret_cast<uint32_t *>(w.rec), *vw = kw + 4 * D;
    uint16_t *sw = reinterpret_cast<uint16_t *>(w.rec + 32 * D);
    const bool full = w.hi - w.lo == kBlock;
    if (full) {
        for (int i = threadIdx.x; i < D; i += kThreads)
            reinterpret_cast<u32x4 *>(kw)[i] = reinterpret_cast<const u32x4 *>(kc)[i];
        for (int i = threadIdx.x; i < D; i += kThreads)
            reinterpret_cast<uint32_t *>(sw)[i] = reinterpret_cast<const uint32_t *>(sc)[i];
    } else {
        for (int i = threadIdx.x; i < (w.hi - w.lo) * (D / 8); i += kThreads) {
            const int t = w.lo + i / (D / 8), n = i % (D / 8);
            const int at = word_at((t >> 4) * W + n / 4, (n & 3) * 16 + (t & 15));
            kw[at] = kc[at];
        }
        for (int i = threadIdx.x; i < (w.hi - w.lo) * (D / 16); i += kThreads) {
            const int at = (i % (D / 16)) * 32 + scale_at(w.lo + i / (D / 16));
            sw[at] = sc[at];
        }
    }
    // V words: 8 tokens of a column each; tokens that are not the call's keep
    // their bits
    for (int i = threadIdx.x; i < 4 * D; i += kThreads) {
        const int n = i >> 6, lane = i & 63, at = word_at(n, lane);
        const int col = n * 16 + (lane & 15), g = lane >> 4;
        uint32_t mask = 0, word = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int t = (k >> 2) * 16 + g * 4 + (k & 3);
            if (full || (t >= w.lo && t < w.hi)) {
                mask |= 15u << nibble_at(k);
                word |= ((vc[t][col >> 3] >> (4 * (col & 7))) & 15u) << nibble_at(k);
            }
        }
        if (mask == 0xFFFFFFFFu)
            vw[at] = word;
        else if (mask)
            vw[at] = (vw[at] & ~mask) | word;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(MoveArgs a) {
    constexpr int LPT = D / 8, TPP = kThreads / LPT, W = D / 32;
    __shared__ __attribute__((aligned(16))) uint32_t codes[8 * D];
    __shared__ uint16_t sc[D / 64 * 128];
    const Span w = span_of<D>(a);
    const int e = a.bf16 ? 2 : 4;
    // rows before position 0 lie in no record
    for (int i = threadIdx.x; i < w.before * LPT; i += kThreads) {
        const f32x8 zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const int64_t row = w.row0 + i / LPT;
        if (a.K)
            store8<true>(static_cast<char *>(a.K) + (row * a.ldk + w.head * a.k_head) * e, a.bf16,
                         i % LPT * 8, D, zero);
        if (a.V)
            store8<true>(static_cast<char *>(a.V) + (row * a.ldv + w.head * a.v_head) * e, a.bf16,
                         i % LPT * 8, D, zero);
    }
    if (w.hi <= w.lo)
        return;
    if (w.rec) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(w.rec);
        for (int e = threadIdx.x; e < 2 * D; e += kThreads)
            reinterpret_cast<u32x4 *>(codes)[e] = reinterpret_cast<const u32x4 *>(src)[e];
        for (int e = threadIdx.x; e < D; e += kThreads)
            reinterpret_cast<uint32_t *>(sc)[e] = src[8 * D + e];
    }
    __syncthreads();
    const int cl = threadIdx.x % LPT;
    for (int t0 = 0; t0 < kBlock; t0 += TPP) {
        const int t = t0 + threadIdx.x / LPT;
        if (t < w.lo || t >= w.hi)
            continue;
        f32x8 k = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v = k;
        if (w.rec) {
            const uint16_t *g = sc + (cl / 8) * 128 + scale_at(t);
            const float sk = bf16_lo(g[0]), bk = bf16_lo(g[32]);
            const float sv = bf16_lo(g[64]), bv = bf16_lo(g[96]);
            const uint32_t word = codes[word_at((t >> 4) * W + cl / 4, (cl & 3) * 16 + (t & 15))];
            const int lane = ((t & 15) >> 2) * 16, shift = nibble_at((t >> 4) * 4 + (t & 3));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = cl * 8 + i;
                const uint32_t x = codes[4 * D + word_at(col >> 4, lane + (col & 15))];
                k[i] = fmaf(sk, (float)((word >> nibble_at(i)) & 15u), bk);
                v[i] = fmaf(sv, (float)((x >> shift) & 15u), bv);
            }
        }
        const int64_t row = w.row + t;
        if (a.K)
            store8<true>(static_cast<char *>(a.K) + (row * a.ldk + w.head * a.k_head) * e, a.bf16,
                         cl * 8, D, k);
        if (a.V)
            store8<true>(static_cast<char *>(a.V) + (row * a.ldv + w.head * a.v_head) * e, a.bf16,
                         cl * 8, D, v);
    }
}

} // namespace

hipError_t launch_cache_append(int head_dim, const MoveArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.c.n_kv_heads * a.seq_blocks), (unsigned)a.c.n_seqs);
    if (head_dim == 64)
        hipLaunchKernelGGL(append_kernel<64>, grid, dim3(kThreads), 0, stream, a);
    else if (head_dim == 128)
        hipLaunchKernelGGL(append_kernel<128>, grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(append_kernel<256>, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_cache_read(int head_dim, const MoveArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.c.n_kv_heads * a.seq_blocks), (unsigned)a.c.n_seqs);
    if (head_dim == 64)
        hipLaunchKernelGGL(read_kernel<64>, grid, dim3(kThreads), 0, stream, a);
    else if (head_dim == 128)
        hipLaunchKernelGGL(read_kernel<128>, grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(read_kernel<256>, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

} // namespace tsl
