// Attention of query rows over the paged 4-bit cache, for many rows a sequence
// (prompts and their chunks): the same pass over the tokens as attend.hip, with
// each expanded token shared by up to 256 query rows.
//
// A workgroup takes 256 query rows of one sequence and K/V head (32 a wave) and
// walks the records they see, TB at a time: the codes of the next TB records, in
// registers since the step before, are expanded to binary16 into one half of
// LDS while the other half is multiplied.  S^T = K Q^T and O^T = V^T P^T on
// 32x32x16 MFMAs, so a lane holds one query row (column l % 32) throughout and
// the probabilities leave S^T as O^T's operand.  A record at a time, each
// product runs beside vector work that does not wait for it: the logits of the
// next record beside the exponentials of this, the weighted sum beside the
// expansion of the next step's codes.
//
// Binary16 has 11 bits where bf16 has 8: a bf16 K would move a logit by 2^-9 of
// its terms, which the exponential passes on to the result at the size of the
// result's own rounding.  Its range is met with powers of two, as the 4-bit
// GEMM's is: a row of Q by its largest element, the K and the V values of the
// records in hand by a bound of theirs (15 |s| + |b|), V's never below that of
// earlier ones, which the accumulators carry.  Probabilities are 2^9 times their
// value relative to the running reference, which moves only when a sum of 16 of
// them comes to 2^15 (none is lost above 2^-33 of the largest): the common step
// looks for no maximum.
#include "attn.hpp"

namespace tsl {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kProbScale = 9.f;     // log2
constexpr float kProbMost = 32768.f;  // of a lane's 16 probabilities together
constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;
static_assert(kRows == kPromptRows, "rows of a tile");

// 4-bit word -> four pairs of binary16 codes (0 .. 15, exact): 1024 + c has c in
// its low mantissa bits, 1024 + 16 c four bits up.
__device__ __forceinline__ void codes16(uint32_t w, f16x2 (&c)[4]) {
    uint32_t lo, hi, o;
    asm("v_mov_b32 %0, 0x000f000f" : "=v"(lo));
    asm("v_mov_b32 %0, 0x00f000f0" : "=v"(hi));
    asm("s_mov_b32 %0, 0x64006400" : "=s"(o));
    const uint32_t w8 = w >> 8;
    const f16x2 base = {(_Float16)-1024.f, (_Float16)-1024.f};
    const f16x2 base16 = {(_Float16)-64.f, (_Float16)-64.f};
    const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    c[0] = __builtin_bit_cast(f16x2, (w & lo) | o) + base;
    c[1] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (w & hi) | o), sixteenth, base16);
    c[2] = __builtin_bit_cast(f16x2, (w8 & lo) | o) + base;
    c[3] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (w8 & hi) | o), sixteenth, base16);
}

__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

// The larger halves of all lanes' words, wave-uniform: rotations within rows of
// 16 lanes, then a lane of each row.
__device__ __forceinline__ uint32_t wave_pk_max(uint32_t v) {
    v = pk_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true)); // row_ror:8
    v = pk_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, true));
    v = pk_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, true));
    v = pk_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, true));
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r);
        lo = (w & 0xFFFFu) > lo ? w & 0xFFFFu : lo;
        hi = (w >> 16) > hi ? w >> 16 : hi;
    }
    return lo | hi << 16;
}

// Nothing is scheduled across.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Place of a 16-byte piece of a row of LDS: 16 neighbouring rows spread over all
// 64 banks.
template <int ROW> __device__ __forceinline__ int piece_at(int row, int piece) {
    return row * ROW + ((piece ^ (ROW == 128 ? row >> 1 & 7 : row & 15)) << 4);
}

template <int D>
__global__ void __launch_bounds__(64 * kWaves, 2) attend_prompt_kernel(AttendArgs a) {
    constexpr int G = D / 64, W = D / 32, ST = D / 16, DT = D / 32;
    constexpr int TB = 8 / G;                         // records of a step
    constexpr int KROW = D * 2, VROW = 64 * TB;       // bytes of a token, of a column
    constexpr int BUF = 32 * TB * KROW;               // 32 KB: K, or V, of a step
    extern __shared__ __attribute__((aligned(16))) char lds[]; // K, K, V, V

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, h = lane >> 5;

    // Later tiles see more tokens and start first; neighbouring workgroups take
    // different heads, whose tokens stay in the L2 of one XCD.  The sequences of
    // a tile take turns: workgroups go to the engines of an XCD in turn too, and
    // a long sequence at the same place of each round would keep to one of them
    // (prompts of 2500, 267, 1756 and 1630 tokens ran in 651 us that way, in
    // 423 us so).
    int b = quotient(blockIdx.x, a.by_splits);
    const int split = blockIdx.x - b * a.splits;
    const int heads = a.c.n_seqs * a.c.n_kv_heads;
    const int tile = a.tiles - 1 - b / heads;
    b %= heads;
    const int turn = quotient(b, a.by_heads), head = b - turn * a.c.n_kv_heads;
    const int s = (turn + tile) % a.c.n_seqs;
    const int unit = (s * a.c.n_kv_heads + head) * a.tiles + tile;
    const SeqRows q = seq_rows(a.c, s);
    const int rows = rows_of(a, q) - tile * kRows;
    if (rows <= 0)
        return;
    const int start = q.ctx - q.n;
    const int last_rho = tile * kRows + (rows < kRows ? rows : kRows) - 1;
    TileView view = view_of(a, q, tile, kRows, rows);
    divide(a, view);
    const int begin = split * view.share;
    const int stop = begin + view.share < view.count ? begin + view.share : view.count;
    if (begin >= stop && split > 0)
        return;
    const int steps = begin < stop ? (stop - begin + TB - 1) / TB : 0;

    // the lane's query row and the wave's positions
    const int mine = wave * 32 + c;
    const bool live = mine < rows;
    const int rho = live ? tile * kRows + mine : last_rho;
    const int i = quotient(rho, a.by_group), hq = head * a.group + rho - i * a.group;
    const int pos = start + i, lo = window_start(a, pos);
    const bool idle = wave * 32 >= rows;
    const int wave_last = wave * 32 + 31 < rows ? tile * kRows + wave * 32 + 31 : last_rho;
    TileView wv = view;
    wv.first = __builtin_amdgcn_readfirstlane(start + quotient(tile * kRows + wave * 32, a.by_group));
    wv.last = __builtin_amdgcn_readfirstlane(start + quotient(wave_last, a.by_group));

    // Q as binary16, its largest element in 2^14 .. 2^15; the scale's sign goes
    // to it, so that the largest product is the largest logit
    f16x8 qr[ST];
    int qe;
    {
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
        const uint16_t *qp = a.Q + (int64_t)(q.row0 + i) * a.ldq + hq * a.q_head + 8 * h;
        u32x4 raw[ST];
        uint32_t top = 0;
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            raw[t] = *reinterpret_cast<const u32x4 *>(qp + 16 * t) ^ flip;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = pk_max(top, raw[t][j] & 0x7FFF7FFFu);
        }
        top = pk_max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const uint32_t e = ((top & 0xFFFFu) > (top >> 16) ? top & 0xFFFFu : top >> 16) >> 7;
        qe = e == 255 ? 0 : (int)e - 127 - 14;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                qr[t][2 * j] = (_Float16)ldexpf(bf16_lo(raw[t][j]), -qe);
                qr[t][2 * j + 1] = (_Float16)ldexpf(bf16_hi(raw[t][j]), -qe);
            }
    }

    f32x16 o[DT];
    float m = kNoMax, l = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            o[t][r] = 0.f;
    uint32_t taint = 0; // groups in which a visible V is not finite

    // ---- a step's records ----
    // record t of a step; past the range a token that no row sees
    auto block_at = [&](int step, int t) {
        const int r = begin + step * TB + t;
        return r < stop ? view_block(view, r) : (kMaxContext >> 5) + 1;
    };
    // tokens that some row of the tile sees: the others enter LDS as zeros
    auto any_sees = [&](int j) {
        return (j <= view.last) & (!a.window | (j > view.first - a.window) | (j < a.sinks));
    };
    // Eight lanes (times G) look after a record: its page, loaded a step before
    // its codes, and who sees it.  Bit 8 G t of a mask is record t's.
    const int lt = (lane >> 3) / G;
    auto bit = [](uint64_t w, int t) { return (w >> (8 * G * t)) & 1; };
    auto page_of = [&](int step) {
        const int blk = block_at(step, lt), page = blk >> a.c.shift;
        const bool in = begin + step * TB + lt < stop && page < a.c.max_pages;
        return in ? a.c.page_table[s * a.c.ld_table + page] : -1;
    };
    // records whose tokens all rows of the wave see, and those whose every token
    // some row of the tile does
    auto seen_by = [&](int step, uint64_t there, uint64_t &clear, bool &full) {
        const int blk = block_at(step, lt), j = blk * kBlock;
        clear = there & __ballot(sees_all(a, wv, blk));
        full = (there & __ballot((j + 31 <= view.last) &
                                 (!a.window | (j > view.first - a.window) | (j + 31 < a.sinks)))) == ~0ull;
    };

    // ---- what a wave holds of the step after the next: one piece of the K codes
    // (1 KB: D = 128 16 tokens, D = 64 32) and one of the V codes (32 tokens of
    // 64 columns) ----
    const int pt = wave / G, pc = wave % G; // their record and piece
    u32x4 kraw, vraw, vs, vb, kx, vx;
    uint32_t ks[4];
    auto fetch = [&](int step, int page, uint64_t &there) {
        const bool in = page >= 0 && page < a.c.n_pages;
        there = __ballot(in);
        const int64_t at = page * a.c.page_bytes + head * a.c.head_bytes +
                           (int64_t)(block_at(step, lt) & ((1 << a.c.shift) - 1)) * record_bytes(D);
        kraw = vraw = vs = vb = kx = vx = u32x4{0, 0, 0, 0};
        ks[0] = ks[1] = ks[2] = ks[3] = 0;
        if (bit(there, pt)) {
            const uint32_t lo32 = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)at, 8 * G * pt);
            const uint32_t hi32 = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(at >> 32), 8 * G * pt);
            const char *own = a.c.pages + (int64_t)((uint64_t)hi32 << 32 | lo32);
            const u32x4 *p = reinterpret_cast<const u32x4 *>(own);
            kraw = p[pc * 64 + lane];
            vraw = p[D + pc * 64 + lane];
            const u32x4 *g = p + 2 * D + pc * 16 + (lane >> 4);
            vs = g[8];
            vb = g[12];
            // D = 128: both groups of one token; D = 64: two tokens of one group
            const int tk = lane & 15;
            const uint16_t *sc = reinterpret_cast<const uint16_t *>(own + 32 * D) + (tk >> 2) * 8 +
                                 (tk & 3) + (D == 128 ? pc * 4 : 0);
            constexpr int kSecond = D == 128 ? 128 : 4;
            ks[0] = sc[0];
            ks[1] = sc[32];
            ks[2] = sc[kSecond];
            ks[3] = sc[kSecond + 32];
        }
        // scales and biases of all the step's tokens, 8 a lane
        if (in) {
            const u32x4 *p = reinterpret_cast<const u32x4 *>(a.c.pages + at + 32 * D + (lane >> 3) % G * 256) +
                             (lane & 7);
            kx = p[0];
            vx = p[8];
        }
    };
    // exponents of the step's K and V: all |values| < 2^(e + 15)
    auto exponents = [&](int step, bool full, int &ek, int &ev, bool &bad) {
        u32x4 k = kx & 0x7FFF7FFFu, v = vx & 0x7FFF7FFFu;
        if (!full) {
            rare();
            const int j = block_at(step, lt) * kBlock + (lane & 3) * 4;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t drop = any_sees(j + (e >> 2) * 16 + (e & 3)) ? 0u : (e & 1 ? 0xFFFF0000u : 0xFFFFu);
                k[e >> 1] &= ~drop;
                v[e >> 1] &= ~drop;
            }
        }
        auto reduce = [&]() {
            const uint32_t mk = pk_max(pk_max(k[0], k[1]), pk_max(k[2], k[3]));
            const uint32_t mv = pk_max(pk_max(v[0], v[1]), pk_max(v[2], v[3]));
            const uint32_t a1 = (mk & 0xFFFFu) > (mk >> 16) ? mk & 0xFFFFu : mk >> 16;
            const uint32_t b1 = (mv & 0xFFFFu) > (mv >> 16) ? mv & 0xFFFFu : mv >> 16;
            uint32_t both = a1 | b1 << 16;
            both += (lane & 7) < 4 ? 0x02000200u : 0u; // 16 |s|
            return wave_pk_max(both);
        };
        uint32_t both = reduce();
        bad = false;
        if ((both & 0xFFFFu) >= 0x7F80u || (both >> 16) >= 0x7F80u) {
            // values that are not finite say nothing of the others'
            rare();
            bool off = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t half = e & 1 ? 0xFFFF0000u : 0xFFFFu, inf = 0x7F807F80u & half;
                off = off | ((v[e >> 1] & half) >= inf);
                k[e >> 1] = (k[e >> 1] & half) >= inf ? k[e >> 1] & ~half : k[e >> 1];
                v[e >> 1] = (v[e >> 1] & half) >= inf ? v[e >> 1] & ~half : v[e >> 1];
            }
            bad = __any(off);
            both = reduce();
        }
        ek = (int)((both & 0xFFFFu) >> 7) - 127 - 13;
        ev = (int)(both >> 23) - 127 - 13;
    };

    auto expand_k = [&](int step, bool full, int ek, char *buf) {
        const int tk = lane & 15;
        f16x2 sk[2], bk[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            uint32_t sw = ks[2 * d], bw = ks[2 * d + 1];
            if (!full) {
                rare();
                // D = 128: group d of token 16 pc + tk; D = 64: token 16 d + tk
                const bool ok = any_sees(block_at(step, pt) * kBlock + 16 * (D == 128 ? pc : d) + tk);
                sw = ok ? sw : 0u;
                bw = ok ? bw : 0u;
            }
            const _Float16 x = (_Float16)ldexpf(bf16_lo(sw), -ek), y = (_Float16)ldexpf(bf16_lo(bw), -ek);
            sk[d] = f16x2{x, x};
            bk[d] = f16x2{y, y};
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int d = D == 128 ? k / 2 : k / W; // group; token half
            const int ww = D == 128 ? k : k % W, uu = D == 128 ? pc : k / W;
            f16x2 cd[4];
            codes16(kraw[k], cd);
            u32x4 out;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(cd[j], sk[d], bk[d]));
            const int tok = pt * 32 + uu * 16 + tk, chunk = 4 * ww + (lane >> 4);
            *reinterpret_cast<u32x4 *>(buf + piece_at<KROW>(tok, chunk)) = out;
        }
    };
    auto expand_v = [&](int step, bool plain, int ev, char *buf) {
        u32x4 sw = vs, bw = vb;
        if (!plain) {
            rare();
            // what no row sees, and what is not finite (its rows are marked
            // instead), must not meet a probability of zero
            const int blk = block_at(step, pt);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t half = e & 1 ? 0xFFFF0000u : 0xFFFFu, inf = 0x7F807F80u & half;
                const int tok = blk * kBlock + (e >> 2) * 16 + (lane >> 4) * 4 + (e & 3);
                const bool ok = any_sees(tok) & ((sw[e >> 1] & inf) != inf) & ((bw[e >> 1] & inf) != inf);
                sw[e >> 1] = ok ? sw[e >> 1] : sw[e >> 1] & ~half;
                bw[e >> 1] = ok ? bw[e >> 1] : bw[e >> 1] & ~half;
            }
        }
        f16x2 sv[4], bv[4];
        auto scaled = [&](float x) { return (_Float16)ldexpf(x, -ev); };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sv[j] = f16x2{scaled(bf16_lo(sw[j])), scaled(bf16_hi(sw[j]))};
            bv[j] = f16x2{scaled(bf16_lo(bw[j])), scaled(bf16_hi(bw[j]))};
        }
        const int g = lane >> 4; // tokens 4 g ..: operand half h = g % 2, place g / 2
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int col = (pc * 4 + k) * 16 + (lane & 15);
            f16x2 cd[4];
            codes16(vraw[k], cd);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                cd[j] = __builtin_elementwise_fma(cd[j], sv[j], bv[j]);
#pragma unroll
            for (int kap = 0; kap < 2; ++kap) {
                const int chunk = pt * 4 + kap * 2 + (g & 1);
                *reinterpret_cast<u32x2 *>(buf + piece_at<VROW>(col, chunk) + (g >> 1) * 8) =
                    u32x2{__builtin_bit_cast(uint32_t, cd[2 * kap]),
                          __builtin_bit_cast(uint32_t, cd[2 * kap + 1])};
            }
        }
    };

    // ---- the products of a record ----
    constexpr int HS = ST / 2; // half of a record's K operands, in registers at a time
    auto read_k = [&](const char *buf, int t, int half, f16x8 (&k)[HS]) {
#pragma unroll
        for (int st = 0; st < HS; ++st)
            k[st] = *reinterpret_cast<const f16x8 *>(buf + t * 32 * KROW +
                                                     piece_at<KROW>(c, 2 * (half * HS + st) + h));
    };
    auto read_v = [&](const char *buf, int t, int kap, f16x8 (&v)[DT]) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
            v[d] = *reinterpret_cast<const f16x8 *>(buf + d * 32 * VROW +
                                                    piece_at<VROW>(c, t * 4 + kap * 2 + h));
    };
    auto logits = [&](const f16x8 (&k)[HS], int half, f32x16 &x) {
#pragma unroll
        for (int st = 0; st < HS; ++st)
            x = half + st == 0 ? mfma32(k[st], qr[0], f32x16{}) : mfma32(k[st], qr[half * HS + st], x);
    };
    // logits of tokens that a row does not see: -inf
    auto mask = [&](int step, int t, uint64_t there, uint64_t clear, f32x16 &x) {
        if (bit(clear, t))
            return;
        rare();
        const int blk = block_at(step, t);
        const bool here = bit(there, t);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int j = blk * kBlock + 8 * (r >> 2) + 4 * h + (r & 3);
            x[r] = here && sees(a, pos, lo, j) ? x[r] : -__builtin_inff();
        }
    };
    auto probabilities = [&](const f32x16 &x, float f, f16x8 (&p)[2]) {
        const float ref = kProbScale - m;
        float t = 0.f;
        const f16x2 one = {(_Float16)1.f, (_Float16)1.f};
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
            const f16x2 w = {(_Float16)exp2_fast(fmaf(x[r], f, ref)),
                             (_Float16)exp2_fast(fmaf(x[r + 1], f, ref))};
            p[r >> 3][r & 7] = w[0];
            p[r >> 3][(r & 7) + 1] = w[1];
            t = __builtin_amdgcn_fdot2(w, one, t, false);
        }
        return t;
    };
    auto raise = [&](const f32x16 &x, float f) { // the reference to the maximum
        float top = x[0];
#pragma unroll
        for (int r = 1; r < 16; ++r)
            top = fmaxf(top, x[r]);
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float to = fmaxf(m, top * f), g = exp2_fast(m - to);
        m = to;
        l *= g;
#pragma unroll
        for (int t = 0; t < DT; ++t)
            o[t] *= g;
    };

    // ---- the walk ----
    uint64_t there = 0, there1 = 0, clear = 0, clear1 = 0; // of this step, the next
    int ek = 0, ev = 0, ek1 = 0, ev1 = 0, page = -1;
    bool bad = false, bad1 = false, full1 = false;
    f32x16 x[2];
    if (steps > 0) {
        bool full;
        const int page0 = page_of(0), page1 = page_of(1);
        page = page_of(2);
        fetch(0, page0, there);
        seen_by(0, there, clear, full);
        exponents(0, full, ek, ev, bad);
        expand_k(0, full, ek, lds);
        expand_v(0, full && !bad, ev, lds + 2 * BUF);
        fetch(1, page1, there1);
        __syncthreads();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f16x8 k[HS];
            read_k(lds, 0, half, k);
            logits(k, half, x[0]);
        }
        mask(0, 0, there, clear, x[0]);
    }
    for (int step = 0; step < steps; ++step) {
        char *kb = lds + (step & 1) * BUF, *vbuf = lds + (2 + (step & 1)) * BUF;
        char *kb1 = lds + (~step & 1) * BUF, *vb1 = lds + (2 + (~step & 1)) * BUF;
        // not 0: it meets infinities
        const float f = fmaxf(ldexpf(fabsf(a.scale), qe + ek), 1.17549435e-38f);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            f32x16 &now = x[t & 1], &then = x[~t & 1];
            const char *kn = t + 1 < TB ? kb : kb1;
            const int tn = (t + 1) % TB;
            f16x8 k0[HS], k1[HS], v0[DT], v1[DT], p[2];
            read_k(kn, tn, 0, k0);
            fence();
            float sum = probabilities(now, f, p);
            if (__any(!(sum < kProbMost))) {
                raise(now, f);
                sum = probabilities(now, f, p);
            }
            l += sum;
            read_k(kn, tn, 1, k1);
            fence();
            logits(k0, 0, then);
            read_v(vbuf, t, 0, v0);
            fence();
            logits(k1, 1, then);
            read_v(vbuf, t, 1, v1);
            fence();
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[d] = mfma32(v0[d], p[0], o[d]);
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[d] = mfma32(v1[d], p[1], o[d]);
            if (t == TB - 2) {
                seen_by(step + 1, there1, clear1, full1);
                exponents(step + 1, full1, ek1, ev1, bad1);
                ev1 = ev1 > ev ? ev1 : ev;
                expand_k(step + 1, full1, ek1, kb1);
                __syncthreads();
            } else if (t == TB - 1) {
                expand_v(step + 1, full1 && !bad1, ev1, vb1);
                __syncthreads();
            }
            if (t + 1 < TB)
                mask(step, t + 1, there, clear, then);
            else
                mask(step + 1, 0, there1, clear1, then);
        }
        if (bad && !idle) // rare: which rows see a V that is not finite, and in which group
            for (int t = 0; t < TB; ++t) {
                const int blk = block_at(step, t);
                const char *rec = bit(there, t) ? record_of(a.c, s, head, blk, record_bytes(D)) : nullptr;
                if (!rec)
                    continue;
                for (int e = 0; e < 32 * G; ++e) {
                    const int tok = e & 31, g = e >> 5;
                    const uint16_t *sc = reinterpret_cast<const uint16_t *>(rec + 32 * D) + g * 128 + 64 +
                                         ((tok & 15) >> 2) * 8 + (tok >> 4) * 4 + (tok & 3);
                    if (((sc[0] & 0x7F80u) == 0x7F80u || (sc[32] & 0x7F80u) == 0x7F80u) &&
                        sees(a, pos, lo, blk * kBlock + tok))
                        taint |= 1u << g;
                }
            }
        if (ev1 != ev) {
            const float g = ldexpf(1.f, ev - ev1);
#pragma unroll
            for (int t = 0; t < DT; ++t)
                o[t] *= g;
        }
        ek = ek1;
        ev = ev1;
        bad = bad1;
        there = there1;
        clear = clear1;
        fetch(step + 2, page, there1);
        page = page_of(step + 3);
    }

    l += __shfl_xor(l, 32, 64);
    if (!live)
        return;
    const float inv = a.splits > 1 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
    const int64_t slot = ((int64_t)unit * a.splits + split) * kRows + mine;
    if (a.splits > 1 && h == 0) {
        a.part_ml[2 * slot] = m;
        a.part_ml[2 * slot + 1] = l;
    }
    auto each = [&](auto put) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                f32x4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    v[r] = ldexpf(o[d][4 * r4 + r] * inv, ev);
                    v[r] = (taint >> (d / 2)) & 1 ? __builtin_nanf("") : v[r];
                }
                put(d * 32 + 8 * r4 + 4 * h, v);
            }
    };
    const int64_t at = (int64_t)(q.row0 + i) * a.ldo + hq * a.o_head;
    if (a.splits > 1)
        each([&](int col, f32x4 v) { *reinterpret_cast<f32x4 *>(a.part + slot * D + col) = v; });
    else if (a.o_bf16)
        each([&](int col, f32x4 v) {
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.O) + at + col) =
                u32x2{pack_pair(v[0], v[1]), pack_pair(v[2], v[3])};
        });
    else
        each([&](int col, f32x4 v) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.O) + at + col) = v;
        });
}

} // namespace

// K and V of two steps.
constexpr int kPromptLds = 4 * 32768;

hipError_t launch_attend_prompt(int head_dim, const AttendArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.c.n_seqs * a.c.n_kv_heads * a.tiles * a.splits));
    const void *f = head_dim == 64 ? reinterpret_cast<const void *>(attend_prompt_kernel<64>)
                                   : reinterpret_cast<const void *>(attend_prompt_kernel<128>);
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kPromptLds);
    if (e != hipSuccess)
        return e;
    if (head_dim == 64)
        hipLaunchKernelGGL(attend_prompt_kernel<64>, grid, dim3(64 * kWaves), kPromptLds, stream, a);
    else
        hipLaunchKernelGGL(attend_prompt_kernel<128>, grid, dim3(64 * kWaves), kPromptLds, stream, a);
    return hipGetLastError();
}

} // namespace tsl
