// Attention of query rows over the paged 4-bit cache, for many rows a sequence
// (prompts and their chunks): the same pass over the tokens as attend.hip, with
// each expanded token shared by up to 128 query rows.
//
// A workgroup takes 128 query rows of one sequence and K/V head (32 a wave) and
// walks the records they see.  S^T = K Q^T and O^T = V^T P^T on 32x32x16 MFMAs, so
// a lane holds one query row (column l % 32) throughout and the probabilities
// leave S^T as O^T's operand.  The logits of a record are multiplied while the
// exponentials of the one before it are formed.  Two workgroups share a CU, so
// that one reads Q and writes O beside the other's products (256 rows, one a CU:
// prompts of 2500 tokens 264 us, so 247).
//
// With three tiles of rows or more, and enough records to be worth a launch,
// attend_images expands the records of a sequence once for all of them, to the two products' operands as they are read;
// a workgroup copies them into four stages of LDS (global_load_lds), two ahead.
// A 4-bit cache's operands are 3.6 times its bytes, but every tile reads them
// again out of the L2, and expanding them there had been 29% of the time (a chunk
// of 512 rows after 16000 tokens, 32 heads over 4 of 128: 189 us that way, 153 us
// so, 890 TFLOP/s where a large library product reaches 1220).  What is left is
// bound by the matrix and the vector units, which overlap in part: of 158 us, 138
// were left without the softmax, 139 without the operands' reads, 148 without the
// copies, 119 of the products alone.
// With fewer tiles, or where there is no room for the images, the codes of the
// next TB records, in registers since the step before, are expanded into one half
// of LDS while the other half is multiplied.
//
// Binary16 has 11 bits where bf16 has 8: a bf16 K would move a logit by 2^-9 of
// its terms, which the exponential passes on to the result at the size of the
// result's own rounding.  Its range is met with powers of two, as the 4-bit
// GEMM's is: a row of Q by its largest element, the K and the V values of the
// records in hand by a bound of theirs (15 |s| + |b|); the accumulators follow
// V's, each row's as far down as what it holds allows (2^-90 of a value that it
// gave weight to); what is left between them the probabilities take.  Few neighbours
// differ: images have even exponents, and one step below is left to the
// probabilities.  Values keep their 11 bits 22 octaves below the largest of a
// record, or of a step's records.
// Probabilities are 2^9 times their value relative to the running reference,
// which moves only when a sum of 16 of them comes to 65000 (above 2^-23 of the
// largest they keep their 11 bits, above 2^-31 some): the common step looks for no
// maximum.  The row's sum is of the rounded ones, in binary32, so that the weights of
// a row add up to 1.
#include "attn.hpp"
#include "gemm_common.hpp"

namespace tsl {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kProbScale = 9.f;     // log2
constexpr float kProbMost = 65000.f;  // of a lane's 16 probabilities together: binary16 holds each
constexpr int kWaves = 4; // a workgroup's; two share a CU
constexpr int kRows = 32 * kWaves;
static_assert(kRows == kPromptRows, "rows of a tile");

// 4-bit word -> four pairs of binary16 sixteenths of codes (0 .. 15 / 16, exact): 64
// + c / 16 has c in its low mantissa bits, 64 + c four bits up.  They meet 16 s, which
// keeps its bits in binary16 four octaves further down than s.
__device__ __forceinline__ void codes16(uint32_t w, f16x2 (&c)[4]) {
    uint32_t lo, hi, o;
    asm("v_mov_b32 %0, 0x000f000f" : "=v"(lo));
    asm("v_mov_b32 %0, 0x00f000f0" : "=v"(hi));
    asm("s_mov_b32 %0, 0x54005400" : "=s"(o));
    const uint32_t w8 = w >> 8;
    const f16x2 base = {(_Float16)-64.f, (_Float16)-64.f};
    const f16x2 base16 = {(_Float16)-4.f, (_Float16)-4.f};
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

// Clears what `drop` names of eight bf16.
template <typename F> __device__ __forceinline__ void drop_where(u32x4 &w, F drop) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w[e >> 1] &= drop(e) ? ~(e & 1 ? 0xFFFF0000u : 0xFFFFu) : 0xFFFFFFFFu;
}

// Exponents of K and V values, all |15 s| + |b| < 2^(e + 15), from scales and biases
// (|.|, eight a lane; lanes l % 8 < 4 hold scales); `bad`: some of V's are not finite.
__device__ __forceinline__ void bounds(u32x4 k, u32x4 v, int lane, int &ek, int &ev, bool &bad) {
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
}

template <int D, bool IMAGES>
__global__ void __launch_bounds__(64 * kWaves, 2) attend_prompt_kernel(AttendArgs a) {
    constexpr int G = D / 64, W = D / 32, ST = D / 16, DT = D / 32;
    constexpr int TB = kWaves / G;                    // records of a step
    constexpr int KROW = D * 2, VROW = 64 * TB;       // bytes of a token, of a column
    constexpr int BUF = 32 * TB * KROW;               // 16 KB: K, or V, of a step
    __shared__ __attribute__((aligned(1024))) char lds[4 * BUF]; // K, K, V, V; or four stages of images

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, h = lane >> 5;

    PromptTile at;
    if (!prompt_tile(a, blockIdx.x, true, at))
        return;
    const int s = at.s, head = at.head, tile = at.tile, splits = at.splits;
    const SeqRows q = at.q;
    const int rows = rows_of(a, q) - tile * kRows;
    const int start = q.ctx - q.n;
    const int last_rho = tile * kRows + (rows < kRows ? rows : kRows) - 1;
    TileView view = view_of(a, q, tile, kRows, rows);
    divide(a, splits, view);
    const int begin = at.split * view.share;
    const int stop = begin + view.share < view.count ? begin + view.share : view.count;
    if (begin >= stop && at.split > 0)
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
    // Eight lanes (times G) look after a record: its page, loaded a step before
    // its codes, and who sees it.  Bit 8 G t of a mask is record t's; the upper
    // half of the lanes looks after none.
    const int lt = (lane >> 3) / G;
    auto bit = [](uint64_t w, int t) { return (w >> (8 * G * t)) & 1; };
    auto page_of = [&](int step) {
        const int blk = block_at(step, lt), page = blk >> a.c.shift;
        const bool in = lt < TB && begin + step * TB + lt < stop && page < a.c.max_pages;
        return in ? a.c.page_table[s * a.c.ld_table + page] : -1;
    };
    // records whose tokens all rows of the wave see, and those whose every token
    // some row of the tile does
    auto seen_by = [&](int step, uint64_t there, uint64_t &clear, bool &full) {
        const int blk = block_at(step, lt);
        clear = there & __ballot(sees_all(a, wv, blk));
        full = (there & __ballot(any_sees_all(a, view, blk))) == (1ull << 8 * kWaves) - 1;
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
    auto exponents = [&](int step, bool full, int &ek, int &ev, bool &bad) {
        u32x4 k = kx & 0x7FFF7FFFu, v = vx & 0x7FFF7FFFu;
        if (!full) {
            rare();
            const int j = block_at(step, lt) * kBlock + (lane & 3) * 4;
            auto unseen = [&](int e) { return !any_sees(a, view, j + (e >> 2) * 16 + (e & 3)); };
            drop_where(k, unseen);
            drop_where(v, unseen);
        }
        bounds(k, v, lane, ek, ev, bad);
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
                const bool ok = any_sees(a, view, block_at(step, pt) * kBlock + 16 * (D == 128 ? pc : d) + tk);
                sw = ok ? sw : 0u;
                bw = ok ? bw : 0u;
            }
            const _Float16 x = (_Float16)ldexpf(bf16_lo(sw), 4 - ek), y = (_Float16)ldexpf(bf16_lo(bw), -ek);
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
            // what no row of the tile sees, and what is not finite (its rows are marked
            // instead), must not meet a probability of zero
            const int tok = block_at(step, pt) * kBlock + (lane >> 4) * 4;
            const u32x4 s0 = sw, b0 = bw;
            auto out = [&](int e) {
                const uint32_t inf = e & 1 ? 0x7F800000u : 0x7F80u;
                return !any_sees(a, view, tok + (e >> 2) * 16 + (e & 3)) | ((s0[e >> 1] & inf) == inf) |
                       ((b0[e >> 1] & inf) == inf);
            };
            drop_where(sw, out);
            drop_where(bw, out);
        }
        f16x2 sv[4], bv[4];
        auto scaled = [&](float x, int e) { return (_Float16)ldexpf(x, e); };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sv[j] = f16x2{scaled(bf16_lo(sw[j]), 4 - ev), scaled(bf16_hi(sw[j]), 4 - ev)};
            bv[j] = f16x2{scaled(bf16_lo(bw[j]), -ev), scaled(bf16_hi(bw[j]), -ev)};
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
    auto mask_record = [&](int blk, bool here, f32x16 &x) {
        rare();
        // bits of the record's tokens: those below n
        const int j = blk * kBlock;
        auto below = [&](int n) { return n - j >= 32 ? ~0u : n > j ? (1u << (n - j)) - 1 : 0u; };
        const uint32_t seen = (here ? below(pos + 1) & (~below(lo) | below(a.sinks)) : 0u) >> 4 * h;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int keep = (int)(seen << (31 - (8 * (r >> 2) + (r & 3)))) >> 31;
            x[r] = __uint_as_float((__float_as_uint(x[r]) & keep) | (0xFF800000u & ~keep));
        }
    };
    auto mask = [&](int step, int t, uint64_t there, uint64_t clear, f32x16 &x) {
        if (!bit(clear, t))
            mask_record(block_at(step, t), bit(there, t), x);
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

    // rare: which rows see a V of the record that is not finite, and in which group
    auto find_taint = [&](int blk) {
        const char *rec = record_of(a.c, s, head, blk, record_bytes(D));
        for (int e = 0; e < 32 * G && rec; ++e) {
            const int tok = e & 31, g = e >> 5;
            const uint16_t *sc = reinterpret_cast<const uint16_t *>(rec + 32 * D) + g * 128 + 64 +
                                 ((tok & 15) >> 2) * 8 + (tok >> 4) * 4 + (tok & 3);
            if (((sc[0] & 0x7F80u) == 0x7F80u || (sc[32] & 0x7F80u) == 0x7F80u) &&
                sees(a, pos, lo, blk * kBlock + tok))
                taint |= 1u << g;
        }
    };
    int ev = 0; // the row's accumulators' exponent
    // ... becomes that of a record's values, or as near as leaves what is there below
    // 2^100 (a row may hold larger values, or have passed over them without weight:
    // behind the reference's moves); the probabilities take what is left between the two
    auto follow = [&](int to) {
        float big = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                big = fmaxf(big, fabsf(o[d][r]));
        big = fmaxf(big, __shfl_xor(big, 32, 64));
        const int low = ev + __builtin_amdgcn_frexp_expf(big) - 100;
        to = to > low || big == 0.f ? to : low;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                o[d][r] = ldexpf(o[d][r], ev - to);
        ev = to;
    };
    auto meet = [&](int e, f16x8 (&p)[2]) {
        rare();
        if (__any(e > ev || e < ev - 2))
            follow(e);
        const _Float16 g = (_Float16)ldexpf(1.f, e - ev);
        p[0] *= g;
        p[1] *= g;
    };

    // ---- the walk over images ----
    const TileView all = IMAGES ? sequence_view(a, q) : view;
    const bool laid_out = IMAGES && at.rank < a.image_seqs && all.count <= a.image_records;
    if (laid_out && steps > 0) {
        constexpr int PER = TB / 2, IMG = 128 * D, STAGE = BUF, SLOTS = 4; // records of a stage
        const int count = stop - begin, stages = (count + PER - 1) / PER;
        const int64_t base = (int64_t)(at.rank * a.c.n_kv_heads + head) * a.image_records;
        auto image_of = [&](int n) {
            return place_of(all, view_block(view, begin + n));
        };
        const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
        auto copy = [&](int st) { // the wave's 4 KB of a stage
            const int n = st * PER + wave * 4096 / IMG;
            const char *from = a.images + (base + image_of(n < count ? n : count - 1)) * IMG + (wave * 4096) % IMG;
            from = reinterpret_cast<const char *>(
                (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint64_t)from) |
                (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)((uint64_t)from >> 32)) << 32);
            const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane(
                (int)(lds0 + (st % SLOTS) * STAGE + wave * 4096));
#pragma unroll
            for (int p = 0; p < 4; ++p)
                dma16(from + p * 1024, (uint32_t)lane * 16, to + p * 1024);
        };
        // the stage is there for all waves; two more are on their way
        auto arrive = [&](int st) {
            if (st + 1 < stages)
                wait_vmcnt<4>();
            else
                wait_vmcnt<0>();
            barrier();
            if (st + 2 < stages)
                copy(st + 2);
        };
        uint32_t words = 0; // exponents and flags of 64 records, one a lane
        uint64_t clear = 0;
        auto look_up = [&](int n) {
            const int k = n + lane;
            words = k < count ? a.image_info[base + image_of(k)] : 0;
            clear = __ballot(((words >> 21) & 1) & sees_all(a, wv, view_block(view, begin + k)));
        };
        auto word_of = [&](int n) { return (uint32_t)__builtin_amdgcn_readlane((int)words, n & 63); };
        auto image = [&](int n) { return lds + (n / PER % SLOTS) * STAGE + (n % PER) * IMG + lane * 16; };
        auto read_k = [&](const char *img, int half, f16x8 (&k)[HS]) {
#pragma unroll
            for (int st = 0; st < HS; ++st)
                k[st] = *reinterpret_cast<const f16x8 *>(img + (half * HS + st) * 1024);
        };
        auto read_v = [&](const char *img, int kap, f16x8 (&v)[DT]) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
                v[d] = *reinterpret_cast<const f16x8 *>(img + 64 * D + (2 * d + kap) * 1024);
        };
        f32x16 x[2];
        look_up(0);
        copy(0);
        if (stages > 1)
            copy(1);
        uint32_t word = word_of(0);
        ev = (int)(word >> 10 & 1023) - 256;
        arrive(0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f16x8 k[HS];
            read_k(image(0), half, k);
            logits(k, half, x[0]);
        }
        if (!(clear & 1))
            mask_record(view_block(view, begin), word >> 21 & 1, x[0]);
        for (int n0 = 0; n0 < count; n0 += 2) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int n = n0 + t;
                if (t && n >= count)
                    break;
                f32x16 &now = x[t], &then = x[t ^ 1];
                if ((n + 1) % PER == 0 && n + 1 < count)
                    arrive((n + 1) / PER);
                const int ek = (int)(word & 1023) - 256, er = (int)(word >> 10 & 1023) - 256;
                const float f = fmaxf(ldexpf(fabsf(a.scale), qe + ek), 1.17549435e-38f);
                f16x8 k0[HS], k1[HS], v0[DT], v1[DT], p[2];
                read_k(image(n + 1), 0, k0);
                fence();
                float sum = probabilities(now, f, p);
                read_k(image(n + 1), 1, k1);
                fence();
                logits(k0, 0, then);
                read_v(image(n), 0, v0);
                fence();
                logits(k1, 1, then);
                read_v(image(n), 1, v1);
                fence();
                if (__any(!(sum < kProbMost))) {
                    raise(now, f);
                    sum = probabilities(now, f, p);
                }
                l += sum;
                if (__any(er != ev))
                    meet(er, p);
                if (word >> 20 & 1 && !idle)
                    find_taint(view_block(view, begin + n));
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = mfma32(v0[d], p[0], o[d]);
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = mfma32(v1[d], p[1], o[d]);
                if (((n + 1) & 63) == 0)
                    look_up(n + 1);
                word = word_of(n + 1);
                if (!(clear >> ((n + 1) & 63) & 1))
                    mask_record(view_block(view, begin + n + 1), word >> 21 & 1, then);
            }
        }
    }

    // ---- the walk over codes ----
    if (!laid_out) {
        uint64_t there = 0, there1 = 0, clear = 0, clear1 = 0; // of this step, the next
        int ek = 0, ek1 = 0, er = 0, er1 = 0, page = -1; // er: of the step's values
        bool bad = false, bad1 = false, full1 = false;
        f32x16 x[2];
        if (steps > 0) {
            bool full;
            const int page0 = page_of(0), page1 = page_of(1);
            page = page_of(2);
            fetch(0, page0, there);
            seen_by(0, there, clear, full);
            exponents(0, full, ek, ev, bad);
            er = ev;
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
                if (__any(er != ev))
                    meet(er, p);
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = mfma32(v0[d], p[0], o[d]);
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = mfma32(v1[d], p[1], o[d]);
                if (t == TB - 2) {
                    seen_by(step + 1, there1, clear1, full1);
                    exponents(step + 1, full1, ek1, er1, bad1);
                    expand_k(step + 1, full1, ek1, kb1);
                    __syncthreads();
                } else if (t == TB - 1) {
                    expand_v(step + 1, full1 && !bad1, er1, vb1);
                    __syncthreads();
                }
                if (t + 1 < TB)
                    mask(step, t + 1, there, clear, then);
                else
                    mask(step + 1, 0, there1, clear1, then);
            }
            if (bad && !idle)
                for (int t = 0; t < TB; ++t)
                    if (bit(there, t))
                        find_taint(block_at(step, t));
            ek = ek1;
            er = er1;
            bad = bad1;
            there = there1;
            clear = clear1;
            fetch(step + 2, page, there1);
            page = page_of(step + 3);
        }
    }

    l += __shfl_xor(l, 32, 64);
    if (!live)
        return;
    const float inv = splits > 1 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
    const int64_t slot = (int64_t)blockIdx.x * kRows + mine;
    if (splits > 1 && h == 0) {
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
    // (its place again, rather than in registers through the walk)
    int again = tile * kRows + mine;
    asm volatile("" : "+v"(again));
    const int oi = quotient(again, a.by_group), oh = head * a.group + again - oi * a.group;
    const int64_t to = (int64_t)(q.row0 + oi) * a.ldo + oh * a.o_head;
    if (splits > 1)
        each([&](int col, f32x4 v) { *reinterpret_cast<f32x4 *>(a.part + slot * D + col) = v; });
    else if (a.o_bf16)
        each([&](int col, f32x4 v) {
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.O) + to + col) =
                u32x2{pack_pair(v[0], v[1]), pack_pair(v[2], v[3])};
        });
    else
        each([&](int col, f32x4 v) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.O) + to + col) = v;
        });
}

// One wave expands one record that some row of its sequence sees: K as the
// operands of its first product, ST pieces of 1 KB in the order in which a wave
// reads them (lane 32 h + c holds 8 columns of token c), then V as those of the
// second (column c, 8 tokens), in binary16 by exponents of the record's own (16500
// tokens of 4 heads of 128: 9.6 us for 33 MB, mostly latency).
template <int D> __global__ void __launch_bounds__(256) attend_images_kernel(AttendArgs a) {
    constexpr int G = D / 64, W = D / 32;
    const int lane = threadIdx.x & 63;
    const int at = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int unit = quotient(at, a.by_images), k = at - unit * a.image_records;
    const int rank = quotient(unit, a.by_heads), head = unit - rank * a.c.n_kv_heads;
    int s;
    SeqRows q;
    if (rank >= a.image_seqs || !prompt_of_rank(a, rank, s, q))
        return;
    const TileView all = sequence_view(a, q);
    if (k >= all.count || all.count > a.image_records)
        return;
    const int blk = view_block(all, k);
    const char *rec = record_of(a.c, s, head, blk, record_bytes(D));
    char *img = a.images + (int64_t)at * (128 * D);
    if (!rec) {
        for (int i = lane; i < 8 * D; i += 64)
            reinterpret_cast<u32x4 *>(img)[i] = u32x4{0, 0, 0, 0};
        if (lane == 0)
            a.image_info[at] = 120 | 120 << 10; // (exponents as those of zeros)
        return;
    }
    const u32x4 *p = reinterpret_cast<const u32x4 *>(rec);
    u32x4 kraw[G], vraw[G], vs[G], vb[G], kx = {0, 0, 0, 0}, vx = {0, 0, 0, 0};
    uint32_t ks[G][2][2]; // group, token half, scale and bias
    const int tk = lane & 15, g = lane >> 4;
#pragma unroll
    for (int pc = 0; pc < G; ++pc) {
        kraw[pc] = p[pc * 64 + lane];
        vraw[pc] = p[D + pc * 64 + lane];
        vs[pc] = p[2 * D + pc * 16 + 8 + g];
        vb[pc] = p[2 * D + pc * 16 + 12 + g];
        const uint16_t *sc = reinterpret_cast<const uint16_t *>(rec + 32 * D) + pc * 128 + (tk >> 2) * 8 + (tk & 3);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            ks[pc][u][0] = sc[4 * u];
            ks[pc][u][1] = sc[4 * u + 32];
        }
    }
    if (lane < 8 * G) {
        kx = p[2 * D + (lane >> 3) * 16 + (lane & 7)];
        vx = p[2 * D + (lane >> 3) * 16 + (lane & 7) + 8];
    }
    const bool full = any_sees_all(a, all, blk);
    kx &= 0x7FFF7FFFu;
    vx &= 0x7FFF7FFFu;
    if (!full) {
        const int j = blk * kBlock + (lane & 3) * 4;
        auto unseen = [&](int e) { return !any_sees(a, all, j + (e >> 2) * 16 + (e & 3)); };
        drop_where(kx, unseen);
        drop_where(vx, unseen);
    }
    int ek, ev;
    bool bad;
    bounds(kx, vx, lane, ek, ev, bad);
    ev = (ev + 1) & ~1; // (neighbours differ less often)
    if (lane == 0)
        a.image_info[at] = (uint32_t)(ek + 256) | (uint32_t)(ev + 256) << 10 | (uint32_t)bad << 20 | 1u << 21;
#pragma unroll
    for (int pc = 0; pc < G; ++pc) {
        // K: word n of a lane's four is 8 columns (4 g + 16 .. of 32 ww) of token 16 u + tk
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int at16 = pc * 4 + n, u = at16 / W, ww = at16 % W, tok = 16 * u + tk;
            const bool ok = full || any_sees(a, all, blk * kBlock + tok);
            const uint32_t sw = ok ? ks[ww / 2][u][0] : 0u, bw = ok ? ks[ww / 2][u][1] : 0u;
            const _Float16 x = (_Float16)ldexpf(bf16_lo(sw), 4 - ek), y = (_Float16)ldexpf(bf16_lo(bw), -ek);
            f16x2 cd[4];
            codes16(kraw[pc][n], cd);
            u32x4 out;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(cd[j], f16x2{x, x}, f16x2{y, y}));
            const int chunk = 4 * ww + g;
            *reinterpret_cast<u32x4 *>(img + (chunk >> 1) * 1024 + ((chunk & 1) * 32 + tok) * 16) = out;
        }
        // V: tokens 4 g .. and 16 + 4 g .. of column 16 (4 pc + n) + tk
        u32x4 sw = vs[pc], bw = vb[pc];
        if (!full | bad) {
            const int tok = blk * kBlock + g * 4;
            const u32x4 s0 = sw, b0 = bw;
            auto out = [&](int e) {
                const uint32_t inf = e & 1 ? 0x7F800000u : 0x7F80u;
                return !any_sees(a, all, tok + (e >> 2) * 16 + (e & 3)) | ((s0[e >> 1] & inf) == inf) |
                       ((b0[e >> 1] & inf) == inf);
            };
            drop_where(sw, out);
            drop_where(bw, out);
        }
        f16x2 sv[4], bv[4];
        auto scaled = [&](float v, int e) { return (_Float16)ldexpf(v, e); };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sv[j] = f16x2{scaled(bf16_lo(sw[j]), 4 - ev), scaled(bf16_hi(sw[j]), 4 - ev)};
            bv[j] = f16x2{scaled(bf16_lo(bw[j]), -ev), scaled(bf16_hi(bw[j]), -ev)};
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int col = (pc * 4 + n) * 16 + tk;
            f16x2 cd[4];
            codes16(vraw[pc][n], cd);
            u32x2 half[2]; // of the tokens' two operands
#pragma unroll
            for (int j = 0; j < 4; ++j)
                half[j >> 1][j & 1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(cd[j], sv[j], bv[j]));
            // lanes 32 apart hold the two halves of a lane's 8 tokens: the lower
            // takes those of the first operand, the upper of the second
            const int up = g >> 1;
            const u32x2 mine = up ? half[1] : half[0], give = up ? half[0] : half[1];
            const u32x2 got = {(uint32_t)__shfl_xor((int)give[0], 32, 64), (uint32_t)__shfl_xor((int)give[1], 32, 64)};
            const u32x4 out = up ? u32x4{got[0], got[1], mine[0], mine[1]} : u32x4{mine[0], mine[1], got[0], got[1]};
            *reinterpret_cast<u32x4 *>(img + 64 * D + ((col >> 5) * 2 + up) * 1024 + ((g & 1) * 32 + (col & 31)) * 16) = out;
        }
    }
}

} // namespace

namespace {
template <int D> hipError_t prompt(const AttendArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)a.parts);
    if (a.image_records > 0)
        hipLaunchKernelGGL((attend_prompt_kernel<D, true>), grid, dim3(64 * kWaves), 0, stream, a);
    else
        hipLaunchKernelGGL((attend_prompt_kernel<D, false>), grid, dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}
} // namespace

hipError_t launch_attend_prompt(int head_dim, const AttendArgs &a, hipStream_t stream) {
    return head_dim == 64 ? prompt<64>(a, stream) : prompt<128>(a, stream);
}

hipError_t launch_attend_images(int head_dim, const AttendArgs &a, hipStream_t stream) {
    const int64_t n = (int64_t)a.image_seqs * a.c.n_kv_heads * a.image_records;
    const dim3 grid((unsigned)((n + 3) / 4));
    if (head_dim == 64)
        hipLaunchKernelGGL(attend_images_kernel<64>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(attend_images_kernel<128>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

} // namespace tsl
