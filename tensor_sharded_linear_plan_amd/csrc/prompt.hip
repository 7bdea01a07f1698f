// Attention of query rows over the paged 4-bit cache, for many rows a sequence
// (prompts and their chunks): the same pass over the tokens as attend.hip, with
// each expanded token shared by up to 256 query rows.
//
// A workgroup takes NW x 32 query rows of one sequence and K/V head (32 a wave)
// and walks the records they see, TB at a time: the codes of the next TB
// records, in registers since the step before, are expanded to binary16 into
// one half of LDS while the other half is multiplied.  S^T = K Q^T and
// O^T = V^T P^T on 32x32x16 MFMAs, so a lane holds one query row (column
// l % 32) throughout and the probabilities leave S^T as O^T's operand.
//
// Binary16 has 11 bits where bf16 has 8: a bf16 K would move a logit by 2^-9 of
// its terms, which the exponential passes on to the result at the size of the
// result's own rounding.  Its range is met with powers of two, as the 4-bit
// GEMM's is: a row of Q by its largest element, the K and the V values of the
// records in hand by a bound of theirs (15 |s| + |b|), V's never below that of
// earlier ones, which the accumulators carry.  Probabilities are kept between
// 2^14 and 2^-24, 2^6 times their value relative to the running reference.
#include "attn.hpp"

namespace tsl {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kProbScale = 6.f; // log2

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

template <int D, int NW, int TB>
__global__ void __launch_bounds__(64 * NW, 2) attend_prompt_kernel(AttendArgs a) {
    constexpr int G = D / 64, W = D / 32, CH = D / 64, ST = D / 16, DT = D / 32;
    constexpr int KROW = D * 2, VROW = 64 * TB; // bytes of a token, of a column
    constexpr int KBYTES = 32 * TB * KROW, BUF = 2 * KBYTES;
    constexpr int UNITS = TB * CH; // 1 KB pieces of the K codes (and of the V codes)
    constexpr int PER = 2 * UNITS / NW;
    static_assert(2 * UNITS % NW == 0 && TB * G == 4, "pieces and waves");
    __shared__ __attribute__((aligned(16))) char lds[2 * BUF];
    constexpr int kRows = 32 * NW;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, h = lane >> 5;

    // later tiles see more tokens and start first; neighbouring workgroups take
    // different heads, whose tokens stay in the L2 of one XCD
    int b = blockIdx.x;
    const int split = b % a.splits;
    b /= a.splits;
    const int heads = a.c.n_seqs * a.c.n_kv_heads;
    const int tile = a.tiles - 1 - b / heads;
    b %= heads;
    const int head = b % a.c.n_kv_heads, s = b / a.c.n_kv_heads;
    const int unit = (s * a.c.n_kv_heads + head) * a.tiles + tile;
    const SeqRows q = seq_rows(a.c, s);
    const int n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
    const int rows = n * a.group - tile * kRows;
    if (rows <= 0)
        return;
    const int start = q.ctx - q.n;
    const int last_rho = tile * kRows + (rows < kRows ? rows : kRows) - 1;
    const TileView view = tile_view(a, start + tile * kRows / a.group, start + last_rho / a.group);
    const int begin = split * view.share;
    const int stop = begin + view.share < view.count ? begin + view.share : view.count;
    if (begin >= stop && split > 0)
        return;
    const int steps = begin < stop ? (stop - begin + TB - 1) / TB : 0;

    // the lane's query row and the wave's positions
    const int mine = wave * 32 + c;
    const bool live = mine < rows;
    const int rho = live ? tile * kRows + mine : last_rho;
    const int i = rho / a.group, hq = head * a.group + rho % a.group;
    const int pos = start + i, lo = window_start(a, pos);
    const bool idle = wave * 32 >= rows;
    const int wave_last = wave * 32 + 31 < rows ? tile * kRows + wave * 32 + 31 : last_rho;
    TileView wv = view;
    wv.first = start + (tile * kRows + wave * 32) / a.group;
    wv.last = start + wave_last / a.group;

    // Q as binary16, its largest element in 2^14 .. 2^15
    f16x8 qr[ST];
    int qe;
    {
        const uint16_t *qp = a.Q + (int64_t)(q.row0 + i) * a.ldq + hq * a.q_head + 8 * h;
        u32x4 raw[ST];
        uint32_t top = 0;
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            raw[t] = *reinterpret_cast<const u32x4 *>(qp + 16 * t);
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
    struct Where {
        const char *rec[TB];
        int blk[TB];
    };
    auto locate = [&](int step, Where &w) {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const int r = begin + step * TB + t;
            w.blk[t] = r < stop ? view_block(view, r) : (kMaxContext >> 5) + 1;
            w.rec[t] = r < stop ? record_of(a.c, s, head, w.blk[t], record_bytes(D)) : nullptr;
        }
    };
    // tokens that some row of the tile sees: the others are not read from LDS as
    // anything but zero
    auto any_sees = [&](int j) {
        return j <= view.last && (!a.window || j > view.first - a.window || j < a.sinks);
    };
    auto whole = [&](const Where &w, int t) {
        const int j = w.blk[t] * kBlock;
        return w.rec[t] && j + 31 <= view.last &&
               (!a.window || j > view.first - a.window || j + 31 < a.sinks);
    };

    // ---- what a wave holds of the next step ----
    u32x4 raw[PER];
    u32x4 aux[PER][2]; // V: scales, biases of 8 tokens; K: four 16-bit values
    u32x2 ek_raw, ev_raw;
    auto fetch = [&](const Where &w) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int u = wave + p * NW;
            const bool is_v = u >= UNITS;
            const int t = (is_v ? u - UNITS : u) / CH, ch = (is_v ? u - UNITS : u) % CH;
            const char *rec = nullptr;
#pragma unroll
            for (int k = 0; k < TB; ++k)
                rec = k == t ? w.rec[k] : rec;
            if (!rec)
                continue;
            raw[p] = reinterpret_cast<const u32x4 *>(rec)[(is_v ? D : 0) + ch * 64 + lane];
            const char *sc = rec + 32 * D;
            if (is_v) {
                const u32x4 *g = reinterpret_cast<const u32x4 *>(sc + ch * 256) + (lane >> 4);
                aux[p][0] = g[8];
                aux[p][1] = g[12];
            } else {
                // D = 128: both groups of one token; D = 64: two tokens of one group
                const int tk = lane & 15;
                const uint16_t *g = reinterpret_cast<const uint16_t *>(sc) + (tk >> 2) * 8 + (tk & 3);
                const int o0 = D == 128 ? ch * 4 : 0, o1 = D == 128 ? 128 + ch * 4 : 4;
                aux[p][0] = u32x4{g[o0], g[o0 + 32], g[o1], g[o1 + 32]};
            }
        }
        // scales and biases of all tokens, 4 a lane
        const int part = lane >> 4;
        const char *rec = nullptr;
#pragma unroll
        for (int k = 0; k < TB; ++k)
            rec = k == part / G ? w.rec[k] : rec;
        ek_raw = ev_raw = u32x2{0, 0};
        if (rec) {
            const char *p = rec + 32 * D + part % G * 256 + (lane & 15) * 8;
            ek_raw = *reinterpret_cast<const u32x2 *>(p);
            ev_raw = *reinterpret_cast<const u32x2 *>(p + 128);
        }
    };
    // exponents of the step's K and V: all |values| < 2^(e + 15)
    auto exponents = [&](const Where &w, int &ek, int &ev, bool &bad) {
        u32x2 k = ek_raw & 0x7FFF7FFFu, v = ev_raw & 0x7FFF7FFFu;
        bool part_seen = false;
#pragma unroll
        for (int t = 0; t < TB; ++t)
            part_seen = part_seen || !whole(w, t);
        if (part_seen) {
            int blk = 0;
#pragma unroll
            for (int t = 0; t < TB; ++t)
                blk = t == (lane >> 4) / G ? w.blk[t] : blk;
            const int q8 = lane & 7, j = blk * kBlock + (q8 & 1) * 16 + (q8 >> 1) * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t keep = any_sees(j + e) ? 0u : (e & 1 ? 0xFFFF0000u : 0xFFFFu);
                k[e >> 1] &= ~keep;
                v[e >> 1] &= ~keep;
            }
        }
        auto reduce = [&](u32x2 x, u32x2 y) {
            const uint32_t mx = pk_max(x[0], x[1]), my = pk_max(y[0], y[1]);
            const uint32_t a1 = (mx & 0xFFFFu) > (mx >> 16) ? mx & 0xFFFFu : mx >> 16;
            const uint32_t b1 = (my & 0xFFFFu) > (my >> 16) ? my & 0xFFFFu : my >> 16;
            uint32_t both = a1 | b1 << 16;
            both += (lane & 15) < 8 ? 0x02000200u : 0u; // 16 |s|
#pragma unroll
            for (int o = 1; o < 64; o <<= 1)
                both = pk_max(both, (uint32_t)__shfl_xor((int)both, o, 64));
            return (uint32_t)__builtin_amdgcn_readfirstlane((int)both);
        };
        uint32_t both = reduce(k, v);
        bad = false;
        if ((both & 0xFFFFu) >= 0x7F80u || (both >> 16) >= 0x7F80u) {
            // values that are not finite say nothing of the others'
            bool off = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t half = e & 1 ? 0xFFFF0000u : 0xFFFFu, inf = 0x7F807F80u & half;
                off = off || (v[e >> 1] & half) >= inf;
                k[e >> 1] = (k[e >> 1] & half) >= inf ? k[e >> 1] & ~half : k[e >> 1];
                v[e >> 1] = (v[e >> 1] & half) >= inf ? v[e >> 1] & ~half : v[e >> 1];
            }
            bad = __any(off);
            both = reduce(k, v);
        }
        ek = (int)((both & 0xFFFFu) >> 7) - 127 - 13;
        ev = (int)(both >> 23) - 127 - 13;
    };
    auto expand = [&](const Where &w, int ek, int ev, char *buf) {
        auto half2 = [&](uint32_t bf, int e) { // one bf16 twice
            const _Float16 x = (_Float16)ldexpf(__uint_as_float(bf << 16), -e);
            return f16x2{x, x};
        };
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int u = wave + p * NW;
            const bool is_v = u >= UNITS;
            const int t = (is_v ? u - UNITS : u) / CH, ch = (is_v ? u - UNITS : u) % CH;
            int blk = 0;
            bool full = false, there = false;
#pragma unroll
            for (int k = 0; k < TB; ++k)
                if (k == t) {
                    blk = w.blk[k];
                    full = whole(w, k);
                    there = w.rec[k] != nullptr;
                }
            if (!there)
                raw[p] = u32x4{0, 0, 0, 0};
            if (is_v) {
                f16x2 sv[4], bv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float sc[2], bi[2];
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        sc[d] = d ? bf16_hi(aux[p][0][j]) : bf16_lo(aux[p][0][j]);
                        bi[d] = d ? bf16_hi(aux[p][1][j]) : bf16_lo(aux[p][1][j]);
                        const int e = 2 * j + d;
                        const int tok = blk * kBlock + (e >> 2) * 16 + (lane >> 4) * 4 + (e & 3);
                        // what no row sees, and what is not finite (its rows are
                        // marked instead), must not meet a probability of zero
                        const bool ok = (full || (there && any_sees(tok))) &&
                                        __builtin_isfinite(sc[d]) && __builtin_isfinite(bi[d]);
                        sc[d] = ok ? ldexpf(sc[d], -ev) : 0.f;
                        bi[d] = ok ? ldexpf(bi[d], -ev) : 0.f;
                    }
                    sv[j] = f16x2{(_Float16)sc[0], (_Float16)sc[1]};
                    bv[j] = f16x2{(_Float16)bi[0], (_Float16)bi[1]};
                }
                const int g = lane >> 4; // tokens 4 g ..: operand half h = g % 2, place g / 2
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int col = (ch * 4 + k) * 16 + (lane & 15);
                    f16x2 cd[4];
                    codes16(raw[p][k], cd);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        cd[j] = __builtin_elementwise_fma(cd[j], sv[j], bv[j]);
#pragma unroll
                    for (int kap = 0; kap < 2; ++kap) {
                        const int chunk = t * 4 + kap * 2 + (g & 1);
                        *reinterpret_cast<u32x2 *>(buf + KBYTES + col * VROW +
                                                   ((chunk ^ (col & 7)) << 4) + (g >> 1) * 8) =
                            u32x2{__builtin_bit_cast(uint32_t, cd[2 * kap]),
                                  __builtin_bit_cast(uint32_t, cd[2 * kap + 1])};
                    }
                }
            } else {
                const int tk = lane & 15;
                f16x2 sk[2], bk[2];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    // D = 128: group d of token 16 ch + tk; D = 64: token 16 d + tk
                    const int tok = blk * kBlock + 16 * (D == 128 ? ch : d) + tk;
                    const bool ok = full || (there && any_sees(tok));
                    sk[d] = half2(ok ? aux[p][0][2 * d] : 0u, ek);
                    bk[d] = half2(ok ? aux[p][0][2 * d + 1] : 0u, ek);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int nw = ch * 4 + k, uu = nw / W, ww = nw % W;
                    const int d = D == 128 ? ww / 2 : uu;
                    f16x2 cd[4];
                    codes16(raw[p][k], cd);
                    u32x4 out;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        out[j] = __builtin_bit_cast(uint32_t,
                                                    __builtin_elementwise_fma(cd[j], sk[d], bk[d]));
                    const int tok = t * 32 + uu * 16 + tk, chunk = 4 * ww + (lane >> 4);
                    *reinterpret_cast<u32x4 *>(buf + tok * KROW + ((chunk ^ (tok & 7)) << 4)) = out;
                }
            }
        }
    };

    // ---- the walk ----
    Where cur, nxt, after;
    int ek = 0, ev = -1000, ek_next = 0, ev_next = 0;
    bool bad = false, bad_next = false;
    if (steps > 0) {
        locate(0, cur);
        fetch(cur);
        exponents(cur, ek, ev, bad);
        expand(cur, ek, ev, lds);
        if (steps > 1) {
            locate(1, nxt);
            fetch(nxt);
        }
        if (steps > 2)
            locate(2, after);
    }
    for (int step = 0; step < steps; ++step) {
        char *buf = lds + (step & 1) * BUF;
        __syncthreads();
        int ev_was = ev;
        if (step + 1 < steps) {
            exponents(nxt, ek_next, ev_next, bad_next);
            ev_next = ev_next > ev ? ev_next : ev;
            expand(nxt, ek_next, ev_next, lds + ((step + 1) & 1) * BUF);
        }
        Where later;
        if (step + 2 < steps) {
            fetch(after);
            if (step + 3 < steps)
                locate(step + 3, later);
        }
        (void)ev_was;
        if (!idle) {
            const float f = ldexpf(a.scale, qe + ek);
#pragma unroll
            for (int t0 = 0; t0 < TB; t0 += 2) {
                bool see = false, all = true;
#pragma unroll
                for (int t = t0; t < t0 + 2; ++t) {
                    const int j = cur.blk[t] * kBlock;
                    see = see || (cur.rec[t] && j <= wv.last &&
                                  (!a.window || j + 31 > wv.first - a.window || j < a.sinks));
                    all = all && cur.rec[t] && sees_all(a, wv, cur.blk[t]);
                }
                if (!see)
                    continue;
                f32x16 sa[2];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        sa[t][r] = 0.f;
#pragma unroll
                for (int st = 0; st < ST; ++st)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int tok = (t0 + t) * 32 + c, chunk = 2 * st + h;
                        const f16x8 k = *reinterpret_cast<const f16x8 *>(
                            buf + tok * KROW + ((chunk ^ (tok & 7)) << 4));
                        sa[t] = mfma32(k, qr[st], sa[t]);
                    }
                if (!all) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int j = cur.blk[t0 + t] * kBlock + 8 * (r >> 2) + 4 * h + (r & 3);
                            const bool v = cur.rec[t0 + t] && sees(a, pos, lo, j);
                            // -inf whatever the sign of the scale
                            sa[t][r] = v ? sa[t][r] * f : -__builtin_inff();
                        }
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        sa[t] *= f;
                }
                float top = sa[0][0];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        top = fmaxf(top, sa[t][r]);
                if (__any(top > m + 8.f)) {
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    const float to = fmaxf(m, top), g = exp2_fast(m - to);
                    m = to;
                    l *= g;
#pragma unroll
                    for (int t = 0; t < DT; ++t)
                        o[t] *= g;
                }
                const float ref = m - kProbScale;
                f16x8 pr[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float p = exp2_fast(sa[t][r] - ref);
                        l += p;
                        pr[t][r >> 3][r & 7] = (_Float16)p;
                    }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int kap = 0; kap < 2; ++kap)
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            const int col = d * 32 + c, chunk = (t0 + t) * 4 + kap * 2 + h;
                            const f16x8 v = *reinterpret_cast<const f16x8 *>(
                                buf + KBYTES + col * VROW + ((chunk ^ (col & 7)) << 4));
                            o[d] = mfma32(v, pr[t][kap], o[d]);
                        }
            }
            if (bad) { // rare: which rows see a V that is not finite, and in which group
                for (int t = 0; t < TB; ++t) {
                    const char *rec = nullptr;
                    int blk = 0;
#pragma unroll
                    for (int k = 0; k < TB; ++k)
                        if (k == t) {
                            rec = cur.rec[k];
                            blk = cur.blk[k];
                        }
                    if (!rec)
                        continue;
                    for (int x = 0; x < 32 * G; ++x) {
                        const int tok = x & 31, g = x >> 5;
                        const uint16_t *sc = reinterpret_cast<const uint16_t *>(rec + 32 * D) +
                                             g * 128 + 64 + ((tok & 15) >> 2) * 8 + (tok >> 4) * 4 +
                                             (tok & 3);
                        if (((sc[0] & 0x7F80u) == 0x7F80u || (sc[32] & 0x7F80u) == 0x7F80u) &&
                            sees(a, pos, lo, blk * kBlock + tok))
                            taint |= 1u << g;
                    }
                }
            }
            if (step + 1 < steps && ev_next != ev) {
                const float g = ldexpf(1.f, ev - ev_next < -1000 ? -1000 : ev - ev_next);
#pragma unroll
                for (int t = 0; t < DT; ++t)
                    o[t] *= g;
            }
        }
        ek = ek_next;
        ev = step + 1 < steps ? ev_next : ev;
        bad = bad_next;
        cur = nxt;
        nxt = after;
        after = later;
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
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int col = d * 32 + 8 * r4 + 4 * h;
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                v[r] = ldexpf(o[d][4 * r4 + r] * inv, ev);
                v[r] = (taint >> (d / 2)) & 1 ? __builtin_nanf("") : v[r];
            }
            if (a.splits > 1) {
                *reinterpret_cast<f32x4 *>(a.part + slot * D + col) = v;
            } else {
                const int64_t at = (int64_t)(q.row0 + i) * a.ldo + hq * a.o_head + col;
                if (a.o_bf16)
                    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.O) + at) =
                        u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                else
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.O) + at) = v;
            }
        }
}

} // namespace

hipError_t launch_attend_prompt(int head_dim, int tile_rows, const AttendArgs &a,
                                hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.c.n_seqs * a.c.n_kv_heads * a.tiles * a.splits));
    const dim3 block((unsigned)(tile_rows * 2));
    if (head_dim == 64 && tile_rows == 256)
        hipLaunchKernelGGL((attend_prompt_kernel<64, 8, 4>), grid, block, 0, stream, a);
    else if (head_dim == 64)
        hipLaunchKernelGGL((attend_prompt_kernel<64, 4, 4>), grid, block, 0, stream, a);
    else if (tile_rows == 256)
        hipLaunchKernelGGL((attend_prompt_kernel<128, 8, 2>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((attend_prompt_kernel<128, 4, 2>), grid, block, 0, stream, a);
    return hipGetLastError();
}

} // namespace tsl
