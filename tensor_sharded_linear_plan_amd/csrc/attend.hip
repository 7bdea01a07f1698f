// Attention of query rows over the paged 4-bit cache, for few rows a sequence
// (generated tokens): o_i = sum_j p_ij v_j, p = softmax over the visible j of
// scale q_i . k_j, one pass over the tokens with a running maximum and sum.
//
// A wave takes up to 16 query rows of one sequence and K/V head (the heads that
// share it, of one or several tokens) and walks a range of the records they see.
// All records of a call in a row, tile after tile, are cut into as many equal
// parts as waves fit on the chip, so that sequences of any lengths end together
// and a wave starts once; where a part runs over the end of a tile the wave goes
// on with the next, and attend_join adds what two or more waves have of a tile.
// Waves do not wait for each other: a start, from the first instruction to the
// first product, takes 3 to 5 us, mostly of three reads that follow from each
// other (lengths, page, record).
//
// The products run on 16x16x32 MFMAs, transposed: S^T = K Q^T and O^T = V^T P^T,
// so a lane holds one query row throughout (column l % 16) and the
// probabilities that leave S^T are the registers that O^T takes in.  Codes are
// expanded to the exact bf16 z + c, z an offset that costs no instruction (128; of
// V three times in four 16); a group's scale and bias enter in binary32,
//     q . k = sum_g s_g (q_g . (128 + c_g)) + (b_g - 128 s_g) sum(q_g)
//     o_g   = sum_j (p_j s_jg) (z + c_jg) - sum_j (p_j s_jg) z + sum_j p_j b_jg,
// with p s as a bf16 and what its rounding left as another: 16 bits of it (8 more
// MFMAs a record, in a kernel that waits for memory and the vector units).
//
// The three sums of o_g are some 50 times their result's terms, so each would keep
// a rounding of its own length: every kSettle records they are made one, which is
// then a sum of values.  What is left does not grow with the tokens that a wave
// walks (near-equal weights, normal values, error in the 2-norm relative to the
// result's: 1e-5 to 3e-5 over 8192, 131072 or 500000 tokens in one wave; settled at
// the end alone 1.5e-3 over 8192, 1.2e-2 over 131072).
//
// Records come by direct copies into LDS (global_load_lds), each wave its own
// three stages: two records are on their way while one is multiplied.
//
// One row each of 32 sequences of up to 32767 tokens, 64 / 8 heads of 128: 123 us
// with the join's 6, 4.5 TB/s, the vector units 65% busy; of one of 131000, 28 / 4
// heads, 30 us with the join's 8; of 64 with windows of 4096, heads of 64, 40 us.
#include "attn.hpp"
#include "gemm_common.hpp"

namespace tsl {
namespace {

constexpr int kWaves = 4; // of a workgroup

constexpr int kStages = 3; // 2 .. 4 (the waits below)
constexpr int kSettle = 8; // records between two settlements (a power of two)

// 4-bit word -> four bf16 pairs holding z + c: 128 + c as it lies, and 16 + c with
// the code three bits up, where a shift is needed anyway.
__device__ __forceinline__ bf16x8 v_codes(uint32_t w) {
    uint32_t m0, m1, z0, z1;
    asm("v_mov_b32 %0, 0x000f000f" : "=v"(m0));
    asm("v_mov_b32 %0, 0x00780078" : "=v"(m1));
    asm("s_mov_b32 %0, 0x43004300" : "=s"(z0));
    asm("s_mov_b32 %0, 0x41804180" : "=s"(z1));
    const u32x4 r = {(w & m0) | z0, ((w >> 1) & m1) | z1, ((w >> 5) & m1) | z1, ((w >> 9) & m1) | z1};
    return __builtin_bit_cast(bf16x8, r);
}

// At most N of the wave's copies into LDS are still under way.
template <int N> __device__ __forceinline__ void wait_copies() {
    wait_vmcnt<N>();
    asm volatile("" ::: "memory");
}

// The part of a wave, of all records in a row cut into equal parts: it begins
// `skip` records into sequence s (rows q).  64 sequences at a time (the host lets
// at most kMaxShared share).
struct Part {
    int s, skip, left, per_seq;
    SeqRows q;
};
template <int ROWS> __device__ __forceinline__ Part part_of(const AttendArgs &a, int me) {
    const int lane = threadIdx.x & 63;
    Part part = {0, 0, 0, 0, {0, 0, 0}};
    int total = 0, begin = 0, before = 0;
    bool finding = false;
    for (int base = 0;;) {
        SeqRows q = {0, 0, 0};
        int own = 0;
        if (base + lane < a.c.n_seqs) {
            q = seq_rows(a.c, base + lane);
            int rows = rows_of(a, q);
            for (int t = 0; rows > 0; ++t, rows -= ROWS)
                own += view_of(a, q, t, ROWS, rows).count;
        }
        own *= a.c.n_kv_heads;
        const int upto = wave_scan(own), all = __builtin_amdgcn_readlane(upto, 63);
        if (!finding) {
            total += all;
            base += 64;
            if (base < a.c.n_seqs)
                continue;
            int share = quotient(total + a.parts - 1, a.by_parts);
            share = share > a.min_share ? share : a.min_share;
            if ((int64_t)share * me >= total)
                return part;
            begin = share * me;
            part.left = total - begin < share ? total - begin : share;
            finding = true;
            base = 0;
            if (a.c.n_seqs > 64)
                continue;
        }
        // the first sequence that ends behind the beginning
        const uint64_t past = __ballot(before + upto > begin);
        if (past) {
            const int at = __builtin_ctzll(past);
            part.s = base + at;
            part.per_seq = __builtin_amdgcn_readlane(own, at);
            part.skip = begin - before - (__builtin_amdgcn_readlane(upto, at) - part.per_seq);
            part.q.row0 = __builtin_amdgcn_readlane(q.row0, at);
            part.q.n = __builtin_amdgcn_readlane(q.n, at);
            part.q.ctx = __builtin_amdgcn_readlane(q.ctx, at);
            return part;
        }
        before += all;
        base += 64;
    }
}

// Rotation of the lanes of a row of 16 by 16 / P ... 8, added or compared: what the
// P groups of columns of a row have, in each of them.
template <int P, class F> __device__ __forceinline__ float over_groups(float v, F f) {
    if (P >= 2)
        v = f(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, true)));
    if (P >= 4)
        v = f(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, true)));
    return v;
}

// The 16 columns of a product are P times the tile's 16 / P rows, and a lane keeps
// of each product 8 / P of its tokens: with few rows the vector work on logits and
// probabilities, which is more than half of all, is divided among the columns
// instead of repeated.
template <int D, int P>
__global__ void __launch_bounds__(64 * kWaves, attend_groups(D)) attend_decode_kernel(AttendArgs a) {
    constexpr int G = D / 64, W = D / 32, DT = D / 16, ROWS = 16 / P;
    constexpr int REC = record_bytes(D), PIECES = REC / 16; // 16 bytes a lane
    constexpr int COPIES = (PIECES + 63) / 64, TPL = 8 / P; // tokens of a lane
    __shared__ __attribute__((aligned(16))) char ring[kWaves][kStages * REC]; // a wave's stages
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int own = c / ROWS, cr = c % ROWS; // the lane's tokens of a record, its row

    // Whole: the wave's (sequence, head, tile).  Shared: its part of all records
    // of the call in a row, tiles innermost, then heads, then sequences.
    const int me = blockIdx.x * kWaves + wave;
    int s, head = 0, tile = 0, at = 0; // at: the record of the tile's list to start at
    int left = INT32_MAX;              // records of the part
    SeqRows q;
    if (!a.shared) {
        if (me >= a.units)
            return;
        const int b = quotient(me, a.by_tiles);
        tile = me - b * a.tiles;
        s = quotient(b, a.by_heads);
        head = b - s * a.c.n_kv_heads;
        q = seq_rows(a.c, s);
    } else {
        const Part part = part_of<ROWS>(a, me);
        if (part.left <= 0)
            return;
        s = part.s;
        q = part.q;
        left = part.left;
        // at most 2^10 heads: the quotient is off by at most one
        const int per_head = quotient(part.per_seq, a.by_heads);
        head = __builtin_amdgcn_readfirstlane(
            (int)((float)part.skip * __builtin_amdgcn_rcpf((float)per_head)));
        head -= head * per_head > part.skip;
        head += (head + 1) * per_head <= part.skip;
        at = part.skip - head * per_head;
    }

    auto next_tile = [&] {
        if (++tile == a.tiles) {
            tile = 0;
            if (++head == a.c.n_kv_heads) {
                head = 0;
                q = seq_rows(a.c, ++s);
            }
        }
    };
    while (true) {
        const int unit = (s * a.c.n_kv_heads + head) * a.tiles + tile;
        const int rows = rows_of(a, q) - tile * ROWS; // of this tile and later ones
        TileView view = {0, 0, 0, 0, 0, 0, 0};
        if (rows > 0)
            view = view_of(a, q, tile, ROWS, rows);
        else if (!a.shared)
            return;
        // on to the tile where the part begins, past those without records
        if (a.shared && at >= view.count) {
            at -= view.count;
            next_tile();
            continue;
        }
        const int start = q.ctx - q.n;
        const int begin = at;
        const int stop = view.count - at < left ? view.count : at + left;
        const bool complete = begin == 0 && stop == view.count;

        // the wave's next 64 records, one a lane: where they lie, and as bits which
        // are there and which all rows of the tile see all of
        const int n_mine = stop - begin;
        uint32_t at_lo = 0, at_hi = 0;
        uint64_t there = 0, clear = 0, next_there = 0, next_clear = 0;
        auto look_up = [&](int k0) {
            const int r = begin + k0 + lane;
            const int blk = view_block(view, r);
            const char *rec = r < stop ? record_of(a.c, s, head, blk, REC) : nullptr;
            next_there = __ballot(rec != nullptr);
            next_clear = __ballot(sees_all(a, view, blk));
            // one that is not there is read from page 0, and passed over
            const uint64_t p = reinterpret_cast<uint64_t>(rec ? rec : a.c.pages);
            at_lo = (uint32_t)p;
            at_hi = (uint32_t)(p >> 32);
        };
        const uint32_t lds0 = (uint32_t)(uintptr_t)&ring[wave][0];
        auto issue = [&](int k) { // record k of the wave into its stage
            if ((k & 63) == 0)
                look_up(k);
            const uint64_t p = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)at_hi, k & 63) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((int)at_lo, k & 63);
            const char *rec = reinterpret_cast<const char *>(p);
            const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + (k % kStages) * REC));
#pragma unroll
            for (int i = 0; i < COPIES; ++i)
                if ((i + 1) * 64 <= PIECES || lane < PIECES - i * 64)
                    dma16(rec + i * 1024, (uint32_t)lane * 16, to + i * 1024);
        };
        // the lane's query row
        const bool live = cr < rows;
        const int rho = tile * ROWS + (live ? cr : 0);
        const int i = quotient(rho, a.by_group), hq = head * a.group + rho - i * a.group;
        const int pos = start + i, lo = window_start(a, pos);
        const uint16_t *qp = a.Q + (int64_t)(q.row0 + i) * a.ldq + hq * a.q_head + 8 * g;
        bf16x8 qr[W];
#pragma unroll
        for (int w = 0; w < W; ++w) // the scale's sign goes to Q: the largest product
            qr[w] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(qp + 32 * w) ^
                                                   (a.scale < 0.f ? 0x80008000u : 0u)); // is the largest logit
        const float scale = fmaxf(fabsf(a.scale), 1.17549435e-38f); // not 0: it meets infinities

        f32x4 o[DT], off[G], base[G];
        float ob[G], qsum[G], m = kNoMax, l = 0.f;
        const bf16x8 all128 = __builtin_bit_cast(bf16x8, u32x4{0x43004300u, 0x43004300u, 0x43004300u, 0x43004300u});
        const bf16x8 offsets = __builtin_bit_cast(bf16x8, u32x4{0x43004300u, 0x41804180u, 0x41804180u, 0x41804180u});
#pragma unroll
        for (int t = 0; t < DT; ++t)
            o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < G; ++d) {
            ob[d] = 0.f;
            off[d] = base[d] = f32x4{0.f, 0.f, 0.f, 0.f};
            // -128 sum(q), in every row of the product: what a product begins with
#pragma unroll
            for (int w = 2 * d; w < 2 * d + 2; ++w)
                base[d] = mfma_bf16(all128, qr[w], base[d]);
            base[d] = -base[d];
            qsum[d] = base[d][0] * -0.0078125f;
        }

        auto settle = [&] {
            rare();
#pragma unroll
            for (int d = 0; d < G; ++d) {
                ob[d] += __shfl_xor(ob[d], 16, 64);
                ob[d] += __shfl_xor(ob[d], 32, 64);
#pragma unroll
                for (int t = 4 * d; t < 4 * d + 4; ++t)
                    o[t] = (o[t] - off[d]) + ob[d];
                ob[d] = 0.f;
                off[d] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        };

        // (one place that looks up and copies: cold code is what a start takes long over)
        for (int k = 1 - kStages; k < n_mine; ++k) {
            if (k > 0 && k % kSettle == 0)
                settle();
            if (k + kStages - 1 < n_mine) {
                wait_lgkm0(); // the stage was read
                issue(k + kStages - 1);
                if (k < 0)
                    continue;
                wait_copies<(kStages - 1) * COPIES>();
            } else if (k < 0) {
                continue;
            } else if (kStages > 3 && k + 2 < n_mine) {
                wait_copies<2 * COPIES>();
            } else if (kStages > 2 && k + 1 < n_mine) {
                wait_copies<COPIES>();
            } else {
                wait_copies<0>();
            }
            if ((k & 63) == 0) { // (looked up kStages - 1 records ago)
                there = next_there;
                clear = next_clear;
            }
            if (!(there >> (k & 63) & 1))
                continue;
            const u32x4 *rec = reinterpret_cast<const u32x4 *>(&ring[wave][(k % kStages) * REC]);
            // scales of the lane's tokens, in pairs
            typedef uint32_t pairs __attribute__((ext_vector_type(TPL / 2)));
            auto scales = [&](int d, int kind) {
                const pairs v = *reinterpret_cast<const pairs *>(reinterpret_cast<const char *>(rec + 2 * D) +
                                                                 d * 256 + kind * 64 + g * 16 + own * TPL * 2);
                return v;
            };

            float x[TPL]; // products, the scale not yet in them
#pragma unroll
            for (int d = 0; d < G; ++d) {
                f32x4 acc[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    acc[u] = base[d];
#pragma unroll
                    for (int w = 2 * d; w < 2 * d + 2; ++w) {
                        const int n = u * W + w;
                        acc[u] = mfma_bf16(q4_to_bf16_plus128(rec[(n >> 2) * 64 + lane][n & 3]), qr[w], acc[u]);
                    }
                }
                const pairs ks = scales(d, 0), kb = scales(d, 1);
#pragma unroll
                for (int e = 0; e < TPL; ++e) {
                    float t = acc[e >> 2][e & 3];
                    if (P == 2)
                        t = own ? acc[1][e] : acc[0][e];
                    if (P == 4) {
                        const float lo2 = own & 2 ? acc[1][e] : acc[0][e], hi2 = own & 2 ? acc[1][2 + e] : acc[0][2 + e];
                        t = own & 1 ? hi2 : lo2;
                    }
                    const float s1 = e & 1 ? bf16_hi(ks[e >> 1]) : bf16_lo(ks[e >> 1]);
                    const float b1 = e & 1 ? bf16_hi(kb[e >> 1]) : bf16_lo(kb[e >> 1]);
                    x[e] = d ? fmaf(b1, qsum[d], x[e]) : b1 * qsum[d];
                    x[e] = fmaf(s1, t, x[e]);
                }
            }
            pairs keep; // of the V scales: a hidden token's may be NaN
#pragma unroll
            for (int e = 0; e < TPL / 2; ++e)
                keep[e] = ~0u;
            const bool all = clear >> (k & 63) & 1;
            if (!all) {
                rare();
                const int blk = view_block(view, begin + k);
#pragma unroll
                for (int e = 0; e < TPL; ++e) {
                    const int at = own * TPL + e;
                    const bool v = sees(a, pos, lo, blk * kBlock + (at >> 2) * 16 + g * 4 + (at & 3));
                    x[e] = v ? x[e] : -__builtin_inff();
                    keep[e >> 1] &= v ? ~0u : (e & 1 ? 0xFFFFu : 0xFFFF0000u);
                }
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < TPL; ++e)
                top = fmaxf(top, x[e]);
            top *= scale;
            // the reference exponent follows the maximum at a distance of 2^8:
            // binary32 sums have room for it, and rescaling becomes rare
            if (__any(top > m + 8.f)) {
                rare();
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float to = fmaxf(m, top), f = exp2_fast(m - to);
                m = to;
                l *= f;
#pragma unroll
                for (int t = 0; t < DT; ++t)
                    o[t] *= f;
#pragma unroll
                for (int d = 0; d < G; ++d) {
                    ob[d] *= f;
                    off[d] *= f;
                }
            }
            float pr[TPL];
#pragma unroll
            for (int e = 0; e < TPL; ++e) {
                pr[e] = exp2_fast(fmaf(x[e], scale, -m));
                l += pr[e];
            }
#pragma unroll
            for (int d = 0; d < G; ++d) {
                pairs vs = scales(d, 2), vb = scales(d, 3);
                if (!all) {
                    rare();
                    vs &= keep;
                    vb &= keep;
                }
                u32x4 hi = {0, 0, 0, 0}, rem = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < TPL / 2; ++h) {
                    const float w0 = pr[2 * h] * bf16_lo(vs[h]), w1 = pr[2 * h + 1] * bf16_hi(vs[h]);
                    ob[d] = fmaf(pr[2 * h], bf16_lo(vb[h]), ob[d]);
                    ob[d] = fmaf(pr[2 * h + 1], bf16_hi(vb[h]), ob[d]);
                    const uint32_t p16 = pack_pair(w0, w1);
                    const uint32_t r16 = pack_pair(w0 - bf16_lo(p16), w1 - bf16_hi(p16));
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        hi[k * (TPL / 2) + h] = P == 1 || own == k ? p16 : 0u;
                        rem[k * (TPL / 2) + h] = P == 1 || own == k ? r16 : 0u;
                    }
                }
                const bf16x8 wh = __builtin_bit_cast(bf16x8, hi), wl = __builtin_bit_cast(bf16x8, rem);
                // what z + c has over c: the same products with a tile of z
                off[d] = mfma_bf16(offsets, wh, off[d]);
                off[d] = mfma_bf16(offsets, wl, off[d]);
                const u32x4 vc = rec[D + d * 64 + lane];
#pragma unroll
                for (int t = 4 * d; t < 4 * d + 4; ++t) {
                    const bf16x8 v = v_codes(vc[t & 3]);
                    o[t] = mfma_bf16(v, wh, o[t]);
                    o[t] = mfma_bf16(v, wl, o[t]);
                }
            }
        }

        // join the lanes and columns of a row
        settle();
        {
            auto more = [](float u, float v) { return fmaxf(u, v); };
            auto sum = [](float u, float v) { return u + v; };
            const float top = over_groups<P>(m, more);
            float f = exp2_fast(m - top);
            l += __shfl_xor(l, 16, 64);
            l += __shfl_xor(l, 32, 64);
            l = over_groups<P>(l * f, sum);
            const float inv = !complete ? 1.f : (l == 0.f ? 0.f : 1.f / l);
            const int64_t slot = (int64_t)(begin == 0 ? a.parts + me : me) * ROWS + c;
            const int64_t to = (int64_t)(q.row0 + i) * a.ldo + hq * a.o_head + 4 * g;
            const bool mine = live && !own;
            if (!complete && mine && g == 0) {
                a.part_ml[2 * slot] = top;
                a.part_ml[2 * slot + 1] = l;
            }
#pragma unroll
            for (int d = 0; d < G; ++d) {
#pragma unroll
                for (int t = 4 * d; t < 4 * d + 4; ++t) {
                    f32x4 v = o[t] * f;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = over_groups<P>(v[e], sum) * inv;
                    if (!mine)
                        continue;
                    if (!complete)
                        *reinterpret_cast<f32x4 *>(a.part + slot * D + 16 * t + 4 * g) = v;
                    else if (a.o_bf16)
                        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.O) + to + 16 * t) =
                            u32x2{pack_pair(v[0], v[1]), pack_pair(v[2], v[3])};
                    else
                        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.O) + to + 16 * t) = v;
                }
            }
        }
        if (!a.shared)
            return;
        if (lane == 0) { // for the join: the waves that share the tile
            if (begin == 0)
                a.spans[2 * unit] = me;
            if (stop == view.count)
                a.spans[2 * unit + 1] = me;
        }
        left -= stop - begin;
        if (left <= 0)
            return;
        at = 0;
        next_tile();
    }
}

// The ranges of a row added: by a wave, four rows a workgroup, or where they are
// many by 16 waves and then one over those waves' results.  D / 8 lanes take a
// range, eight columns each, so that a wave has 512 / D ranges at a time, four
// times over; each group of lanes has a running reference as over tokens.  Bound
// by latency, that of instructions not yet in the cache among it: the code is
// short, and walks the ranges and the waves' results in one place.
template <int D, int WPR, bool MANY>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) attend_join_kernel(AttendArgs a, int tile_rows) {
    constexpr int LPR = D / 8, AT_ONCE = 64 / LPR, AHEAD = 4, RPW = WPR == 1 ? 4 : 1;
    __shared__ __attribute__((aligned(16))) float sums[WPR][D];
    __shared__ float2 sums_ml[WPR];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int s, head, tile, rho, used;
    int64_t slot0;
    SeqRows q;
    if (MANY) {
        PromptTile at;
        const int me = blockIdx.x; // (WPR 16)
        if (!prompt_tile(a, me / kPromptRows, false, at) || at.splits == 1)
            return; // (its workgroup has written the result)
        s = at.s, head = at.head, tile = at.tile, q = at.q;
        rho = tile * kPromptRows + me % kPromptRows;
        const int rows = rows_of(a, q);
        if (rho >= rows)
            return;
        TileView view = view_of(a, q, tile, kPromptRows, rows - tile * kPromptRows);
        divide(a, at.splits, view);
        used = view.used;
        slot0 = (int64_t)at.unit * at.splits;
    } else {
        s = blockIdx.z, head = blockIdx.y;
        rho = blockIdx.x * RPW + (WPR == 1 ? wave : 0);
        if (rho >= a.rows)
            return;
        tile = quotient(rho, a.by_tile_rows);
        const int unit = (s * a.c.n_kv_heads + head) * a.tiles + tile;
        const int from = a.spans[2 * unit], last = a.spans[2 * unit + 1];
        q = seq_rows(a.c, s);
        const int rows = rows_of(a, q);
        if (rho >= rows)
            return;
        // the waves that shared it (one that had all of it has written the result)
        slot0 = from;
        used = last - from + 1;
        if (view_of(a, q, tile, tile_rows, rows - tile * tile_rows).count == 0)
            used = 0;
        else if (used == 1)
            return;
    }
    slot0 = slot0 * tile_rows + rho - tile * tile_rows;
    const float *part = a.part + slot0 * D;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + slot0;
    int64_t step = tile_rows;
    int first = WPR == 1 ? 0 : wave, stride = WPR;

    f32x4 v0, v1;
    float top, sum;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        v0 = v1 = f32x4{0.f, 0.f, 0.f, 0.f};
        top = kNoMax;
        sum = 0.f;
#pragma unroll 1
        for (int k0 = first * AT_ONCE + lane / LPR; k0 - lane / LPR < used; k0 += stride * AT_ONCE * AHEAD) {
            f32x4 w[AHEAD][2];
            float2 f[AHEAD];
            float to = top;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int k = k0 + i * stride * AT_ONCE, of = k < used ? k : 0;
                const int at = !MANY && pass == 0 && of == 0 ? a.parts : of; // (attn.hpp, `part`)
                const f32x4 *p = reinterpret_cast<const f32x4 *>(part + at * step * D) + lane % LPR * 2;
                f[i] = ml[at * step];
                w[i][0] = p[0];
                w[i][1] = p[1];
                if (k >= used)
                    f[i].x = -__builtin_inff();
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                to = fmaxf(to, f[i].x);
            const float g = exp2_fast(top - to);
            top = to;
            v0 *= g;
            v1 *= g;
            sum *= g;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float e = exp2_fast(f[i].x - top);
                if (k0 + i * stride * AT_ONCE < used) { // (not 0 times what is not a number)
                    v0 += w[i][0] * e;
                    v1 += w[i][1] * e;
                    sum += f[i].y * e;
                }
            }
        }
        // over the groups of lanes
#pragma unroll 1
        for (int o = LPR; o < 64; o <<= 1) {
            const float other = __shfl_xor(top, o, 64), to = fmaxf(top, other);
            const float e = exp2_fast(top - to), g = exp2_fast(other - to);
            top = to;
            sum = sum * e + __shfl_xor(sum, o, 64) * g;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v0[j] = v0[j] * e + __shfl_xor(v0[j], o, 64) * g;
                v1[j] = v1[j] * e + __shfl_xor(v1[j], o, 64) * g;
            }
        }
        if (WPR == 1 || pass == 1)
            break;
        if (lane < LPR) {
            reinterpret_cast<f32x4 *>(sums[wave])[lane * 2] = v0;
            reinterpret_cast<f32x4 *>(sums[wave])[lane * 2 + 1] = v1;
            sums_ml[wave] = make_float2(top, sum);
        }
        __syncthreads();
        if (wave)
            return;
        part = sums[0];
        ml = sums_ml;
        step = 1;
        used = WPR;
        first = 0;
        stride = 1;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i = quotient(rho, a.by_group);
    const int64_t at = (int64_t)(q.row0 + i) * a.ldo + (head * a.group + rho - i * a.group) * a.o_head +
                       lane * 8;
    if (lane >= LPR)
        return;
    v0 *= inv;
    v1 *= inv;
    if (a.o_bf16) {
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.O) + at) =
            u32x4{pack_pair(v0[0], v0[1]), pack_pair(v0[2], v0[3]), pack_pair(v1[0], v1[1]), pack_pair(v1[2], v1[3])};
    } else {
        f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(a.O) + at);
        o[0] = v0;
        o[1] = v1;
    }
}

// The same with many rows and up to kJoinLanes ranges: D / 8 lanes add up a row's,
// eight at a time.  256 rows of 8 heads in 32 ranges: the call 51 us so, 63 us with
// 16 waves a row; 128 rows of 4 heads in 128 ranges 62 and 51.
template <int D> __global__ void __launch_bounds__(256) prompt_join_kernel(AttendArgs a) {
    constexpr int LPR = D / 8, ROWS = 256 / LPR, AHEAD = 8;
    const int col = threadIdx.x % LPR * 8, me = blockIdx.x * ROWS;
    PromptTile at;
    if (!prompt_tile(a, me / kPromptRows, false, at) || at.splits == 1)
        return; // (its workgroup has written the result)
    const int mine = me % kPromptRows + threadIdx.x / LPR, rho = at.tile * kPromptRows + mine;
    const int rows = rows_of(a, at.q);
    if (rho >= rows)
        return;
    TileView view = view_of(a, at.q, at.tile, kPromptRows, rows - at.tile * kPromptRows);
    divide(a, at.splits, view);
    const int64_t slot = (int64_t)at.unit * at.splits * kPromptRows + mine;
    const float *part = a.part + slot * D + col;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + slot;
    f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
    float top = kNoMax, sum = 0.f;
    for (int k0 = 0; k0 < view.used; k0 += AHEAD) {
        f32x4 w[AHEAD][2];
        float2 f[AHEAD];
        float to = top;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int k = k0 + i < view.used ? k0 + i : k0;
            const f32x4 *p = reinterpret_cast<const f32x4 *>(part + (int64_t)k * (kPromptRows * D));
            f[i] = ml[(int64_t)k * kPromptRows];
            w[i][0] = p[0];
            w[i][1] = p[1];
            to = fmaxf(to, f[i].x);
        }
        const float g = exp2_fast(top - to);
        top = to;
        v0 *= g;
        v1 *= g;
        sum *= g;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (k0 + i < view.used) {
                const float e = exp2_fast(f[i].x - top);
                v0 += w[i][0] * e;
                v1 += w[i][1] * e;
                sum += f[i].y * e;
            }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i = quotient(rho, a.by_group);
    const int64_t to = (int64_t)(at.q.row0 + i) * a.ldo + (at.head * a.group + rho - i * a.group) * a.o_head + col;
    v0 *= inv;
    v1 *= inv;
    if (a.o_bf16) {
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.O) + to) =
            u32x4{pack_pair(v0[0], v0[1]), pack_pair(v0[2], v0[3]), pack_pair(v1[0], v1[1]), pack_pair(v1[2], v1[3])};
    } else {
        f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(a.O) + to);
        o[0] = v0;
        o[1] = v1;
    }
}

template <int D, int P> hipError_t decode(const AttendArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.parts + kWaves - 1) / kWaves));
    hipLaunchKernelGGL((attend_decode_kernel<D, P>), grid, dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

template <int D> hipError_t join(int tile_rows, AttendArgs a, hipStream_t stream) {
    const bool many = a.parts / a.units > kJoinWave;
    const unsigned rows = (unsigned)(many ? a.rows : (a.rows + 3) / 4);
    const dim3 grid(rows, (unsigned)a.c.n_kv_heads, (unsigned)a.c.n_seqs);
    a.by_tile_rows = make_div((uint32_t)tile_rows);
    if (many)
        hipLaunchKernelGGL((attend_join_kernel<D, 16, false>), grid, dim3(1024), 0, stream, a, tile_rows);
    else
        hipLaunchKernelGGL((attend_join_kernel<D, 1, false>), grid, dim3(256), 0, stream, a, tile_rows);
    return hipGetLastError();
}

template <int D> hipError_t prompt_join(const AttendArgs &a, hipStream_t stream) {
    // (tiles in two ranges or more)
    const unsigned rows = (unsigned)(a.units < kPromptPlaces / 2 ? a.units : kPromptPlaces / 2) * kPromptRows;
    if (a.splits > kJoinLanes)
        hipLaunchKernelGGL((attend_join_kernel<D, 16, true>), dim3(rows), dim3(1024), 0, stream, a, kPromptRows);
    else
        hipLaunchKernelGGL((prompt_join_kernel<D>), dim3(rows / (256 / (D / 8))), dim3(256), 0, stream, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_attend_decode(int head_dim, int tile_rows, const AttendArgs &a, hipStream_t stream) {
    if (head_dim == 64)
        return tile_rows == 4 ? decode<64, 4>(a, stream)
                              : (tile_rows == 8 ? decode<64, 2>(a, stream) : decode<64, 1>(a, stream));
    if (head_dim == 128)
        return tile_rows == 4 ? decode<128, 4>(a, stream)
                              : (tile_rows == 8 ? decode<128, 2>(a, stream) : decode<128, 1>(a, stream));
    return tile_rows == 8 ? decode<256, 2>(a, stream) : decode<256, 1>(a, stream);
}

hipError_t launch_attend_join(int head_dim, int tile_rows, const AttendArgs &a, hipStream_t stream) {
    return head_dim == 64 ? join<64>(tile_rows, a, stream)
                          : (head_dim == 128 ? join<128>(tile_rows, a, stream) : join<256>(tile_rows, a, stream));
}

hipError_t launch_prompt_join(int head_dim, const AttendArgs &a, hipStream_t stream) {
    return head_dim == 64 ? prompt_join<64>(a, stream) : prompt_join<128>(a, stream);
}

} // namespace tsl
