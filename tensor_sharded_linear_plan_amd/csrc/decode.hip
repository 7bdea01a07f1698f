// Products of a few token rows (up to 64) with an epilogue, in one launch:
// one rank's Y = act(X W + bias) + residual, a sum set of row shards, or a
// gated pair act(X W_0) * (X W_1) (mlxcel manual "Tensor parallelism",
// "Column Parallel" / "Row Parallel").
//
// At these sizes a call streams some tens of MB of weights, and its time is
// the launch and a few memory latencies as much as bytes; a second launch
// that adds k-partials costs as much as the products.  So the k-range is
// split inside a workgroup: it owns one 16-column tile (gated: that tile of
// both weights) and its W waves take consecutive runs of the whole k-range --
// a sum set's members laid end to end in item order -- which meet in LDS, are
// added in wave order (so in k order) and go through the epilogue in
// registers.  Nothing returns to memory but the result; no workspace, no
// atomics, the same bits every time.  W is 16 for up to 256 tiles (and 16
// rows: more need the registers of 8 waves), 8 up to 512, else 4: about 4096
// waves fill the chip's 1024 SIMDs fourfold.
//
// A wave reads its weights as the streaming kernel does (contiguous 1 KB wave
// loads in MFMA operand order, 4-bit groups applied exactly: skinny.hip), in
// units of 128 k of 4-bit or 64 k of bf16 weights, and its activation
// fragments straight from global memory -- a wave reads only its own k-run of
// X, from L2, so there is nothing to share through LDS and no barrier before
// the sum.  Products of one weight (4-bit: up to 32 rows) and bf16 pairs of
// more than 16 rows hold a second unit, whose loads are in flight while the
// first is computed; the other pairs and 4-bit calls of more rows load the
// next unit once the one before is in the matrix cores, and the SIMD's other
// waves fill the gap.  Most of those loads are activations (16 rows of 32 k
// are 1 KB, as the weights of 128 k), so calls of up to 8 rows pack several
// k-slices into one operand (RG below).  Measured: one rank's 4-bit gate and
// up, 1 row, 3584 -> 2 x 4736 (19 MB), 8.2 us; 4 ranks' down shards, 4 rows,
// 18944 -> 3584 (38 MB), 14.5 us with whole operands, 11.5 with packed ones
// (3.3 TB/s; with whole ones and a separate launch for the k-partials 19.0).
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "epilogue.hpp"
#include "internal.hpp"

namespace tsl {
namespace {

constexpr int kItems = 64, kMembers = 128;

struct Member {
    const char *B;       // packed weights
    const uint16_t *X;
    const int32_t *ridx; // row m reads X row ridx[m] (zeros outside [0, x_rows)); null: row m
    int64_t x_rows, ldx;
    int32_t Ks, units;   // k, and units of it
    int32_t KC, pad_;    // chunks per column tile in B
};
struct Item {
    void *Y;
    int64_t ldy;
    int32_t M, Ns;
    int32_t first, units; // its members from `first` on; their units together
    int32_t start, y_bf16;
};
struct Group : Epilogues<kItems> {
    int32_t n, pad_;
    Item it[kItems];
    Member mb[kMembers];
};

template <bool Q4> struct Unit {
    static constexpr int K = Q4 ? 128 : 64;
    static constexpr int CHUNKS = Q4 ? 1 : 2;          // 16-byte weight loads per lane
    static constexpr int64_t CS = Q4 ? kQ4Record : 1024; // bytes per chunk
    static constexpr int FR = K / 32;                  // activation fragments
};

// MT 16-row tiles; more than one needs the registers of 8 waves.  RG: rows of
// a call of few rows (4 or 8; 4-bit weights), else 16.  Of the 16 rows an MFMA
// takes, rows RG s .. RG s + RG - 1 are then the call's rows at 32-k slice s of
// 16 / RG, so that one load holds several slices' activations.  Against the
// weights of slice t the results in slice t's rows are its product (the others
// mean nothing): each lane keeps its own slice's and adds them up, and the
// lanes of one row meet at the end.
template <bool Q4, bool DUAL, int MT, int RG>
__global__ void __launch_bounds__(MT == 1 ? 1024 : 512) decode_kernel(Group grp) {
    constexpr bool FEW = RG < 16;
    static_assert(!FEW || (Q4 && MT == 1), "one tile of slices");
    using C = Unit<Q4>;
    constexpr int NS = 16 / RG;       // slices of a load
    constexpr int XR = C::FR / NS;    // activation loads per unit
    constexpr int NT = DUAL ? 2 : 1;
    extern __shared__ __attribute__((aligned(16))) f32x4 red[]; // [waves][MT][NT][64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int W = blockDim.x >> 6;
    const int bid = blockIdx.x;
    int lo = 0, hi = grp.n - 1; // last item whose first workgroup is <= bid
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (grp.it[mid].start <= bid)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Item &a = grp.it[lo];
    const int64_t tile = bid - a.start;
    const int u0 = wave * a.units / W, u1 = (wave + 1) * a.units / W;
    const int kg = lane >> 4;
    const int row = lane & (RG - 1);      // this lane's activation row
    const int slice = (lane & 15) / RG;   // and slice of a load; its results':
    const int rslice = kg * 4 / RG;
    const int64_t up = DUAL ? static_cast<const char *>(grp.ep(lo).up) - grp.mb[a.first].B : 0;

    // where the next unit comes from: unit lu of member r.  Rows past M read
    // row 0 (finite or not, their results are not stored; masking their lanes
    // off measured 16.1 against 15.2 us, 4 rows x 18944 x 3584); a row whose
    // index lies outside X reads row 0 and is masked to zeros.
    int r = a.first, lu = u0;
    const char *wp[NT];
    const uint16_t *xp[MT]; // this lane's rows and k-run
    uint32_t keep[MT];
    bool masked = false; // some row of the wave may be (uniform)
    int Ks = 0;
    auto enter = [&]() __attribute__((always_inline)) {
        const Member &b = grp.mb[r];
        Ks = b.Ks;
        wp[0] = b.B + tile * b.KC * C::CS;
        if constexpr (DUAL)
            wp[1] = wp[0] + up;
        masked = b.ridx != nullptr;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            int64_t s = 16 * i + row < a.M ? 16 * i + row : 0;
            keep[i] = ~0u;
            if (masked) {
                s = b.ridx[s];
                const bool ok = s >= 0 && s < b.x_rows;
                keep[i] = ok ? ~0u : 0u;
                s = ok ? s : 0;
            }
            xp[i] = b.X + s * b.ldx + 8 * kg;
        }
    };
    struct Regs {
        u32x4 w[NT][C::CHUNKS];
        u32x2 sb[NT]; // (RG 4: the one pair of this lane's results)
        u32x4 x[MT][XR];
    };
    auto load = [&](Regs &g) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const char *rec = wp[j] + (int64_t)lu * C::CHUNKS * C::CS;
#pragma unroll
            for (int l = 0; l < C::CHUNKS; ++l)
                g.w[j][l] = *reinterpret_cast<const u32x4 *>(rec + l * C::CS + lane * 16);
            if constexpr (RG == 4)
                g.sb[j].x = *reinterpret_cast<const uint32_t *>(rec + kQ4PairsAt + (lane & 15) * 8 +
                                                                (rslice >> 1) * 4);
            else if constexpr (Q4)
                g.sb[j] = *reinterpret_cast<const u32x2 *>(rec + kQ4PairsAt + (lane & 15) * 8);
        }
        // 4-bit k-ranges are whole 64-k groups and bf16 units 64 k, so that
        // every condition here is uniform but in a ragged last bf16 unit
        const int left = Ks - lu * C::K;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint16_t *x = xp[i] + lu * C::K + 32 * slice;
            if (left >= C::K) {
#pragma unroll
                for (int f = 0; f < XR; ++f)
                    g.x[i][f] = *reinterpret_cast<const u32x4 *>(x + 32 * NS * f);
            } else {
#pragma unroll
                for (int f = 0; f < XR; ++f) {
                    const int k = 32 * (NS * f + slice) + 8 * kg;
                    u32x4 v = {0, 0, 0, 0};
                    if (k + 8 <= left) {
                        v = *reinterpret_cast<const u32x4 *>(x + 32 * NS * f);
                    } else if (k < left) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t l0 = k + 2 * e < left ? x[32 * NS * f + 2 * e] : 0u;
                            const uint32_t h0 = k + 2 * e + 1 < left ? x[32 * NS * f + 2 * e + 1] : 0u;
                            v[e] = l0 | (h0 << 16);
                        }
                    }
                    g.x[i][f] = v;
                }
            }
            if (masked) {
#pragma unroll
                for (int f = 0; f < XR; ++f)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        g.x[i][f][e] &= keep[i];
            }
        }
        ++lu;
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Regs &g) __attribute__((always_inline)) {
        if constexpr (FEW) {
            const bf16x8 ones = __builtin_bit_cast(
                bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int f = 0; f < XR; ++f) {
                const bf16x8 xa = __builtin_bit_cast(bf16x8, g.x[0][f]);
                const f32x4 xs = mfma_bf16(xa, ones, zero); // of the slice of each lane's results
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    f32x4 ag[NS];
#pragma unroll
                    for (int t = 0; t < NS; ++t)
                        ag[t] = mfma_bf16(xa, q4_to_bf16_plus128(g.w[j][0][NS * f + t]), zero);
                    // as below: s sum(x (128 + q)) + (b - 128 s) sum(x)
                    const uint32_t sbp = g.sb[j][f];
                    const float sc = bf16_lo(sbp);
                    const float cb = __builtin_fmaf(-128.f, sc, bf16_hi(sbp));
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float v = rslice & 1 ? ag[1][q] : ag[0][q];
                        if constexpr (NS == 4) {
                            const float v1 = rslice & 1 ? ag[3][q] : ag[2][q];
                            v = rslice & 2 ? v1 : v;
                        }
                        acc[0][j][q] = __builtin_fmaf(sc, v, acc[0][j][q]);
                        acc[0][j][q] = __builtin_fmaf(cb, xs[q], acc[0][j][q]);
                    }
                }
            }
        } else if constexpr (!Q4) {
#pragma unroll
            for (int f = 0; f < C::FR; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        acc[i][j] = mfma_bf16(__builtin_bit_cast(bf16x8, g.x[i][f]),
                                              __builtin_bit_cast(bf16x8, g.w[j][f]), acc[i][j]);
        } else {
            const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u,
                                                                 0x3F803F80u, 0x3F803F80u});
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            f32x4 xs[MT], ag[MT][NT];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                bf16x8 xa[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    xa[i] = __builtin_bit_cast(bf16x8, g.x[i][t]);
                    xs[i] = mfma_bf16(xa[i], ones, (t & 1) ? xs[i] : zero);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const bf16x8 bq = q4_to_bf16_plus128(g.w[j][0][t]);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        ag[i][j] = mfma_bf16(xa[i], bq, (t & 1) ? ag[i][j] : zero);
                }
                if (t & 1) { // end of a group: y += s sum(x (128 + q)) + (b - 128 s) sum(x)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint32_t sbp = g.sb[j][t >> 1];
                        const float sc = bf16_lo(sbp);
                        const float cb = __builtin_fmaf(-128.f, sc, bf16_hi(sbp));
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                acc[i][j][q] = __builtin_fmaf(sc, ag[i][j][q], acc[i][j][q]);
                                acc[i][j][q] = __builtin_fmaf(cb, xs[i][q], acc[i][j][q]);
                            }
                    }
                }
            }
        }
    };
    if (u0 < u1) {
        while (lu >= grp.mb[r].units) {
            lu -= grp.mb[r].units;
            ++r;
        }
        enter();
        auto next = [&](Regs &g) __attribute__((always_inline)) {
            if (lu == grp.mb[r].units) { // the next member's k-range
                lu = 0;
                ++r;
                enter();
            }
            load(g);
        };
        Regs g0, g1;
        load(g0);
        // One unit at a time where a second one's registers spill or leave a SIMD
        // fewer waves, whose loads overlap as well (one at a time / two, 3584 ->
        // 2 x 4736, 4-bit: M 1 8.3 / 8.7 us, 77 and 110 registers; M 8 9.7 / 10.2,
        // spills; M 32 19.8 / 22.0; one weight, M 48 24.8 / 26.3; bf16 pairs, M 1
        // 16.2 / 15.8)
        if constexpr (MT == 1 ? DUAL : Q4 && MT * NT > 2) {
            for (int u = u0 + 1; u < u1; ++u) {
                compute(g0);
                next(g0);
            }
            compute(g0);
        } else {
            int u = u0;
            // steady state: each step's prefetch exists, so that the wait
            // counts at the loop head are exact
            for (; u + 2 < u1; u += 2) {
                next(g1);
                compute(g0);
                next(g0);
                compute(g1);
            }
            if (u + 1 < u1) {
                next(g1);
                compute(g0);
                compute(g1);
            } else {
                compute(g0);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            red[((wave * MT + i) * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    // wave i adds up and stores row tile i
    for (int i = wave; i < MT; i += W) {
        f32x4 v[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            v[j] = red[(i * NT + j) * 64 + lane];
            for (int w = 1; w < W; ++w) {
                const f32x4 p = red[((w * MT + i) * NT + j) * 64 + lane];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[j][q] += p[q];
            }
        }
        if constexpr (FEW) { // the slices' sums
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[j][q] += __shfl_xor(v[j][q], 32, 64);
                    if constexpr (RG == 4)
                        v[j][q] += __shfl_xor(v[j][q], 16, 64);
                }
                if constexpr (RG == 4) { // each lane's one row to its first place
                    const float a0 = kg & 1 ? v[j][1] : v[j][0], a1 = kg & 1 ? v[j][3] : v[j][2];
                    v[j][0] = kg & 2 ? a1 : a0;
                }
            }
        }
        // lane holds rows 16 i + 4 (lane / 16) + q (RG 4: row lane / 16; RG 8:
        // lanes from 32 on repeat the others) of column lane % 16
        const int64_t col = tile * 16 + (lane & 15);
        if (col >= a.Ns)
            return;
        const Epilogue e = grp.ep(lo);
#pragma unroll
        for (int q = 0; q < (RG == 4 ? 1 : 4); ++q) {
            const int64_t m = RG == 4 ? kg : 16 * i + 4 * kg + q;
            if (m >= a.M) // (RG 8: so are the repeated lanes' rows)
                continue;
            float y;
            if constexpr (DUAL)
                y = ep_gate(e, v[0][q], v[1][q], m, col);
            else
                y = ep_apply(e, v[0][q], m, col);
            ep_put(a.Y, a.y_bf16, m * a.ldy + col, y);
        }
    }
}

typedef void (*DecodeFn)(Group);

template <bool Q4, bool DUAL> DecodeFn pick(int64_t M) {
    if constexpr (Q4) {
        if (M <= 8)
            return M <= 4 ? decode_kernel<true, DUAL, 1, 4> : decode_kernel<true, DUAL, 1, 8>;
    }
    return M <= 16   ? decode_kernel<Q4, DUAL, 1, 16>
           : M <= 32 ? decode_kernel<Q4, DUAL, 2, 16>
           : M <= 48 ? decode_kernel<Q4, DUAL, 3, 16>
                     : decode_kernel<Q4, DUAL, 4, 16>;
}

// Waves of a workgroup.
int wave_count(int64_t tiles, int64_t M) {
    return tiles <= 256 && M <= 16 ? 16 : (tiles <= 512 ? 8 : 4);
}

} // namespace

// Each tile's waves read the call's X again (from L2), which the streaming
// kernel's workgroups share among four or eight tiles, so this form is for
// calls of few tiles or few rows: with T tiles (of one weight) and M rows, up
// to 32 rows T M <= 9472 (gated: twice that, for a tile of X serves both
// weights), and T <= 1200.  Either side of it, K 3584, this form / the other:
// 4-bit lone T 592: M 16 15.1 / 14.9 us, M 32 25.7 / 22.2; T 1184: M 16 22.2 /
// 18.4; T 1280: M 8 15.0 / 16.6; T 2048: M 6 23.8 / 20.8; gated T 1184: M 16
// 24.2 / 25.7, M 32 39.7 / 36.9; bf16 lone T 592: M 16 16.5 / 17.9, M 32 25.2
// / 22.4.  (The rule does not read k; along others the border lies elsewhere:
// 4-bit lone T 592, M 16, K 1024 6.3 / 8.5, K 8192 27.6 / 19.0, bf16 7.2 /
// 10.4 and 38.1 / 36.8.)  Up to 4 rows of 4-bit weights, whose activations are
// one load a unit, and up to 64 lone items or sets (of up to 8 members): T <=
// 1536, and any T (a launch's workgroups countable) from 3 rows on: T 1280: M
// 1 10.1 / 14.1, M 4 10.2 / 15.8; T 2048: M 1 17.6 / 16.5, M 4 18.6 / 20.9; T
// 9504: M 4 63.4 / 65.7; experts of 2048 -> 768, rows through an index: 32 of
// them, M 2 10.1 / 14.7, 64, M 1 17.5 / 15.6, M 4 18.0 / 19.1, 128, M 4 34.3 /
// 30.4.  A launch closes at 128 members too, but sets gain more than its end
// costs: 48 sets of 4 shards of 192 -> 2048 (two launches), M 4 24.0 / 60.7;
// 40 of 4, 192 -> 512, M 1 9.8 / 24.5; 64 of 8, 512 -> 256 (four launches), M
// 4 34.8 / 91.0.  From 33 to 64 rows 4-bit weights always (T 1184: M 48 53 /
// 63, gated 57 / 78; T 2048: M 48 82 / 75), bf16 only gated pairs of few tiles
// (T 224, K 4096: M 64 20.8 / 23.1; T 592: 52.9 / 40.8; lone T 256: 20.1 /
// 15.5).  Few tiles of a long k leave a 4-bit wave of more than one row tile a
// chain of loads that only the split over workgroups shortens: with less than
// half the chip's waves, up to 8 units a wave (T 46, 106 units over 8 waves, M
// 42: 39.2 / 23.9 us; 64 units, M 24: 17.0 / 15.4; one row tile, 256 units
// over 16 waves, M 1: 16.5 / 21.3).
bool decode_applies(const std::vector<LinearItem> &items, tsl_dtype wdtype, int64_t M) {
    if (wdtype == TSL_F32 || M > kDecodeRows)
        return false;
    int64_t tiles = 0, sets = 0, units = 0, set = 0; // units: the longest set's
    bool any = false;
    for (const LinearItem &L : items) {
        set = (L.set_pos == 0 ? 0 : set) + (wdtype == TSL_Q4G64 ? L.g.KT : L.g.KT / 2);
        units = set > units ? set : units;
        any = any || L.ep;
        if (L.accumulate || L.set_len > kSetParts)
            return false;
        if (L.set_len > 0) {
            tiles += L.g.Nt;
            ++sets;
        }
    }
    if (any && wdtype == TSL_Q4G64 && M <= 4 && sets <= kItems)
        return tiles <= 1536 || (M > 2 && tiles < (1 << 20));
    if (!any || tiles > 1200)
        return false;
    const int waves = wave_count(tiles, M);
    if (wdtype == TSL_Q4G64 && M > 16 && tiles * waves < 2048 && units > 8 * waves)
        return false;
    const bool two = dual(items[0]);
    if (M <= 32)
        return tiles * M <= (two ? 18944 : 9472);
    return wdtype == TSL_Q4G64 || (two && tiles * M <= 14336);
}

hipError_t launch_decode(const std::vector<LinearItem> &items, tsl_dtype wdtype, int64_t M,
                         hipStream_t stream) {
    const bool q4 = wdtype == TSL_Q4G64, two = dual(items[0]);
    const int mt = (int)((M + 15) / 16);
    const DecodeFn fn = q4 ? (two ? pick<true, true>(M) : pick<true, false>(M))
                           : (two ? pick<false, true>(M) : pick<false, false>(M));
    int64_t tiles = 0;
    for (const LinearItem &L : items)
        if (L.set_len > 0)
            tiles += L.g.Nt;
    const int waves = wave_count(tiles, M);
    const size_t lds = (size_t)waves * mt * (two ? 2 : 1) * 64 * 16;
    for (size_t i = 0; i < items.size();) {
        Group grp{};
        int members = 0;
        int64_t blocks = 0;
        for (; i < items.size() && grp.n < kItems && members + items[i].set_len <= kMembers;
             i += items[i].set_len) {
            const LinearItem &L = items[i];
            grp.set_ep(grp.n, L.ep);
            Item &a = grp.it[grp.n++];
            a.Y = L.Y;
            a.ldy = L.ldy;
            a.M = (int32_t)L.M;
            a.Ns = (int32_t)L.g.Ns;
            a.first = members;
            a.y_bf16 = L.ydtype == TSL_BF16;
            a.start = (int32_t)blocks;
            blocks += L.g.Nt;
            for (int r = 0; r < L.set_len; ++r) {
                const LinearItem &P = items[i + r];
                Member &m = grp.mb[members++];
                m.B = static_cast<const char *>(P.packed);
                m.X = static_cast<const uint16_t *>(P.X);
                m.ridx = P.ridx;
                m.x_rows = P.x_rows;
                m.ldx = P.ldx;
                m.Ks = (int32_t)P.g.Ks;
                m.KC = (int32_t)P.g.KT;
                m.units = (int32_t)(q4 ? P.g.KT : P.g.KT / 2);
                a.units += m.units;
            }
        }
        hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(64 * waves), lds, stream, grp);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace tsl
