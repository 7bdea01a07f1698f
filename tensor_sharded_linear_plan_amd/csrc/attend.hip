// Attention of query rows over the paged 4-bit cache, for few rows a sequence
// (generated tokens): o_i = sum_j p_ij v_j, p = softmax over the visible j of
// scale q_i . k_j, one pass over the tokens with a running maximum and sum.
//
// A workgroup takes up to 16 query rows of one sequence and K/V head (the heads
// that share it, of one or several tokens) and a range of the records they see;
// its four waves take records in turn and join at the end through LDS.  Where the
// tiles are few the ranges are many, and attend_join adds them.
//
// The products run on 16x16x32 MFMAs, transposed: S^T = K Q^T and O^T = V^T P^T,
// so a lane holds one query row throughout (column l % 16) and the
// probabilities that leave S^T are the registers that O^T takes in.  Codes are
// expanded to the exact bf16 128 + c; a group's scale and bias enter in
// binary32,
//     q . k = sum_g s_g (q_g . (128 + c_g)) + (b_g - 128 s_g) sum(q_g)
//     o_g   = sum_j (p_j s_jg) (128 + c_jg) + sum_j p_j (b_jg - 128 s_jg),
// with p s as a bf16 and what its rounding left as another, so that neither
// shows in the result (8 more MFMAs a record, in a kernel that waits for
// memory and the vector units).
//
// Records come by direct copies into LDS (global_load_lds), each wave its own
// two stages: the next record is on its way while this one is multiplied, and
// the registers that a prefetch would hold are free, so that four workgroups
// share a CU.
#include "attn.hpp"
#include "gemm_common.hpp"

namespace tsl {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ float pick(u32x4 w, int e) {
    return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
}

constexpr int kStages = 2;

// At most N of the wave's copies into LDS are still under way.
template <int N> __device__ __forceinline__ void wait_copies() {
    wait_vmcnt<N>();
    asm volatile("" ::: "memory");
}

// P records a step: the 16 columns of a product are P times the tile's 16 / P
// rows, and a lane keeps of each product what is of its own record.
template <int D, int P>
__global__ void __launch_bounds__(64 * kWaves, attend_groups(D, P)) attend_decode_kernel(AttendArgs a) {
    constexpr int G = D / 64, W = D / 32, DT = D / 16, ROWS = 16 / P;
    constexpr int REC = record_bytes(D), PIECES = REC / 16; // 16 bytes a lane
    constexpr int COPIES = (PIECES + 63) / 64, STEP = P * REC;
    // a wave's stages, and after the walk its sums
    __shared__ __attribute__((aligned(16))) char ring[kWaves][kStages * STEP];
    __shared__ float red_m[kWaves][16], red_l[kWaves][16];
    static_assert(kStages * STEP >= DT * 1024, "sums of a wave");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int own = c / ROWS, cr = c % ROWS; // the lane's record of a step, its row

    int b = blockIdx.x;
    const int split = b % a.splits;
    b /= a.splits;
    const int unit = b; // (sequence, head, tile)
    const int tile = b % a.tiles;
    b /= a.tiles;
    const int head = b % a.c.n_kv_heads, s = b / a.c.n_kv_heads;
    const SeqRows q = seq_rows(a.c, s);
    const int n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
    const int rows = n * a.group - tile * ROWS; // of this tile and later ones
    if (rows <= 0)
        return;
    const int start = q.ctx - q.n;
    const int last_rho = tile * ROWS + (rows < ROWS ? rows : ROWS) - 1;
    const TileView view = tile_view(a, start + tile * ROWS / a.group, start + last_rho / a.group);
    const int begin = split * view.share;
    const int stop = begin + view.share < view.count ? begin + view.share : view.count;
    if (begin >= stop && split > 0)
        return;

    // pages of the wave's next 64 records, one a lane
    const int mine = begin + wave * P;
    const int n_mine = mine < stop ? (stop - mine + kWaves * P - 1) / (kWaves * P) : 0; // steps
    auto index_at = [&](int k, int p) { return mine + k * (kWaves * P) + p; };
    int pages = -1;
    auto look_up = [&](int k0) {
        const int r = index_at(k0 + lane / P, lane % P);
        const int page = r < stop ? view_block(view, r) >> a.c.shift : a.c.max_pages;
        pages = page < a.c.max_pages ? a.c.page_table[s * a.c.ld_table + page] : -1;
        pages = pages < a.c.n_pages ? pages : -1;
    };
    const uint32_t lds0 = (uint32_t)(uintptr_t)&ring[wave][0];
    // the records of step k into their stage; one that is not there is read from
    // page 0, and its tokens are hidden
    auto copy = [&](int k) {
        constexpr int kSteps = 64 / P;
        if (k % kSteps == 0)
            look_up(k);
        uint32_t there = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int page = __builtin_amdgcn_readlane(pages, k % kSteps * P + p);
            const int blk = view_block(view, index_at(k, p));
            const char *rec = a.c.pages + head * a.c.head_bytes;
            if (page >= 0) {
                there |= 1u << p;
                rec += page * a.c.page_bytes + (int64_t)(blk & ((1 << a.c.shift) - 1)) * REC;
            }
            const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane(
                (int)(lds0 + (k % kStages) * STEP + p * REC));
#pragma unroll
            for (int i = 0; i < COPIES; ++i)
                if ((i + 1) * 64 <= PIECES || lane < PIECES - i * 64)
                    dma16(rec + i * 1024, (uint32_t)lane * 16, to + i * 1024);
        }
        return there;
    };
    uint32_t there = 0, there1 = 0;
    if (n_mine > 0)
        there1 = copy(0);

    // the lane's query row
    const bool live = cr < rows;
    const int rho = tile * ROWS + (live ? cr : 0);
    const int i = rho / a.group, hq = head * a.group + rho % a.group;
    const int pos = start + i, lo = window_start(a, pos);
    const uint16_t *qp = a.Q + (int64_t)(q.row0 + i) * a.ldq + hq * a.q_head + 8 * g;
    bf16x8 qr[W];
    float qsum[G];
#pragma unroll
    for (int w = 0; w < W; ++w) // the scale's sign goes to Q: the largest product
        qr[w] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(qp + 32 * w) ^
                                               (a.scale < 0.f ? 0x80008000u : 0u)); // is the largest logit
    const float scale = fmaxf(fabsf(a.scale), 1.17549435e-38f); // not 0: it meets infinities
#pragma unroll
    for (int k = 0; k < G; ++k) {
        float t = 0.f;
#pragma unroll
        for (int w = 2 * k; w < 2 * k + 2; ++w)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                t += (float)qr[w][j];
        t += __shfl_xor(t, 16, 64);
        t += __shfl_xor(t, 32, 64);
        qsum[k] = t;
    }

    f32x4 o[DT], off[G], base[G];
    float ob[G], m = kNoMax, l = 0.f;
    const bf16x8 all128 = __builtin_bit_cast(bf16x8, u32x4{0x43004300u, 0x43004300u, 0x43004300u, 0x43004300u});
#pragma unroll
    for (int t = 0; t < DT; ++t)
        o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < G; ++k) {
        ob[k] = 0.f;
        off[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        const float z = -128.f * qsum[k];
        base[k] = f32x4{z, z, z, z};
    }

    for (int k = 0; k < n_mine; ++k) {
        there = there1;
        if (k + 1 < n_mine) {
            wait_lgkm0(); // the stage was read
            there1 = copy(k + 1);
            wait_copies<P * COPIES>();
        } else {
            wait_copies<0>();
        }
        const u32x4 *rec = reinterpret_cast<const u32x4 *>(&ring[wave][(k % kStages) * STEP]);
        // scales of the lane's 8 tokens
        const u32x4 *sc = rec + own * (REC / 16) + 2 * D + g;

        f32x4 acc[2][G];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            u32x4 kc[G];
#pragma unroll
            for (int d = 0; d < G; ++d)
                kc[d] = rec[p * (REC / 16) + d * 64 + lane];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int d = 0; d < G; ++d) {
                    f32x4 t = base[d];
#pragma unroll
                    for (int w = 2 * d; w < 2 * d + 2; ++w)
                        t = mfma_bf16(q4_to_bf16_plus128(kc[(u * W + w) >> 2][(u * W + w) & 3]), qr[w], t);
                    if (p == 0)
                        acc[u][d] = t;
                    else
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[u][d][e] = own == p ? t[e] : acc[u][d][e];
                }
        }
        float x[8]; // products, the scale not yet in them
#pragma unroll
        for (int d = 0; d < G; ++d) {
            const u32x4 ks = sc[d * 16], kb = sc[d * 16 + 4];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = pick(kb, e) * qsum[d];
                x[e] = fmaf(pick(ks, e), acc[e >> 2][d][e & 3], d ? x[e] + t : t);
            }
        }
        u32x4 keep = {~0u, ~0u, ~0u, ~0u}; // of the V scales: a hidden token's may be NaN
        bool all = there == (1u << P) - 1;
#pragma unroll
        for (int p = 0; p < P; ++p)
            all = all && sees_all(a, view, view_block(view, index_at(k, p)));
        if (!all) {
            rare();
            const int blk = view_block(view, index_at(k, own));
            const bool here = there >> own & 1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool v = here & sees(a, pos, lo, blk * kBlock + (e >> 2) * 16 + g * 4 + (e & 3));
                x[e] = v ? x[e] : -__builtin_inff();
                keep[e >> 1] &= v ? ~0u : (e & 1 ? 0xFFFFu : 0xFFFF0000u);
            }
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 8; ++e)
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
        float pr[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            pr[e] = exp2_fast(fmaf(x[e], scale, -m));
            l += pr[e];
        }
#pragma unroll
        for (int d = 0; d < G; ++d) {
            u32x4 vs = sc[d * 16 + 8], vb = sc[d * 16 + 12];
            if (!all) {
                rare();
                vs &= keep;
                vb &= keep;
            }
            u32x4 hi, rem;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float w0 = pr[2 * h] * bf16_lo(vs[h]), w1 = pr[2 * h + 1] * bf16_hi(vs[h]);
                ob[d] = fmaf(pr[2 * h], bf16_lo(vb[h]), ob[d]);
                ob[d] = fmaf(pr[2 * h + 1], bf16_hi(vb[h]), ob[d]);
                hi[h] = pack_pair(w0, w1);
                rem[h] = pack_pair(w0 - bf16_lo(hi[h]), w1 - bf16_hi(hi[h]));
            }
            // what 128 + c has over c: the same products with a tile of 128
            off[d] = mfma_bf16(all128, __builtin_bit_cast(bf16x8, hi), off[d]);
            off[d] = mfma_bf16(all128, __builtin_bit_cast(bf16x8, rem), off[d]);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const u32x4 vc = rec[p * (REC / 16) + D + d * 64 + lane];
                const uint32_t take = P == 1 || own == p ? ~0u : 0u;
                const bf16x8 wh = __builtin_bit_cast(bf16x8, hi & take), wl = __builtin_bit_cast(bf16x8, rem & take);
#pragma unroll
                for (int t = 4 * d; t < 4 * d + 4; ++t) {
                    const bf16x8 v = q4_to_bf16_plus128(vc[t & 3]);
                    o[t] = mfma_bf16(v, wh, o[t]);
                    o[t] = mfma_bf16(v, wl, o[t]);
                }
            }
        }
    }

    // join the lanes of a row, then the waves and their columns
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
#pragma unroll
    for (int d = 0; d < G; ++d) {
        ob[d] += __shfl_xor(ob[d], 16, 64);
        ob[d] += __shfl_xor(ob[d], 32, 64);
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
        reinterpret_cast<f32x4 *>(ring[wave])[t * 64 + lane] = (o[t] - off[t >> 2]) + ob[t >> 2];
    if (g == 0) {
        red_m[wave][c] = m;
        red_l[wave][c] = l;
    }
    __syncthreads();
    if (!live || own)
        return;
    float top = red_m[0][c];
#pragma unroll
    for (int w = 0; w < kWaves * P; ++w)
        top = fmaxf(top, red_m[w / P][c + w % P * ROWS]);
    float sum = 0.f, f[kWaves * P];
#pragma unroll
    for (int w = 0; w < kWaves * P; ++w) {
        f[w] = exp2_fast(red_m[w / P][c + w % P * ROWS] - top);
        sum += f[w] * red_l[w / P][c + w % P * ROWS];
    }
    const float inv = a.splits > 1 ? 1.f : (sum == 0.f ? 0.f : 1.f / sum);
    const int64_t slot = ((int64_t)unit * a.splits + split) * ROWS + c;
    if (a.splits > 1 && wave == 0 && g == 0) {
        a.part_ml[2 * slot] = top;
        a.part_ml[2 * slot + 1] = sum;
    }
#pragma unroll
    for (int t0 = 0; t0 < DT; t0 += kWaves) {
        const int t = t0 + wave;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves * P; ++w)
            v += reinterpret_cast<const f32x4 *>(ring[w / P])[t * 64 + lane + w % P * ROWS] * f[w];
        v *= inv;
        const int col = 16 * t + 4 * g;
        if (a.splits > 1) {
            *reinterpret_cast<f32x4 *>(a.part + slot * D + col) = v;
        } else {
            const int64_t at = (int64_t)(q.row0 + i) * a.ldo + hq * a.o_head + col;
            if (a.o_bf16)
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.O) + at) =
                    u32x2{pack_pair(v[0], v[1]), pack_pair(v[2], v[3])};
            else
                *reinterpret_cast<f32x4 *>(static_cast<float *>(a.O) + at) = v;
        }
    }
}

// The ranges of a row added, by 256 / 64 / WPR rows a workgroup, WPR waves each: a
// row's threads take its ranges' references and sums together, then its waves
// the ranges in turn, D / 64 columns a lane, eight rows of partial sums on their
// way at a time.
template <int D, int WPR>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendArgs a, int tile_rows) {
    constexpr int V = D / 64, kAhead = 8, RPW = 4 / WPR, N = 64 * WPR;
    typedef float vec __attribute__((ext_vector_type(V)));
    __shared__ float fac[RPW][kMaxSplits], red[2][4];
    __shared__ vec sums[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int me = threadIdx.x % N, mw = wave % WPR, slot_row = wave / WPR;
    const int per_unit = (a.c.max_rows * a.group + RPW - 1) / RPW;
    int b = blockIdx.x / per_unit;
    const int rho = blockIdx.x % per_unit * RPW + slot_row;
    const int tile = rho / tile_rows, unit = b * a.tiles + tile;
    const int head = b % a.c.n_kv_heads, s = b / a.c.n_kv_heads;
    const SeqRows q = seq_rows(a.c, s);
    const int n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
    const bool live = rho < n * a.group;
    if (WPR == 4 && !live)
        return;
    const int end = n * a.group < (tile + 1) * tile_rows ? n * a.group : (tile + 1) * tile_rows;
    const int start = q.ctx - q.n;
    TileView view = tile_view(a, start + tile * tile_rows / a.group, start + (end - 1) / a.group);
    if (!live)
        view.used = 0;
    const int64_t slot0 = (int64_t)unit * a.splits * tile_rows + rho % tile_rows;

    float top = kNoMax;
    for (int k = me; k < view.used; k += N)
        top = fmaxf(top, a.part_ml[2 * (slot0 + (int64_t)k * tile_rows)]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        top = fmaxf(top, __shfl_xor(top, o, 64));
    if (WPR > 1) {
        red[0][wave] = top;
        __syncthreads();
        top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    }
    float sum = 0.f;
    for (int k = me; k < view.used; k += N) {
        const float *ml = a.part_ml + 2 * (slot0 + (int64_t)k * tile_rows);
        const float f = exp2_fast(ml[0] - top);
        fac[slot_row][k] = f;
        sum += f * ml[1];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        sum += __shfl_xor(sum, o, 64);
    red[1][wave] = sum;
    __syncthreads();
    if (WPR > 1)
        sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);

    const float *part = a.part + slot0 * D + lane * V;
    const int64_t step = (int64_t)tile_rows * D;
    vec v;
#pragma unroll
    for (int j = 0; j < V; ++j)
        v[j] = 0.f;
    for (int k = mw; k < view.used; k += WPR * kAhead) {
        vec w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int at = k + WPR * i;
            w[i] = *reinterpret_cast<const vec *>(part + (at < view.used ? at : k) * step);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (k + WPR * i < view.used)
                v += w[i] * fac[slot_row][k + WPR * i];
    }
    if (WPR > 1) {
        sums[wave][lane] = v;
        __syncthreads();
        if (wave)
            return;
        v = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
    }
    if (!live)
        return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t at = (int64_t)(q.row0 + rho / a.group) * a.ldo +
                       (head * a.group + rho % a.group) * a.o_head + lane * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (a.o_bf16)
            static_cast<uint16_t *>(a.O)[at + j] = (uint16_t)pack_pair(v[j] * inv, 0.f);
        else
            static_cast<float *>(a.O)[at + j] = v[j] * inv;
    }
}

template <int D, int P> hipError_t decode(const AttendArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.c.n_seqs * a.c.n_kv_heads * a.tiles * a.splits));
    hipLaunchKernelGGL((attend_decode_kernel<D, P>), grid, dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

template <int D> hipError_t join(int tile_rows, const AttendArgs &a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.c.max_rows * a.group, units = (int64_t)a.c.n_seqs * a.c.n_kv_heads;
    if (a.splits > kJoinWave)
        hipLaunchKernelGGL((attend_join_kernel<D, 4>), dim3((unsigned)(units * rows)), dim3(256), 0, stream,
                           a, tile_rows);
    else
        hipLaunchKernelGGL((attend_join_kernel<D, 1>), dim3((unsigned)(units * ((rows + 3) / 4))), dim3(256),
                           0, stream, a, tile_rows);
    return hipGetLastError();
}

} // namespace

hipError_t launch_attend_decode(int head_dim, int tile_rows, const AttendArgs &a, hipStream_t stream) {
    if (head_dim == 64)
        return tile_rows == 4 ? decode<64, 4>(a, stream)
                              : (tile_rows == 8 ? decode<64, 2>(a, stream) : decode<64, 1>(a, stream));
    if (head_dim == 128)
        return tile_rows == 8 ? decode<128, 2>(a, stream) : decode<128, 1>(a, stream);
    return decode<256, 1>(a, stream);
}

hipError_t launch_attend_join(int head_dim, int tile_rows, const AttendArgs &a, hipStream_t stream) {
    return head_dim == 64 ? join<64>(tile_rows, a, stream)
                          : (head_dim == 128 ? join<128>(tile_rows, a, stream) : join<256>(tile_rows, a, stream));
}

} // namespace tsl
