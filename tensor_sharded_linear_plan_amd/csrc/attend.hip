// Attention of query rows over the paged 4-bit cache, for few rows a sequence
// (generated tokens): o_i = sum_j p_ij v_j, p = softmax over the visible j of
// scale q_i . k_j, one pass over the tokens with a running maximum and sum.
//
// A workgroup takes 16 query rows of one sequence and K/V head (the heads that
// share it, of one or several tokens) and a range of the records they see; its
// four waves take records in turn and join at the end through LDS.  Where the
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

template <int D>
__global__ void __launch_bounds__(64 * kWaves, D == 256 ? 2 : 4) attend_decode_kernel(AttendArgs a) {
    constexpr int G = D / 64, W = D / 32, DT = D / 16;
    constexpr int REC = record_bytes(D), PIECES = REC / 16; // 16 bytes a lane
    constexpr int COPIES = (PIECES + 63) / 64;
    // a wave's stages, and after the walk its sums
    __shared__ __attribute__((aligned(16))) char ring[kWaves][kStages * REC];
    __shared__ float red_m[kWaves][16], red_l[kWaves][16];
    static_assert(kStages * REC >= DT * 1024, "sums of a wave");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;

    int b = blockIdx.x;
    const int split = b % a.splits;
    b /= a.splits;
    const int unit = b; // (sequence, head, tile)
    const int tile = b % a.tiles;
    b /= a.tiles;
    const int head = b % a.c.n_kv_heads, s = b / a.c.n_kv_heads;
    const SeqRows q = seq_rows(a.c, s);
    const int n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
    const int rows = n * a.group - tile * kTileRows; // of this tile and later ones
    if (rows <= 0)
        return;
    const int start = q.ctx - q.n;
    const int last_rho = tile * kTileRows + (rows < kTileRows ? rows : kTileRows) - 1;
    const TileView view = tile_view(a, start + tile * kTileRows / a.group, start + last_rho / a.group);
    const int begin = split * view.share;
    const int stop = begin + view.share < view.count ? begin + view.share : view.count;
    if (begin >= stop && split > 0)
        return;

    // the lane's query row
    const bool live = c < rows;
    const int rho = tile * kTileRows + (live ? c : 0);
    const int i = rho / a.group, hq = head * a.group + rho % a.group;
    const int pos = start + i, lo = window_start(a, pos);
    const uint16_t *qp = a.Q + (int64_t)(q.row0 + i) * a.ldq + hq * a.q_head + 8 * g;
    bf16x8 qr[W];
    float qsum[G];
#pragma unroll
    for (int w = 0; w < W; ++w)
        qr[w] = *reinterpret_cast<const bf16x8 *>(qp + 32 * w);
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

    f32x4 o[DT];
    float ob[G], m = kNoMax, l = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
        o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < G; ++k)
        ob[k] = 0.f;

    // pages of the wave's next 64 records, one a lane
    const int mine = begin + wave;
    const int n_mine = mine < stop ? (stop - mine + kWaves - 1) / kWaves : 0;
    int pages = -1;
    auto look_up = [&](int k0) {
        const int r = mine + (k0 + lane) * kWaves;
        const int page = r < stop ? view_block(view, r) >> a.c.shift : a.c.max_pages;
        pages = page < a.c.max_pages ? a.c.page_table[s * a.c.ld_table + page] : -1;
        pages = pages < a.c.n_pages ? pages : -1;
    };
    const uint32_t lds0 = (uint32_t)(uintptr_t)&ring[wave][0];
    // record k of the wave into its stage; one that is not there is read from
    // page 0, and passed over
    auto copy = [&](int k) {
        if ((k & 63) == 0)
            look_up(k);
        const int p = __builtin_amdgcn_readlane(pages, k & 63);
        const int blk = view_block(view, mine + k * kWaves);
        const char *rec = a.c.pages + (p < 0 ? 0 : p) * a.c.page_bytes + head * a.c.head_bytes +
                          (int64_t)(blk & ((1 << a.c.shift) - 1)) * REC;
#pragma unroll
        for (int i = 0; i < COPIES; ++i)
            if ((i + 1) * 64 <= PIECES || lane < PIECES - i * 64)
                dma16(rec + i * 1024, (uint32_t)lane * 16, lds0 + (k % kStages) * REC + i * 1024);
        return p >= 0;
    };
    bool there = false, there1 = false;
    if (n_mine > 0)
        there1 = copy(0);
    for (int k = 0; k < n_mine; ++k) {
        there = there1;
        if (k + 1 < n_mine) {
            wait_lgkm0(); // the stage was read
            there1 = copy(k + 1);
            wait_copies<COPIES>();
        } else {
            wait_copies<0>();
        }
        if (!there)
            continue;
        const int blk = view_block(view, mine + k * kWaves);
        const u32x4 *rec = reinterpret_cast<const u32x4 *>(&ring[wave][(k % kStages) * REC]);
        const u32x4 *sc = rec + 2 * D + g; // scales of the lane's 8 tokens

        float y[8];
        u32x4 kc[G], ks[G], kb[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            kc[i] = rec[i * 64 + lane];
            ks[i] = sc[i * 16];
            kb[i] = sc[i * 16 + 4];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x4 acc[G];
#pragma unroll
            for (int k = 0; k < G; ++k) {
                const float z = -128.f * qsum[k];
                acc[k] = f32x4{z, z, z, z};
#pragma unroll
                for (int w = 2 * k; w < 2 * k + 2; ++w)
                    acc[k] = mfma_bf16(q4_to_bf16_plus128(kc[(u * W + w) >> 2][(u * W + w) & 3]),
                                       qr[w], acc[k]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = 0.f;
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    x = fmaf(pick(ks[k], u * 4 + e), acc[k][e], x);
                    x = fmaf(pick(kb[k], u * 4 + e), qsum[k], x);
                }
                y[u * 4 + e] = x * a.scale;
            }
        }
        bool vis[8];
        const bool all = sees_all(a, view, blk);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            vis[e] = true;
            if (!all) {
                vis[e] = sees(a, pos, lo, blk * kBlock + (e >> 2) * 16 + g * 4 + (e & 3));
                y[e] = vis[e] ? y[e] : -__builtin_inff();
            }
        }
        float top = y[0];
#pragma unroll
        for (int e = 1; e < 8; ++e)
            top = fmaxf(top, y[e]);
        // the reference exponent follows the maximum at a distance of 2^8:
        // binary32 sums have room for it, and rescaling becomes rare
        if (__any(top > m + 8.f)) {
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float to = fmaxf(m, top), f = exp2_fast(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int t = 0; t < DT; ++t)
                o[t] *= f;
#pragma unroll
            for (int k = 0; k < G; ++k)
                ob[k] *= f;
        }
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = exp2_fast(y[e] - m);
            l += p[e];
        }
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const u32x4 vs = sc[k * 16 + 8], vb = sc[k * 16 + 12], vc = rec[D + k * 64 + lane];
            u32x4 hi, lo16;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                float w[2];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int e = 2 * h + d;
                    // what a token out of sight holds may be NaN
                    w[d] = vis[e] ? p[e] * pick(vs, e) : 0.f;
                    ob[k] += vis[e] ? fmaf(p[e], pick(vb, e), -128.f * w[d]) : 0.f;
                }
                hi[h] = pack_bf16(w[0], w[1]);
                lo16[h] = pack_bf16(w[0] - bf16_lo(hi[h]), w[1] - bf16_hi(hi[h]));
            }
            const bf16x8 wh = __builtin_bit_cast(bf16x8, hi), wl = __builtin_bit_cast(bf16x8, lo16);
#pragma unroll
            for (int t = 4 * k; t < 4 * k + 4; ++t) {
                const bf16x8 v = q4_to_bf16_plus128(vc[t & 3]);
                o[t] = mfma_bf16(v, wh, o[t]);
                o[t] = mfma_bf16(v, wl, o[t]);
            }
        }
    }

    // join the lanes of a row, then the waves
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
#pragma unroll
    for (int k = 0; k < G; ++k) {
        ob[k] += __shfl_xor(ob[k], 16, 64);
        ob[k] += __shfl_xor(ob[k], 32, 64);
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
        reinterpret_cast<f32x4 *>(ring[wave])[t * 64 + lane] = o[t] + ob[t >> 2];
    if (g == 0) {
        red_m[wave][c] = m;
        red_l[wave][c] = l;
    }
    __syncthreads();
    float top = red_m[0][c];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        top = fmaxf(top, red_m[w][c]);
    float sum = 0.f, f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        f[w] = exp2_fast(red_m[w][c] - top);
        sum += f[w] * red_l[w][c];
    }
    if (!live)
        return;
    const float inv = a.splits > 1 ? 1.f : (sum == 0.f ? 0.f : 1.f / sum);
    const int64_t slot = ((int64_t)unit * a.splits + split) * kTileRows + c;
    if (a.splits > 1 && wave == 0 && g == 0) {
        a.part_ml[2 * slot] = top;
        a.part_ml[2 * slot + 1] = sum;
    }
#pragma unroll
    for (int t0 = 0; t0 < DT; t0 += kWaves) {
        const int t = t0 + wave;
        f32x4 v = reinterpret_cast<const f32x4 *>(ring[0])[t * 64 + lane] * f[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            v += reinterpret_cast<const f32x4 *>(ring[w])[t * 64 + lane] * f[w];
        v *= inv;
        const int col = 16 * t + 4 * g;
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

// The ranges of a tile's rows added: a workgroup a row.  Its threads take the
// ranges' references and sums together, then its waves the ranges in turn, D /
// 64 columns a lane, four rows of partial sums on their way at a time.
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendArgs a, int tile_rows) {
    constexpr int V = D / 64, kAhead = 4;
    typedef float vec __attribute__((ext_vector_type(V)));
    __shared__ float fac[kMaxSplits], red[8];
    __shared__ vec sums[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int unit = blockIdx.x / tile_rows, c = blockIdx.x % tile_rows;
    int b = unit;
    const int tile = b % a.tiles;
    b /= a.tiles;
    const int head = b % a.c.n_kv_heads, s = b / a.c.n_kv_heads;
    const SeqRows q = seq_rows(a.c, s);
    const int n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
    const int rows = n * a.group - tile * tile_rows;
    if (c >= rows)
        return;
    const int start = q.ctx - q.n;
    const int last_rho = tile * tile_rows + (rows < tile_rows ? rows : tile_rows) - 1;
    const TileView view = tile_view(a, start + tile * tile_rows / a.group, start + last_rho / a.group);
    const int64_t slot0 = (int64_t)unit * a.splits * tile_rows + c;

    float top = kNoMax;
    for (int k = threadIdx.x; k < view.used; k += 256)
        top = fmaxf(top, a.part_ml[2 * (slot0 + (int64_t)k * tile_rows)]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        top = fmaxf(top, __shfl_xor(top, o, 64));
    if (lane == 0)
        red[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float sum = 0.f;
    for (int k = threadIdx.x; k < view.used; k += 256) {
        const float *ml = a.part_ml + 2 * (slot0 + (int64_t)k * tile_rows);
        const float f = exp2_fast(ml[0] - top);
        fac[k] = f;
        sum += f * ml[1];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        sum += __shfl_xor(sum, o, 64);
    if (lane == 0)
        red[4 + wave] = sum;
    __syncthreads();
    sum = (red[4] + red[5]) + (red[6] + red[7]);

    const float *part = a.part + slot0 * D + lane * V;
    const int64_t step = (int64_t)tile_rows * D;
    vec v;
#pragma unroll
    for (int j = 0; j < V; ++j)
        v[j] = 0.f;
    int k = wave;
    for (; k + 4 * (kAhead - 1) < view.used; k += 4 * kAhead) {
        vec w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            w[i] = *reinterpret_cast<const vec *>(part + (k + 4 * i) * step);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            v += w[i] * fac[k + 4 * i];
    }
    for (; k < view.used; k += 4)
        v += *reinterpret_cast<const vec *>(part + k * step) * fac[k];
    sums[wave][lane] = v;
    __syncthreads();
    if (wave)
        return;
    v = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int rho = tile * tile_rows + c;
    const int64_t at = (int64_t)(q.row0 + rho / a.group) * a.ldo +
                       (head * a.group + rho % a.group) * a.o_head + lane * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (a.o_bf16)
            static_cast<uint16_t *>(a.O)[at + j] = (uint16_t)pack_bf16(v[j] * inv, 0.f);
        else
            static_cast<float *>(a.O)[at + j] = v[j] * inv;
    }
}

} // namespace

hipError_t launch_attend_decode(int head_dim, const AttendArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.c.n_seqs * a.c.n_kv_heads * a.tiles * a.splits));
    const dim3 block(64 * kWaves);
    if (head_dim == 64)
        hipLaunchKernelGGL(attend_decode_kernel<64>, grid, block, 0, stream, a);
    else if (head_dim == 128)
        hipLaunchKernelGGL(attend_decode_kernel<128>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(attend_decode_kernel<256>, grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_attend_join(int head_dim, int tile_rows, const AttendArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.c.n_seqs * a.c.n_kv_heads * a.tiles * tile_rows));
    if (head_dim == 64)
        hipLaunchKernelGGL(attend_join_kernel<64>, grid, dim3(256), 0, stream, a, tile_rows);
    else if (head_dim == 128)
        hipLaunchKernelGGL(attend_join_kernel<128>, grid, dim3(256), 0, stream, a, tile_rows);
    else
        hipLaunchKernelGGL(attend_join_kernel<256>, grid, dim3(256), 0, stream, a, tile_rows);
    return hipGetLastError();
}

} // namespace tsl
