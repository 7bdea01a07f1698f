// Internal interface between the C ABI of tsl_attn.h (attn.cpp) and its HIP
// kernels, and what those kernels share on the device: where a token of the
// cache lies and which tokens a tile of query rows sees.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "tsl_attn.h"

namespace tsl {

constexpr int kMaxRotateItems = 8;
constexpr int kMaxHeadDim = 512; // of rotate_heads

struct RotateArgs {
    struct Item {
        const void *X;
        void *Y;
        int64_t ldx, x_head, ldy, y_head;
        int32_t n_heads, x_bf16, y_bf16;
    } item[kMaxRotateItems];
    const int32_t *positions;
    const float *freq;
    int64_t ld_pos, M;
    int32_t heads; // of all items
    int32_t rot_dim, head_dim, pairs, inverse;
    int32_t wide; // every item takes the vector form
    uint32_t axis[kMaxHeadDim / 2 / 16]; // two bits a pair
};

hipError_t launch_rotate(const RotateArgs &a, hipStream_t stream);

// One record holds kBlock tokens of one head (tsl_attn.h, tsl_cache).
constexpr int kBlock = 32;
constexpr int record_bytes(int head_dim) { return 36 * head_dim; }

// Longest context; windows and first tokens are no longer either, so that
// positions and their differences fit 32 bits.
constexpr int kMaxContext = 1 << 30;

struct CacheArgs {
    char *pages;
    int64_t page_bytes, head_bytes;
    int32_t n_pages, shift; // records of a page and head: 1 << shift
    int32_t n_kv_heads;
    // sequences
    const int32_t *row_start, *context, *page_table;
    int64_t ld_table;
    int32_t rows, n_seqs, max_rows, max_pages;
};

// Division of numbers below 2^31 by one that the host knows: a product's upper
// half and a shift, where the compiler's division takes 35 instructions -- of
// which a workgroup's start would have a dozen.
struct Div {
    uint32_t mul, shift;
};
inline Div make_div(uint32_t d) {
    Div v = {0, 0};
    while ((uint64_t(1) << v.shift) < d)
        ++v.shift;
    v.mul = (uint32_t)((((uint64_t(1) << v.shift) - d) << 32) / d + 1);
    return v;
}
__host__ __device__ __forceinline__ int quotient(int n, Div d) {
    const uint32_t hi = (uint32_t)(((uint64_t)(uint32_t)n * d.mul) >> 32);
    return (int)((hi + (uint32_t)n) >> d.shift);
}

struct MoveArgs {
    CacheArgs c;
    void *K, *V;
    int64_t ldk, k_head, ldv, v_head;
    int32_t bf16;
    int32_t seq_blocks; // records a sequence's rows may span
    Div by_heads;
};

hipError_t launch_cache_append(int head_dim, const MoveArgs &a, hipStream_t stream);
hipError_t launch_cache_read(int head_dim, const MoveArgs &a, hipStream_t stream);

struct AttendArgs {
    CacheArgs c;
    const uint16_t *Q;
    void *O;
    int64_t ldq, q_head, ldo, o_head;
    float scale; // times log2 e
    int32_t group, window, sinks, o_bf16;
    Div by_group, by_tiles, by_heads, by_parts; // heads: of the cache
    int32_t rows;      // query rows of a sequence and K/V head, at most
    int32_t rows_min, rows_max; // sequences with fewer or more are another kernel's
    int32_t tiles;     // row tiles of a sequence and K/V head
    int32_t splits;    // many rows: ranges of tokens a tile is divided into at most
    int32_t shared;    // few rows: all records of the call in a row, cut into parts
    int32_t parts;     // few rows: waves
    int32_t units;     // sequences * heads * tiles; many rows: heads * tiles, at most
    int32_t min_share; // records of a range or part at least
    // sums of ranges: [range][tile rows][head_dim], and of each row its reference
    // exponent and sum.  Many rows: range = workgroup.  Few: a wave has sums of its
    // own of two tiles at most, the one that it goes on with (range = wave) and the
    // one that it begins and does not end (parts + wave)
    float *part, *part_ml;
    int32_t *spans; // shared: the first and last wave of each unit, (sequence * heads + head) * tiles + tile
    // many rows, where records are expanded once for the call: of image_seqs
    // sequences and each head up to image_records images of 128 head_dim bytes
    // (0: none), and of each its exponents and flags
    char *images;
    uint32_t *image_info;
    int32_t image_records, image_seqs;
    Div by_images;
    Div by_tile_rows; // the join
};

constexpr int kMaxShared = 1024; // sequences of a shared call
constexpr int kJoinWave = 16;  // ranges that one wave adds; 16 waves more
constexpr int kJoinLanes = 64; // ... that the lanes of a row add, with many rows
// attend_decode: tiles of 16 / P query rows (P 1, 2, or with head_dim up to 128 4),
// three stages of a record for each of four waves in a CU's 160 KB of LDS.
// Workgroups that share a CU (four: a start more a CU does not hide better):
constexpr int attend_groups(int head_dim) {
    const int n = 160 * 1024 / (4 * 3 * record_bytes(head_dim));
    return n > 4 ? 4 : n;
}

hipError_t launch_attend_decode(int head_dim, int tile_rows, const AttendArgs &a, hipStream_t stream);
constexpr int kPromptRows = 128; // of attend_prompt, head_dim 64 or 128
hipError_t launch_attend_prompt(int head_dim, const AttendArgs &a, hipStream_t stream);
hipError_t launch_attend_images(int head_dim, const AttendArgs &a, hipStream_t stream);
hipError_t launch_prompt_join(int head_dim, const AttendArgs &a, hipStream_t stream);
hipError_t launch_attend_join(int head_dim, int tile_rows, const AttendArgs &a, hipStream_t stream);

// ---- where tokens lie and which are seen ------------------------------------------
// (host code too, for tests without a GPU)

// A sequence's rows, clamped to what the operands have.
struct SeqRows {
    int row0, n, ctx;
};
__host__ __device__ __forceinline__ SeqRows seq_rows(const CacheArgs &c, int s) {
    SeqRows r;
    const int a = c.row_start[s], b = c.row_start[s + 1];
    r.row0 = a < 0 ? 0 : (a > c.rows ? c.rows : a);
    const int end = b < r.row0 ? r.row0 : (b > c.rows ? c.rows : b);
    r.n = end - r.row0;
    const int ctx = c.context[s];
    r.ctx = ctx < 0 ? 0 : (ctx > kMaxContext ? kMaxContext : ctx);
    return r;
}

// The record of a sequence's tokens 32 blk .. 32 blk + 31 (blk >= 0), or null
// where they are not there.
__host__ __device__ __forceinline__ char *record_of(const CacheArgs &c, int s, int head, int blk,
                                           int rec_bytes) {
    const int page = blk >> c.shift;
    if (page >= c.max_pages)
        return nullptr;
    const int p = c.page_table[s * c.ld_table + page];
    if (p < 0 || p >= c.n_pages)
        return nullptr;
    return c.pages + p * c.page_bytes + head * c.head_bytes +
           (int64_t)(blk & ((1 << c.shift) - 1)) * rec_bytes;
}

// What a tile of query rows sees: positions first .. last (of its rows), and
// the records that hold a visible token of any row, as a list: `lead` records
// from 0 on (first tokens that stay visible), then those from `from` on.
struct TileView {
    int first, last;
    int lead, from, count;
    int share, used; // of a tile in ranges: records of one, ranges with any
};
__host__ __device__ __forceinline__ TileView tile_view(const AttendArgs &a, int first, int last) {
    TileView v;
    v.first = first;
    v.last = last;
    const int cap = a.c.max_pages << (a.c.shift + 5); // at most 2^30
    const int end = last + 1 < cap ? last + 1 : cap;  // tokens below it
    v.lead = v.from = v.count = 0;
    if (end > 0) {
        int lo = a.window && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
        lo = lo < end ? lo : end;
        const int keep = a.sinks < end ? a.sinks : end;
        v.from = lo >> 5;
        const int lead = (keep + 31) >> 5;
        v.lead = lead < v.from ? lead : v.from;
        v.count = v.lead + ((end + 31) >> 5) - v.from;
    }
    return v;
}
// Query rows of a sequence and K/V head, 0 where they are not this kernel's.
__host__ __device__ __forceinline__ int rows_of(const AttendArgs &a, const SeqRows &q) {
    const int rows = (q.n < a.c.max_rows ? q.n : a.c.max_rows) * a.group;
    return rows < a.rows_min || rows > a.rows_max ? 0 : rows;
}
// What tile `tile` of `tile_rows` query rows sees; `rows` of it and later ones.
__host__ __device__ __forceinline__ TileView view_of(const AttendArgs &a, const SeqRows &q, int tile,
                                                     int tile_rows, int rows) {
    const int last = tile * tile_rows + (rows < tile_rows ? rows : tile_rows) - 1, start = q.ctx - q.n;
    return tile_view(a, start + quotient(tile * tile_rows, a.by_group), start + quotient(last, a.by_group));
}
// What all rows of a sequence together see.
__host__ __device__ __forceinline__ TileView sequence_view(const AttendArgs &a, const SeqRows &q) {
    const int n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
    return tile_view(a, q.ctx - q.n, q.ctx - q.n + n - 1);
}
// ... and at most so many records of `cap` tokens.
inline int64_t most_records(int64_t cap, int64_t rows, int64_t window, int64_t sinks) {
    const int64_t all = (cap + kBlock - 1) / kBlock;
    const int64_t some = (window + rows) / kBlock + 2 + (sinks + kBlock - 1) / kBlock;
    return window && some < all ? some : all;
}
// Where a record that a tile sees stands in its sequence's list.
__host__ __device__ __forceinline__ int place_of(const TileView &all, int blk) {
    return blk < all.lead ? blk : blk - all.from + all.lead;
}
__host__ __device__ __forceinline__ int view_block(const TileView &v, int i) {
    return i < v.lead ? i : v.from + i - v.lead;
}
// Whether some row of the tile may see token j (first tokens and a window between them).
__host__ __device__ __forceinline__ bool any_sees(const AttendArgs &a, const TileView &v, int j) {
    return (j <= v.last) & (!a.window | (j > v.first - a.window) | (j < a.sinks));
}
// ... and all of a record's.
__host__ __device__ __forceinline__ bool any_sees_all(const AttendArgs &a, const TileView &v, int blk) {
    const int j = blk * kBlock;
    return (j + 31 <= v.last) & (!a.window | (j > v.first - a.window) | (j + 31 < a.sinks));
}
// Whether every row of the tile sees all tokens of a record.
__host__ __device__ __forceinline__ bool sees_all(const AttendArgs &a, const TileView &v, int blk) {
    const int lo = blk * kBlock, hi = lo + kBlock - 1;
    return hi <= v.first && (!a.window || lo > v.last - a.window || hi < a.sinks);
}
// Whether a row at position pos (its window starting at lo) sees token j.
__host__ __device__ __forceinline__ bool sees(const AttendArgs &a, int pos, int lo, int j) {
    return j <= pos && (j >= lo || j < a.sinks);
}
__host__ __device__ __forceinline__ int window_start(const AttendArgs &a, int pos) {
    return a.window ? pos - a.window + 1 : 0;
}

// Two binary32 values as a pair of bf16, to nearest even (one instruction).
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// The sum of the lanes up to each: within rows of 16, then over the rows.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true); // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    const int a = __builtin_amdgcn_readlane(v, 15), b = __builtin_amdgcn_readlane(v, 31),
              c = __builtin_amdgcn_readlane(v, 47);
    const int row = (int)((threadIdx.x & 63) >> 4);
    return v + (row > 0 ? a : 0) + (row > 1 ? b : 0) + (row > 2 ? c : 0);
}

// Many rows: a workgroup's tile.  The tiles that there are, of all sequences in a
// row and in each the later ones first (they see more tokens), heads innermost;
// each in as many ranges as let the workgroups fit the CUs.
struct PromptTile {
    int s, head, tile, unit, split, splits;
    int rank; // of the sequence among those that have tiles
    SeqRows q;
};
constexpr int kPromptPlaces = 512; // workgroups that run at once
// `index`: unit * splits + split, or of the join the unit.
__device__ __forceinline__ bool prompt_tile(const AttendArgs &a, int index, bool ranges, PromptTile &t) {
    const int lane = threadIdx.x & 63;
    int total = 0, before = 0, f = 0;
    t.rank = 0;
    t.splits = 1;
    t.split = 0;
    t.unit = index;
    bool finding = a.splits == 1; // (no need to know how many there are)
    if (finding)
        f = quotient(index, a.by_heads);
    for (int base = 0;;) {
        SeqRows q = {0, 0, 0};
        int own = 0;
        if (base + lane < a.c.n_seqs) {
            q = seq_rows(a.c, base + lane);
            own = (rows_of(a, q) + kPromptRows - 1) / kPromptRows;
        }
        const int upto = wave_scan(own), all = __builtin_amdgcn_readlane(upto, 63);
        if (!finding) {
            total += all;
            base += 64;
            if (base < a.c.n_seqs)
                continue;
            const int units = total * a.c.n_kv_heads;
            if (units < kPromptPlaces) { // (exact: the quotients are below 2^10)
                const float n = (float)kPromptPlaces + 0.5f;
                const int fit = units ? (int)(n * __builtin_amdgcn_rcpf((float)units)) : 1;
                t.splits = __builtin_amdgcn_readfirstlane(fit < a.splits ? fit : a.splits);
            }
            if (ranges && t.splits > 1) {
                if (index >= kPromptPlaces)
                    return false;
                t.unit = __builtin_amdgcn_readfirstlane(
                    (int)(((float)index + 0.5f) * __builtin_amdgcn_rcpf((float)t.splits)));
                t.split = index - t.unit * t.splits;
            }
            if (t.unit >= units)
                return false;
            f = quotient(t.unit, a.by_heads);
            finding = true;
            base = 0;
            if (a.c.n_seqs > 64)
                continue;
        }
        const uint64_t past = __ballot(before + upto > f);
        if (past) {
            const int at = __builtin_ctzll(past);
            t.s = base + at;
            t.rank += __builtin_popcountll(__ballot(own > 0) & ((1ull << at) - 1));
            t.head = t.unit - f * a.c.n_kv_heads;
            t.tile = before + __builtin_amdgcn_readlane(upto, at) - 1 - f;
            // (row_start that descends may give any sum)
            if (t.tile < 0 || t.tile >= __builtin_amdgcn_readlane(own, at))
                return false;
            t.q.row0 = __builtin_amdgcn_readlane(q.row0, at);
            t.q.n = __builtin_amdgcn_readlane(q.n, at);
            t.q.ctx = __builtin_amdgcn_readlane(q.ctx, at);
            return true;
        }
        before += all;
        t.rank += __builtin_popcountll(__ballot(own > 0));
        base += 64;
        if (base >= a.c.n_seqs)
            return false;
    }
}
// The sequence with tiles of that rank.
__device__ __forceinline__ bool prompt_of_rank(const AttendArgs &a, int rank, int &s, SeqRows &of) {
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < a.c.n_seqs; base += 64) {
        SeqRows q = {0, 0, 0};
        if (base + lane < a.c.n_seqs)
            q = seq_rows(a.c, base + lane);
        uint64_t have = __ballot(rows_of(a, q) > 0);
        const int n = __builtin_popcountll(have);
        if (rank < n) {
            while (rank--)
                have &= have - 1;
            const int at = __builtin_ctzll(have);
            s = base + at;
            of.row0 = __builtin_amdgcn_readlane(q.row0, at);
            of.n = __builtin_amdgcn_readlane(q.n, at);
            of.ctx = __builtin_amdgcn_readlane(q.ctx, at);
            return true;
        }
        rank -= n;
    }
    return false;
}
// A tile's ranges.
__host__ __device__ __forceinline__ void divide(const AttendArgs &a, int splits, TileView &v) {
    v.share = (int)(((uint32_t)v.count + splits - 1) / (uint32_t)splits);
    v.share = v.share > a.min_share ? v.share : a.min_share;
    v.used = (v.count + v.share - 1) / v.share;
}

// Keeps a branch that few steps take from being made part of all of them.
__device__ __forceinline__ void rare() { asm volatile(""); }

// Where no running maximum was set yet; its exponentials of it are zero.
constexpr float kNoMax = -3.0e38f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

} // namespace tsl
