// The C ABI of tsl_attn.h.  Checks run before anything is enqueued; no exception leaves an
// entry point.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cstddef>

#include "attn.hpp"
#include "group.hpp"
#include "tsl_attn.h"

using namespace tsl;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxTokens = int64_t(1) << 30; // of a page table's row
constexpr int kMaxSeqs = 65535;
constexpr int kMaxHeads = 1024;
constexpr float kLog2e = 1.44269504088896340736f;

bool dense_type(int d) { return d == TSL_F32 || d == TSL_BF16; }
size_t elem(int d) { return d == TSL_F32 ? 4 : 2; }

// A [rows][heads][cols] operand (tsl_attn.h, "Heads").
struct Heads {
    const void *p;
    int64_t rows, heads, cols, ld, head;
    size_t e;

    // strides that keep its elements apart, in either nesting
    bool sound() const {
        if (ld >= kMaxStride || head >= kMaxStride)
            return false;
        if (rows <= 1 && heads <= 1)
            return true;
        if (rows <= 1)
            return head >= cols;
        if (heads <= 1)
            return ld >= cols;
        return (head >= cols && ld >= (heads - 1) * head + cols) ||
               (ld >= cols && head >= (rows - 1) * ld + cols);
    }
    size_t bytes() const {
        return (size_t)((rows - 1) * ld + (heads - 1) * head + cols) * e;
    }
    bool wide() const { // 16-byte aligned runs throughout
        const int64_t run = 16 / (int64_t)e;
        return aligned(p, 16) && (rows <= 1 || ld % run == 0) && (heads <= 1 || head % run == 0);
    }
};

// Whether two operands share a byte: their spans, and where those meet (slices
// of one array) the rows of each pair of heads.
bool clash(const Heads &a, const Heads &b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || !overlaps(a.p, a.bytes(), b.p, b.bytes()))
        return false;
    // a lone row's stride says nothing
    const int64_t la = a.rows > 1 ? a.ld : a.cols, lb = b.rows > 1 ? b.ld : b.cols;
    for (int64_t i = 0; i < a.heads; ++i)
        for (int64_t j = 0; j < b.heads; ++j)
            if (matrices_overlap(static_cast<const char *>(a.p) + i * a.head * (int64_t)a.e, a.rows,
                                 a.cols, la, a.e,
                                 static_cast<const char *>(b.p) + j * b.head * (int64_t)b.e, b.rows,
                                 b.cols, lb, b.e))
                return true;
    return false;
}

tsl_status cache_check(const tsl_cache *c, bool with_pages) {
    if (!c || c->n_pages < 1 || c->page_tokens < 1 || c->n_kv_heads < 1 || c->head_dim < 1 ||
        (with_pages && !c->pages))
        return TSL_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) ||
        c->page_tokens < kBlock || c->page_tokens > 4096 ||
        (c->page_tokens & (c->page_tokens - 1)) || c->n_kv_heads > kMaxHeads ||
        c->n_pages > INT32_MAX)
        return TSL_ERR_UNSUPPORTED;
    if (with_pages && !aligned(c->pages, 256))
        return TSL_ERR_MISALIGNED;
    return TSL_OK;
}

size_t page_size(const tsl_cache &c) {
    return (size_t)c.n_kv_heads * (size_t)(c.page_tokens / kBlock) * record_bytes(c.head_dim);
}

tsl_status seqs_check(const tsl_cache &c, const tsl_seqs *q, bool with_arrays) {
    if (!q || q->n_seqs < 0 || q->rows < 0 || q->max_rows < 0 || q->max_context < 0 ||
        q->max_pages < 0)
        return TSL_ERR_INVALID_ARG;
    if (with_arrays && q->n_seqs > 0) {
        if (!q->row_start || !q->context || (q->max_pages > 0 && !q->page_table))
            return TSL_ERR_INVALID_ARG;
        if (q->n_seqs > 1 && q->ld_table < q->max_pages)
            return TSL_ERR_INVALID_ARG;
    }
    if (q->n_seqs > kMaxSeqs || q->rows >= kMaxRows || q->ld_table >= kMaxStride ||
        (int64_t)q->max_pages * c.page_tokens > kMaxTokens)
        return TSL_ERR_UNSUPPORTED;
    if (with_arrays &&
        (!aligned(q->row_start, 4) || !aligned(q->context, 4) || !aligned(q->page_table, 4)))
        return TSL_ERR_MISALIGNED;
    return TSL_OK;
}

bool nothing(const tsl_seqs &q) { return q.n_seqs == 0 || q.rows == 0 || q.max_rows == 0; }

CacheArgs cache_args(const tsl_cache &c, const tsl_seqs &q) {
    CacheArgs a{};
    a.pages = static_cast<char *>(c.pages);
    a.page_bytes = (int64_t)page_size(c);
    a.head_bytes = a.page_bytes / c.n_kv_heads;
    a.n_pages = (int32_t)c.n_pages;
    a.shift = 0;
    while ((kBlock << a.shift) < c.page_tokens)
        ++a.shift;
    a.n_kv_heads = c.n_kv_heads;
    a.row_start = q.row_start;
    a.context = q.context;
    a.page_table = q.page_table;
    a.ld_table = q.n_seqs > 1 ? q.ld_table : 0;
    a.rows = (int32_t)q.rows;
    a.n_seqs = q.n_seqs;
    a.max_rows = (int32_t)std::min<int64_t>(q.max_rows, q.rows);
    a.max_pages = q.max_pages;
    return a;
}

// Whether an operand of the caller's touches the cache or the arrays that
// the kernels read.
bool meets_cache(const Heads &h, const tsl_cache &c, const tsl_seqs &q, bool arrays) {
    if (!h.p)
        return false;
    const size_t pages = page_size(c) * (size_t)c.n_pages;
    if (overlaps(h.p, h.bytes(), c.pages, pages))
        return true;
    if (!arrays)
        return false;
    return overlaps(h.p, h.bytes(), q.row_start, 4 * ((size_t)q.n_seqs + 1)) ||
           overlaps(h.p, h.bytes(), q.context, 4 * (size_t)q.n_seqs) ||
           (q.max_pages > 0 &&
            overlaps(h.p, h.bytes(), q.page_table,
                     4 * ((size_t)(q.n_seqs - 1) * (size_t)(q.n_seqs > 1 ? q.ld_table : 0) +
                          (size_t)q.max_pages)));
}

// Checks and arguments that cache_append and cache_read share.
tsl_status move_args(const tsl_cache *cache, const tsl_seqs *seqs, tsl_dtype dtype, const void *K,
                     int64_t ldk, int64_t k_head, const void *V, int64_t ldv, int64_t v_head,
                     bool read, MoveArgs *out) {
    tsl_status st = cache_check(cache, true);
    if (st != TSL_OK)
        return st;
    if ((st = seqs_check(*cache, seqs, true)) != TSL_OK)
        return st;
    if (!dense_type(dtype) || (read ? !K && !V : !K || !V))
        return TSL_ERR_INVALID_ARG;
    const size_t e = elem(dtype);
    const Heads k = {K, seqs->rows, cache->n_kv_heads, cache->head_dim, ldk, k_head, e};
    const Heads v = {V, seqs->rows, cache->n_kv_heads, cache->head_dim, ldv, v_head, e};
    for (const Heads *h : {&k, &v}) {
        if (!h->p)
            continue;
        if (h->ld < 0 || h->head < 0 || !h->sound())
            return TSL_ERR_INVALID_ARG;
        if (!h->wide())
            return TSL_ERR_MISALIGNED;
    }
    MoveArgs a{};
    a.c = cache_args(*cache, *seqs);
    // a run of n rows touches at most so many records, wherever it starts
    a.seq_blocks = a.c.max_rows > 0 ? (a.c.max_rows + kBlock - 2) / kBlock + 1 : 0;
    if ((int64_t)a.c.n_kv_heads * a.seq_blocks > kMaxBlocks) // (of a sequence)
        return TSL_ERR_UNSUPPORTED;
    if (!nothing(*seqs) &&
        (meets_cache(k, *cache, *seqs, read) || meets_cache(v, *cache, *seqs, read) ||
         (read && clash(k, v))))
        return TSL_ERR_INVALID_ARG;
    a.K = const_cast<void *>(K);
    a.V = const_cast<void *>(V);
    a.ldk = ldk;
    a.k_head = k_head;
    a.ldv = ldv;
    a.v_head = v_head;
    a.bf16 = dtype == TSL_BF16;
    a.by_heads = make_div((uint32_t)a.c.n_kv_heads);
    *out = a;
    return TSL_OK;
}

// How one of cache_attention's kernels divides its work; a function of sizes alone.
struct AttendPlan {
    int32_t rows;      // query rows of a sequence and K/V head, at most
    int32_t tile_rows, tiles, splits, min_share;
    int32_t shared, parts;
    int64_t units, ranges; // (sequence, head, tile); ranges with sums of their own
    // records of a sequence and head that are expanded once (0: none), sequences
    int32_t images, image_seqs;
    size_t image_bytes;
    size_t bytes;
};

// Query rows of a sequence and K/V head up to which the kernel of few rows takes
// it, where every tile of 16 expands the records it reads anew.  Of one sequence
// of 4000 tokens, heads of 128, 48 rows took 22.7 us with it and 24.2 with the
// other, 64 24.7 and 25.2, 128 32 and 26; of 16000 tokens 64 33 and 40, 96 41 and
// 38; of 16 sequences of 4000 48 56 and 65, 64 69 and 66, 128 118 and 72.
constexpr int64_t kFewRows = 64;
constexpr int64_t kCUs = 256;
constexpr int64_t kMaxWaves = 4 * kMaxBlocks; // of the kernel of few rows
// Records that a wave takes alone, with no join after it: 4 and 8 of them took
// 9.0 and 12.7 us so, 10.4 and 10.6 divided.
constexpr int kWholeRecords = 6;
// Records that are worth a wave of their own with few rows, and a workgroup's
// range with many (128 rows over 4000 tokens: 32 us with ranges of 4, 25 of 8, 31
// of 16).
constexpr int kAttendShare = 1, kPromptShare = 8;

// Expanding the records of the sequences once costs a launch and about what two
// tiles' expansion does: it is done for so many records times the tiles beyond two
// (8 heads, 500 records: 3 tiles 29.3 us so and 26.7 without, 4 34.2 and 31.3, 5
// 33.8 and 33.6; 4000 records: 2 tiles 53.8 and 52.2, 3 59.1 and 62.2, 4 66.6 and
// 76.5, 5 75 and 93), and this is the most memory it takes.
constexpr int64_t kImageWork = 2048;
constexpr int64_t kImageBytes = int64_t(1) << 30;

// The plan of the images: for as many sequences as there is room for.
void plan_images(const tsl_cache &c, const tsl_seqs &q, int64_t group, int32_t window, int32_t sinks,
                 bool few, AttendPlan *p) {
    p->images = p->image_seqs = 0;
    p->image_bytes = 0;
    const int64_t n =
        most_records(std::min<int64_t>(q.max_context, (int64_t)q.max_pages * c.page_tokens),
                     std::min<int64_t>(q.max_rows, q.rows), window, sinks);
    if (few || p->tiles <= 2 || n == 0)
        return;
    // (of sequences with more rows than the other kernel's, one has max_rows)
    const int64_t others = std::max<int64_t>(0, q.rows * group - p->rows) / (kFewRows + 1);
    const int64_t one = n * c.n_kv_heads, image = 128 * c.head_dim;
    const int64_t seqs = std::min({(int64_t)q.n_seqs, 1 + others, kImageBytes / (one * image)});
    if (seqs * one * (p->tiles - 2) < kImageWork)
        return;
    p->images = (int32_t)n;
    p->image_seqs = (int32_t)seqs;
    p->image_bytes = round_up((size_t)(one * seqs * image), 256) + round_up((size_t)(one * seqs) * 4, 256);
}

tsl_status plan_kernel(const tsl_cache &c, const tsl_seqs &q, int64_t group, int64_t rows, bool few,
                       int tile_rows, int32_t window, int32_t sinks, AttendPlan *p) {
    p->rows = (int32_t)rows;
    p->tile_rows = tile_rows;
    int64_t seen = std::min<int64_t>(q.max_context, (int64_t)q.max_pages * c.page_tokens);
    if (window)
        seen = std::min<int64_t>(seen, (int64_t)window + sinks + tile_rows + 2 * kBlock);
    const int64_t records = (seen + kBlock - 1) / kBlock;
    p->tiles = (int32_t)((rows + tile_rows - 1) / tile_rows);
    p->units = (int64_t)q.n_seqs * c.n_kv_heads * p->tiles;
    if (!few && q.n_seqs > 1) { // tiles that the rows of the call may come to
        const int64_t all = q.rows * group;
        p->units = std::min(p->units, (all / tile_rows + std::min<int64_t>(q.n_seqs, all / (kFewRows + 1))) *
                                          c.n_kv_heads);
    }
    p->min_share = few ? kAttendShare : kPromptShare;
    const int64_t most = std::max<int64_t>(1, (records + p->min_share - 1) / p->min_share);
    p->shared = 0;
    p->splits = 1;
    p->parts = (int32_t)std::min<int64_t>(p->units, kMaxWaves + 1);
    p->ranges = 0;
    // (a call of more sequences than that has several tiles for every wave as it
    // is; records, and the waves' number beside them, are counted in 32 bits)
    const int64_t held = ((int64_t)q.max_pages * c.page_tokens + kBlock - 1) / kBlock;
    const int64_t places = kCUs * 4 * attend_groups(c.head_dim); // waves that fit
    if (few && records > kWholeRecords && q.n_seqs <= kMaxShared && p->units * held <= INT32_MAX - places) {
        p->shared = 1;
        p->parts = (int32_t)std::min(places, p->units * most);
        p->ranges = 2 * p->parts;
    }
    if (!few) {
        // one sequence has max_rows; how many ranges there are is for the kernel to say,
        // which cuts tiles only while all their ranges fit the places
        p->splits = (int32_t)std::max<int64_t>(
            1, std::min(most, kPromptPlaces / std::max<int64_t>(1, (int64_t)p->tiles * c.n_kv_heads)));
        if (p->splits > 1)
            p->ranges = std::min<int64_t>(kPromptPlaces, p->units * p->splits);
        p->parts = (int32_t)std::min<int64_t>(std::max(p->units, p->ranges), kMaxBlocks + 1);
    }
    // workgroups of a launch: four waves with few rows, and four rows of the join's
    // (whose other dimensions are heads and sequences)
    if (few ? p->parts > kMaxWaves || (p->ranges && rows > kMaxBlocks)
            : p->parts > kMaxBlocks)
        return TSL_ERR_UNSUPPORTED;
    plan_images(c, q, group, window, sinks, few, p);
    p->bytes = p->image_bytes + round_up((size_t)p->ranges * tile_rows * (size_t)(c.head_dim + 2) * 4 +
                            (p->shared ? (size_t)p->units * 8 : 0),
                        256);
    return TSL_OK;
}

// The kernels of a call: of few rows, of many, or both, each for the sequences of
// its kind.  A lone sequence goes by max_rows.
struct AttendPlans {
    bool few, many;
    AttendPlan f, m;
    size_t bytes() const { return (few ? f.bytes : 0) + (many ? m.bytes : 0); }
};

tsl_status attend_plan(const tsl_cache &c, const tsl_seqs &q, int32_t n_q_heads, int32_t window,
                       int32_t sinks, AttendPlans *p) {
    const int64_t group = n_q_heads / c.n_kv_heads;
    const int64_t rows = std::min<int64_t>(q.max_rows, q.rows) * group;
    if (rows > kMaxContext)
        return TSL_ERR_UNSUPPORTED;
    p->many = rows > kFewRows && c.head_dim <= 128;
    p->few = !p->many || q.n_seqs > 1;
    if (p->few) {
        // beside long sequences most of the others have one row
        const int64_t most = p->many ? kFewRows : rows, typical = p->many ? group : rows;
        const int tile = typical > 8 ? 16 : (typical > 4 || c.head_dim > 128 ? 8 : 4);
        const tsl_status st = plan_kernel(c, q, group, most, true, tile, window, sinks, &p->f);
        if (st != TSL_OK)
            return st;
    }
    return p->many ? plan_kernel(c, q, group, rows, false, kPromptRows, window, sinks, &p->m) : TSL_OK;
}

tsl_status attend_check(const tsl_cache *cache, const tsl_seqs *seqs, int32_t n_q_heads,
                        int32_t window, int32_t sinks, bool run) {
    tsl_status st = cache_check(cache, run);
    if (st != TSL_OK)
        return st;
    if ((st = seqs_check(*cache, seqs, run)) != TSL_OK)
        return st;
    if (n_q_heads < 1 || window < 0 || sinks < 0)
        return TSL_ERR_INVALID_ARG;
    if (n_q_heads % cache->n_kv_heads)
        return TSL_ERR_NOT_DIVISIBLE;
    if (n_q_heads > kMaxHeads || window > kMaxContext || sinks > kMaxContext)
        return TSL_ERR_UNSUPPORTED;
    return TSL_OK;
}

} // namespace

extern "C" tsl_status rotate_heads(int32_t n_items, const tsl_rotate_item *items, int64_t M,
                                   const tsl_rotary *rotary, int inverse, void *stream) {
    if (!items || !rotary || n_items < 1 || M < 0 || (inverse != 0 && inverse != 1))
        return TSL_ERR_INVALID_ARG;
    const tsl_rotary &r = *rotary;
    if (!r.positions || !r.freq || r.axes < 1 || r.head_dim < 2 || r.rot_dim < 2 ||
        r.rot_dim % 2 || r.rot_dim > r.head_dim ||
        (r.style != TSL_ROTARY_HALVES && r.style != TSL_ROTARY_PAIRS))
        return TSL_ERR_INVALID_ARG;
    if (n_items > kMaxRotateItems || r.axes > 4 || r.head_dim > kMaxHeadDim || M >= kMaxRows)
        return TSL_ERR_UNSUPPORTED;
    if (r.axes > 1 && (r.ld_pos < M || r.ld_pos >= kMaxStride))
        return TSL_ERR_INVALID_ARG;
    if (!aligned(r.positions, 4) || !aligned(r.freq, 4))
        return TSL_ERR_MISALIGNED;
    RotateArgs a{};
    for (int p = 0; p < r.rot_dim / 2 && r.pair_axis; ++p) {
        if (r.pair_axis[p] >= r.axes)
            return TSL_ERR_INVALID_ARG;
        a.axis[p >> 4] |= (uint32_t)r.pair_axis[p] << (2 * (p & 15));
    }
    const int half = r.rot_dim / 2;
    bool wide = r.head_dim % 8 == 0 &&
                (r.style == TSL_ROTARY_HALVES ? half % 8 == 0 : r.rot_dim % 8 == 0);
    int64_t heads = 0;
    Heads x[kMaxRotateItems], y[kMaxRotateItems];
    for (int i = 0; i < n_items; ++i) {
        const tsl_rotate_item &it = items[i];
        if (!it.X || !it.Y || it.n_heads < 1 || !dense_type(it.xdtype) || !dense_type(it.ydtype) ||
            it.ldx < 0 || it.x_head < 0 || it.ldy < 0 || it.y_head < 0)
            return TSL_ERR_INVALID_ARG;
        if (it.n_heads > kMaxHeads)
            return TSL_ERR_UNSUPPORTED;
        x[i] = Heads{it.X, M, it.n_heads, r.head_dim, it.ldx, it.x_head, elem(it.xdtype)};
        y[i] = Heads{it.Y, M, it.n_heads, r.head_dim, it.ldy, it.y_head, elem(it.ydtype)};
        if (!x[i].sound() || !y[i].sound())
            return TSL_ERR_INVALID_ARG;
        if (!aligned(it.X, x[i].e) || !aligned(it.Y, y[i].e))
            return TSL_ERR_MISALIGNED;
        wide = wide && x[i].wide() && y[i].wide();
        heads += it.n_heads;
        a.item[i] = RotateArgs::Item{it.X,       it.Y,      it.ldx, it.x_head,
                                     it.ldy,     it.y_head, it.n_heads, it.xdtype == TSL_BF16,
                                     it.ydtype == TSL_BF16};
    }
    if (M == 0)
        return TSL_OK;
    const Heads pos = {r.positions, r.axes, 1, M, r.axes > 1 ? r.ld_pos : M, 0, 4};
    const Heads freq = {r.freq, 1, 1, half, half, 0, 4};
    for (int i = 0; i < n_items; ++i) {
        if (clash(y[i], pos) || clash(y[i], freq))
            return TSL_ERR_INVALID_ARG;
        for (int j = 0; j < n_items; ++j) {
            const bool own = i == j && y[i].p == x[i].p && y[i].e == x[i].e &&
                             (M == 1 || y[i].ld == x[i].ld) &&
                             (y[i].heads == 1 || y[i].head == x[i].head);
            if ((!own && clash(y[i], x[j])) || (i < j && clash(y[i], y[j])))
                return TSL_ERR_INVALID_ARG;
        }
    }
    a.positions = r.positions;
    a.freq = r.freq;
    a.ld_pos = r.ld_pos;
    a.M = M;
    a.heads = (int32_t)heads;
    a.rot_dim = r.rot_dim;
    a.head_dim = r.head_dim;
    a.pairs = r.style == TSL_ROTARY_PAIRS;
    a.inverse = inverse;
    a.wide = wide;
    return from_hip(launch_rotate(a, static_cast<hipStream_t>(stream)));
}

extern "C" tsl_status cache_size(const tsl_cache *cache, size_t *bytes) {
    if (!bytes)
        return TSL_ERR_INVALID_ARG;
    const tsl_status st = cache_check(cache, false);
    if (st == TSL_OK)
        *bytes = page_size(*cache) * (size_t)cache->n_pages;
    return st;
}

extern "C" tsl_status cache_append(const tsl_cache *cache, const tsl_seqs *seqs, tsl_dtype dtype,
                                   const void *K, int64_t ldk, int64_t k_head, const void *V,
                                   int64_t ldv, int64_t v_head, void *stream) {
    MoveArgs a;
    const tsl_status st =
        move_args(cache, seqs, dtype, K, ldk, k_head, V, ldv, v_head, false, &a);
    if (st != TSL_OK || nothing(*seqs))
        return st;
    return from_hip(launch_cache_append(cache->head_dim, a, static_cast<hipStream_t>(stream)));
}

extern "C" tsl_status cache_read(const tsl_cache *cache, const tsl_seqs *seqs, tsl_dtype dtype,
                                 void *K, int64_t ldk, int64_t k_head, void *V, int64_t ldv,
                                 int64_t v_head, void *stream) {
    MoveArgs a;
    const tsl_status st = move_args(cache, seqs, dtype, K, ldk, k_head, V, ldv, v_head, true, &a);
    if (st != TSL_OK || nothing(*seqs))
        return st;
    return from_hip(launch_cache_read(cache->head_dim, a, static_cast<hipStream_t>(stream)));
}

extern "C" tsl_status cache_attention_workspace_size(const tsl_cache *cache, const tsl_seqs *seqs,
                                                     int32_t n_q_heads, int32_t window,
                                                     int32_t sinks, size_t *bytes) {
    if (!bytes)
        return TSL_ERR_INVALID_ARG;
    tsl_status st = attend_check(cache, seqs, n_q_heads, window, sinks, false);
    AttendPlans p;
    if (st == TSL_OK && (st = attend_plan(*cache, *seqs, n_q_heads, window, sinks, &p)) == TSL_OK)
        *bytes = p.bytes();
    return st;
}

extern "C" tsl_status cache_attention(const tsl_cache *cache, const tsl_seqs *seqs,
                                      int32_t n_q_heads, const void *Q, int64_t ldq, int64_t q_head,
                                      float scale, int32_t window, int32_t sinks, tsl_dtype odtype,
                                      void *O, int64_t ldo, int64_t o_head, void *workspace,
                                      size_t ws_bytes, void *stream) {
    tsl_status st = attend_check(cache, seqs, n_q_heads, window, sinks, true);
    if (st != TSL_OK)
        return st;
    if (!Q || !O || !dense_type(odtype) || !isfinite(scale * kLog2e) || ldq < 0 || q_head < 0 || ldo < 0 ||
        o_head < 0)
        return TSL_ERR_INVALID_ARG;
    const Heads q = {Q, seqs->rows, n_q_heads, cache->head_dim, ldq, q_head, 2};
    const Heads o = {O, seqs->rows, n_q_heads, cache->head_dim, ldo, o_head, elem(odtype)};
    if (!q.sound() || !o.sound())
        return TSL_ERR_INVALID_ARG;
    if (!q.wide() || !o.wide())
        return TSL_ERR_MISALIGNED;
    AttendPlans p;
    if ((st = attend_plan(*cache, *seqs, n_q_heads, window, sinks, &p)) != TSL_OK)
        return st;
    if (nothing(*seqs))
        return TSL_OK;
    if (p.bytes()) {
        if (!workspace || ws_bytes < p.bytes())
            return TSL_ERR_BUFFER_TOO_SMALL;
        if (!aligned(workspace, 256))
            return TSL_ERR_MISALIGNED;
        const Heads ws = {workspace, 1, 1, (int64_t)p.bytes(), (int64_t)p.bytes(), 0, 1};
        if (clash(ws, q) || clash(ws, o) || meets_cache(ws, *cache, *seqs, true))
            return TSL_ERR_INVALID_ARG;
    }
    if (clash(o, q) || meets_cache(o, *cache, *seqs, true))
        return TSL_ERR_INVALID_ARG;
    AttendArgs a{};
    a.c = cache_args(*cache, *seqs);
    a.Q = static_cast<const uint16_t *>(Q);
    a.O = O;
    a.ldq = ldq;
    a.q_head = q_head;
    a.ldo = ldo;
    a.o_head = o_head;
    a.scale = scale * kLog2e;
    a.group = n_q_heads / cache->n_kv_heads;
    a.window = window;
    a.sinks = sinks;
    a.o_bf16 = odtype == TSL_BF16;
    a.by_group = make_div((uint32_t)a.group);
    a.by_heads = make_div((uint32_t)cache->n_kv_heads);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    for (const bool few : {true, false}) {
        if (few ? !p.few : !p.many)
            continue;
        const AttendPlan &k = few ? p.f : p.m;
        // query rows of a sequence and head that this kernel takes
        a.rows_min = few || !p.few ? 0 : (int32_t)kFewRows + 1;
        a.rows_max = few && p.many ? (int32_t)kFewRows : INT32_MAX;
        a.rows = k.rows;
        a.by_tiles = make_div((uint32_t)k.tiles);
        a.by_parts = make_div((uint32_t)k.parts);
        a.tiles = k.tiles;
        a.splits = k.splits;
        a.shared = k.shared;
        a.parts = k.parts;
        a.units = (int32_t)k.units;
        a.min_share = k.min_share;
        a.image_records = k.images;
        a.image_seqs = k.image_seqs;
        if (k.images) {
            a.by_images = make_div((uint32_t)k.images);
            a.images = ws;
            a.image_info = reinterpret_cast<uint32_t *>(
                ws + k.image_bytes -
                round_up((size_t)k.images * k.image_seqs * cache->n_kv_heads * 4, 256));
        }
        if (k.ranges) {
            char *const at = ws + k.image_bytes;
            a.part = reinterpret_cast<float *>(at);
            a.part_ml = a.part + k.ranges * k.tile_rows * cache->head_dim;
            a.spans = reinterpret_cast<int32_t *>(a.part_ml + k.ranges * k.tile_rows * 2);
        }
        ws += k.bytes;
        hipError_t e = k.images ? launch_attend_images(cache->head_dim, a, hs) : hipSuccess;
        if (e == hipSuccess)
            e = few ? launch_attend_decode(cache->head_dim, k.tile_rows, a, hs)
                           : launch_attend_prompt(cache->head_dim, a, hs);
        if (e == hipSuccess && k.ranges)
            e = few ? launch_attend_join(cache->head_dim, k.tile_rows, a, hs)
                    : launch_prompt_join(cache->head_dim, a, hs);
        if (e != hipSuccess)
            return from_hip(e);
    }
    return TSL_OK;
}

extern "C" const char *tsl_attn_last_hip_error_string(void) {
    return hipGetErrorString(g_last_hip);
}
