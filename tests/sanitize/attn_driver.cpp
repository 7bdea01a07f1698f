// The host side of tsl_attn.h, and the index arithmetic that its kernels share
// (which record a token lies in, which records a tile of rows sees), under
// AddressSanitizer and UndefinedBehaviorSanitizer; no GPU is touched.  Exits 0
// when everything held.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "attn.hpp"

using namespace tsl;

static int failures = 0;
#define EXPECT(cond)                                                                               \
    do {                                                                                           \
        if (!(cond)) {                                                                             \
            fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #cond);                             \
            ++failures;                                                                            \
        }                                                                                          \
    } while (0)

static void *addr(uint64_t a) { return reinterpret_cast<void *>(a); }
static uint32_t state = 12345;
static int pick(int n) { // 0 .. n - 1
    state = state * 1664525u + 1013904223u;
    return (int)((state >> 8) % (uint32_t)n);
}

// A record is inside the cache, its first byte where the layout says, and null
// for every page index that is not one.
static void records() {
    const int odd[] = {-1, INT32_MIN, INT32_MAX, -5};
    for (int round = 0; round < 2000; ++round) {
        CacheArgs c{};
        const int d = 64 << pick(3);
        c.shift = pick(8);
        c.n_kv_heads = 1 + pick(5);
        c.n_pages = 1 + pick(6);
        c.head_bytes = (int64_t)record_bytes(d) << c.shift;
        c.page_bytes = c.head_bytes * c.n_kv_heads;
        c.max_pages = pick(5);
        c.n_seqs = 1 + pick(3);
        c.ld_table = c.max_pages + pick(3);
        std::vector<int32_t> table((size_t)(c.n_seqs - 1) * c.ld_table + c.max_pages);
        for (int32_t &t : table)
            t = pick(4) ? pick(c.n_pages) : (pick(2) ? odd[pick(4)] : c.n_pages + pick(3));
        c.page_table = table.data();
        c.pages = static_cast<char *>(addr(1 << 20));
        for (int i = 0; i < 50; ++i) {
            const int s = pick(c.n_seqs), h = pick(c.n_kv_heads);
            const int blk = pick(3) ? pick((c.max_pages + 2) << c.shift) : pick(1 << 26);
            const char *r = record_of(c, s, h, blk, record_bytes(d));
            const int page = blk >> c.shift;
            const int32_t p = page < c.max_pages ? table[s * c.ld_table + page] : -1;
            EXPECT((r != nullptr) == (p >= 0 && p < c.n_pages));
            if (r)
                EXPECT(r >= c.pages && r + record_bytes(d) <= c.pages + c.n_pages * c.page_bytes &&
                       r == c.pages + p * c.page_bytes + h * c.head_bytes +
                                (int64_t)(blk % (1 << c.shift)) * record_bytes(d));
        }
    }
}

// A tile's list names every record with a token that a row sees, once, in order,
// and its ranges cover the list.
static void views() {
    for (int round = 0; round < 20000; ++round) {
        AttendArgs a{};
        a.c.shift = pick(4);
        a.c.max_pages = pick(12);
        a.window = pick(3) ? 0 : 1 + pick(200);
        if (!pick(20))
            a.window = kMaxContext;
        a.sinks = pick(2) ? 0 : pick(150);
        if (!pick(20))
            a.sinks = kMaxContext;
        const int splits = 1 + pick(9);
        a.min_share = 1 + pick(9);
        const int first = pick(500) - 20, last = first + pick(70);
        TileView v = tile_view(a, first, last);
        divide(a, splits, v);
        const int cap = a.c.max_pages << (a.c.shift + 5);
        std::vector<int> list;
        for (int i = 0; i < v.count; ++i)
            list.push_back(view_block(v, i));
        EXPECT(std::is_sorted(list.begin(), list.end()));
        EXPECT(std::adjacent_find(list.begin(), list.end()) == list.end());
        for (int blk = 0; blk < 24; ++blk) {
            bool any = false, all = true;
            for (int pos = first; pos <= last; ++pos)
                for (int j = 32 * blk; j < 32 * blk + 32; ++j) {
                    const bool plain = j <= pos && (!a.window || j > (int64_t)pos - a.window || j < a.sinks);
                    EXPECT(plain == sees(a, pos, window_start(a, pos), j));
                    any = any || (plain && j < cap);
                    all = all && plain;
                }
            const bool listed = std::find(list.begin(), list.end(), blk) != list.end();
            EXPECT(!any || listed);
            EXPECT(!sees_all(a, v, blk) || all);
        }
        for (int b : list)
            EXPECT(b >= 0 && 32 * b < cap);
        EXPECT(v.used <= splits && (v.count == 0) == (v.used == 0));
        EXPECT((int64_t)v.used * v.share >= v.count && (v.used == 0 || (v.used - 1) * v.share < v.count));
    }
    // every tile's records stand in its sequence's list, each once, and the list is
    // no longer than the bound
    for (int round = 0; round < 20000; ++round) {
        AttendArgs a{};
        a.c.shift = pick(3);
        a.c.max_pages = 1 + pick(12);
        a.window = pick(3) ? 1 + pick(300) : 0;
        a.sinks = pick(2) ? 0 : pick(200);
        a.group = 1 + pick(9);
        a.by_group = make_div((uint32_t)a.group);
        a.c.max_rows = 1 + pick(90);
        a.rows_max = INT32_MAX;
        const int cap = a.c.max_pages << (a.c.shift + 5);
        const SeqRows q = {0, 1 + pick(100), pick(cap + 40)};
        const TileView all = sequence_view(a, q);
        const int rows = rows_of(a, q), n = q.n < a.c.max_rows ? q.n : a.c.max_rows;
        EXPECT(all.count <= most_records(q.ctx < cap ? q.ctx : cap, n, a.window, a.sinks));
        for (int tile = 0; tile * 16 < rows; ++tile) {
            const TileView v = view_of(a, q, tile, 16, rows - tile * 16);
            for (int i = 0; i < v.count; ++i) {
                const int at = place_of(all, view_block(v, i));
                EXPECT(at >= 0 && at < all.count && view_block(all, at) == view_block(v, i));
            }
            for (int j = 0; j < cap; ++j) // what a row sees, the sequence's rows do
                if (sees(a, v.last, window_start(a, v.last), j))
                    EXPECT(any_sees(a, all, j));
        }
        for (int blk = 0; blk < 24; ++blk) {
            bool every = true;
            for (int j = 32 * blk; j < 32 * blk + 32; ++j)
                every = every && any_sees(a, all, j);
            EXPECT(!any_sees_all(a, all, blk) || every);
        }
    }
    // the ends of the ranges of positions
    AttendArgs a{};
    a.c.shift = 7;
    a.c.max_pages = 1 << 18;
    for (int w : {0, 1, kMaxContext})
        for (int f : {-(1 << 22), -1, 0, kMaxContext - 64}) {
            a.window = w;
            const TileView v = tile_view(a, f, f + 63);
            EXPECT(v.count >= 0 && v.count <= (kMaxContext >> 5));
            EXPECT(window_start(a, f) <= f + 1 || !w);
        }
    // sequences whose arrays are out of order or out of bounds
    const int32_t start[] = {-7, 5, 3, 900, INT32_MAX}, ctx[] = {INT32_MIN, -1, INT32_MAX, 12};
    CacheArgs c{};
    c.row_start = start;
    c.context = ctx;
    c.rows = 100;
    for (int s = 0; s < 4; ++s) {
        const SeqRows r = seq_rows(c, s);
        EXPECT(r.row0 >= 0 && r.n >= 0 && r.row0 + r.n <= c.rows && r.ctx >= 0 && r.ctx <= kMaxContext);
    }
}

// Division by the host's multipliers is exact below 2^31.
static void divisions() {
    for (int round = 0; round < 200000; ++round) {
        const uint32_t d = round < 5000 ? 1 + round : 1 + (state >> 1) % (1u << (1 + pick(30)));
        const Div v = make_div(d);
        for (int k = 0; k < 4; ++k) {
            state = state * 1664525u + 1013904223u;
            const int n = k == 0 ? INT32_MAX : (int)(state >> 1);
            EXPECT(quotient(n, v) == (int)((uint32_t)n / d));
            const int m = (int)(n / d * d); // a multiple, and the number before it
            EXPECT(quotient(m, v) == (int)(m / d) && (m == 0 || quotient(m - 1, v) == (int)((m - 1) / d)));
        }
    }
}

static void calls() {
    size_t b = 0;
    tsl_cache c = {addr(1 << 20), 10, 64, 2, 128};
    EXPECT(cache_size(&c, &b) == TSL_OK && b == 10u * 2 * 2 * 36 * 128);
    EXPECT(cache_size(&c, nullptr) == TSL_ERR_INVALID_ARG && cache_size(nullptr, &b) == TSL_ERR_INVALID_ARG);
    tsl_seqs q = {static_cast<int32_t *>(addr(1 << 30)), static_cast<int32_t *>(addr((1 << 30) + 4096)),
                  static_cast<int32_t *>(addr((1 << 30) + 8192)), 8, 0, 3, 5, 500, 8};
    for (int d : {64, 128, 256})
        for (int hq : {2, 14, 64})
            for (int rows : {0, 1, 5, 5000})
                for (int ctx : {0, 1, 500, 100000000})
                    for (int w : {0, 1, 4096, 1 << 30}) {
                        c.head_dim = d;
                        q.rows = q.max_rows = rows;
                        q.max_context = ctx;
                        EXPECT(cache_attention_workspace_size(&c, &q, hq, w, 4, &b) == TSL_OK);
                        EXPECT(b % 4 == 0);
                    }
    c.head_dim = 128;
    q.rows = 0;
    q.max_rows = 5;
    // no rows: accepted, nothing enqueued
    EXPECT(cache_append(&c, &q, TSL_BF16, addr(1 << 28), 256, 128, addr(1 << 29), 256, 128, nullptr) == TSL_OK);
    EXPECT(cache_attention(&c, &q, 4, addr(1 << 28), 512, 128, 1.f, 0, 0, TSL_F32, addr(1 << 29), 512, 128,
                           nullptr, 0, nullptr) == TSL_OK);
    EXPECT(cache_attention(&c, &q, 3, addr(1 << 28), 512, 128, 1.f, 0, 0, TSL_F32, addr(1 << 29), 512, 128,
                           nullptr, 0, nullptr) == TSL_ERR_NOT_DIVISIBLE);
}

int main() {
    records();
    views();
    divisions();
    calls();
    if (!failures)
        printf("all checks passed\n");
    return failures != 0;
}
