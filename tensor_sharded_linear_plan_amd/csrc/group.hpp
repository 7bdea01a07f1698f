// The host side of a (grouped) shard product, shared by the library's entry
// points: argument checks, packed-layout geometry, and the planning and
// launch sequence of a validated group.  Every check runs before anything
// is enqueued, so a rejected call has no side effects.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstddef>
#include <vector>

#include "internal.hpp"
#include "tsl.h"

namespace tsl {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool valid_dtype(int d) { return d == TSL_F32 || d == TSL_BF16 || d == TSL_Q4G64; }

// Shard descriptor sanity: the block lies inside W and matches its strategy.
inline tsl_status check_shard(const tsl_shard *s) {
    if (!s)
        return TSL_ERR_INVALID_ARG;
    if (s->K < 1 || s->N < 1 || s->k_len < 1 || s->n_len < 1 || s->k_off < 0 || s->n_off < 0)
        return TSL_ERR_INVALID_ARG;
    if (s->k_off + s->k_len > s->K || s->n_off + s->n_len > s->N)
        return TSL_ERR_INVALID_ARG;
    switch (s->strategy) {
    case TSL_COLUMN:
        if (s->k_off != 0 || s->k_len != s->K)
            return TSL_ERR_INVALID_ARG;
        break;
    case TSL_ROW:
        if (s->n_off != 0 || s->n_len != s->N)
            return TSL_ERR_INVALID_ARG;
        break;
    case TSL_REPLICATED:
    case TSL_EXPERT:
        if (s->k_off != 0 || s->k_len != s->K || s->n_off != 0 || s->n_len != s->N)
            return TSL_ERR_INVALID_ARG;
        break;
    default:
        return TSL_ERR_INVALID_ARG;
    }
    return TSL_OK;
}

// The HIP error behind the calling thread's latest TSL_ERR_HIP.
inline thread_local hipError_t g_last_hip = hipSuccess;

inline tsl_status from_hip(hipError_t e) {
    if (e == hipSuccess)
        return TSL_OK;
    g_last_hip = e;
    return TSL_ERR_HIP;
}

inline tsl_status geometry(const tsl_shard &s, tsl_dtype wdtype, PackGeom *g) {
    tsl_status st = check_shard(&s);
    if (st != TSL_OK)
        return st;
    if (!valid_dtype(wdtype))
        return TSL_ERR_INVALID_ARG;
    PackGeom r;
    r.Ks = s.k_len;
    r.Ns = s.n_len;
    r.Nt = (r.Ns + 15) / 16;
    const int64_t k64 = (r.Ks + 63) / 64;
    switch (wdtype) {
    case TSL_F32:
        r.KT = k64 * 4;
        r.Kpad = k64 * 64;
        r.total_bytes = (size_t)r.Nt * (size_t)r.KT * 64 * 16;
        break;
    case TSL_BF16:
        r.KT = k64 * 2;
        r.Kpad = k64 * 64;
        r.total_bytes = (size_t)r.Nt * (size_t)r.KT * 64 * 16;
        break;
    default: // TSL_Q4G64
        if (s.k_len % 64 || s.k_off % 64)
            return TSL_ERR_GROUP_ALIGN;
        r.KT = (r.Ks + 127) / 128;
        r.Kpad = r.KT * 128;
        r.exp_off = round_up((size_t)r.Nt * (size_t)r.KT * kQ4Record, 256);
        r.total_bytes = r.exp_off + round_up((size_t)r.Nt * 16 * 4, 256);
        break;
    }
    *g = r;
    return TSL_OK;
}

// Bytes from the first to one past the last element of an [M][n] matrix
// with row stride ld (M, n > 0).
inline size_t span(int64_t M, int64_t n, int64_t ld, size_t elem) {
    return (size_t)((M - 1) * ld + n) * elem;
}

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Whether an [Ma][wa] and an [Mb][wb] row-strided matrix share a byte
// (Ma, Mb > 0).  With equal strides this is exact -- column blocks or row
// blocks of one matrix held by different owners do not overlap -- otherwise
// it compares address ranges.
inline bool matrices_overlap(const void *pa, int64_t Ma, int64_t wa, int64_t lda, size_t ea,
                      const void *pb, int64_t Mb, int64_t wb, int64_t ldb, size_t eb) {
    const int64_t L = lda * (int64_t)ea;
    const int64_t Wa = wa * (int64_t)ea, Wb = wb * (int64_t)eb;
    if (L != ldb * (int64_t)eb || Wa > L || Wb > L)
        return overlaps(pa, span(Ma, wa, lda, ea), pb, span(Mb, wb, ldb, eb));
    // b - a = q L + rem, 0 <= rem < L: rows r1 - r2 = q need rem < Wa, rows
    // r1 - r2 = q + 1 need L - rem < Wb, each with -Mb < r1 - r2 < Ma
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(pb) - reinterpret_cast<uintptr_t>(pa));
    int64_t q = d / L, rem = d % L;
    if (rem < 0) {
        rem += L;
        q -= 1;
    }
    const bool same_row = (q > -Mb && q < Ma) && rem < Wa;
    const bool next_row = (q + 1 > -Mb && q + 1 < Ma) && L - rem < Wb;
    return same_row || next_row;
}

// Which kernel family serves a product of M rows.
inline bool use_skinny(tsl_dtype wdtype, int64_t M) {
    return wdtype == TSL_F32 || M <= (wdtype == TSL_BF16 ? kSkinnyMaxMBf16 : kSkinnyMaxM);
}

// Most items one grouped call takes.
constexpr int32_t kMaxItems = 4096;
// Workgroups per launch: the dispatch grid counts work-items in 32 bits.
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;

inline tsl_status check_types(tsl_dtype wdtype, tsl_dtype xdtype) {
    if (!valid_dtype(wdtype) || !valid_dtype(xdtype) || xdtype == TSL_Q4G64)
        return TSL_ERR_INVALID_ARG;
    // (weights, activations) pairs the kernels implement
    const bool pair_ok = (wdtype == TSL_F32 && xdtype == TSL_F32) ||
                         (wdtype == TSL_BF16 && xdtype == TSL_BF16) ||
                         (wdtype == TSL_Q4G64 && xdtype == TSL_BF16);
    return pair_ok ? TSL_OK : TSL_ERR_UNSUPPORTED;
}

// Validates one shard product (weight and activation types already
// checked) and fills its item.
// A member of a sum set after its first item has no output of its own
// (need_y false): its Y fields are not checked.
inline tsl_status check_item(const tsl_shard *shard, tsl_dtype wdtype, const void *packed,
                      size_t packed_bytes, tsl_dtype xdtype, const void *X, int64_t ldx, int64_t M,
                      int ydtype, void *Y, int64_t ldy, int accumulate, LinearItem *out,
                      bool need_y = true) {
    if (!need_y) {
        Y = reinterpret_cast<void *>(uintptr_t(256));
        ydtype = TSL_F32;
        accumulate = 0;
        ldy = INT64_MAX;
    }
    if (!shard || !packed || !X || !Y)
        return TSL_ERR_INVALID_ARG;
    if (ydtype != TSL_F32 && ydtype != TSL_BF16)
        return TSL_ERR_INVALID_ARG;
    PackGeom g;
    tsl_status st = geometry(*shard, wdtype, &g);
    if (st != TSL_OK)
        return st;
    if (accumulate != 0 && accumulate != 1)
        return TSL_ERR_INVALID_ARG;
    if (accumulate && ydtype != TSL_F32)
        return TSL_ERR_UNSUPPORTED;
    if (ldx < g.Ks || ldy < g.Ns)
        return TSL_ERR_INVALID_ARG;
    if (packed_bytes < g.total_bytes)
        return TSL_ERR_BUFFER_TOO_SMALL;
    const int64_t xa = xdtype == TSL_F32 ? 4 : 8;
    const uintptr_t ya = ydtype == TSL_F32 ? 4 : 2;
    if (!aligned(packed, 256) || !aligned(X, 16) || ldx % xa || !aligned(Y, ya))
        return TSL_ERR_MISALIGNED;
    // the kernels' item tables hold shard sizes in 32 bits, and the GEMM
    // addresses a tile's operands with 32-bit offsets
    if (g.Kpad >= INT32_MAX || g.Ns >= INT32_MAX)
        return TSL_ERR_UNSUPPORTED;
    if (!use_skinny(wdtype, M) && (ldx >= kPrefillMaxStride || g.Kpad >= kPrefillMaxStride))
        return TSL_ERR_UNSUPPORTED;
    out->g = g;
    out->M = M;
    out->packed = packed;
    out->X = X;
    out->ldx = ldx;
    out->Y = Y;
    out->ldy = ldy;
    out->ydtype = (tsl_dtype)ydtype;
    out->accumulate = accumulate;
    if (!need_y) {
        out->Y = nullptr;
        out->ldy = 0;
    }
    return TSL_OK;
}

// Launch order of a group: longest k first, so the longest tiles are
// dispatched first and the short ones fill in at the end.
inline std::vector<LinearItem> launch_order(const std::vector<LinearItem> &items) {
    // sum sets move as units (first item, then its members in order)
    struct Unit {
        size_t first, len;
        int64_t kpad;
    };
    std::vector<Unit> units;
    for (size_t i = 0; i < items.size(); i += items[i].set_len) {
        Unit u{i, (size_t)items[i].set_len, 0};
        for (size_t r = 0; r < u.len; ++r)
            u.kpad = items[i + r].g.Kpad > u.kpad ? items[i + r].g.Kpad : u.kpad;
        units.push_back(u);
    }
    std::stable_sort(units.begin(), units.end(),
                     [](const Unit &a, const Unit &b) { return a.kpad > b.kpad; });
    std::vector<LinearItem> v;
    v.reserve(items.size());
    for (const Unit &u : units)
        for (size_t r = 0; r < u.len; ++r)
            v.push_back(items[u.first + r]);
    return v;
}

// A set of two whose results the gate combines (act(X W_0) * (X W_1)).
inline bool gated(const LinearItem &L) { return L.ep && (L.ep->flags & kEpGated); }

// The GEMM regime: a sum set whose members have equal k-ranges becomes one
// product over the members' k-ranges laid end to end in set order,
// Y = [X_0 X_1 ...] [W_0; W_1; ...] -- the rank sum accumulated inside the
// GEMM, with no binary32 partials and no sum launch.  4-bit weights: k-
// ranges of whole 128-k records (the activation pass writes each member's
// binary16 activations at its k offset of the joined row, and the GEMM
// reads each 128-k block's records from its member's packed buffer).
// bf16 weights: k-ranges of whole 64-k stages, activations not read through
// a row index (the GEMM reads each stage's activations, at their member's
// row stride, and weights from the member's own buffers).  The rule reads
// nothing the workspace query does not see.  Other sets, and every set of
// fp32 weights or of the decode regime, pass unchanged.
inline std::vector<LinearItem> concat_sets(const std::vector<LinearItem> &in, tsl_dtype wdtype,
                                    int64_t M) {
    if ((wdtype != TSL_Q4G64 && wdtype != TSL_BF16) || use_skinny(wdtype, M))
        return in;
    const int64_t unit = wdtype == TSL_Q4G64 ? 128 : 64;
    std::vector<LinearItem> out;
    out.reserve(in.size());
    for (size_t i = 0; i < in.size();) {
        const size_t len = in[i].set_len;
        bool join = len > 1 && len <= (size_t)kSetParts && !gated(in[i]) &&
                    (int64_t)len * in[i].g.Kpad < kPrefillMaxStride;
        for (size_t r = 0; join && r < len; ++r)
            join = in[i + r].g.Ks % unit == 0 && in[i + r].g.Ks == in[i].g.Ks &&
                   (wdtype == TSL_Q4G64 || !in[i + r].ridx);
        if (!join) {
            for (size_t r = 0; r < len; ++r)
                out.push_back(in[i + r]);
            i += len;
            continue;
        }
        LinearItem c = in[i];
        c.cat = (int)len;
        c.set_len = 1;
        c.set_pos = 0;
        c.g.Ks *= (int64_t)len;
        c.g.KT *= (int64_t)len;
        c.g.Kpad *= (int64_t)len;
        c.g.total_bytes = 0; // no packed buffer of its own
        c.packed = nullptr;
        c.X = nullptr; // never shares an activation copy
        c.ldx = 0;
        c.ridx = nullptr;
        c.x_rows = 0;
        for (size_t r = 0; r < len; ++r) {
            c.seg_packed[r] = in[i + r].packed;
            c.seg_X[r] = in[i + r].X;
            c.seg_ldx[r] = in[i + r].ldx;
            c.seg_ridx[r] = in[i + r].ridx;
            c.seg_xrows[r] = in[i + r].x_rows;
        }
        out.push_back(c);
        i += len;
    }
    return out;
}

// Sum sets: each member of a set runs into its own binary32 partial (in
// the workspace, ahead of what the plan needs), balanced with every other
// product of the group; one more launch then adds the partials of all sets
// in order.

// Rewrites every sum set of *items into lone items writing binary32
// partials at ws, ws + ...; returns the bytes used.  Call it once: the
// items it leaves are no longer sets.  With ws == nullptr the partials'
// addresses are null (for sizing; such items are never launched).
inline size_t split_sets(std::vector<LinearItem> *items, char *ws) {
    size_t off = 0;
    for (size_t i = 0; i < items->size();) {
        const size_t len = (*items)[i].set_len;
        if (len > 1) {
            void *const sY = (*items)[i].Y;
            const int64_t sldy = (*items)[i].ldy;
            const tsl_dtype sy = (*items)[i].ydtype;
            const Epilogue *const ep = (*items)[i].ep;
            // a gated pair's results are combined by the sum launch
            const int flen = gated((*items)[i]) ? 0 : (int)len;
            for (size_t r = 0; r < len; ++r) {
                LinearItem &L = (*items)[i + r];
                L.fset_len = flen;
                L.fset_pos = (int)r;
                L.fset_Y = sY;
                L.fset_ldy = sldy;
                L.fset_ydtype = sy;
                L.Y = ws ? ws + off : nullptr;
                L.ldy = L.g.Ns;
                L.ydtype = TSL_F32;
                L.accumulate = 0;
                L.set_len = 1;
                L.set_pos = 0;
                L.ep = nullptr; // the whole set's, once its products are added
                L.fset_ep = flen > 0 && r == 0 ? ep : nullptr;
                L.no_split = len > (size_t)kSetParts; // summed by launch_combine_sum

                off += ((size_t)L.M * (size_t)L.g.Ns * 4 + 255) / 256 * 256;
            }
        }
        i += len;
    }
    return off;
}

// The last columns of a lone product as a piece of its own where the GEMM
// plan wants that (prefill.hip, tail_choice): *items becomes the two pieces.
// eps receives the second's epilogue, which the caller keeps until the launch.
inline void split_tail(std::vector<LinearItem> *items, tsl_dtype wdtype, int64_t M, Epilogue *ep) {
    if constexpr (kEpilogue) {
        if (items->size() != 1 || use_skinny(wdtype, M))
            return;
        const int64_t n0 = tail_columns((*items)[0], wdtype);
        if (n0 == 0)
            return;
        LinearItem a = (*items)[0], b = a;
        const size_t ye = a.ydtype == TSL_F32 ? 4 : 2;
        auto past = [](auto *p, int64_t bytes) {
            typedef decltype(p) P;
            return p ? reinterpret_cast<P>(reinterpret_cast<uintptr_t>(p) + bytes) : p;
        };
        a.g.Ns = n0;
        b.g.Ns -= n0;
        b.tail = true;
        b.Y = past(b.Y, n0 * ye);
        const int64_t bytes = n0 / 16 * (a.g.KT / a.cat) * 1024; // of the columns before
        if (wdtype == TSL_Q4G64) {
            b.tile_off = n0 / 16; // the column exponents lie behind all the records
        } else {
            a.g.Nt = n0 / 16;
            b.g.Nt -= n0 / 16;
            b.packed = past(b.packed, bytes);
            for (int r = 0; r < b.cat; ++r)
                b.seg_packed[r] = past(b.seg_packed[r], bytes);
        }
        if (b.ep) {
            *ep = *b.ep;
            ep->bias = past(ep->bias, n0 * (ep->flags & kEpBiasBf16 ? 2 : 4));
            ep->res = past(ep->res, n0 * (ep->flags & kEpResBf16 ? 2 : 4));
            ep->pre = past(ep->pre, n0 * (ep->flags & kEpPreBf16 ? 2 : 4));
            ep->pre2 = past(ep->pre2, n0 * (ep->flags & kEpPreBf16 ? 2 : 4));
            if (wdtype != TSL_Q4G64)
                ep->up = past(ep->up, bytes);
            b.ep = ep;
        }
        items->assign({a, b});
    }
}

// Rows read through an index.  The 4-bit activation pass (GEMM regime) and
// the resident streaming kernel (a few decode rows, bf16 and 4-bit
// weights) read them where they lie; the other kernels read X rows at
// fixed strides, so for them each distinct (X, ldx, k_len, row index,
// rows) is first gathered into a dense copy at the front of the workspace
// (all of a call's gathers in one launch), and the items read the copy.
// Rewrites the indexed items of *items that need a gathered copy to read
// it (ws + ...; null ws: sizing, every item its own copy) and returns the
// bytes the copies take; *jobs receives the gathers to enqueue.
inline size_t plan_row_gathers(std::vector<LinearItem> *items, tsl_dtype wdtype, int64_t M, char *ws,
                        std::vector<RowGather> *jobs) {
    // the 4-bit activation pass reads through the index itself, and so do
    // the streaming kernels that hold a call's rows in LDS (a few rows: the
    // plan's resident calls, decided by the items' shapes alone)
    if (wdtype == TSL_Q4G64 && !use_skinny(wdtype, M))
        return 0;
    if (wdtype != TSL_F32 && use_skinny(wdtype, M) &&
        skinny_plan(items->data(), (int)items->size(), wdtype, M).resident)
        return 0;
    const size_t e = wdtype == TSL_F32 ? 4 : 2;
    const int64_t xa = wdtype == TSL_F32 ? 4 : 8; // row strides of 16 bytes
    size_t off = 0;
    for (LinearItem &L : *items) {
        if (!L.ridx)
            continue;
        const int64_t Kc = (L.g.Ks + xa - 1) / xa * xa;
        const RowGather *same = nullptr;
        for (const RowGather &j : *jobs)
            if (ws && j.X == L.X && j.ldx == L.ldx && j.ridx == L.ridx && j.x_rows == L.x_rows &&
                j.M == L.M && j.Ks == L.g.Ks)
                same = &j;
        if (!same) {
            jobs->push_back(RowGather{L.X, L.ldx, L.ridx, L.x_rows, L.M, L.g.Ks,
                                      ws ? ws + off : nullptr, Kc});
            off += ((size_t)L.M * (size_t)Kc * e + 255) / 256 * 256;
            same = &jobs->back();
        }
        L.X = same->out;
        L.ldx = Kc;
        L.ridx = nullptr;
        L.x_rows = 0;
    }
    return off;
}

// Workspace bytes of a validated group.
inline size_t group_workspace(const std::vector<LinearItem> &in, tsl_dtype wdtype, int64_t M) {
    if (M == 0 || in.empty())
        return 0;
    if constexpr (kEpilogue) {
        if (decode_applies(in, wdtype, M))
            return 0;
    }
    std::vector<LinearItem> src = in;
    std::vector<RowGather> jobs;
    const size_t gathered = plan_row_gathers(&src, wdtype, M, nullptr, &jobs);
    std::vector<LinearItem> items = launch_order(concat_sets(src, wdtype, M));
    Epilogue tail_ep;
    split_tail(&items, wdtype, M, &tail_ep);
    const size_t parts = split_sets(&items, nullptr);
    if (use_skinny(wdtype, M))
        return gathered + parts + skinny_plan(items.data(), (int)items.size(), wdtype, M).ws_bytes;
    return gathered + parts + prefill_plan(items.data(), (int)items.size(), wdtype, M).ws_bytes;
}

// Plans and enqueues a validated group.
inline tsl_status run_group(const std::vector<LinearItem> &in, tsl_dtype wdtype, int64_t M,
                     void *workspace, size_t ws_bytes, void *stream) {
    if (M == 0)
        return TSL_OK;
    if constexpr (kEpilogue) {
        if (decode_applies(in, wdtype, M))
            return from_hip(launch_decode(in, wdtype, M, static_cast<hipStream_t>(stream)));
    }
    // (a null or short workspace is rejected below, before any launch)
    char *const ws0 = static_cast<char *>(workspace);
    std::vector<LinearItem> src = in;
    std::vector<RowGather> gathers;
    const size_t gathered = plan_row_gathers(&src, wdtype, M, ws0, &gathers);
    char *ws = ws0 ? ws0 + gathered : nullptr; // the rank partials, then the plan's
    std::vector<LinearItem> ordered = launch_order(concat_sets(src, wdtype, M));
    Epilogue tail_ep;
    split_tail(&ordered, wdtype, M, &tail_ep);
    std::vector<LinearItem> items = ordered;
    const size_t parts = split_sets(&items, ws);
    const int n = (int)items.size();
    hipStream_t s = static_cast<hipStream_t>(stream);
    size_t need;
    int64_t blocks;
    SkinnyPlan sp;
    PrefillPlan pp;
    const bool skinny = use_skinny(wdtype, M);
    if (skinny) {
        sp = skinny_plan(items.data(), n, wdtype, M);
        need = gathered + parts + sp.ws_bytes;
        blocks = skinny_blocks(sp, items.data(), n);
    } else {
        pp = prefill_plan(items.data(), n, wdtype, M);
        need = gathered + parts + pp.ws_bytes;
        blocks = prefill_blocks(pp, items.data(), n, M);
    }
    if (blocks > kMaxBlocks)
        return TSL_ERR_UNSUPPORTED;
    if (need > 0) {
        if (!workspace || ws_bytes < need)
            return TSL_ERR_BUFFER_TOO_SMALL;
        if (!aligned(workspace, 256))
            return TSL_ERR_MISALIGNED;
    }
    // every product that is launched writes somewhere
    for (const LinearItem &L : items)
        if (!L.Y)
            return TSL_ERR_INVALID_ARG;
    // the rows read through an index, gathered (an index outside [0, x_rows)
    // gives a row of zeros)
    if (!gathers.empty()) {
        const hipError_t ge = launch_row_gathers(gathers, wdtype == TSL_F32 ? 4 : 2, s);
        if (ge != hipSuccess)
            return from_hip(ge);
    }
    hipError_t e = skinny ? launch_skinny(sp, items.data(), n, wdtype, M, ws + parts, s)
                          : launch_prefill(pp, items.data(), n, wdtype, M, ws + parts, s);
    if (e != hipSuccess)
        return from_hip(e);
    // k-split GEMM products: each product's k-partials, in k order
    // k-split products (decode regime: those that neither accumulate into
    // Y nor belong to a sum set too long for one sum launch; launch_skinny
    // finished the others)
    auto kcount = [&](size_t i) {
        return !skinny ? pp.ks[i]
                       : (items[i].accumulate || items[i].no_split ? 1 : sp.ks[i]);
    };
    auto kparts = [&](size_t i) {
        return kcount(i) > 1 ? reinterpret_cast<const float *>(
                                   ws + parts + (skinny ? sp.ws_off[i] : pp.p_off[i]))
                             : static_cast<const float *>(items[i].Y);
    };
    std::vector<SumSpec> sums;
    for (size_t i = 0; i < ordered.size();) {
        const size_t len = ordered[i].set_len;
        if (len == 1 && kcount(i) > 1) { // a lone product: its k-partials into its Y
            SumSpec sp1;
            sp1.parts[0] = kparts(i);
            sp1.ks[0] = kcount(i);
            sp1.n_parts = 1;
            if (dual(items[i])) { // the second weight's partials follow the first's
                sp1.parts[1] = sp1.parts[0] + (int64_t)kcount(i) * items[i].M * items[i].g.Ns;
                sp1.ks[1] = kcount(i);
                sp1.n_parts = 2;
            }
            sp1.M = items[i].M;
            sp1.n = items[i].g.Ns;
            sp1.Y = items[i].Y;
            sp1.ldy = items[i].ldy;
            sp1.ydtype = items[i].ydtype;
            sp1.ep = items[i].ep;
            sums.push_back(sp1);
        }
        i += len;
    }
    if (!parts) {
        if (!sums.empty())
            e = launch_sum_sets((int)sums.size(), sums.data(), M, s);
        return from_hip(e);
    }
    // the rank sums of the split sets, in item order: sets of up to
    // kSetParts members share one launch, longer ones get their own
    for (size_t i = 0; i < ordered.size(); i += ordered[i].set_len) {
        const LinearItem &L = ordered[i];
        if (L.set_len == 1)
            continue;
        if (skinny && sp.fset[i] >= 0)
            continue; // added up by the streaming launch itself
        if (L.set_len > kSetParts) {
            const float *p[kMaxParts];
            for (int r = 0; r < L.set_len; ++r)
                p[r] = static_cast<const float *>(items[i + r].Y);
            // with an epilogue: added into the first partial, which then goes
            // through it
            if (L.ep)
                e = launch_combine_sum(L.set_len, p, L.M, L.g.Ns, L.g.Ns, TSL_F32, items[i].Y,
                                       L.g.Ns, s);
            else
                e = launch_combine_sum(L.set_len, p, L.M, L.g.Ns, L.g.Ns, L.ydtype, L.Y, L.ldy, s);
            if (e != hipSuccess)
                return from_hip(e);
            if (!L.ep)
                continue;
        }
        SumSpec sp;
        sp.n_parts = L.set_len > kSetParts ? 1 : L.set_len;
        for (int r = 0; r < sp.n_parts; ++r) {
            sp.parts[r] = kparts(i + r);
            sp.ks[r] = kcount(i + r);
        }
        sp.ep = L.ep;
        sp.M = L.M;
        sp.n = L.g.Ns;
        sp.Y = L.Y;
        sp.ldy = L.ldy;
        sp.ydtype = L.ydtype;
        sums.push_back(sp);
    }
    if (!sums.empty())
        e = launch_sum_sets((int)sums.size(), sums.data(), M, s);
    return from_hip(e);
}

// Gathers and validates the items of a grouped call.
inline tsl_status gather(int32_t n_items, const tsl_linear_item *items, tsl_dtype wdtype,
                  tsl_dtype xdtype, int64_t M, std::vector<LinearItem> *out) {
    if (!items || n_items < 1 || n_items > kMaxItems || M < 0)
        return TSL_ERR_INVALID_ARG;
    tsl_status st = check_types(wdtype, xdtype);
    if (st != TSL_OK)
        return st;
    out->resize(n_items);
    int32_t first = 0; // first item of the current sum set
    for (int32_t i = 0; i < n_items; ++i) {
        const tsl_linear_item &it = items[i];
        const bool member = i > first;
        if ((it.sum_next != 0 && it.sum_next != 1) || it.rows < 0 || it.rows > M)
            return TSL_ERR_INVALID_ARG;
        if (it.sum_next && i == n_items - 1)
            return TSL_ERR_INVALID_ARG;
        st = check_item(it.shard, wdtype, it.packed, it.packed_bytes, xdtype, it.X, it.ldx, M,
                        it.ydtype, it.Y, it.ldy, it.accumulate, &(*out)[i], !member);
        if (st != TSL_OK)
            return st;
        LinearItem &L = (*out)[i];
        L.set_pos = i - first;
        L.M = it.rows ? it.rows : M;
        if (it.row_index) { // rows read through an index
            if (it.x_rows < 1 || it.x_rows > INT32_MAX)
                return TSL_ERR_INVALID_ARG;
            if (!aligned(it.row_index, 4))
                return TSL_ERR_MISALIGNED;
            L.ridx = it.row_index;
            L.x_rows = it.x_rows;
        }
        if (member && (L.g.Ns != (*out)[first].g.Ns || L.M != (*out)[first].M))
            return TSL_ERR_INVALID_ARG;
        if (!it.sum_next) { // the set [first, i] is complete
            (*out)[first].set_len = i - first + 1;
            if (i > first && (*out)[first].accumulate)
                return TSL_ERR_INVALID_ARG;
            if (i - first + 1 > kMaxParts)
                return TSL_ERR_INVALID_ARG;
            for (int32_t r = first + 1; r <= i; ++r)
                (*out)[r].set_len = 0;
            first = i + 1;
        }
    }
    if (M == 0)
        return TSL_OK;
    // the products run in no particular order: no output may overlap
    // another output or any input
    const size_t xe = xdtype == TSL_F32 ? 4 : 2;
    for (int32_t i = 0; i < n_items; ++i) {
        const LinearItem &a = (*out)[i];
        if (!a.Y)
            continue; // a sum-set member writes into its set's output
        const size_t ea = a.ydtype == TSL_F32 ? 4 : 2;
        for (int32_t j = 0; j < n_items; ++j) {
            const LinearItem &b = (*out)[j];
            const size_t eb = b.ydtype == TSL_F32 ? 4 : 2;
            if (matrices_overlap(a.Y, a.M, a.g.Ns, a.ldy, ea, b.X, b.ridx ? b.x_rows : b.M, b.g.Ks,
                                 b.ldx, xe))
                return TSL_ERR_INVALID_ARG;
            if (b.ridx && overlaps(a.Y, span(a.M, a.g.Ns, a.ldy, ea), b.ridx, (size_t)b.M * 4))
                return TSL_ERR_INVALID_ARG;
            if (j > i && b.Y &&
                matrices_overlap(a.Y, a.M, a.g.Ns, a.ldy, ea, b.Y, b.M, b.g.Ns, b.ldy, eb))
                return TSL_ERR_INVALID_ARG;
        }
    }
    return TSL_OK;
}

} // namespace tsl
