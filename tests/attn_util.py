"""Shared by the tests of the attention operators: a plain numpy form of each in
binary64, the cache's page layout read bit by bit, and device operands in the
strides a test asks for."""
import numpy as np

from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": tsl.F32, "bf16": tsl.BF16}
U = 2.0 ** -24


def tt(kind):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16}[kind]


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def rne(x, kind):
    """binary64 values rounded to binary32, then to the type."""
    t = torch()
    with np.errstate(over="ignore"):
        x32 = np.asarray(x, np.float64).astype(np.float32)
    return t.from_numpy(np.ascontiguousarray(x32)).to(tt(kind)).double().numpy()


class Operand:
    """[rows][heads][d] on the device with chosen strides inside a buffer
    filled with `fill`; `tokens` outermost, or heads outermost."""

    def __init__(self, rows, heads, d, kind, pad=0, head_major=False, fill=7.0, values=None, strides=None):
        t = torch()
        run = 8 if kind == "bf16" else 4
        pad = pad * run
        if head_major:
            self.ld, self.head = d + pad, max(rows, 1) * (d + pad) + pad
        else:
            self.head, self.ld = d + pad, heads * (d + pad) + pad
        if strides:
            self.ld, self.head = strides
        n = max(rows - 1, 0) * self.ld + (heads - 1) * self.head + d + 64
        self.buf = t.full((n,), fill, dtype=tt(kind), device=DEV)
        self.view = self.buf.as_strided((max(rows, 0), heads, d), (self.ld, self.head, 1))
        self.fill, self.kind = fill, kind
        if values is not None:
            self.view.copy_(t.from_numpy(np.ascontiguousarray(values, dtype=np.float32)).to(tt(kind)))

    def get(self):
        return self.view.detach().double().cpu().numpy()

    def rest_untouched(self, rows=None):
        """Nothing was written outside the operand (or outside these rows of it)."""
        b = self.buf.clone()
        v = b.as_strided(self.view.shape, self.view.stride())
        if rows is None:
            v.fill_(self.fill)
        elif len(rows):
            v[torch().as_tensor(rows, device=DEV)] = self.fill
        return bool((b == self.fill).all())


def quantise(x):
    """[..., d] binary64 -> (codes, scales, biases) of its runs of 64, as
    cache_append says."""
    r = x.reshape(x.shape[:-1] + (x.shape[-1] // 64, 64))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        b = rne(r.min(-1), "bf16")
        d = (r.max(-1).astype(np.float32) - b.astype(np.float32)).astype(np.float32)
        s = rne((d / np.float32(15)).astype(np.float64), "bf16")
        bad = ~(np.isfinite(r).all(-1) & np.isfinite(s) & np.isfinite(b))
        q = (r - b[..., None]) / np.where(s > 0, s, 1.0)[..., None]
        c = np.where(((s > 0) & ~bad)[..., None], np.clip(np.rint(q), 0, 15), 0)
    s, b = np.where(bad, np.nan, s), np.where(bad, np.nan, b)
    return c.reshape(x.shape).astype(np.int64), s, b


def values(c, s, b):
    return c * np.repeat(s, 64, -1) + np.repeat(b, 64, -1)


def held(x):
    """What the cache holds for x."""
    return values(*quantise(x))


class Pages:
    """A cache on the device, its pages filled with 0xFF (codes of 15, scales
    and biases of NaN) unless `fill` says otherwise."""

    def __init__(self, n_pages, page_tokens, heads, d, fill=0xFF):
        t = torch()
        self.n_pages, self.page_tokens, self.heads, self.d = n_pages, page_tokens, heads, d
        self.dict = dict(pages=None, n_pages=n_pages, page_tokens=page_tokens, n_kv_heads=heads,
                         head_dim=d)
        self.bytes = tsl.cache_size(self.dict)
        self.buf = t.full((self.bytes + 256,), fill, dtype=t.uint8, device=DEV)
        self.dict["pages"] = self.buf
        self.fill = fill

    def unpack(self):
        """(K codes, V codes) [page][token][head][d] and (K, V) (scale, bias)
        [page][token][head][d / 64], from the layout's description."""
        raw = self.buf[:self.bytes].cpu().numpy()
        d, w = self.d, self.d // 32
        rec = raw.reshape(self.n_pages, self.heads, self.page_tokens // 32, 36 * d)
        words = np.ascontiguousarray(rec[..., :32 * d]).view("<u4").astype(np.int64)
        sc = np.ascontiguousarray(rec[..., 32 * d:]).view("<u2").astype(np.uint32) << 16
        sc = sc.view(np.float32).astype(np.float64).reshape(rec.shape[:3] + (d // 64, 4, 32))
        t = np.arange(32)
        u, g, r = t // 16, t % 16 // 4, t % 4
        col = np.arange(d)
        at = lambda n, lane: n // 4 * 256 + lane * 4 + n % 4  # noqa: E731
        nib = lambda i: 4 * (i // 2 + 4 * (i % 2))  # noqa: E731
        ki = at(u[:, None] * w + col // 32, 16 * (col % 32 // 8) + (t % 16)[:, None])
        vi = 4 * d + at(col // 16, 16 * g[:, None] + col % 16)
        kc = words[..., ki] >> nib(col % 8) & 15
        vc = words[..., vi] >> nib(4 * u + r)[:, None] & 15
        scales = sc[..., 8 * g + 4 * u + r]  # [page][head][rec][run][4][token]

        def tokens(x):  # [page][head][rec][token][...] -> [page][token][head][...]
            x = x.reshape((self.n_pages, self.heads, self.page_tokens) + x.shape[4:])
            return np.moveaxis(x, 1, 2)
        part = [tokens(np.moveaxis(scales[..., k, :], -1, 3)) for k in range(4)]
        return tokens(kc), tokens(vc), (part[0], part[1]), (part[2], part[3])


class Batch:
    """Sequences with `rows` new tokens at the end of `context` ones, on a
    shuffled page table."""

    def __init__(self, rows, context, page_tokens, seed=0, spare=2, lead=0, tail=0, extra_cols=1):
        t = torch()
        self.n, self.ctx, self.page_tokens = list(rows), list(context), page_tokens
        need = [-(-max(c, 0) // page_tokens) for c in context]
        self.n_pages = max(sum(need) + spare, 1)
        order = rng(seed + 77).permutation(self.n_pages)
        self.max_pages = max(need + [0])
        self.table = np.full((len(rows), max(self.max_pages + extra_cols, 1)), -1, np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = order[at:at + k]
            at += k
        self.start = lead + np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.rows = int(self.start[-1]) + tail
        self.lead = lead
        self.dev = [t.from_numpy(x).to(DEV) for x in
                    (self.start, np.asarray(context, np.int32).reshape(-1), self.table)]

    def dict(self, **kw):
        d = dict(n_seqs=len(self.n), rows=self.rows, max_rows=max(self.n + [0]),
                 max_context=max(self.ctx + [0]), row_start=self.dev[0], context=self.dev[1],
                 page_table=self.dev[2], ld_table=self.table.shape[1], max_pages=self.max_pages)
        d.update(kw)
        return d

    def whole(self):
        """The batch whose rows are all of the contexts (to fill a cache)."""
        b = Batch.__new__(Batch)
        b.__dict__.update(self.__dict__)
        t = torch()
        b.n = [max(c, 0) for c in self.ctx]
        b.start = np.concatenate([[0], np.cumsum(b.n)]).astype(np.int32)
        b.rows, b.lead = int(b.start[-1]), 0
        b.dev = [t.from_numpy(b.start).to(DEV), self.dev[1], self.dev[2]]
        return b

    def live(self):
        return np.arange(self.start[0], self.start[-1])


def fill(pages, batch, K, V, kind="bf16"):
    """All tokens of the batch's contexts into the cache; K, V [tokens][h][d]."""
    w = batch.whole()
    if not w.rows:
        return
    k = Operand(w.rows, pages.heads, pages.d, kind, values=K)
    v = Operand(w.rows, pages.heads, pages.d, kind, values=V)
    tsl.cache_append(pages.dict, w.dict(), DT[kind], k.view, k.ld, k.head, v.view, v.ld, v.head)


def attend(q, K, V, scale, window, sinks, start):
    """Rows q [n][hq][d] from position `start` on over tokens K, V [ctx][h][d]:
    outputs, and the bound sum_j p_j |v_j| (binary64)."""
    n, hq, d = q.shape
    ctx, h, _ = K.shape
    g = hq // h
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    pos = start + np.arange(n)[:, None]
    j = np.arange(ctx)[None]
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sinks)
    for x in range(hq):
        k, v = K[:, x // g], V[:, x // g]
        ok_k = np.where(np.isfinite(k), k, 0.0)
        s = q[:, x] @ ok_k.T * scale
        s = np.where(np.isfinite(k).all(1)[None], s, np.nan)
        s = np.where(see, s, -np.inf)
        top = np.max(np.where(np.isnan(s), -np.inf, s), 1, keepdims=True, initial=-np.inf)
        p = np.exp(s - np.where(np.isfinite(top), top, 0))
        p = np.where(see, p, 0.0)
        tot = p.sum(1, keepdims=True)
        p = p / np.where(tot == 0, 1, tot)
        fv = np.where(np.isfinite(v), v, 0.0)
        out[:, x], mag[:, x] = p @ fv, p @ np.abs(fv)
        taint = see.astype(float) @ (~np.isfinite(v)).astype(float) > 0
        out[:, x][taint] = np.nan
    return out, mag


def within(got, want, lim, what=""):
    """|got - want| <= lim everywhere, NaN where the reference has NaN."""
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, "NaN places")
    d, lim = np.nan_to_num(np.abs(got - want)), np.broadcast_to(np.nan_to_num(lim), got.shape)
    bad = d > lim
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], d[bad][:3], lim[bad][:3])
