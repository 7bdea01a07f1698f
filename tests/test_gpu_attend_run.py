"""The attention operators together, as an attention layer uses them on two ranks:
q, k and v column shards -> rotation -> the rank's cache -> attention over it ->
output row shards, summed; prompts, then generated tokens; captured in graphs that
share a workspace; on another stream than the current one.

The cache's values are compared with the rotated keys and the values that went in
(at most half a step of 4 bits of the run's range, its scale and bias rounded to
bf16: s / 2 + (15 s + |b|) / 2^8 + the operands' own), and the layer's output with
the same layer in binary64 over what the cache holds.  Four tensors of that are
rounded to bf16 (q, rotated q, the heads' output, the result), each by half a step
h = 2^-8 a value; the softmax amplifies its operand's by no more than 2 at these
inputs, so 2 * 4 h bounds the result's error in the 2-norm."""
import numpy as np
import pytest

import attn_util as au
from block_util import HALF, Weight, f64, out, put, rng
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl
from test_gpu_rotate import reference as rotated

pytestmark = pytest.mark.gpu

TP, D, HQ, HKV, HD, PAGE = 2, 192, 8, 4, 64, 32
B = tsl.BF16


class Layer:
    """Both ranks' share of a layer, and the sequences' state."""

    def __init__(self, lengths, seed=0, window=0, sinks=0):
        t = torch()
        self.window, self.sinks = window, sinks
        self.Wq, self.Wk, self.Wv = (Weight("bf16", D, h * HD, seed + i, False)
                                     for i, h in ((1, HQ), (2, HKV), (3, HKV)))
        self.Wo = Weight("bf16", HQ * HD, D, seed + 4, False)
        plan = lambda n: tsl.plan_linear(D, n, TP, tsl.COLUMN)  # noqa: E731
        self.cols = [plan(h * HD) for h in (HQ, HKV, HKV)]
        self.row = tsl.plan_linear(HQ * HD, D, TP, tsl.ROW)
        self.freq = (1e4 ** (-np.arange(HD // 2) / (HD // 2))).astype(np.float32)
        self.dfreq = t.from_numpy(self.freq).to(DEV)
        self.batch = au.Batch([0] * len(lengths), lengths, PAGE, seed=seed)  # room for so many
        self.pages = [au.Pages(self.batch.n_pages, PAGE, HKV // TP, HD) for _ in range(TP)]
        self.packs = [[w.pack(sh) for sh in c] for w, c in
                      zip((self.Wq, self.Wk, self.Wv), self.cols)]
        self.opack = [self.Wo.pack(r) for r in self.row]
        self.ctx = [0] * len(lengths)

    def begin(self, rows, most=None):
        """The arrays of a step of so many new tokens of each sequence; room for
        `most` rows."""
        t = torch()
        self.ctx = [c + n for c, n in zip(self.ctx, rows)]
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        m = int(start[-1]) if most is None else most
        pos = np.zeros(m, np.int32)
        for s, (n, c) in enumerate(zip(rows, self.ctx)):
            pos[start[s]:start[s] + n] = np.arange(c - n, c)
        return dict(m=m, rows=rows, start=start, pos=pos, dpos=t.from_numpy(pos).to(DEV),
                    dstart=t.from_numpy(start).to(DEV),
                    dctx=t.from_numpy(np.asarray(self.ctx, np.int32)).to(DEV))

    def step(self, st, x, ws=None, stream=None):
        """Layer output [m][D] of the step's rows; intermediate tensors."""
        t, m = torch(), st["m"]
        seqs = dict(n_seqs=len(self.ctx), rows=m, max_rows=st.get("max_rows", max(st["rows"])),
                    max_context=max(self.batch.ctx), row_start=st["dstart"], context=st["dctx"],
                    page_table=self.batch.dev[2], ld_table=self.batch.table.shape[1],
                    max_pages=self.batch.max_pages)
        keep, parts = [], []
        for r in range(TP):
            hq, hkv = HQ // TP, HKV // TP
            q, k, v = (t.empty((m, h * HD), dtype=t.bfloat16, device=DEV) for h in (hq, hkv, hkv))
            for y, c, p in zip((q, k, v), self.cols, self.packs):
                sh, (buf, nb) = c[r], p[r]
                n = tsl.shard_linear_workspace_size(sh, B, m)
                w = t.empty(max(n, 256), dtype=t.uint8, device=DEV)
                tsl.shard_linear(sh, B, buf, nb, B, x, D, m, B, y, y.stride(0), 0, w, n, stream=stream)
                keep.append(w)
            qr, kr = t.empty_like(q), t.empty_like(k)
            items = [dict(X=a, ldx=h * HD, x_head=HD, Y=y, ldy=h * HD, y_head=HD, n_heads=h, xdtype=B,
                          ydtype=B) for a, y, h in ((q, qr, hq), (k, kr, hkv))]
            tsl.rotate_heads(items, m, dict(positions=st["dpos"], ld_pos=m, axes=1, freq=self.dfreq,
                                            rot_dim=HD, head_dim=HD), stream=stream)
            cache = self.pages[r].dict
            tsl.cache_append(cache, seqs, B, kr, hkv * HD, HD, v, hkv * HD, HD, stream=stream)
            n = tsl.cache_attention_workspace_size(cache, seqs, hq, self.window, self.sinks)
            w = ws if ws is not None else t.empty(max(n, 256), dtype=t.uint8, device=DEV)
            assert n <= w.numel()
            o = t.empty_like(q)
            tsl.cache_attention(cache, seqs, hq, qr, hq * HD, HD, HD ** -0.5, self.window, self.sinks, B,
                                o, hq * HD, HD, w, n, stream=stream)
            part = t.empty((m, D), dtype=t.float32, device=DEV)
            buf, nb = self.opack[r]
            n = tsl.shard_linear_workspace_size(self.row[r], B, m)
            w2 = t.empty(max(n, 256), dtype=t.uint8, device=DEV)
            tsl.shard_linear(self.row[r], B, buf, nb, B, o, hq * HD, m, tsl.F32, part, D, 0, w2, n,
                             stream=stream)
            parts.append(part)
            keep.append(dict(k=kr, v=v, o=o, w=(w, w2), q=(q, qr), seqs=seqs))
        y = t.empty((m, D), dtype=t.bfloat16, device=DEV)
        tsl.combine_partials(tsl.COMBINE_SUM, parts, tsl.F32, m, D, D, B, y, D, stream=stream)
        return y, [x for x in keep if isinstance(x, dict)], keep

    def held(self, r):
        """K and V of all sequences' tokens in rank r's cache, as cache_read gives them."""
        t = torch()
        n = sum(self.ctx)
        start = np.concatenate([[0], np.cumsum(self.ctx)]).astype(np.int32)
        k, v = (t.zeros((max(n, 1), HKV // TP, HD), device=DEV) for _ in "kv")
        seqs = dict(n_seqs=len(self.ctx), rows=n, max_rows=max(self.ctx), max_context=max(self.ctx),
                    row_start=t.from_numpy(start).to(DEV),
                    context=t.from_numpy(np.asarray(self.ctx, np.int32)).to(DEV),
                    page_table=self.batch.dev[2], ld_table=self.batch.table.shape[1],
                    max_pages=self.batch.max_pages)
        tsl.cache_read(self.pages[r].dict, seqs, tsl.F32, k, HKV // TP * HD, HD, v, HKV // TP * HD, HD)
        return f64(k), f64(v), start

    def want(self, st, x):
        """The layer in binary64 over what the caches hold."""
        y = np.zeros((st["m"], D))
        xs = f64(x)
        q = (xs @ self.Wq.w).reshape(-1, HQ, HD)
        q, _ = rotated(q, st["pos"][None], self.freq, np.zeros(HD // 2, int), HD, tsl.ROTARY_HALVES, False)
        for r in range(TP):
            k, v, start = self.held(r)
            h = slice(r * HQ // TP, (r + 1) * HQ // TP)
            for s, n in enumerate(st["rows"]):
                a, c0, c1 = int(st["start"][s]), int(start[s]), int(start[s + 1])
                o, _ = au.attend(q[a:a + n, h], k[c0:c1], v[c0:c1], HD ** -0.5, self.window, self.sinks,
                                 c1 - c0 - n)
                y[a:a + n] += o.reshape(n, HQ // TP * HD) @ self.Wo.w[r * HQ // TP * HD:(r + 1) * HQ // TP * HD]
        return y


def cached_is_what_went_in(layer, st, ranks):
    for r, d in enumerate(ranks):
        k, v, start = layer.held(r)
        for name, got in (("k", k), ("v", v)):
            x = f64(d[name]).reshape(st["m"], HKV // TP, HD)
            for s, n in enumerate(st["rows"]):
                a = int(st["start"][s])
                g, w = got[start[s + 1] - n:start[s + 1]], x[a:a + n]
                _, sc, b = au.quantise(w)
                lim = np.repeat(sc / 2 + (15 * sc + np.abs(b)) * HALF["bf16"], 64, -1)
                assert (np.abs(g - w) <= lim).all(), (name, s)


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_prompts_then_generated_tokens(window, sinks):
    layer = Layer([420, 60, 200], 10, window, sinks)
    for i, rows in enumerate([[37, 5, 0], [1, 1, 150], [1, 1, 1], [300, 1, 3], [1, 0, 1]]):
        st = layer.begin(rows)
        x = put(3 * rng(20 + i).standard_normal((st["m"], D)), "bf16")
        y, ranks, keep = layer.step(st, x)
        cached_is_what_went_in(layer, st, ranks)
        want = layer.want(st, x)
        rel = np.linalg.norm(f64(y) - want) / np.linalg.norm(want)
        assert rel <= 8 * HALF["bf16"], (i, rel)


def test_two_graphs_share_a_workspace():
    """A step of generated tokens and one with a prompt, each captured once and
    replayed with new lengths and tokens, between eager steps of another layer in
    the same workspace: every replay gives the bits of an eager twin."""
    t = torch()
    lengths = [700, 300]
    a, twin, other = Layer(lengths, 30), Layer(lengths, 30), Layer([500], 50)
    ws = t.empty(1 << 25, dtype=t.uint8, device=DEV)
    graphs = {}
    most = {"tokens": 2, "prompt": 240}
    for i, rows in enumerate([[130, 3], [1, 1], [1, 1], [200, 1], [1, 1], [110, 130], [1, 0], [9, 100]]):
        kind = "tokens" if sum(rows) <= 2 else "prompt"
        ctx = list(a.ctx)
        st, st2 = a.begin(rows, most[kind]), twin.begin(rows, most[kind])
        for d in (st, st2):
            d["max_rows"] = 1 if kind == "tokens" else 200
        x = put(3 * rng(60 + i).standard_normal((most[kind], D)), "bf16")
        if kind not in graphs:
            st["x"] = x.clone()
            side, g = t.cuda.Stream(), t.cuda.CUDAGraph()
            side.wait_stream(t.cuda.current_stream())
            t.cuda.synchronize()
            with t.cuda.graph(g, stream=side):
                y, ranks, keep = a.step(st, st["x"], ws)
            graphs[kind] = (g, st, y, ranks, keep)
        g, st0, y, ranks, _ = graphs[kind]
        for k in ("dpos", "dstart", "dctx"):
            st0[k].copy_(st[k])
        st0["x"].copy_(x)
        y.fill_(9)
        t.cuda.synchronize()
        g.replay()
        # eager work between: another layer's prompt, in the same workspace
        other.ctx = [0]
        so = other.begin([180])
        xo = put(3 * rng(90).standard_normal((180, D)), "bf16")
        yo, _, keep_o = other.step(so, xo, ws)
        y2, ranks2, keep2 = twin.step(st2, x, t.empty(1 << 25, dtype=t.uint8, device=DEV))
        t.cuda.synchronize()
        n = sum(rows)
        assert t.equal(y[:n], y2[:n]), (i, rows, ctx)
        for r in range(TP):
            assert t.equal(a.pages[r].buf, twin.pages[r].buf)
            assert t.equal(ranks[r]["o"][:n], ranks2[r]["o"][:n])
        want = other.want(so, xo)
        assert np.linalg.norm(f64(yo) - want) <= 8 * HALF["bf16"] * np.linalg.norm(want)


def test_on_another_stream():
    """The calls go to the stream they are given, in its order: behind work that
    makes their operands."""
    t = torch()
    layer, twin = Layer([150, 90], 70), Layer([150, 90], 70)
    side = t.cuda.Stream()
    for rows in ([120, 60], [1, 2]):
        st, st2 = layer.begin(rows), twin.begin(rows)
        x = put(3 * rng(71).standard_normal((st["m"], D)), "bf16")
        y2, ranks2, keep2 = twin.step(st2, x)
        t.cuda.synchronize()
        with t.cuda.stream(side):
            late = t.full_like(x, float("nan"))
            busy = t.randn(2048, 2048, device=DEV)
            for _ in range(20):
                busy = (busy @ busy) * 1e-3
            late.copy_(x)
        y, ranks, keep = layer.step(st, late, stream=side.cuda_stream)
        side.synchronize()
        assert t.equal(y, y2)
        for r in range(TP):
            assert t.equal(layer.pages[r].buf, twin.pages[r].buf)
