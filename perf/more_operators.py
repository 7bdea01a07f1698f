"""Timed cases of the attention operators: rotary positions of the query and key
heads, keys and values written to and read from a paged cache held in 4 bits, and
attention over that cache, in full or within a sliding window with a few first
tokens that stay visible.

``own`` False computes the operators in plain torch operations in binary32 (angles
and 4-bit codes in binary64), rounded once at the end; ``own`` True makes the calls
of the library.  Head counts and widths are those of the layers in
``tensor_sharded_linear_plan_amd/configs.py``.

Fields of a case: ``op`` names the operator; ``hq``, ``hkv``, ``d`` query heads, key
and value heads, head width; ``seqs`` sequences, each with up to ``rows`` new tokens
after up to ``past`` cached ones, the lengths ragged where ``mix`` is not 0 (it seeds
them); ``page`` tokens of a cache page.  Rotation: ``rot`` rotated columns of a head,
``axes`` position axes, ``style``, ``inverse`` the backward direction, ``far`` the
largest position.  Attention: ``window`` visible last tokens (0: all), ``sinks`` first
tokens that stay visible.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- the cases ----------------------------------------------------------------

def listed():
    return [
        # one generated token of a 7B-class layer far into a text
        dict(name="rotate_decode", op="rotate", hq=28, hkv=4, d=128, m=1, rot=128, axes=1,
             style="halves", inverse=False, far=120000, y="bf16"),
        # prefill of 8192 tokens, 27B-class layer
        dict(name="rotate_prompt", op="rotate", hq=64, hkv=8, d=128, m=8192, rot=128, axes=1,
             style="halves", inverse=False, far=32768, y="bf16"),
        # training backward over the frames of a video: time, height and width positions,
        # part of each head rotated, binary32
        dict(name="rotate_video_grad", op="rotate", hq=32, hkv=8, d=64, m=1531, rot=48, axes=3,
             style="pairs", inverse=True, far=4000, y="f32"),
        # a decode step of 48 sequences: one token each into its cache
        dict(name="append_decode", op="append", hq=64, hkv=8, d=128, seqs=48, rows=1, past=9000,
             page=64, mix=11),
        # prompts of a batch, some of them continued, into their caches
        dict(name="append_prompt", op="append", hq=64, hkv=8, d=128, seqs=8, rows=2048, past=500,
             page=128, mix=12),
        # one generated token of one sequence, 7B-class layer
        dict(name="decode_one", op="attend", hq=28, hkv=4, d=128, seqs=1, rows=1, past=4000,
             page=64, mix=0, window=0, sinks=0),
        # a decode step of 32 sequences of very different lengths, 27B-class layer
        dict(name="decode_batch", op="attend", hq=64, hkv=8, d=128, seqs=32, rows=1, past=32767,
             page=64, mix=13, window=0, sinks=0),
        # one generated token after a book-length text, 7B-class layer
        dict(name="decode_long", op="attend", hq=28, hkv=4, d=128, seqs=1, rows=1, past=131000,
             page=128, mix=0, window=0, sinks=0),
        # prefill of four prompts of different lengths, 27B-class layer
        dict(name="prompt_batch", op="attend", hq=64, hkv=8, d=128, seqs=4, rows=2500, past=0,
             page=128, mix=14, window=0, sinks=0),
        # a later chunk of a long prompt, K/V heads replicated on the ranks
        dict(name="prompt_chunk", op="attend", hq=32, hkv=4, d=128, seqs=1, rows=512, past=16000,
             page=256, mix=0, window=0, sinks=0),
        # a decode step of 64 streams with a window and four first tokens, heads of 64
        dict(name="window_decode", op="attend", hq=32, hkv=8, d=64, seqs=64, rows=1, past=16000,
             page=32, mix=15, window=4096, sinks=4),
        # prefill of 8192 tokens with a window and four first tokens, heads of 64
        dict(name="window_prompt", op="attend", hq=32, hkv=8, d=64, seqs=1, rows=8192, past=0,
             page=64, mix=0, window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(28, 4, 128), (64, 8, 128), (32, 8, 64), (32, 4, 128), (8, 8, 64), (7, 1, 128)]


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "window"])
    hq, hkv, d = rng.choice(HEADS)
    c = dict(op=op, hq=hq, hkv=hkv, d=d)
    if op == "rotate":
        axes = rng.choice([1, 1, 2, 3])
        return dict(c, m=_log(rng, 1, 8192), rot=rng.choice([d, d // 2, 3 * d // 4]), axes=axes,
                    style=rng.choice(["halves", "pairs"]), inverse=rng.random() < 0.4,
                    far=_log(rng, 100, 1000000), y=rng.choice(["bf16", "bf16", "f32"]))
    c.update(seqs=_log(rng, 1, 64), page=rng.choice([32, 64, 128, 256]),
             mix=rng.randrange(1, 1 << 20))
    if op == "append":
        return dict(c, rows=_log(rng, 1, max(1, 8192 // c["seqs"])), past=_log(rng, 1, 2000))
    c.update(op="attend", window=0, sinks=0)
    if op == "window":
        c.update(window=_log(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 64]))
    if rng.random() < 0.5:  # generated tokens, or a few proposed ones at once
        rows = rng.choice([1, 1, 1, 2, 5])
        return dict(c, rows=rows, past=_log(rng, 64, min(65536, 262144 // c["seqs"])))
    c["seqs"] = min(c["seqs"], 8)
    rows = _log(rng, 17, 4096 // c["seqs"])
    return dict(c, rows=rows, past=rng.choice([0, 0, _log(rng, 16, 8192 // c["seqs"])]))


# ---- inputs -------------------------------------------------------------------

def _lengths(c):
    """New tokens and cached ones before them, of each sequence."""
    r, n = random.Random(c["mix"]), c["seqs"]
    if not c["mix"]:
        return [c["rows"]] * n, [c["past"]] * n
    cut = lambda top: [top] + [int(round(top * r.random())) for _ in range(n - 1)]  # noqa: E731
    return [max(1, v) for v in cut(c["rows"])], cut(c["past"])


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _kv(g, t, c):
    """Keys with a few strong channels and an offset in each, values of tokens of
    different strength."""
    h, d = c["hkv"], c["d"]
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    strong = 1 + 3 * (torch.rand((h, d), generator=g, device=DEV) < 0.05)
    k = ((rnd(t, h, d) + rnd(h, d)) * strong).to(torch.bfloat16)
    v = (rnd(t, h, d) * (0.25 + torch.rand((t, 1, 1), generator=g, device=DEV))).to(torch.bfloat16)
    return k, v


def _inputs(case, seed):
    c, g = case, _gen(seed)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    heads = hq + 2 * hkv
    if c["op"] == "rotate":
        m, half = c["m"], c["rot"] // 2
        x = torch.randn((m, heads * d), generator=g, device=DEV).to(TYPES[c["y"]])
        pos = torch.randint(0, c["far"] + 1, (c["axes"], m), generator=g, device=DEV,
                            dtype=torch.int32)
        freq = (1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        # the pairs of a head by axis: runs of equal length, the first axis takes the rest
        axis = [max(0, p * c["axes"] // half) for p in range(half)]
        return dict(x=x, q=x[:, :hq * d], k=x[:, hq * d:(hq + hkv) * d], pos=pos, freq=freq,
                    axis=axis)
    rows, past = _lengths(c)
    ctx = [a + b for a, b in zip(rows, past)]
    page = c["page"]
    npages = [-(-n // page) for n in ctx]
    first = [sum(npages[:i]) for i in range(len(ctx))]
    width = max(npages)
    order = torch.randperm(sum(npages) + 3, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None]
    start = torch.tensor(first, device=DEV)[:, None]
    table = torch.where(col < torch.tensor(npages, device=DEV)[:, None],
                        order[(start + col).clamp(max=sum(npages) - 1)], -1).to(torch.int32)
    cum = lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=torch.int32,  # noqa: E731
                                 device=DEV)
    d_ = dict(rows=rows, ctx=ctx, n_pages=sum(npages) + 3, table=table, row_start=cum(rows),
              all_start=cum(ctx), context=torch.tensor(ctx, dtype=torch.int32, device=DEV))
    t = sum(rows)
    x = torch.randn((t, heads * d), generator=g, device=DEV).to(torch.bfloat16)
    if c["op"] == "append":
        k, v = _kv(g, t, c)
        x[:, hq * d:(hq + hkv) * d], x[:, (hq + hkv) * d:] = k.view(t, -1), v.view(t, -1)
        d_.update(k=x[:, hq * d:(hq + hkv) * d], v=x[:, (hq + hkv) * d:])
    else:
        d_.update(q=x[:, :hq * d])
        d_["k"], d_["v"] = _kv(g, sum(ctx), c)
    return d_


# ---- the operators in plain form -------------------------------------------------

def _where(start, context):
    """Of each row: its sequence and its position in it."""
    n = start[1:] - start[:-1]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n.long())
    i = torch.arange(seq.numel(), device=DEV) - start.long()[seq]
    return seq, context.long()[seq] - n.long()[seq] + i


def _quant(x):
    """[..., d] to codes, and a scale and a bias for every 64 of them."""
    x = x.float().unflatten(-1, (-1, GROUP))
    b = x.amin(-1, keepdim=True).to(torch.bfloat16)
    s = ((x.amax(-1, keepdim=True) - b.float()) / 15).to(torch.bfloat16)
    q = (x.double() - b.double()) / torch.where(s > 0, s, torch.ones_like(s)).double()
    q = torch.where(s > 0, q.round().clamp(0, 15), torch.zeros_like(q)).to(torch.uint8)
    return q.flatten(-2), s[..., 0], b[..., 0]


def _values(q, s, b):
    q = q.unflatten(-1, (-1, GROUP)).float()
    return (s.float()[..., None] * q + b.float()[..., None]).flatten(-2)


def _slot(c, d, start):
    """Of each row: its page, and its token in the page."""
    seq, pos = _where(start, d["context"])
    return d["table"].long()[seq, pos // c["page"]], pos % c["page"]


def _cache(c, d, x, start):
    """The paged codes, scales and biases that hold the rows x."""
    shape = (d["n_pages"], c["page"], c["hkv"])
    q = torch.zeros(shape + (c["d"],), dtype=torch.uint8, device=DEV)
    s = torch.zeros(shape + (c["d"] // GROUP,), dtype=torch.bfloat16, device=DEV)
    b = torch.zeros_like(s)
    at = _slot(c, d, start)
    q[at], s[at], b[at] = _quant(x.unflatten(-1, (c["hkv"], c["d"])) if x.dim() == 2 else x)
    return q, s, b


def _plain_rotate(c, d):
    half, t = c["rot"] // 2, TYPES[c["y"]]
    angle = d["pos"].double()[d["axis_t"]].t() * d["freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    sin = -sin if c["inverse"] else sin

    def turn(x):
        x = x.unflatten(-1, (-1, c["d"])).float()
        y = x.clone()
        a = slice(0, half) if c["style"] == "halves" else slice(0, c["rot"], 2)
        b = slice(half, c["rot"]) if c["style"] == "halves" else slice(1, c["rot"], 2)
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        return y.flatten(1).to(t)

    return dict(q=turn(d["q"]), k=turn(d["k"]))


def _plain_append(c, d):
    at = _slot(c, d, d["row_start"])

    def store(x, cache):
        q, s, b = cache
        q[at], s[at], b[at] = _quant(x.unflatten(-1, (c["hkv"], c["d"])))
        return _values(q[at], s[at], b[at])

    return dict(k=store(d["k"], d["kc"]), v=store(d["v"], d["vc"]))


def _plain_attend(c, d):
    hkv, w, g = c["hkv"], c["d"], c["hq"] // c["hkv"]
    page = d["table"].long().clamp(min=0)  # [n][pages]
    gather = lambda cache: _values(*[t[page].flatten(1, 2) for t in cache])  # noqa: E731
    k = gather(d["kc"]).permute(0, 2, 3, 1).contiguous()  # [n][hkv][w][keys]
    v = gather(d["vc"]).permute(0, 2, 1, 3).contiguous()
    n, keys, top = k.shape[0], k.shape[3], max(d["rows"])
    seq, pos = _where(d["row_start"], d["context"])
    i = torch.arange(seq.numel(), device=DEV) - d["row_start"].long()[seq]
    q = torch.zeros((n, top, hkv, g, w), device=DEV)
    q[seq, i] = d["q"].float().unflatten(-1, (hkv, g, w))
    at = torch.full((n, top), -1, device=DEV)
    at[seq, i] = pos
    s = (q.permute(0, 2, 1, 3, 4).reshape(n, hkv, top * g, w) @ k) * w ** -0.5
    j, p = torch.arange(keys, device=DEV), at.repeat_interleave(g, 1)[:, None, :, None]
    seen = j <= p
    if c["window"]:
        seen &= (j > p - c["window"]) | (j < c["sinks"])
    s.masked_fill_(~seen, float("-inf"))
    s -= s.amax(-1, keepdim=True).clamp(min=-3e38)
    s.exp_()
    o = (s @ v) / s.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(n, hkv, top, g, w).permute(0, 2, 1, 3, 4)[seq, i]
    return o.flatten(1).to(torch.bfloat16)


# ---- the library's calls ---------------------------------------------------------

def _tsl():
    from tensor_sharded_linear_plan_amd import binding
    return binding


def _seqs(c, d, start, rows):
    return dict(n_seqs=c["seqs"], rows=sum(rows), max_rows=max(rows), max_context=max(d["ctx"]),
                row_start=start, context=d["context"], page_table=d["table"],
                ld_table=d["table"].stride(0), max_pages=d["table"].shape[1])


def _prepare_own(c, d):
    tsl, s, w = _tsl(), dict(d), c["d"]
    if c["op"] == "rotate":
        t = tsl.F32 if c["y"] == "f32" else tsl.BF16
        ld = d["x"].stride(0)
        s["yq"], s["yk"] = torch.empty_like(d["q"].contiguous()), torch.empty_like(d["k"].contiguous())
        s["items"] = [dict(X=d[n], ldx=ld, x_head=w, xdtype=t, Y=s["y" + n], ldy=s["y" + n].stride(0),
                           y_head=w, ydtype=t, n_heads=c["h" + (n if n == "q" else "kv")])
                      for n in ("q", "k")]
        s["rotary"] = dict(positions=d["pos"], ld_pos=d["pos"].stride(0), axes=c["axes"],
                           pair_axis=d["axis"], freq=d["freq"], rot_dim=c["rot"], head_dim=w,
                           style=tsl.ROTARY_HALVES if c["style"] == "halves" else tsl.ROTARY_PAIRS)
        return s
    cache = dict(pages=None, n_pages=d["n_pages"], page_tokens=c["page"], n_kv_heads=c["hkv"],
                 head_dim=w)
    cache["pages"] = torch.zeros(tsl.cache_size(cache), dtype=torch.uint8, device=DEV)
    s["cache"], s["seqs"] = cache, _seqs(c, d, d["row_start"], d["rows"])
    if c["op"] == "append":
        s["ko"], s["vo"] = (torch.empty((sum(d["rows"]), c["hkv"], w), device=DEV) for _ in "kv")
        return s
    tsl.cache_append(cache, _seqs(c, d, d["all_start"], d["ctx"]), tsl.BF16, s.pop("k"),
                     c["hkv"] * w, w, s.pop("v"), c["hkv"] * w, w)
    s["o"] = torch.empty((sum(d["rows"]), c["hq"] * w), dtype=torch.bfloat16, device=DEV)
    s["nws"] = tsl.cache_attention_workspace_size(cache, s["seqs"], c["hq"], c["window"], c["sinks"])
    s["ws"] = torch.empty(max(s["nws"], 256), dtype=torch.uint8, device=DEV)
    return s


def _call(c, s):
    tsl, w = _tsl(), c["d"]
    if c["op"] == "rotate":
        tsl.rotate_heads(s["items"], c["m"], s["rotary"], int(c["inverse"]))
        return dict(q=s["yq"], k=s["yk"])
    if c["op"] == "append":
        k, v, ko, vo = s["k"], s["v"], s["ko"], s["vo"]
        tsl.cache_append(s["cache"], s["seqs"], tsl.BF16, k, k.stride(0), w, v, v.stride(0), w)
        tsl.cache_read(s["cache"], s["seqs"], tsl.F32, ko, ko.stride(0), w, vo, vo.stride(0), w)
        return dict(k=ko, v=vo)
    q, o = s["q"], s["o"]
    tsl.cache_attention(s["cache"], s["seqs"], c["hq"], q, q.stride(0), w, w ** -0.5, c["window"],
                        c["sinks"], tsl.BF16, o, o.stride(0), w, s["ws"], s["nws"])
    return o


def _prepare_plain(c, d):
    s = dict(d)
    if c["op"] == "rotate":
        s["axis_t"] = torch.tensor(d["axis"], device=DEV)
        return s
    start, rows = ("all_start", "ctx") if c["op"] == "attend" else ("row_start", "rows")
    s["kc"], s["vc"] = _cache(c, d, d["k"], d[start]), _cache(c, d, d["v"], d[start])
    if c["op"] == "attend":
        del s["k"], s["v"]
    return s


def prepare(case, seed):
    d = _inputs(case, seed)
    return case, _prepare_own(case, d) if own else _prepare_plain(case, d)


def run(state):
    case, d = state
    if own:
        return _call(case, d)
    return dict(rotate=_plain_rotate, append=_plain_append, attend=_plain_attend)[case["op"]](case, d)


# ---- what a pass cannot do without -------------------------------------------------

def _visible(c, pos):
    """Keys that the token at a position sees."""
    if not c["window"]:
        return pos + 1
    last = min(pos + 1, c["window"])
    return last + min(c["sinks"], pos + 1 - last)


def work(case):
    c = case
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "rotate":
        e = 4 if c["y"] == "f32" else 2
        return dict(bytes=c["m"] * ((hq + hkv) * d * 2 * e + 4 * c["axes"]) + 2 * c["rot"],
                    flops=c["m"] * (hq + hkv) * c["rot"] * 3)
    rows, past = _lengths(c)
    token = 2 * hkv * (d // 2 + d // GROUP * 4)  # cache bytes of a token
    t = sum(rows)
    if c["op"] == "append":
        return dict(bytes=t * (2 * hkv * d * (2 + 4) + token), flops=t * 2 * hkv * d * 8)
    seen = [sum(_visible(c, p + i) for i in range(r)) for r, p in zip(rows, past)]
    held = [min(p + r, c["sinks"] + c["window"] + r - 1) if c["window"] else p + r
            for r, p in zip(rows, past)]
    return dict(bytes=sum(held) * token + t * hq * d * 4, flops=sum(seen) * hq * d * 4)


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_cache(x, d):
    """What the 4-bit cache holds for heads [t][h][d]."""
    x = x.to(torch.float64).reshape(*x.shape[:2], d // GROUP, GROUP)
    low = x.min(3).values.to(torch.float32).to(torch.bfloat16).to(torch.float64)
    step = ((x.max(3).values - low) / 15).to(torch.float32).to(torch.bfloat16).to(torch.float64)
    n = torch.round((x - low[..., None]) / step[..., None]).nan_to_num(0.0)
    return (torch.clamp(n, 0, 15) * step[..., None] + low[..., None]).reshape(*x.shape[:2], d)


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    hq, hkv, w = c["hq"], c["hkv"], c["d"]
    if c["op"] == "rotate":
        half = c["rot"] // 2
        pos = torch.stack([d["pos"][a] for a in d["axis"]], 1).to(torch.float64)
        turn = torch.polar(torch.ones_like(pos), pos * d["freq"].to(torch.float64))
        turn = (turn.conj() if c["inverse"] else turn)[:, None]
        out = {}
        for name, heads in (("q", hq), ("k", hkv)):
            x = d[name].to(torch.float64).reshape(c["m"], heads, w)
            part = x[..., :c["rot"]].reshape(c["m"], heads, *((2, half) if c["style"] == "halves" else (half, 2)))
            part = part.transpose(2, 3) if c["style"] == "halves" else part
            z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
            z = z.transpose(2, 3) if c["style"] == "halves" else z
            out[name] = torch.cat([z.reshape(c["m"], heads, c["rot"]), x[..., c["rot"]:]], 2).reshape(c["m"], -1)
        return out
    if c["op"] == "append":
        t = sum(d["rows"])
        return {n: _exact_cache(d[n].reshape(t, hkv, w), w) for n in ("k", "v")}
    g, out, row, tok = hq // hkv, [], 0, 0
    for n, ctx in zip(d["rows"], d["ctx"]):
        k, v = (_exact_cache(d[x][tok:tok + ctx], w) for x in ("k", "v"))
        q = d["q"][row:row + n].to(torch.float64).reshape(n, hkv, g, w)
        at = torch.arange(ctx - n, ctx, device=DEV).repeat_interleave(g)[:, None]
        key = torch.arange(ctx, device=DEV)[None]
        hide = key > at
        if c["window"]:
            hide = hide | ((at - key >= c["window"]) & (key >= c["sinks"]))
        heads = []
        for h in range(hkv):
            s = torch.matmul(q[:, h].reshape(n * g, w), k[:, h].t().contiguous()) / math.sqrt(w)
            s[hide] = -math.inf
            p = torch.exp(s - torch.logsumexp(s, 1, keepdim=True))
            heads.append(torch.matmul(p, v[:, h].contiguous()).reshape(n, g * w))
        out.append(torch.cat(heads, 1))
        row, tok = row + n, tok + ctx
    return torch.cat(out)
