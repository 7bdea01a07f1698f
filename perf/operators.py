"""Timed cases of the layer-block operators: the residual-adding root-mean-square
norm (with an 8-bit output and its backward pass), the shard products with bias,
activation and residual in their epilogue (and their backward pass), and the
gated feed-forward block (and its backward pass).

``own`` False computes the operators in plain torch operations in binary32,
rounded once at the end; ``own`` True makes the calls of the library.  Sizes are
those of the workloads in ``tensor_sharded_linear_plan_amd/configs.py``.

Fields of a case: ``op`` names the operator; ``m`` token rows; ``k``, ``n`` the
input and output width of a product (``n`` the width of a norm); ``tp`` the rank
shards summed in one call (norm: the rank partials added); ``w`` the weight
type; ``y`` the output type; ``act`` the activation.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DEV = "cuda"


# ---- the cases ----------------------------------------------------------------

def listed():
    return [
        # one generated token after a row-parallel product of a 7B-class layer on 4
        # ranks: rank partials added, residual stream updated, next input normed
        dict(name="norm_decode", op="norm", m=1, n=3584, tp=4, y="bf16", group=0),
        # the same between the blocks of a 27B-class layer in prefill, the next
        # products' input in 8 bits with a scale per 128 columns
        dict(name="norm_prefill_e4m3", op="norm", m=2048, n=5120, tp=4, y="e4m3", group=128),
        # norm backward, a short fine-tuning batch at width 2048
        dict(name="norm_grad_short", op="norm_grad", m=250, n=2048),
        # norm backward, a full training batch of 8192 tokens at width 4096
        dict(name="norm_grad_batch", op="norm_grad", m=8192, n=4096),
        # a decode step of 4 sequences: the down projection's 4 rank shards, 4-bit
        # weights, summed, with the residual stream added
        dict(name="linear_decode_q4", op="linear", m=4, k=18944, n=3584, tp=4, w="q4", y="bf16",
             act="none", bias=False, res=True),
        # prefill of 2048 tokens, 27B-class down projection, 4 rank shards, residual
        dict(name="linear_prefill_q4", op="linear", m=2048, k=17408, n=5120, tp=4, w="q4",
             y="bf16", act="none", bias=False, res=True),
        # one rank's column shard of a dense (non-gated) feed-forward layer: bias and
        # gelu, a batch of short prompts, ragged row count
        dict(name="linear_bf16_gelu", op="linear", m=250, k=2048, n=2048, tp=1, w="bf16",
             y="bf16", act="gelu", bias=True, res=False),
        # backward of one rank's row shard with bias, gradients kept in binary32
        dict(name="linear_grad", op="linear_grad", m=2048, k=2048, n=4096, act="none", dw="f32"),
        # one generated token through one rank's gate and up shards, 7B-class, 4-bit
        dict(name="gated_decode_q4", op="gated", m=1, k=3584, n=4736, w="q4", act="silu",
             save=False),
        # prefill through one rank's gate and up shards, 27B-class, 4-bit
        dict(name="gated_prefill_q4", op="gated", m=2048, k=5120, n=4352, w="q4", act="silu",
             save=False),
        # training forward of one rank's bf16 shards, pre-activations kept
        dict(name="gated_train", op="gated", m=512, k=4096, n=1792, w="bf16", act="silu",
             save=True),
        # training backward of one rank's bf16 shards over 4096 tokens
        dict(name="gated_grad", op="gated_grad", m=4096, k=4096, n=3584, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear_grad", "gated", "gated_grad"])
    if op == "norm":
        n, tp = _log(rng, 64, 8192), rng.choice([1, 2, 4, 8])
        m = _log(rng, 1, max(1, min(4096, 40_000_000 // (n * tp))))
        return dict(op=op, m=m, n=n, tp=tp, y=rng.choice(["bf16", "e4m3", "f32"]),
                    group=rng.choice([0, 32, 64, 128]))
    if op == "norm_grad":
        n = _log(rng, 64, 8192)
        return dict(op=op, m=_log(rng, 1, min(8192, 30_000_000 // n)), n=n)
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
    if op == "linear":
        w = rng.choice(["q4", "bf16", "f32"])
        if w == "f32":  # the framework's small fp32 layers
            m, k, n, tp = _log(rng, 1, 48), _log(rng, 64, 2048), _log(rng, 64, 2048), 1
        elif w == "q4":
            tp = rng.choice([1, 2, 4])
            m, k, n = _log(rng, 1, 2048), 64 * tp * _log(rng, 4, 64), _log(rng, 128, 5120)
        else:
            tp = rng.choice([1, 2, 4])
            m, k, n = _log(rng, 1, 2048), 16 * tp * _log(rng, 8, 128), _log(rng, 128, 5120)
        return dict(op=op, m=m, k=k, n=n, tp=tp, w=w, y="f32" if w == "f32" else "bf16", act=act,
                    bias=rng.random() < 0.5, res=rng.random() < 0.5)
    if op == "linear_grad":
        return dict(op=op, m=_log(rng, 1, 2048), k=_log(rng, 64, 4096), n=_log(rng, 64, 4096),
                    act=act, dw="f32" if act == "none" else "bf16")
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "gated":
        w = rng.choice(["q4", "bf16"])
        k = 64 * _log(rng, 4, 80) if w == "q4" else _log(rng, 256, 5120)
        return dict(op=op, m=_log(rng, 1, 2048), k=k, n=_log(rng, 128, 4352), w=w, act=act,
                    save=rng.random() < 0.5)
    return dict(op=op, m=_log(rng, 1, 4096), k=_log(rng, 128, 4096), n=_log(rng, 128, 3584),
                act=act)


# ---- inputs -------------------------------------------------------------------

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _up(v, a):
    return (v + a - 1) // a * a


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rows(g, m, n, dtype, std=1.0, ld=None):
    """[m][n] view of rows with a stride of whole 16 bytes (or `ld`)."""
    ld = ld or _up(n, 8)
    return (torch.randn((m, ld), generator=g, device=DEV) * std).to(dtype)[:, :n]


def _inputs(case, seed):
    """What the operator reads, from the seed alone (the same for both forms)."""
    g, c, d = _gen(seed), case, {}
    op, m, n = c["op"], c["m"], c["n"]
    if op == "norm":
        d["parts"] = [_rows(g, m, n, torch.float32, 0.5) for _ in range(c["tp"])]
        d["residual"] = _rows(g, m, n, torch.bfloat16, 2.0)
        d["weight"] = (1 + 0.1 * torch.randn(n, generator=g, device=DEV)).to(torch.bfloat16)
    elif op == "norm_grad":
        d["x"] = _rows(g, m, n, torch.bfloat16, 2.0)
        d["weight"] = (1 + 0.1 * torch.randn(n, generator=g, device=DEV)).to(torch.bfloat16)
        d["rstd"] = torch.rsqrt(d["x"].double().square().mean(1) + EPS).float()
        d["dy"] = _rows(g, m, n, torch.bfloat16)
        d["dres"] = _rows(g, m, n, torch.bfloat16)
    else:
        k = c["k"]
        t = TYPES["f32"] if c.get("w") == "f32" else torch.bfloat16
        d["x"] = _rows(g, m, k, t)
        names = ["gate", "up"] if op.startswith("gated") else ["w"]
        for name in names:
            if c.get("w") == "q4":
                d[name] = (torch.randint(0, 16, (k, n), generator=g, device=DEV, dtype=torch.uint8),
                           (0.005 + 0.015 * torch.rand((k // 64, n), generator=g, device=DEV)).to(torch.bfloat16),
                           (0.05 * torch.randn((k // 64, n), generator=g, device=DEV)).to(torch.bfloat16))
            else:
                d[name] = (torch.randn((k, n), generator=g, device=DEV) * 0.02).to(t)
        if op == "linear":
            d["bias"] = (0.5 * torch.randn(n, generator=g, device=DEV)).to(t) if c["bias"] else None
            d["res"] = _rows(g, m, n, t, 2.0) if c["res"] else None
        if op == "linear_grad":
            d["z"] = _rows(g, m, n, t) if c["act"] != "none" else None
            d["dy"] = _rows(g, m, n, t)
        if op == "gated_grad":
            d["g"], d["u"] = _rows(g, m, n, t), _rows(g, m, n, t)
            d["dh"] = _rows(g, m, n, t)
    return d


# ---- the operators in plain form -------------------------------------------------

def _dense(w):
    """A weight in binary32: 4-bit codes with a scale and a bias per 64 inputs, or dense."""
    if not isinstance(w, tuple):
        return w.float()
    codes, scale, bias = w
    k, n = codes.shape
    q = codes.view(k // 64, 64, n).float()
    return (q * scale.float()[:, None] + bias.float()[:, None]).view(k, n)


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _act_slope(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + \
            v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * a * (1 + 3 * 0.044715 * v * v)
    return torch.ones_like(v)


def _groups(y, group):
    """[m][n] -> [m][groups][group], zero padded; group 0 is the whole row."""
    m, n = y.shape
    w = group or n
    return torch.nn.functional.pad(y, (0, _up(n, w) - n)).view(m, -1, w)


def _plain(case, d):
    c, op = case, case["op"]
    if op == "norm":
        n = c["n"]
        r = torch.stack(d["parts"]).sum(0) + d["residual"].float()
        rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
        y = r * rstd * d["weight"].float()
        out = dict(residual=r.to(torch.bfloat16))
        if c["y"] == "e4m3":
            w = _groups(y, c["group"])
            scale = w.abs().amax(2) / E4M3_MAX
            q = w / torch.where(scale > 0, scale, torch.ones_like(scale))[:, :, None]
            y = q.clamp(-E4M3_MAX, E4M3_MAX).reshape(c["m"], -1)[:, :n]
            out["scales"] = scale
        out["y"] = y.to(TYPES[c["y"]])
        return out
    if op == "norm_grad":
        x, dy = d["x"].float(), d["dy"].float()
        xh = x * d["rstd"][:, None]
        t = dy * d["weight"].float()
        dx = d["rstd"][:, None] * (t - xh * (t * xh).mean(1, keepdim=True)) + d["dres"].float()
        return dict(dx=dx.to(torch.bfloat16), dw=(dy * xh).sum(0))
    x = d["x"].float()
    if op == "linear":
        v = x @ _dense(d["w"])
        if d["bias"] is not None:
            v = v + d["bias"].float()
        v = _act(v, c["act"])
        if d["res"] is not None:
            v = v + d["res"].float()
        return v.to(TYPES[c["y"]])
    if op == "linear_grad":
        dz = d["dy"].float()
        if d["z"] is not None:
            dz = dz * _act_slope(d["z"].float(), c["act"])
        return dict(dx=(dz @ _dense(d["w"]).t()).to(torch.bfloat16),
                    dw=(x.t() @ dz).to(TYPES[c["dw"]]), db=dz.sum(0))
    if op == "gated":
        g, u = x @ _dense(d["gate"]), x @ _dense(d["up"])
        out = dict(h=(_act(g, c["act"]) * u).to(torch.bfloat16))
        if c["save"]:
            out.update(g=g.to(torch.bfloat16), u=u.to(torch.bfloat16))
        return out
    g, u, dh = d["g"].float(), d["u"].float(), d["dh"].float()
    dg, du = dh * u * _act_slope(g, c["act"]), dh * _act(g, c["act"])
    dx = dg @ _dense(d["gate"]).t() + du @ _dense(d["up"]).t()
    return dict(dx=dx.to(torch.bfloat16), dgate=(x.t() @ dg).to(torch.bfloat16),
                dup=(x.t() @ du).to(torch.bfloat16))


# ---- the library's calls ---------------------------------------------------------

def _tsl():
    from tensor_sharded_linear_plan_amd import binding
    return binding


def _acts(tsl, act):
    return dict(none=tsl.ACT_NONE, relu=tsl.ACT_RELU, silu=tsl.ACT_SILU, gelu=tsl.ACT_GELU,
                gelu_tanh=tsl.ACT_GELU_TANH)[act]


def _bytes(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=DEV)


def _pack(tsl, shard, w, transposed=False):
    """A shard's packed copy, as a program lays its weights out once."""
    if isinstance(w, tuple):
        wt, args = tsl.Q4G64, (w[0], w[0].shape[1], 1, w[1], w[2], w[1].shape[1], 1)
    else:
        wt = tsl.F32 if w.dtype == torch.float32 else tsl.BF16
        s = (1, w.shape[1]) if transposed else (w.shape[1], 1)
        args = (w, s[0], s[1], None, None, 0, 0)
    nb = tsl.pack_shard_size(shard, wt)
    buf = _bytes(nb)
    tsl.pack_shard(shard, wt, *args, buf, nb)
    return buf, nb


def _empty(m, n, dtype):
    return torch.empty((m, _up(n, 8)), dtype=dtype, device=DEV)[:, :n]


def _prepare_own(case, d):
    tsl, c, op = _tsl(), case, case["op"]
    m, n, s = c["m"], c["n"], dict(d)
    bf, f32 = torch.bfloat16, torch.float32
    if op == "norm":
        s["sum"], s["y"] = _empty(m, n, bf), _empty(m, n, TYPES[c["y"]])
        groups = -(-n // c["group"]) if c["group"] else 1
        s["scales"] = torch.empty((m, groups), device=DEV) if c["y"] == "e4m3" else None
    elif op == "norm_grad":
        s["dx"], s["dw"] = _empty(m, n, bf), torch.empty(n, device=DEV)
        s["ws"] = _bytes(tsl.add_rms_norm_grad_workspace_size(m, n))
    elif op == "linear":
        k, tp = c["k"], c["tp"]
        s["wt"] = dict(q4=tsl.Q4G64, bf16=tsl.BF16, f32=tsl.F32)[c["w"]]
        s["y"] = _empty(m, n, TYPES[c["y"]])
        yt = tsl.F32 if c["y"] == "f32" else tsl.BF16
        s["items"], s["eps"] = [], []
        for r, sh in enumerate(tsl.plan_linear(k, n, tp, tsl.ROW, 64 if c["w"] == "q4" else 0)):
            buf, nb = _pack(tsl, sh, d["w"])
            s["items"].append(dict(shard=sh, packed=buf, packed_bytes=nb, X=s["x"][:, sh.k_off:],
                                   ldx=s["x"].stride(0), Y=s["y"], ldy=s["y"].stride(0), ydtype=yt,
                                   sum_next=int(r + 1 < tp)))
            s["eps"].append(dict(bias=d["bias"], bias_dtype=yt, act=_acts(tsl, c["act"]),
                                 residual=d["res"], res_dtype=yt,
                                 ld_res=d["res"].stride(0) if d["res"] is not None else 0)
                            if r == 0 else None)
        s["nws"] = tsl.shard_linear_group_epilogue_workspace_size(s["items"], s["eps"], s["wt"], m)
        s["ws"] = _bytes(s["nws"])
        s.pop("w")
    elif op == "gated":
        s["wt"] = tsl.Q4G64 if c["w"] == "q4" else tsl.BF16
        sh = tsl.plan_linear(c["k"], n, 1, tsl.COLUMN, 64 if c["w"] == "q4" else 0)[0]
        (pg, nb), (pu, _) = _pack(tsl, sh, s.pop("gate")), _pack(tsl, sh, s.pop("up"))
        s["h"] = _empty(m, n, bf)
        s["g"], s["u"] = (_empty(m, n, bf), _empty(m, n, bf)) if c["save"] else (None, None)
        s["items"] = [dict(gate=sh, up=sh, packed_gate=pg, packed_up=pu, packed_bytes=nb, X=s["x"],
                           ldx=s["x"].stride(0), H=s["h"], ldh=s["h"].stride(0), hdtype=tsl.BF16,
                           G=s["g"], U=s["u"], ld_gu=s["h"].stride(0))]
        s["nws"] = tsl.shard_gated_group_workspace_size(s["items"], s["wt"], m)
        s["ws"] = _bytes(s["nws"])
    else:
        k = c["k"]
        sh = s["sh"] = tsl.plan_linear(k, n, 1, tsl.COLUMN)[0]
        t = tsl.transpose_shard(sh)
        dwt = TYPES[c.get("dw", "bf16")]
        s["dx"] = _empty(m, k, bf)
        if op == "linear_grad":
            s["wp"], s["nb"] = _pack(tsl, t, s.pop("w"), True)
            s["dw"], s["db"] = _empty(k, n, dwt), torch.empty(n, device=DEV)
            s["nws"] = tsl.shard_linear_grad_workspace_size(sh, tsl.BF16, m)
        else:
            s["gp"], s["nb"] = _pack(tsl, t, s.pop("gate"), True)
            s["up_"], _ = _pack(tsl, t, s.pop("up"), True)
            s["dgate"], s["dup"] = _empty(k, n, dwt), _empty(k, n, dwt)
            s["nws"] = tsl.shard_gated_grad_workspace_size(sh, sh, tsl.BF16, m)
        s["ws"] = _bytes(s["nws"])
    return s


def _call(case, s):
    tsl, c, op = _tsl(), case, case["op"]
    m, n = c["m"], c["n"]
    if op == "norm":
        yt = dict(bf16=tsl.BF16, f32=tsl.F32, e4m3=tsl.E4M3)[c["y"]]
        p, res, w, y = s["parts"], s["residual"], s["weight"], s["y"]
        tsl.add_rms_norm(p, tsl.F32, p[0].stride(0), m, n, res, tsl.BF16, res.stride(0), s["sum"],
                         s["sum"].stride(0), w, tsl.BF16, EPS, yt, y, y.stride(0),
                         scales=s["scales"], group=c["group"] if c["y"] == "e4m3" else 0)
        out = dict(residual=s["sum"], y=y)
        if s["scales"] is not None:
            out["scales"] = s["scales"]
        return out
    if op == "norm_grad":
        x, dy, dres, dx = s["x"], s["dy"], s["dres"], s["dx"]
        tsl.add_rms_norm_grad(m, n, dy, tsl.BF16, dy.stride(0), x, tsl.BF16, x.stride(0),
                              s["weight"], tsl.BF16, EPS, s["rstd"], dres, dres.stride(0), dx,
                              tsl.BF16, dx.stride(0), s["dw"], 0, s["ws"], s["ws"].numel())
        return dict(dx=dx, dw=s["dw"])
    if op == "linear":
        tsl.shard_linear_group_epilogue(s["items"], s["eps"], s["wt"],
                                        tsl.F32 if c["w"] == "f32" else tsl.BF16, m, s["ws"],
                                        s["nws"])
        return s["y"]
    act = _acts(tsl, c["act"])
    if op == "gated":
        tsl.shard_gated_group(s["items"], act, s["wt"], tsl.BF16, m, s["ws"], s["nws"])
        return dict(h=s["h"], g=s["g"], u=s["u"]) if c["save"] else dict(h=s["h"])
    x, dx = s["x"], s["dx"]
    if op == "linear_grad":
        dy, z, dw = s["dy"], s["z"], s["dw"]
        tsl.shard_linear_grad(s["sh"], tsl.BF16, s["wp"], s["nb"], m, x, x.stride(0), act, z,
                              z.stride(0) if z is not None else 0, dy, dy.stride(0), tsl.BF16, dx,
                              dx.stride(0), tsl.F32 if c["dw"] == "f32" else tsl.BF16, dw,
                              dw.stride(0), 1, 0, s["db"], s["ws"], s["nws"])
        return dict(dx=dx, dw=dw, db=s["db"])
    g, u, dh, dg, du = s["g"], s["u"], s["dh"], s["dgate"], s["dup"]
    tsl.shard_gated_grad(s["sh"], s["sh"], tsl.BF16, s["gp"], s["up_"], s["nb"], m, x, x.stride(0),
                         act, g, u, g.stride(0), dh, dh.stride(0), tsl.BF16, dx, dx.stride(0),
                         tsl.BF16, dg, du, dg.stride(0), 1, 0, s["ws"], s["nws"])
    return dict(dx=dx, dgate=dg, dup=du)


def prepare(case, seed):
    d = _inputs(case, seed)
    return case, _prepare_own(case, d) if own else d


def run(state):
    case, d = state
    return _call(case, d) if own else _plain(case, d)


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    c, op, m, n = case, case["op"], case["m"], case["n"]
    ysz = dict(f32=4, bf16=2, e4m3=1).get(c.get("y"), 2)
    if op == "norm":
        groups = (-(-n // c["group"]) if c["group"] else 1) if c["y"] == "e4m3" else 0
        return dict(bytes=m * n * (4 * c["tp"] + 2 + 2 + ysz) + 2 * n + 4 * m * groups,
                    flops=m * n * (c["tp"] + 5))
    if op == "norm_grad":
        return dict(bytes=m * n * 8 + 4 * m + 6 * n, flops=m * n * 10)
    k = c["k"]
    sz = 4 if c.get("w") == "f32" else 2
    wb = k * n * (0.5 + 4 / 64) if c.get("w") == "q4" else k * n * sz
    if op == "linear":
        return dict(bytes=wb + m * k * sz + m * n * ysz * (1 + c["res"]) + n * sz * c["bias"],
                    flops=2 * m * k * n)
    if op == "linear_grad":
        return dict(bytes=wb + 2 * m * k * 2 + m * n * 2 * (1 + (c["act"] != "none")) +
                    k * n * (4 if c["dw"] == "f32" else 2) + 4 * n, flops=4 * m * k * n)
    if op == "gated":
        return dict(bytes=2 * wb + m * k * 2 + m * n * 2 * (3 if c["save"] else 1),
                    flops=4 * m * k * n)
    return dict(bytes=2 * wb + 2 * m * k * 2 + 3 * m * n * 2 + 2 * k * n * 2, flops=8 * m * k * n)


# ---- the definitions in 64 bits ------------------------------------------------------

def exact(case, seed):
    c, d, op = case, _inputs(case, seed), case["op"]
    f = lambda t: t.to(torch.float64)  # noqa: E731

    def weight(w):
        if not isinstance(w, tuple):
            return f(w)
        return f(w[0]) * f(w[1]).repeat_interleave(64, 0) + f(w[2]).repeat_interleave(64, 0)

    def act(v):  # value and slope
        one = torch.ones_like(v)
        if c["act"] == "none":
            return v, one
        if c["act"] == "relu":
            return v.clamp(min=0), (v > 0).double()
        if c["act"] == "silu":
            s = torch.special.expit(v)
            return v * s, s + v * s * (1 - s)
        if c["act"] == "gelu":
            p = torch.special.ndtr(v)
            return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        w = math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)  # (1 + tanh a) / 2 = expit(2 a)
        s = torch.special.expit(w)
        return v * s, s + v * s * (1 - s) * math.sqrt(8 / math.pi) * (1 + 0.134145 * v ** 2)

    if op == "norm":
        r = f(d["residual"])
        for p in d["parts"]:
            r = r + f(p)
        y = r / torch.sqrt(torch.sum(r ** 2, 1, keepdim=True) / c["n"] + EPS) * f(d["weight"])
        out = dict(residual=r, y=y)
        if c["y"] == "e4m3":
            w = c["group"] or c["n"]
            cut = [y[:, i:i + w] for i in range(0, c["n"], w)]
            top = [t.abs().max(1, keepdim=True).values for t in cut]
            out["scales"] = torch.cat(top, 1) / E4M3_MAX
            out["y"] = torch.cat([t / b * E4M3_MAX for t, b in zip(cut, top)], 1)
        return out
    if op == "norm_grad":
        x, dy, w, rs = f(d["x"]), f(d["dy"]), f(d["weight"]), f(d["rstd"])[:, None]
        dot = torch.sum(dy * w * x, 1, keepdim=True)
        return dict(dx=f(d["dres"]) + rs * dy * w - x * rs ** 3 * dot / c["n"],
                    dw=torch.sum(dy * x * rs, 0))
    x = f(d["x"])
    if op == "linear":
        v = torch.matmul(x, weight(d["w"]))
        v = act(v if d["bias"] is None else v + f(d["bias"]))[0]
        return v if d["res"] is None else v + f(d["res"])
    if op == "linear_grad":
        dz = f(d["dy"]) if d["z"] is None else f(d["dy"]) * act(f(d["z"]))[1]
        return dict(dx=torch.matmul(dz, weight(d["w"]).T.contiguous()),
                    dw=torch.matmul(x.T.contiguous(), dz), db=torch.sum(dz, 0))
    if op == "gated":
        g, u = torch.matmul(x, weight(d["gate"])), torch.matmul(x, weight(d["up"]))
        return dict(h=act(g)[0] * u, g=g, u=u) if c["save"] else dict(h=act(g)[0] * u)
    a, slope = act(f(d["g"]))
    dh = f(d["dh"])
    dg, du = dh * f(d["u"]) * slope, dh * a
    wg, wu, xt = weight(d["gate"]), weight(d["up"]), x.T.contiguous()
    return dict(dx=torch.matmul(dg, wg.T.contiguous()) + torch.matmul(du, wu.T.contiguous()),
                dgate=torch.matmul(xt, dg), dup=torch.matmul(xt, du))
