"""Shared by the tests of the layer-block operators: exact inputs in every
weight type, the activations in binary64 and the errors their binary32
evaluation may have."""
import numpy as np
from scipy import special

from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": tsl.F32, "bf16": tsl.BF16, "q4": tsl.Q4G64}
ACTS = {"none": tsl.ACT_NONE, "relu": tsl.ACT_RELU, "silu": tsl.ACT_SILU, "gelu": tsl.ACT_GELU,
        "gelu_tanh": tsl.ACT_GELU_TANH}
SCALE = 2.0 ** -7  # weights are integers times this


def tt(name):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16}[name]


def f64(x):
    return x.detach().cpu().double().numpy()


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def put(a, kind, ld=None, fill=float("nan")):
    """numpy [m][n] -> device rows of `kind` at a stride of ld, padding `fill`."""
    t = torch()
    a = np.atleast_2d(a)
    ld = ld or (a.shape[1] + 7) // 8 * 8
    buf = t.full((a.shape[0], ld), fill, dtype=t.float32)
    buf[:, :a.shape[1]] = t.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return buf.to(tt(kind)).to(DEV)[:, :a.shape[1]]


def out(m, n, kind, ld=None, fill=7.0):
    t = torch()
    ld = ld or (n + 7) // 8 * 8
    buf = t.full((m + 1, ld), fill, dtype=tt(kind), device=DEV)
    return buf, buf[:m, :n]


def untouched(buf, m, n, fill=7.0):
    """Nothing outside the [m][n] block was written."""
    return bool((buf[m:] == fill).all()) and bool((buf[:m, n:] == fill).all())


def ints(seed, shape, lo=-3, hi=3):
    return rng(seed).integers(lo, hi + 1, size=shape).astype(np.float64)


class Weight:
    """W[K][N] = small integers times SCALE, exact in every weight type (4-bit:
    scale SCALE, bias -8 SCALE), or random values when exact is False."""

    def __init__(self, kind, K, N, seed, exact=True):
        t = torch()
        self.kind, self.K, self.N = kind, K, N
        r = rng(seed)
        if kind == "q4":
            q = r.integers(0, 16, size=(K, N)).astype(np.uint8)
            if exact:
                s = np.full((K // 64, N), SCALE)
                b = -8 * s
            else:
                s, b = r.uniform(.005, .02, (K // 64, N)), .05 * r.standard_normal((K // 64, N))
            self.s = t.from_numpy(s.astype(np.float32)).to(t.bfloat16).to(DEV)
            self.b = t.from_numpy(b.astype(np.float32)).to(t.bfloat16).to(DEV)
            self.q = t.from_numpy(q).to(DEV)
            self.w = q * np.repeat(f64(self.s), 64, 0) + np.repeat(f64(self.b), 64, 0)
        else:
            w = r.integers(-8, 8, size=(K, N)) * SCALE if exact else .02 * r.standard_normal((K, N))
            self.d = t.from_numpy(w.astype(np.float32)).to(tt(kind)).to(DEV)
            self.w = f64(self.d)

    def pack(self, sh, transposed=False):
        t = torch()
        nb = tsl.pack_shard_size(sh, DT[self.kind])
        buf = t.empty(nb, dtype=t.uint8, device=DEV)
        if self.kind == "q4":
            tsl.pack_shard(sh, tsl.Q4G64, self.q, self.N, 1, self.s, self.b, self.N, 1, buf, nb)
        else:
            k, n = (1, self.N) if transposed else (self.N, 1)
            tsl.pack_shard(sh, DT[self.kind], self.d, k, n, None, None, 0, 0, buf, nb)
        return buf, nb


def ws(n):
    t = torch()
    return t.full((max(int(n), 256),), 0xAB, dtype=t.uint8, device=DEV) if n else None


def act(v, name):
    """(value, slope, bound on the binary32 value's error) of an activation.

    With u = 2^-24: the logistic s(t) = 1 / (1 + 2^(-t log2 e)) has its
    exponent's argument within 2 u |t| 1.45 (a product and a rounded constant)
    plus, for gelu_tanh, 4 u of t itself; exp2, the sum, the reciprocal and the
    product with v add 1 to 2 u each: (6 |t| + 8) u of the result.  erfc is
    within 16 ulp (32 u) and its argument within 2 u, which it answers 2 x^2
    fold (x^2 = v^2 / 2): (2 v^2 + 40) u.  Results below the smallest normal
    binary32 number may be flushed."""
    one = np.ones_like(v)
    if name == "none":
        return v, one, 0 * v
    if name == "relu":
        return np.maximum(v, 0), (v > 0).astype(float), 0 * v
    if name == "gelu":
        p = 0.5 * special.erfc(-v / np.sqrt(2))
        a = v * p
        return a, p + v * np.exp(-v * v / 2) / np.sqrt(2 * np.pi), \
            (2 * v * v + 40) * U * np.abs(a) + 1e-35
    c0 = 2 * np.sqrt(2 / np.pi)
    t, dt = (v, one) if name == "silu" else (c0 * (v + 0.044715 * v ** 3),
                                             c0 * (1 + 3 * 0.044715 * v ** 2))
    s = special.expit(t)
    return v * s, s + v * s * (1 - s) * dt, (6 * np.abs(t) + 8) * U * np.abs(v * s) + 1e-35


def close(got, want, err, kind):
    """|got - want| within err and the stored type's half step."""
    bad = np.abs(got - want) > err + HALF[kind] * (np.abs(want) + err) + 1e-38
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def rne(x, kind):
    """binary64 values that binary32 holds, rounded to the stored type."""
    t = torch()
    return t.from_numpy(np.asarray(x, dtype=np.float32)).to(tt(kind)).double().numpy()
