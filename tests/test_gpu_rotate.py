"""rotate_heads on the GPU against its formula in binary64.

Tolerance, u = 2^-24: the reduced angle, at most half a turn, is rounded once
(2^-26 of a turn, 2 pi times that in radians: 1.6 u), sine and cosine are within
2 u, so each is off by at most 4 u; a product, a product and their sum add
three roundings: |error| <= 6 u (|x1| + |x2|), then half a step of the output's
type."""
import numpy as np
import pytest

import attn_util as au
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def reference(x, pos, freq, axis, rot, style, inverse):
    """x [m][h][d]; (result, |x1| + |x2| where rotated, else 0)."""
    t = (pos[axis].astype(np.float64) * freq[:, None].astype(np.float64)).T  # [m][pairs]
    c, s = np.cos(t)[:, None], np.sin(t)[:, None] * (-1 if inverse else 1)
    half = rot // 2
    i1 = np.arange(half) if style == tsl.ROTARY_HALVES else 2 * np.arange(half)
    i2 = i1 + (half if style == tsl.ROTARY_HALVES else 1)
    y, mag = x.copy(), np.zeros_like(x)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    mag[..., i1] = mag[..., i2] = np.abs(x[..., i1]) + np.abs(x[..., i2])
    return y, mag


def check(got, want, mag, kind):
    """Columns passed through (mag 0) are rounded once too: not at all where the
    types are the same."""
    err = 6 * au.U * mag
    au.within(got, want, err + au.HALF[kind] * (np.abs(want) + err))


def setup(seed, m, heads, d, rot, axes, far, xk, yk, pad, head_major, in_place):
    r, t = au.rng(seed), torch()
    freq = (1e6 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    pos = r.integers(-far // 3, far + 1, size=(axes, m)).astype(np.int32)
    axis = r.integers(0, axes, size=rot // 2)
    ops, items = [], []
    for h in heads:
        x = au.Operand(m, h, d, xk, pad, head_major, values=r.standard_normal((m, h, d)) * 2)
        y = x if in_place else au.Operand(m, h, d, yk, pad * 2, head_major)
        ops.append((x, y, x.get()))
        items.append(dict(X=x.view, ldx=x.ld, x_head=x.head, Y=y.view, ldy=y.ld, y_head=y.head,
                          n_heads=h, xdtype=au.DT[xk], ydtype=au.DT[yk]))
    ld = m + 3
    dpos = t.zeros((axes, ld), dtype=t.int32, device=DEV)
    dpos[:, :m] = t.from_numpy(pos).to(DEV)
    rotary = dict(positions=dpos, ld_pos=ld, axes=axes, pair_axis=axis.tolist(),
                  freq=t.from_numpy(freq).to(DEV), rot_dim=rot, head_dim=d)
    return ops, items, rotary, pos, freq, axis


@pytest.mark.parametrize("m,heads,d,rot,axes,style,xk,yk,pad,head_major", [
    (1, (28, 4), 128, 128, 1, 0, "bf16", "bf16", 0, False),
    (1, (1,), 64, 64, 1, 1, "bf16", "bf16", 0, False),
    (5, (7, 1), 128, 96, 3, 0, "bf16", "bf16", 1, False),
    (33, (8, 2), 64, 48, 3, 1, "f32", "f32", 0, False),
    (130, (3, 3, 1), 256, 256, 2, 0, "f32", "bf16", 2, True),
    (17, (2,), 512, 512, 4, 1, "bf16", "f32", 0, True),
    (9, (3,), 80, 20, 2, 0, "bf16", "bf16", 0, False),   # half no multiple of 8
    (9, (3,), 36, 6, 2, 1, "f32", "f32", 0, False),      # odd widths
    (4, (5,), 64, 2, 1, 0, "bf16", "bf16", 0, False),    # one pair
    (700, (16, 8), 128, 64, 1, 0, "bf16", "bf16", 0, False),
])
@pytest.mark.parametrize("inverse", [0, 1])
def test_rotate(m, heads, d, rot, axes, style, xk, yk, pad, head_major, inverse):
    ops, items, rotary, pos, freq, axis = setup(m * 7 + d, m, heads, d, rot, axes, 100000, xk, yk,
                                                pad, head_major, False)
    rotary["style"] = style
    tsl.rotate_heads(items, m, rotary, inverse)
    for x, y, x0 in ops:
        want, mag = reference(x0, pos, freq, axis, rot, style, inverse)
        check(y.get(), want, mag, yk)
        if rot < d:
            assert np.array_equal(y.get()[..., rot:], au.rne(x0[..., rot:], yk))
        assert y.rest_untouched() and np.array_equal(x.get(), x0)


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("odd", [False, True])
def test_in_place_and_there_and_back(style, odd):
    d, rot = (36, 22) if odd else (128, 64)
    ops, items, rotary, pos, freq, axis = setup(3, 50, (6, 2), d, rot, 2, 5000, "f32", "f32", 1,
                                                False, True)
    rotary["style"] = style
    tsl.rotate_heads(items, 50, rotary, 0)
    first = [x.get() for x, _, _ in ops]
    for (x, _, x0), f in zip(ops, first):
        want, mag = reference(x0, pos, freq, axis, rot, style, 0)
        check(f, want, mag, "f32")
        assert x.rest_untouched()
    tsl.rotate_heads(items, 50, rotary, 1)
    for (x, _, x0), f in zip(ops, first):  # two rotations' errors
        _, mag = reference(x0, pos, freq, axis, rot, style, 0)
        # |x1| + |x2| = mag; the first result's columns are each off by 7 u mag (formula
        # and rounding) and together at most 1.5 mag: the second turn passes on both
        # columns' errors (14 u mag) and adds 6 u 1.5 mag and half a step (u 1.5 mag)
        assert (np.abs(x.get() - x0) <= 25 * au.U * mag).all()


def test_inverse_is_the_gradient():
    """The inverse call against differences of the forward one: for a linear map
    <dy, R (x + h e) - R x> / h = (R^T dy)_e up to binary32 rounding."""
    t, m, h, d = torch(), 3, 2, 64
    ops, items, rotary, pos, freq, axis = setup(5, m, (h,), d, 48, 3, 300, "f32", "f32", 0, False, False)
    x, y, x0 = ops[0]
    dy = au.rng(8).standard_normal((m, h, d)).astype(np.float32).astype(np.float64)
    g = au.Operand(m, h, d, "f32", values=dy)
    dx = au.Operand(m, h, d, "f32")
    tsl.rotate_heads([dict(items[0], X=g.view, ldx=g.ld, x_head=g.head, Y=dx.view, ldy=dx.ld,
                           y_head=dx.head)], m, rotary, 1)
    step = 2.0 ** 6
    for col in (0, 5, 24, 29, 47, 48, 63):
        out = []
        for sign in (1, -1):
            v = x0.copy()
            v[..., col] += sign * step
            x.view.copy_(t.from_numpy(v.astype(np.float32)))
            tsl.rotate_heads(items, m, rotary, 0)
            out.append(y.get())
        diff = ((out[0] - out[1]) * dy).sum(-1) / (2 * step)
        # |x| <= 2^7 + 10: each output off by 6 u 2 2^7.2 and half a step of it, two of them count
        bound = 2 * (12 + 1) * au.U * 2 ** 7.2 * np.abs(dy).max() * 2 / (2 * step) + 12 * au.U * np.abs(dy).max()
        assert (np.abs(diff - dx.get()[..., col]) <= bound).all(), col


def test_far_positions():
    """Positions next to 2^31: the angle is the binary64 product's."""
    t = torch()
    pos = np.array([[2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 1234567]], np.int32)
    freq = np.array([1.0, 0.7310585, 1e-3, 1e-6], np.float32)
    x = au.Operand(4, 1, 8, "f32", values=au.rng(1).standard_normal((4, 1, 8)))
    y = au.Operand(4, 1, 8, "f32")
    tsl.rotate_heads([dict(X=x.view, ldx=x.ld, x_head=x.head, Y=y.view, ldy=y.ld, y_head=y.head,
                           n_heads=1, xdtype=0, ydtype=0)], 4,
                     dict(positions=t.from_numpy(pos).to(DEV), freq=t.from_numpy(freq).to(DEV),
                          rot_dim=8, head_dim=8))
    from fractions import Fraction
    import math
    # 2 pi to 40 digits: exact reduction of the exact product
    two_pi = Fraction(62831853071795864769252867665590057683943, 10 ** 40)
    ang = np.array([[float(Fraction(int(p)) * Fraction(float(f)) -
                           two_pi * math.floor(Fraction(int(p)) * Fraction(float(f)) / two_pi))
                     for f in freq] for p in pos[0]])
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    x0 = x.get()
    want = np.concatenate([x0[..., :4] * c - x0[..., 4:] * s, x0[..., 4:] * c + x0[..., :4] * s], -1)
    # the turns (3.5e8 at most) carry three binary64 roundings, 2^-53 of them each
    extra = 2 * np.pi * 3.5e8 * 3 * 2.0 ** -53
    mag = np.abs(x0[..., :4]) + np.abs(x0[..., 4:])
    mag = np.concatenate([mag, mag], -1)
    assert (np.abs(y.get() - want) <= (7 * au.U + extra) * mag).all()


def test_no_rows_and_grouped_layout_in_place():
    """M = 0 enqueues nothing; q and k heads lying in turns ([q q k] per K/V head)
    rotate in place, v between them left alone."""
    t, m, d, kv, g = torch(), 11, 64, 3, 2
    per = (g + 2) * d  # q, q, k, v
    x = t.randn((m, kv * per), device=DEV).to(t.bfloat16)
    x0 = x.clone()
    freq = t.rand(32, device=DEV)
    pos = t.arange(m, dtype=t.int32, device=DEV)
    rot = dict(positions=pos, freq=freq, rot_dim=64, head_dim=d)
    items = [dict(X=x[:, i * d:], ldx=kv * per, x_head=per, Y=x[:, i * d:], ldy=kv * per, y_head=per,
                  n_heads=kv, xdtype=tsl.BF16, ydtype=tsl.BF16) for i in (0, 1, 2)]
    tsl.rotate_heads(items, 0, rot)
    assert t.equal(x, x0)
    tsl.rotate_heads(items, m, rot)
    a, b = (v.double().cpu().numpy().reshape(m, kv, g + 2, d) for v in (x, x0))
    want, mag = reference(b[:, :, :3].reshape(m, -1, d), pos.cpu().numpy()[None],
                          freq.cpu().numpy(), np.zeros(32, int), 64, 0, 0)
    check(a[:, :, :3].reshape(m, -1, d), want, mag, "bf16")
    assert np.array_equal(a[:, :, 3], b[:, :, 3])
