"""The e4m3 output of add_rms_norm bit for bit.  Rows of +-1 with eps 0 have
rstd exactly 1, so y is +-weight exactly and the scale max |y| / 448 and the
codes y / scale follow from binary32 divisions, each rounded to nearest even,
and one rounding to e4m3: nothing is left to a tolerance."""
import numpy as np
import pytest

from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu

f4 = np.float32
TOP = f4(448)


def codes(y, s):
    """Of one run: RNE_e4m3(y / s), zeros where s is zero."""
    t = torch()
    with np.errstate(divide="ignore", invalid="ignore"):
        x = np.where(s > 0, np.clip((y / s).astype(f4), -TOP, TOP), f4(0)).astype(f4)
    return t.from_numpy(x).to(t.float8_e4m3fn).float().numpy()


def run(w, group):
    """Codes and scales of a row of alternating signs and weight w."""
    t = torch()
    n = w.size
    sign = np.where(np.arange(n) % 2, -1, 1).astype(f4)
    P, W = t.from_numpy(sign[None]).to(DEV), t.from_numpy(w).to(DEV)
    Y = t.empty((1, n), dtype=t.float8_e4m3fn, device=DEV)
    sc = t.empty((1, -(-n // group) if group else 1), device=DEV)
    rs = t.empty(1, device=DEV)
    tsl.add_rms_norm([P], tsl.F32, n, 1, n, None, tsl.F32, 0, None, 0, W, tsl.F32, 0.0, tsl.E4M3, Y,
                     n, sc, group, rs)
    assert float(rs) == 1.0
    return Y.float().cpu().numpy()[0], sc.cpu().numpy()[0], sign * w


def check(w, group):
    got, sc, y = run(w, group)
    g = group or w.size
    for i in range(sc.size):
        b = slice(i * g, (i + 1) * g)
        s = f4(np.abs(y[b]).max() / TOP)
        assert sc[i] == s
        assert np.array_equal(got[b], codes(y[b], s)), (i, y[b], s)


def near_ties(rng, top, count):
    """A run's maximum and values within a step of where two codes meet."""
    s = f4(top / TOP)
    tie = (rng.integers(8, 16, count) + .5) * 2.0 ** rng.integers(-9, 5, count)
    v = (np.minimum(tie, 440) * np.float64(s)).astype(f4)
    step = rng.integers(-1, 2, count)
    v = np.where(step < 0, np.nextafter(v, f4(0)), np.where(step > 0, np.nextafter(v, f4(np.inf)), v))
    return np.concatenate([[top], v]).astype(f4)


@pytest.mark.parametrize("group", [32, 64, 128, 0])
def test_codes_next_to_ties(group):
    rng = np.random.default_rng(group)
    g = group or 512
    for _ in range(4):
        check(np.concatenate([near_ties(rng, f4(2.0 ** rng.integers(-3, 4) * (1 + rng.random())), g - 1)
                              for _ in range(8192 // g if group else 1)]), group)


@pytest.mark.parametrize("group", [32, 0])
@pytest.mark.parametrize("top", [2.0 ** -100, 2.0 ** -117, 2.0 ** -126, 2.0 ** -135, 2.0 ** -139,
                                 2.0 ** -140, 2.0 ** -141, 2.0 ** -149, 2.0 ** 120])
def test_scales_near_the_ends_of_the_range(group, top):
    """Scales that are subnormal, round up to the smallest subnormal or down to
    zero, and ones whose reciprocal is subnormal."""
    rng = np.random.default_rng(1)
    check(np.concatenate([near_ties(rng, f4(top * k), 31) for k in (1, 1.25, 1.5, 1.75)]), group)
