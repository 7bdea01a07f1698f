"""Rows so far apart that element offsets pass 2^31 (and bytes 2^32): the same
bits as from dense rows."""
import pytest

import gpu_util  # noqa: F401
from block_util import DEV, Weight, torch, tsl, ws

pytestmark = pytest.mark.gpu

M, LD = 2200, 1 << 20  # 2.3e9 elements


def far(cols, kind, src=None):
    t = torch()
    buf = t.empty((M, LD), dtype=kind, device=DEV)[:, :cols]
    buf.fill_(float("nan")) if src is None else buf.copy_(src)
    return buf


def rand(cols, kind, seed):
    t = torch()
    g = t.Generator(device=DEV).manual_seed(seed)
    return t.randn((M, cols), device=DEV, generator=g).to(kind)


def test_norm_and_its_backward():
    t = torch()
    n, bf = 1024, t.bfloat16
    p, r, dy = (rand(n, bf, s) for s in range(3))
    w = rand(n, bf, 3)[0].contiguous()
    res = []
    for f in (False, True):
        P, R, DY = (far(n, bf, x) if f else x for x in (p, r, dy))
        S, Y, DX = (far(n, bf) if f else t.empty((M, n), dtype=bf, device=DEV) for _ in range(3))
        ld = LD if f else n
        rstd = t.empty(M, device=DEV)
        tsl.add_rms_norm([P, P], tsl.BF16, ld, M, n, R, tsl.BF16, ld, S, ld, w, tsl.BF16, 1e-6,
                         tsl.BF16, Y, ld, rstd=rstd)
        nb = tsl.add_rms_norm_grad_workspace_size(M, n)
        dw = t.empty(n, device=DEV)
        tsl.add_rms_norm_grad(M, n, DY, tsl.BF16, ld, S, tsl.BF16, ld, w, tsl.BF16, 1e-6, rstd, R,
                              ld, DX, tsl.BF16, ld, dw, 0, ws(nb), nb)
        res.append([x.clone() for x in (S, Y, DX, dw, rstd)])
    for a, b in zip(*res):
        assert bool(t.isfinite(a).all()) and bool((a == b).all())


@pytest.mark.parametrize("kind", ["bf16", "q4"])
def test_products(kind):
    t = torch()
    K, N, bf = 192, 160, t.bfloat16
    dt = {"bf16": tsl.BF16, "q4": tsl.Q4G64}[kind]
    W = Weight(kind, K, N, 5)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN, 64)[0]
    buf, nb = W.pack(sh)
    x, r = rand(K, bf, 6), rand(N, bf, 7)
    res = []
    for f in (False, True):
        X, R = (far(x_.shape[1], bf, x_) if f else x_ for x_ in (x, r))
        Y, P, H, G, U = (far(N, bf) if f else t.empty((M, N), dtype=bf, device=DEV)
                         for _ in range(5))
        lx, ln = (LD, LD) if f else (K, N)
        it = [dict(shard=sh, packed=buf, packed_bytes=nb, X=X, ldx=lx, Y=Y, ldy=ln,
                   ydtype=tsl.BF16)]
        ep = [dict(act=tsl.ACT_SILU, residual=R, res_dtype=tsl.BF16, ld_res=ln, pre=P,
                   pre_dtype=tsl.BF16, ld_pre=ln)]
        need = tsl.shard_linear_group_epilogue_workspace_size(it, ep, dt, M)
        w = ws(need)
        tsl.shard_linear_group_epilogue(it, ep, dt, tsl.BF16, M, w, need)
        it = [dict(gate=sh, up=sh, packed_gate=buf, packed_up=buf, packed_bytes=nb, X=X, ldx=lx,
                   H=H, ldh=ln, hdtype=tsl.BF16, G=G, U=U, ld_gu=ln)]
        need = tsl.shard_gated_group_workspace_size(it, dt, M)
        w2 = ws(need)
        tsl.shard_gated_group(it, tsl.ACT_SILU, dt, tsl.BF16, M, w2, need)
        res.append([x_.clone() for x_ in (Y, P, H, G, U)])
        del X, R, Y, P, H, G, U
    for a, b in zip(*res):
        assert bool(t.isfinite(a).all()) and bool((a == b).all())


def test_backward_products():
    t = torch()
    K, N, bf = 192, 160, t.bfloat16
    W = Weight("bf16", K, N, 8)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    tr = tsl.transpose_shard(sh)
    nb = tsl.pack_shard_size(tr, tsl.BF16)
    packed = t.empty(nb, dtype=t.uint8, device=DEV)
    tsl.pack_shard(tr, tsl.BF16, W.d, 1, N, None, None, 0, 0, packed, nb)
    x, z, dy = rand(K, bf, 9), rand(N, bf, 10), rand(N, bf, 11)
    res = []
    for f in (False, True):
        X, Z, DY = (far(s.shape[1], bf, s) if f else s for s in (x, z, dy))
        lx, ln = (LD, LD) if f else (K, N)
        DX = far(K, bf) if f else t.empty((M, K), dtype=bf, device=DEV)
        dW, db = t.empty((K, N), device=DEV), t.empty(N, device=DEV)
        n = tsl.shard_linear_grad_workspace_size(sh, tsl.BF16, M)
        w = ws(n)
        tsl.shard_linear_grad(sh, tsl.BF16, packed, nb, M, X, lx, tsl.ACT_GELU, Z, ln, DY, ln,
                              tsl.BF16, DX, lx, tsl.F32, dW, N, 1, 0, db, w, n)
        res.append([s.clone() for s in (DX, dW, db)])
        n = tsl.shard_gated_grad_workspace_size(sh, sh, tsl.BF16, M)
        w2 = ws(n)
        dU = t.empty_like(dW)
        tsl.shard_gated_grad(sh, sh, tsl.BF16, packed, packed, nb, M, X, lx, tsl.ACT_SILU, Z, Z,
                             ln, DY, ln, tsl.BF16, DX, lx, tsl.F32, dW, dU, N, 1, 0, w2, n)
        res[-1] += [s.clone() for s in (DX, dW, dU)]
    for a, b in zip(*res):
        assert bool(t.isfinite(a).all()) and bool((a == b).all())
