"""The layer-block operators together, as a feed-forward block uses them on
two ranks: norm of (rank partials + residual) -> gate/up column shards with the
gate -> down row shards, summed, with the residual -- and the backward pass
through all of it -- against the same block in binary64.

Every stored value is bf16 (half step h = 2^-8), and every stage rounds its
result once, so each output's error is a handful of independent h-sized
relative errors carried through the block.  Carried linearly, a stage's
relative (2-norm) error is at most the sum over the rounded tensors that feed
it; forward that is 4 roundings (stream, norm, H, output), backward up to 12
(the forward's three, each gradient tensor's and each dZ pair's).  A rounding's
2-norm error is at most h, and the nonlinear steps (norm, silu) amplify by no
more than 2 at these inputs, so 2 * 4 h and 2 * 12 h bound the two."""
import numpy as np
import pytest

from block_util import HALF, Weight, act, f64, out, put, rng, ws
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu

TP, D, F, EPS = 2, 192, 256, 1e-5
B = tsl.BF16


class Block:
    def __init__(self, M):
        t = torch()
        self.M = M
        self.G, self.U_, self.D_ = (Weight("bf16", *s, seed, False)
                                    for s, seed in (((D, F), 1), ((D, F), 2), ((F, D), 3)))
        self.w = put(1 + 0.1 * rng(4).standard_normal((1, D)), "bf16")[0]
        self.parts = [put(rng(5 + r).standard_normal((M, D)), "f32") for r in range(TP)]
        self.res = put(rng(9).standard_normal((M, D)), "bf16")
        self.dy = put(rng(10).standard_normal((M, D)), "bf16")
        self.col = tsl.plan_linear(D, F, TP, tsl.COLUMN)
        self.row = tsl.plan_linear(F, D, TP, tsl.ROW)
        self.fwd = [(self.G.pack(c), self.U_.pack(c), self.D_.pack(r))
                    for c, r in zip(self.col, self.row)]
        self.bwd = [(self.G.pack(tsl.transpose_shard(c), True),
                     self.U_.pack(tsl.transpose_shard(c), True),
                     self.D_.pack(tsl.transpose_shard(r), True))
                    for c, r in zip(self.col, self.row)]
        new = lambda n, k="bf16": out(M, n, k)[1]  # noqa: E731
        self.stream, self.x, self.y = new(D), new(D), new(D)
        self.rstd = t.empty(M, device=DEV)
        self.h, self.g, self.u, self.dh = new(F), new(F), new(F), new(F)
        self.dparts = [new(D, "f32") for _ in range(TP)]
        self.dxn, self.dx = new(D), new(D)
        self.dwn = t.empty(D, device=DEV)
        self.dg, self.du, self.dd = (t.empty(s, device=DEV) for s in ((D, F), (D, F), (F, D)))

    def forward(self):
        M, f = self.M, F // TP
        tsl.add_rms_norm(self.parts, tsl.F32, self.parts[0].stride(0), M, D, self.res, B, D,
                         self.stream, D, self.w, B, EPS, B, self.x, D, rstd=self.rstd)
        items = [dict(gate=c, up=c, packed_gate=p[0][0], packed_up=p[1][0], packed_bytes=p[0][1],
                      X=self.x, ldx=D, H=self.h[:, r * f:], ldh=F, hdtype=B, G=self.g[:, r * f:],
                      U=self.u[:, r * f:], ld_gu=F)
                 for r, (c, p) in enumerate(zip(self.col, self.fwd))]
        n = tsl.shard_gated_group_workspace_size(items, B, M)
        keep = [ws(n)]
        tsl.shard_gated_group(items, tsl.ACT_SILU, B, B, M, keep[0], n)
        items = [dict(shard=s, packed=p[2][0], packed_bytes=p[2][1], X=self.h[:, r * f:], ldx=F,
                      Y=self.y, ldy=D, ydtype=B, sum_next=int(r + 1 < TP))
                 for r, (s, p) in enumerate(zip(self.row, self.fwd))]
        eps = [dict(residual=self.stream, res_dtype=B, ld_res=D)] + [None] * (TP - 1)
        n = tsl.shard_linear_group_epilogue_workspace_size(items, eps, B, M)
        keep.append(ws(n))
        tsl.shard_linear_group_epilogue(items, eps, B, B, M, keep[1], n)
        return keep

    def backward(self):
        M, f = self.M, F // TP
        keep = []
        for r in range(TP):
            s, c, (pg, pu, pd) = self.row[r], self.col[r], self.bwd[r]
            n = tsl.shard_linear_grad_workspace_size(s, B, M)
            keep.append(ws(n))
            tsl.shard_linear_grad(s, B, *pd, M, self.h[:, r * f:], F, tsl.ACT_NONE, None, 0, self.dy,
                                  D, B, self.dh[:, r * f:], F, tsl.F32, self.dd[r * f:], D, 1, 0,
                                  None, keep[-1], n)
            n = tsl.shard_gated_grad_workspace_size(c, c, B, M)
            keep.append(ws(n))
            tsl.shard_gated_grad(c, c, B, pg[0], pu[0], pg[1], M, self.x, D, tsl.ACT_SILU,
                                 self.g[:, r * f:], self.u[:, r * f:], F, self.dh[:, r * f:], F,
                                 tsl.F32, self.dparts[r], D, tsl.F32, self.dg[:, r * f:],
                                 self.du[:, r * f:], F, 1, 0, keep[-1], n)
        tsl.combine_partials(tsl.COMBINE_SUM, self.dparts, tsl.F32, M, D, D, B, self.dxn, D)
        n = tsl.add_rms_norm_grad_workspace_size(M, D)
        keep.append(ws(n))
        tsl.add_rms_norm_grad(M, D, self.dxn, B, D, self.stream, B, D, self.w, B, EPS, self.rstd,
                              self.dy, D, self.dx, B, D, self.dwn, 0, keep[-1], n)
        return keep

    def outputs(self):
        return dict(stream=self.stream, y=self.y, dx=self.dx, dwn=self.dwn, dg=self.dg, du=self.du,
                    dd=self.dd)


def reference(b):
    wg, wu, wd, w, dy = b.G.w, b.U_.w, b.D_.w, f64(b.w), f64(b.dy)
    s = f64(b.res) + sum(f64(p) for p in b.parts)
    rstd = 1 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + EPS)
    x = s * rstd * w
    g, u = x @ wg, x @ wu
    a, d, _ = act(g, "silu")
    h = a * u
    dh = dy @ wd.T
    dg, du = dh * u * d, dh * a
    dx = dg @ wg.T + du @ wu.T
    t, xh = dx * w, s * rstd
    return dict(stream=s, y=h @ wd + s, dd=h.T @ dy, dg=x.T @ dg, du=x.T @ du,
                dwn=np.sum(dx * xh, 0),
                dx=rstd * (t - xh * np.mean(t * xh, axis=1, keepdims=True)) + dy)


@pytest.mark.parametrize("M", [1, 5, 48, 200])
def test_forward_and_backward(M):
    b = Block(M)
    keep = b.forward(), b.backward()
    want = reference(b)
    for k, v in b.outputs().items():
        rel = np.linalg.norm(f64(v) - want[k]) / np.linalg.norm(want[k])
        assert rel <= (8 if k in ("stream", "y") else 24) * HALF["bf16"], (k, rel)
    del keep


def test_captured_beside_eager_runs():
    """Forward and backward in one captured graph, replayed between eager runs
    of another block with buffers of its own: each keeps its results."""
    t = torch()
    a, b = Block(40), Block(7)
    keep = [a.forward(), a.backward(), b.forward(), b.backward()]
    wa, wb = ({k: v.clone() for k, v in c.outputs().items()} for c in (a, b))
    graph, side = t.cuda.CUDAGraph(), t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.graph(graph, stream=side):
        keep += [a.forward(), a.backward()]
    for _ in range(3):
        for c in (a, b):
            for v in c.outputs().values():
                v.zero_()
        graph.replay()
        keep += [b.forward(), b.backward()]
        t.cuda.synchronize()
        for c, w in ((a, wa), (b, wb)):
            assert all(t.equal(v, w[k]) for k, v in c.outputs().items())
