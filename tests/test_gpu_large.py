"""4-bit weights of more than 4 GiB packed: every column reads its own
records.

All codes and scales are zero, so W[k][n] = bias[k / 64][n], and each row of X
holds a single one: a product is one bias, exactly."""
import pytest

import gpu_util  # noqa: F401
from block_util import DEV, torch, tsl, ws

pytestmark = pytest.mark.gpu

K, N = 65536, 120000


@pytest.fixture(scope="module")
def weight():
    t = torch()
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN, 64)[0]
    nb = tsl.pack_shard_size(sh, tsl.Q4G64)
    assert nb > 1 << 32
    col = t.arange(N, device=DEV)
    # 1 .. 127 eighths, another value every 16 columns and every group of k
    bias = ((col // 16 * 7 + 13 * t.arange(K // 64, device=DEV)[:, None]) % 127 + 1).float() / 8
    bias = bias.bfloat16()
    codes = t.zeros((K, N), dtype=t.uint8, device=DEV)
    scales = t.zeros_like(bias)
    buf = t.empty(nb, dtype=t.uint8, device=DEV)
    tsl.pack_shard(sh, tsl.Q4G64, codes, N, 1, scales, bias, N, 1, buf, nb)
    t.cuda.synchronize()
    return sh, buf, nb, bias.float()


def rows(M):
    t = torch()
    at = (t.arange(M, device=DEV) * 997) % K
    x = t.zeros((M, K), dtype=t.bfloat16, device=DEV)
    x[t.arange(M, device=DEV), at] = 1
    return x, at // 64


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_products(weight, M):
    t = torch()
    sh, buf, nb, bias = weight
    x, g = rows(M)
    want = bias[g]
    n = tsl.shard_linear_workspace_size(sh, tsl.Q4G64, M)
    y = t.empty((M, N), device=DEV)
    w = ws(n)
    tsl.shard_linear(sh, tsl.Q4G64, buf, nb, tsl.BF16, x, K, M, tsl.F32, y, N, 0, w, n)
    assert bool((y == want).all()), "plain"
    y.fill_(float("nan"))
    res = t.ones((M, N), device=DEV)
    it = [dict(shard=sh, packed=buf, packed_bytes=nb, X=x, ldx=K, Y=y, ldy=N, ydtype=tsl.F32)]
    ep = [dict(residual=res, res_dtype=tsl.F32, ld_res=N)]
    n = tsl.shard_linear_group_epilogue_workspace_size(it, ep, tsl.Q4G64, M)
    w = ws(n)
    tsl.shard_linear_group_epilogue(it, ep, tsl.Q4G64, tsl.BF16, M, w, n)
    assert bool((y == want + 1).all()), "epilogue"
    y.fill_(float("nan"))
    it = [dict(gate=sh, up=sh, packed_gate=buf, packed_up=buf, packed_bytes=nb, X=x, ldx=K, H=y,
               ldh=N, hdtype=tsl.F32)]
    n = tsl.shard_gated_group_workspace_size(it, tsl.Q4G64, M)
    w = ws(n)
    tsl.shard_gated_group(it, tsl.ACT_NONE, tsl.Q4G64, tsl.BF16, M, w, n)
    assert bool((y == want * want).all()), "gated"
