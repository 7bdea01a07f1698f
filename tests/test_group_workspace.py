"""Grouped products accept the workspace their size query asks for, with items
that accumulate among the others, on the host alone: the workspace's address is
odd, so a call of enough bytes ends in TSL_ERR_MISALIGNED and one of too few in
TSL_ERR_BUFFER_TOO_SMALL."""
import pytest

A = 1 << 44  # addresses far apart; never read
STEP = 1 << 36


def items_of(t, units):
    """units: (members, k_len, n_len, accumulate, rows)."""
    items = []
    for members, K, N, acc, rows in units:
        sh = t.plan_linear(K, N, 1, t.COLUMN, 64)[0]
        for r in range(members):
            a = A + 3 * len(items) * STEP
            items.append(dict(shard=sh, packed=a, packed_bytes=STEP, X=a + STEP, ldx=K,
                              Y=a + 2 * STEP, ldy=N, ydtype=t.F32, accumulate=acc,
                              sum_next=int(r + 1 < members), rows=rows))
    return items


# an accumulating product is not split along k; the planner may then split
# another of the call further than it would without
CALLS = [("q4", 2807, [(1, 2880, 1113, 1, 0), (1, 256, 61, 0, 0), (1, 2240, 162, 0, 654),
                       (1, 6720, 166, 0, 1311)]),
         ("bf16", 64, [(1, 2432, 394, 0, 0), (4, 192, 274, 0, 14), (4, 1728, 3932, 0, 30),
                       (1, 1536, 3724, 1, 0)]),
         ("q4", 73, [(2, 7040, 111, 0, 23), (2, 4992, 223, 0, 0), (1, 1472, 4854, 1, 0)]),
         ("bf16", 3313, [(4, 1024, 319, 0, 0), (1, 2112, 38, 1, 70), (1, 2112, 133, 1, 0),
                         (1, 1664, 30, 0, 0)]),
         ("q4", 1331, [(1, 3136, 65, 0, 0), (1, 1408, 272, 1, 0), (4, 704, 2757, 0, 0),
                       (4, 5760, 257, 0, 590)])]


@pytest.mark.parametrize("kind,M,units", CALLS)
@pytest.mark.parametrize("accumulating", [True, False])
def test_calls_fit_their_query(tsl_lib, kind, M, units, accumulating):
    t = tsl_lib
    wdtype = {"q4": t.Q4G64, "bf16": t.BF16}[kind]
    items = items_of(t, [(m, K, N, acc if accumulating else 0, rows) for m, K, N, acc, rows in units])
    n = t.shard_linear_group_workspace_size(items, wdtype, M)
    assert n > 0
    with pytest.raises(t.TslError) as e:
        t.shard_linear_group(items, wdtype, t.BF16, M, A - 1, n, stream=0)
    assert e.value.status == t.ERR_MISALIGNED
    # and the same items storing their products
    plain = [dict(it, accumulate=0) for it in items]
    with pytest.raises(t.TslError) as e:
        t.shard_linear_group(plain, wdtype, t.BF16, M, A - 1, n, stream=0)
    assert e.value.status == t.ERR_MISALIGNED
    none = [None] * len(items)
    n = t.shard_linear_group_epilogue_workspace_size(items, none, wdtype, M)
    assert n > 0
    for its in (items, plain):
        with pytest.raises(t.TslError) as e:
            t.shard_linear_group_epilogue(its, none, wdtype, t.BF16, M, A - 1, n, stream=0)
        assert e.value.status == t.ERR_MISALIGNED
