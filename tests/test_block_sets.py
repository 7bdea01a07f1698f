"""Which calls of many sum sets the few-rows form takes, on the host alone: it
needs no workspace, the streaming form the partials of the sets' members."""
import pytest

A = 1 << 40  # addresses far apart; never read
STEP = 1 << 24


def size(t, sets, members, K, N, M):
    sh = t.plan_linear(K, N, 1, t.COLUMN, 64)[0]
    items, eps = [], []
    for i in range(sets * members):
        a = A + 3 * i * STEP
        items.append(dict(shard=sh, packed=a, packed_bytes=STEP, X=a + STEP, ldx=K, Y=a + 2 * STEP,
                          ldy=N, sum_next=int(i % members + 1 < members)))
        eps.append(dict(act=t.ACT_RELU) if i % members == 0 else None)
    return t.shard_linear_group_epilogue_workspace_size(items, eps, t.Q4G64, M)


@pytest.mark.parametrize("sets,members,N,M,one", [
    # up to 64 sets, whatever their members: several launches of 128 members
    (40, 4, 512, 1, True), (48, 4, 2048, 3, True), (64, 8, 256, 4, True),
    # sets of more than 8 members, wide calls of one or two rows, and of more sets
    (64, 16, 16, 2, False),
    (48, 4, 2048, 1, False), (65, 2, 2048, 4, False), (64, 2, 2048, 2, False)])
def test_sets_of_the_few_rows_form(tsl_lib, sets, members, N, M, one):
    assert (size(tsl_lib, sets, members, 192, N, M) == 0) == one
