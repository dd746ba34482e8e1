"""Pages that a release takes from the table though the pool has no such page: recorded, on the stack as they are, and no
place for anybody afterwards.  Against the plain lists of tests/feed_oracle.py."""
import pytest
import torch

from tests import feed_oracle as fo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


def ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


@pytest.mark.parametrize("entry", [-1, 6, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("width", [5, 5000])  # one launch and two (and room for the 80 tokens below: 5 pages)
def test_an_entry_outside_the_pool_is_recorded(moe, entry, width):
    lens, ended, table = [20, 40, 0], [True, True, False], [[2, entry], [0, 1, 4], []]
    table = [row + [0] * (width - len(row)) for row in table]
    free, n_free = [5, 0, 0, 0, 0, 0], 1
    ln, t, f, nf, ws = ints(lens), ints(table), ints(free), ints([n_free]), moe.pages_workspace(3)
    moe.page_release(ln, torch.tensor(ended).cuda(), t, f, nf, 16, ws)
    assert moe.get_status(ws) == -8
    after, left, stack = fo.release(lens, ended, table, free, n_free, 16)
    assert ln.tolist() == after and nf.tolist() == [left] and f.tolist() == stack
    # five pages given out again: the one that is none has no place, the others have theirs
    plan = moe.page_plan(ln, ints([0, 0, 80]), t, f, nf, 16, 6, 80, ws)
    assert moe.get_status(ws) == -8 and plan.n_free.tolist() == [1]
    want = fo.plan(after, [0, 0, 80], table, stack, left, 16, 80)[2]
    none = [p for p in range(80) if stack[5 - p // 16] == entry]
    assert len(none) == 16
    assert plan.slot.tolist() == [-1 if i in none else p for i, p in enumerate(want)]


def test_entries_that_nobody_holds_are_not_looked_at(moe):
    ws = moe.pages_workspace(2)
    f, ln = ints([0, 0, 0, 0]), ints([16, 5])
    moe.page_release(ln, torch.tensor([True, False]).cuda(), ints([[3, -1], [-9, -1]]), f, ints([0]), 16, ws)
    assert moe.get_status(ws) == 0 and f.tolist() == [3, 0, 0, 0] and ln.tolist() == [0, 5]
