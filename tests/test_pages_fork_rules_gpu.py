"""Which of the forks of one call are refused."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("lens,parent,child,want,after", [
    # a fork whose parent is another fork's child is refused, and that other one done
    ([5, 0, 0], [0, 1], [1, 2], [2, -2], [5, 5, 0]), ([5, 0, 0], [1, 0], [2, 1], [-2, 2], [5, 5, 0]),
    # also where that other one is refused, its child not being empty
    ([5, 3, 0], [0, 1], [1, 2], [-2, -2], [5, 3, 0]),
    # of two forks with one child the first is done; a row is not its own child
    ([5, 3, 0], [1, 0], [2, 2], [3, -2], [5, 3, 3]), ([5, 0, 0], [2, 0], [2, 1], [-2, 2], [5, 5, 0]),
    # one parent of two children
    ([5, 0, 0], [0, 0], [1, 2], [2, 3], [5, 5, 5])])
def test_children_and_parents(lens, parent, child, want, after):
    table, n, refs = torch.full((3, 4), -1, dtype=torch.int32).cuda(), ints([0] * 3), ints([0] * 9)
    pool = torch.zeros((9, 1, 4, 64), device="cuda").half()
    cache = fa.PagedKV(pool, pool.clone(), table, n)
    fa.kv_grow(cache, refs, ints(lens))
    assert fa.kv_fork(cache, refs, ints(parent), ints(child)).tolist() == want
    assert n.tolist() == after
