"""kv_fork() and kv_compact() of caches whose pages cannot be copied: refused as a whole,
with the table, the lengths, the counts and the other layers' pages as they were."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def caches(table, n):
    """A cache that can be copied, and ones that cannot: a head dimension that is no
    multiple of 8, a pool that is not on 16 bytes, and in 4 bits a head dimension of 60."""
    good, odd = (torch.randn((9, 2, 4, D), device="cuda").half() for D in (64, 20))
    off = torch.zeros(9 * 2 * 4 * 64 + 1, device="cuda").half()[1:].view(9, 2, 4, 64)
    four = [torch.zeros((9, 2, 4, w), dtype=torch.uint8, device="cuda") for w in (32, 32, 4, 4)]
    return (fa.PagedKV(good, good.clone(), table, n),
            (fa.PagedKV(odd, odd.clone(), table, n), fa.PagedKV(off, off.clone(), table, n), fa.PagedKV4(*four, table, n, D=60)))


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("alone", [False, True])
def test_nothing_changes(which, alone):
    table, n, refs = torch.full((3, 4), -1, dtype=torch.int32).cuda(), ints([0, 0, 0]), ints([0] * 9)
    good, bad = caches(table, n)
    layers = bad[which] if alone else [good, bad[which]]
    fa.kv_grow(good, refs, ints([6, 5, 0]))
    fa.kv_free(good, refs, ints([0]))               # pages 0 and 1 are holes
    held = [x.clone() for x in (table, n, refs, good.k_cache, good.v_cache)]
    for call in (lambda: fa.kv_fork(layers, refs, ints([1]), ints([2])), lambda: fa.kv_compact(layers, refs)):
        with pytest.raises(fa.FAError):
            call()
        for x, y in zip((table, n, refs, good.k_cache, good.v_cache), held):
            assert torch.equal(x, y)
    assert fa.kv_fork(good, refs, ints([1]), ints([2])).tolist() == [0]
    assert fa.kv_compact(good, refs).tolist()[:4] == [0, -1, 2, 1]
