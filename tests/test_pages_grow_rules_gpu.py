"""Which sequences of one call grow where the free pages do not suffice for all."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


@pytest.mark.parametrize("tokens,want", [
    # four free pages: a need that is refused stands in front of those behind it
    ([9, 1, 1], [-2, -2, -2]), ([1, 1, 9], [1, 1, -2]), ([1, 9, 0], [1, -2, 0]),
    # a row that is too short for its tokens asks for no pages
    ([11, 2, 2], [-2, 2, 2]), ([4, 1, 0], [4, -2, 0])])
def test_needs_in_order(tokens, want):
    table, n, refs = (torch.full(s, v, dtype=torch.int32).cuda() for s, v in (((3, 10), -1), ((3,), 0), ((4,), 0)))
    pool = torch.zeros((4, 1, 1, 64), device="cuda").half()
    cache = fa.PagedKV(pool, pool.clone(), table, n)
    assert fa.kv_grow(cache, refs, torch.tensor(tokens, dtype=torch.int32).cuda()).tolist() == want
    assert n.tolist() == [t if w != -2 else 0 for t, w in zip(tokens, want)]
    assert int(refs.sum()) == sum(max(w, 0) for w in want)
