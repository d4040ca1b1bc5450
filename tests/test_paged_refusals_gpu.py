"""Calls of the paged-cache operators that have to be refused, or answered with nothing."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
from test_paged_gpu import BF16, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()
    fa.load()


@pytest.mark.parametrize("T", [1, 40])
def test_a_prefix_without_its_pages_is_refused(T):
    pool = Pool([50, 3], 2, 64, 16, BF16, seed=1, prefix=40)
    cache, q = pool.gpu(), pool.queries(4, T).cuda()
    with pytest.raises(ValueError, match="prefix_len must lie"):
        fa.forward_shared_prefix(q, cache, None, 40)
    with pytest.raises(ValueError, match="prefix_len must lie"):
        fa.forward_shared_prefix(q, cache, pool.prefix_table[:0].cuda(), 1)
    # no prefix at all: forward_paged()
    want = fa.forward_paged(q, cache)
    for none in (None, pool.prefix_table[:0].cuda(), pool.prefix_table.cuda()):
        got = fa.forward_shared_prefix(q, cache, none, 0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_batch_of_no_sequences():
    pool = Pool([50, 3], 2, 64, 16, BF16, seed=2, prefix=40)
    full = pool.gpu()
    cache = fa.PagedKV(full.k_cache, full.v_cache, torch.empty((0, 7), dtype=torch.int32, device="cuda"),
                       torch.empty(0, dtype=torch.int32, device="cuda"))
    kept = full.k_cache.clone()
    q, kv = (torch.empty((0, h, 3, 64), dtype=BF16, device="cuda") for h in (4, 2))
    for o, lse in (fa.forward_paged(q, cache), fa.forward_shared_prefix(q, cache, pool.prefix_table.cuda(), 40)):
        assert o.shape == (0, 4, 3, 64) and lse.shape == (0, 4, 3)
    assert fa.kv_append(cache, kv, kv, q=q).shape == q.shape
    torch.cuda.synchronize()
    assert torch.equal(full.k_cache.view(torch.int16), kept.view(torch.int16))


@pytest.mark.parametrize("T", [1, 5])
def test_tokens_past_the_table_overwrite_nothing(T):
    """A table of 32 keys: what does not fit is dropped, and its query is turned by its position."""
    D, page, before = 64, 16, [30, 31, 32, 40]
    pool = Pool([32, 32, 32, 32], 2, D, page, BF16, seed=3)
    cache = pool.gpu()
    freq = (1000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    q, k, v = (torch.randn((4, h, T, D), generator=pool.g).to(BF16).cuda() for h in (4, 2, 2))
    cache.seq_len.copy_(torch.tensor(before, dtype=torch.int32) + T)
    old_k, old_v = cache.k_cache.clone(), cache.v_cache.clone()
    got = fa.kv_append(cache, k, v, q=q, inv_freq=freq)
    # the same tokens in a table that has room
    wide = Pool([64] * 4, 2, D, page, BF16, seed=4).gpu()
    wide.seq_len.copy_(cache.seq_len)
    assert torch.equal(got, fa.kv_append(wide, k, v, q=q, inv_freq=freq))
    for new, old, there in ((cache.k_cache, old_k, wide.k_cache), (cache.v_cache, old_v, wide.v_cache)):
        for b, n in enumerate(before):
            for i in range(32):
                page_at = int(cache.block_table[b, i // page]), slice(None), i % page
                want = there[int(wide.block_table[b, i // page]), :, i % page] if n <= i < n + T else old[page_at]
                assert torch.equal(new[page_at], want), (b, i)
