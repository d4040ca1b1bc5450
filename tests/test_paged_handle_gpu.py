"""A PagedKV holds the memory that its calls use: its tensors can be updated in
place, and nothing else can take their place unnoticed."""
import gc

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
from test_paged_gpu import BF16, Pool, run_paged


def test_attributes_are_properties():
    """(no GPU needed)"""
    for name in ("k_cache", "v_cache", "block_table", "seq_len", "batch", "Hkv", "D", "dtype", "device", "c"):
        assert isinstance(fa.PagedKV.__dict__[name], property), name


@pytest.mark.gpu
def test_tensors_cannot_be_replaced():
    fa.build()
    pool = Pool([200, 45], 2, 64, 16, BF16, seed=3)
    q, cache, o, lse = run_paged(pool, 8, 1)
    for name in ("k_cache", "v_cache", "block_table", "seq_len"):
        was = getattr(cache, name)
        with pytest.raises(AttributeError, match="cannot be replaced"):
            setattr(cache, name, was.clone())
        with pytest.raises(AttributeError, match="cannot be replaced"):
            setattr(cache, name, None)
        assert getattr(cache, name) is was
    for name, value in (("batch", 1), ("Hkv", 4), ("D", 128), ("dtype", torch.float16)):
        with pytest.raises(AttributeError, match="cannot be replaced"):
            setattr(cache, name, value)
    with pytest.raises(AttributeError):
        cache.c = cache.c
    # a copy: edits of it change nothing
    cache.c.seq_len = 0
    need = cache.workspace_bytes(8, 1)
    cache.c.table_width = 0
    assert cache.workspace_bytes(8, 1) == need
    again = fa.forward_paged(q.cuda(), cache)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.gpu
def test_tensors_are_updated_in_place():
    fa.build()
    pool = Pool([200, 45], 2, 64, 16, BF16, seed=4)
    q, cache, o, lse = run_paged(pool, 8, 1)
    cache.seq_len -= 7
    pool.lens -= 7
    run_paged(pool, 8, 1, q=q)
    got = fa.forward_paged(q.cuda(), cache)
    want = fa.forward_paged(q.cuda(), pool.gpu())
    assert torch.equal(got[0], want[0]) and not torch.equal(got[0], o)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["k_cache", "v_cache", "block_table", "seq_len"])
def test_a_tensor_with_other_memory_is_refused(name):
    fa.build()
    pool = Pool([200, 45], 2, 64, 16, BF16, seed=5)
    cache, q = pool.gpu(), pool.queries(8, 1).cuda()
    x = torch.randn((2, 2, 1, 64), device="cuda").to(BF16)
    tensor = getattr(cache, name)
    was = tensor.data
    tensor.data = was.clone()
    for call in (lambda: fa.forward_paged(q, cache), lambda: fa.kv_append(cache, x, x),
                 lambda: fa.forward_shared_prefix(q, cache, pool.prefix_table.cuda(), 0)):
        with pytest.raises(ValueError, match="other memory"):
            call()
    tensor.data = was
    assert torch.equal(fa.forward_paged(q, cache)[0], fa.forward_paged(q, pool.gpu())[0])


@pytest.mark.gpu
def test_the_handle_keeps_its_tensors():
    """The memory of tensors that only the handle still holds is not given to others."""
    fa.build()
    pool = Pool([200, 45], 2, 64, 16, BF16, seed=6)
    q = pool.queries(8, 1).cuda()
    want = fa.forward_paged(q, pool.gpu())
    cache = pool.gpu()
    native, sizes = cache._native, [t.numel() * t.element_size() for t in (cache.k_cache, cache.block_table, cache.seq_len)]
    del cache
    gc.collect()
    torch.cuda.synchronize()
    others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    got = fa._BINDING.forward(native, q, None, 0, True, None, None, None, True, None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del others
