"""Calls of no tokens whose positions have no memory, as torch's empty tensors have none."""
import os
import shutil

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

P = 0x10000       # a 16-byte-aligned stand-in address; never dereferenced
cuda_toolkit = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                  reason="CUDA toolkit not present")


@cuda_toolkit
@pytest.mark.parametrize("B,T", [(2, 0), (0, 3), (0, 0)])
def test_no_tokens(B, T):
    fa.build()
    rows = fa.fa_rows(P, 4 * 64, 64, 64)
    none, bad = fa.fa_positions(None, 0, 0, 1, 3, P), fa.fa_positions(None, 0, 0, 1, 0, P)
    c = fa.fa_paged_kv(P, P, 2 * 16 * 64, 16 * 64, 64, 10, 16, 2, 64, P, 4, 4, P)
    c4 = fa.fa_paged_kv4(P, P, 2 * 16 * 32, 16 * 32, 32, P, P, 2 * 16 * 4, 16 * 4, 4, 10, 16, 2, 64, P, 4, 4, P)

    def calls(pos, B, T):
        yield fa.fa_rotary(rows, rows, rows, rows, B, 4, 2, T, 64, P, 64, False, pos, 0, False, False, None)
        yield fa.fa_kv_append_at(c, rows, rows, None, None, B, 0, T, P, 64, False, pos, 0, False, None)
        yield fa.fa_kv_append_q4(c4, rows, rows, None, None, B, 0, T, P, 64, False, pos, 0, False, None)
    assert list(calls(none, B, T)) == [fa.FA_OK] * 3
    assert list(calls(bad, B, T)) == [fa.FA_ERR_INVALID_ARG] * 3       # (axes are checked as ever)
    assert list(calls(none, 2, 1)) == [fa.FA_ERR_INVALID_ARG] * 3


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(2, 0), (0, 3), (0, 0)])
def test_no_tokens_in_torch(B, T):
    fa.build()
    dtype = torch.bfloat16
    x = torch.zeros((B, 2, T, 64), dtype=dtype, device="cuda")
    freq, pair = torch.ones(32, device="cuda"), torch.zeros(32, dtype=torch.int32, device="cuda")
    table, n = torch.zeros((B, 2), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    pool = torch.zeros((3, 2, 16, 64), dtype=dtype, device="cuda")
    four = [torch.zeros((3, 2, 16, w), dtype=torch.uint8, device="cuda") for w in (32, 32, 4, 4)]
    for positions, axis in ((torch.zeros((B, T), dtype=torch.int32, device="cuda"), None),
                            (torch.zeros((3, B, T), dtype=torch.int32, device="cuda"), pair)):
        a, b = fa.rotary(x, freq, positions, k=x, pair_axis=axis)
        assert a.shape == x.shape and b.shape == x.shape
        y = x.clone().requires_grad_()
        (grad,) = torch.autograd.grad(fa.rotary(y, freq, positions, pair_axis=axis), y, x)
        assert grad.shape == x.shape
        for cache in (fa.PagedKV(pool, pool.clone(), table, n), fa.PagedKV4(*four, table, n)):
            q = fa.kv_append(cache, x, x, q=x, inv_freq=freq, positions=positions, pair_axis=axis)
            assert q.shape == x.shape
