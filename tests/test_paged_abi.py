"""Argument checks of the paged-cache entry points, on the host: every call
returns before any CUDA call."""
import os
import shutil

import pytest

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="CUDA toolkit not present")

P = 0x10000       # a 16-byte-aligned stand-in address; never dereferenced
BIG = 1 << 40
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa.build()
    return fa.load()


def cache(**kw):
    a = dict(k=P, v=P, stride_page=2 * 16 * 64, stride_head=16 * 64, stride_slot=64, num_pages=10, page_size=16, Hkv=2,
             D=64, table=P, table_stride=4, table_width=4, seq_len=P)
    a.update(kw)
    return fa.fa_paged_kv(*(a[f] for f, _ in fa.fa_paged_kv._fields_))


def rows(**kw):
    a = dict(ptr=P, stride_b=4 * 64, stride_h=64, stride_n=64)
    a.update(kw)
    return fa.fa_rows(*(a[f] for f, _ in fa.fa_rows._fields_))


BAD_CACHES = [
    (dict(k=None), fa.FA_ERR_INVALID_ARG), (dict(v=P + 8), fa.FA_ERR_INVALID_ARG),
    (dict(stride_page=2 * 16 * 64 + 4), fa.FA_ERR_INVALID_ARG), (dict(stride_head=-64), fa.FA_ERR_INVALID_ARG),
    (dict(stride_slot=32), fa.FA_ERR_INVALID_ARG), (dict(num_pages=-1), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=0), fa.FA_ERR_INVALID_ARG), (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(D=0), fa.FA_ERR_INVALID_ARG),
    (dict(D=60), fa.FA_ERR_UNSUPPORTED), (dict(D=136, stride_slot=136), fa.FA_ERR_UNSUPPORTED),
    (dict(table=None), fa.FA_ERR_INVALID_ARG), (dict(table=P + 2), fa.FA_ERR_INVALID_ARG),
    (dict(seq_len=None), fa.FA_ERR_INVALID_ARG), (dict(seq_len=P + 1), fa.FA_ERR_INVALID_ARG),
    (dict(table_width=-1), fa.FA_ERR_INVALID_ARG), (dict(table_stride=3), fa.FA_ERR_INVALID_ARG),
    (dict(table_width=1 << 30, table_stride=1 << 30), fa.FA_ERR_INVALID_ARG),
]


def fwd(c=None, q=None, o=None, B=2, Hq=4, T=1, prefix=0, table=P, ws=P, size=BIG):
    c, q, o = c or cache(), q or rows(), o or rows()
    if prefix is None:
        return fa.fa_fwd_paged(q, c, o, P, B, Hq, T, True, NAN, False, ws, size, None)
    return fa.fa_fwd_shared_prefix(q, c, table, prefix, o, P, B, Hq, T, True, NAN, False, ws, size, None)


def append(c=None, k=None, q=None, qo=None, B=2, Hq=4, T=1, freq=P, rot=64, offset=0):
    k = k or rows()
    return fa.fa_kv_append(c or cache(), k, rows(), q, qo, B, Hq, T, freq, rot, False, offset, False, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches(bad, status):
    c = cache(**bad)
    assert fwd(c, prefix=None) == status
    assert fwd(c, prefix=7) == status
    assert append(c) == status
    assert fa.fa_fwd_paged_workspace_bytes(c, 2, 4, 1) == 0
    assert fa.fa_fwd_shared_prefix_workspace_bytes(c, 7, 2, 4, 1) == 0


@pytest.mark.parametrize("prefix", [None, 7])
def test_forward_checks(prefix):
    bad = fa.FA_ERR_INVALID_ARG
    assert fwd(B=-1, prefix=prefix) == bad
    assert fwd(T=-1, prefix=prefix) == bad
    assert fwd(Hq=3, prefix=prefix) == bad                       # no multiple of Hkv
    assert fwd(q=rows(ptr=None), prefix=prefix) == bad
    assert fwd(q=rows(ptr=P + 8), prefix=prefix) == bad
    assert fwd(q=rows(stride_h=68), prefix=prefix) == bad
    assert fwd(o=rows(stride_n=-64), T=2, prefix=prefix) == bad
    assert fwd(o=rows(stride_b=0), prefix=prefix) == bad          # rows of the output on each other
    assert fwd(ws=None, prefix=prefix) == bad
    assert fwd(ws=P + 4, prefix=prefix) == bad
    need = fa.fa_fwd_shared_prefix_workspace_bytes(cache(), prefix or 0, 2, 4, 1)
    assert need > 0 and fwd(size=need - 1, prefix=prefix) == bad
    assert fwd(B=1 << 20, Hq=1 << 12, prefix=prefix) == bad       # more than 2^31 heads
    for empty in (dict(B=0), dict(T=0), dict(Hq=0)):
        assert fwd(q=rows(ptr=None), ws=None, size=0, prefix=prefix, **empty) == fa.FA_OK


def test_prefix_checks():
    bad = fa.FA_ERR_INVALID_ARG
    assert fwd(prefix=-1) == bad
    assert fwd(prefix=7, table=None) == bad
    assert fwd(prefix=7, table=P + 2) == bad
    assert fwd(prefix=(1 << 31) - 8) == bad                       # positions past 2^31
    assert fa.fa_fwd_shared_prefix_workspace_bytes(cache(), -1, 2, 4, 1) == 0
    assert fa.fa_fwd_shared_prefix_workspace_bytes(cache(), 0, 2, 4, 1) == fa.fa_fwd_paged_workspace_bytes(cache(), 2, 4, 1)


def test_append_checks():
    bad = fa.FA_ERR_INVALID_ARG
    assert append(B=-1) == bad
    assert append(T=-1) == bad
    assert append(rot=63) == bad
    assert append(rot=66) == bad
    assert append(rot=-2) == bad
    assert append(freq=None) == bad
    assert append(freq=P + 2) == bad
    assert append(offset=-1) == bad
    assert append(offset=(1 << 40) + 1) == bad
    assert append(B=1 << 16, T=1 << 16) == bad
    assert append(k=rows(ptr=None)) == bad
    assert append(k=rows(stride_b=4)) == bad
    assert append(q=rows(), qo=None) == bad
    assert append(q=rows(), qo=rows(stride_h=0)) == bad
    assert append(B=0, k=rows(ptr=None)) == fa.FA_OK
    assert append(T=0, k=rows(ptr=None)) == fa.FA_OK


def test_python_refusals():
    torch = pytest.importorskip("torch")
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    table, n = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.PagedKV(kc, kc.clone(), table, n)
    with pytest.raises(ValueError, match="dtype"):
        fa.PagedKV(kc.float(), kc.float(), table, n)
    with pytest.raises(ValueError, match="one shape"):
        fa.PagedKV(kc, kc[:3], table, n)
    with pytest.raises(ValueError, match="one set of strides"):
        fa.PagedKV(kc, kc.transpose(1, 2).contiguous().transpose(1, 2), table, n)
    with pytest.raises(ValueError, match="last dimension"):
        fa.PagedKV(kc.transpose(2, 3), kc.transpose(2, 3), table, n)
    with pytest.raises(ValueError, match="block_table"):
        fa.PagedKV(kc, kc.clone(), table.long(), n)
    with pytest.raises(ValueError, match="rows of block_table"):
        fa.PagedKV(kc, kc.clone(), table.t(), n)
    with pytest.raises(ValueError, match="seq_len"):
        fa.PagedKV(kc, kc.clone(), table, n[:1])
