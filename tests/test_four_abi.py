"""Argument checks of the 4-bit cache, rotary and page entry points, on the host: every
call returns before any CUDA call; and the reference implementations of the tests."""
import os
import random
import shutil

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import four_reference as ref

cuda_toolkit = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                  reason="CUDA toolkit not present")

P = 0x10000       # a 16-byte-aligned stand-in address; never dereferenced
BIG = 1 << 40
NAN = float("nan")
BAD, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


def cache4(**kw):
    a = dict(k=P, v=P, stride_page=2 * 16 * 32, stride_head=16 * 32, stride_slot=32, k_scales=P, v_scales=P,
             scale_stride_page=2 * 16 * 4, scale_stride_head=16 * 4, scale_stride_slot=4, num_pages=10, page_size=16,
             Hkv=2, D=64, table=P, table_stride=4, table_width=4, seq_len=P)
    a.update(kw)
    return fa.fa_paged_kv4(*(a[f] for f, _ in fa.fa_paged_kv4._fields_))


def rows(**kw):
    a = dict(ptr=P, stride_b=4 * 64, stride_h=64, stride_n=64)
    a.update(kw)
    return fa.fa_rows(*(a[f] for f, _ in fa.fa_rows._fields_))


def table(**kw):
    a = dict(table=P, table_stride=4, table_width=4, B=3, seq_len=P, refs=P, num_pages=10, page_size=16)
    a.update(kw)
    return fa.fa_page_table(*(a[f] for f, _ in fa.fa_page_table._fields_))


def positions(**kw):
    a = dict(n=P, stride_axis=100, stride_b=10, stride_t=1, axes=3, pair_axis=P)
    a.update(kw)
    return fa.fa_positions(*(a[f] for f, _ in fa.fa_positions._fields_))


BAD_CACHES = [
    (dict(k=None), BAD), (dict(v=P + 8), BAD), (dict(k_scales=None), BAD), (dict(v_scales=P + 4), BAD),
    (dict(stride_page=2 * 16 * 32 + 8), BAD), (dict(stride_head=-32), BAD), (dict(stride_slot=16), BAD),
    (dict(scale_stride_slot=6), BAD), (dict(scale_stride_page=-4), BAD), (dict(scale_stride_slot=0), BAD),
    (dict(D=128), BAD), (dict(num_pages=-1), BAD), (dict(page_size=0), BAD), (dict(Hkv=0), BAD), (dict(D=0), BAD),
    (dict(D=60), UNSUPPORTED), (dict(D=136), UNSUPPORTED), (dict(table=None), BAD), (dict(table=P + 2), BAD),
    (dict(seq_len=None), BAD), (dict(seq_len=P + 1), BAD), (dict(table_width=-1), BAD), (dict(table_stride=3), BAD),
    (dict(table_width=1 << 30, table_stride=1 << 30), BAD),
]


@cuda_toolkit
@pytest.mark.parametrize("bad, status", BAD_CACHES)
def test_bad_caches(lib, bad, status):
    c = cache4(**bad)
    assert fa.fa_fwd_paged_q4(rows(), c, rows(), P, 2, 4, 1, True, NAN, False, P, BIG, None) == status
    assert fa.fa_fwd_paged_q4_workspace_bytes(c, 2, 4, 1) == 0
    assert fa.fa_kv_append_q4(c, rows(), rows(), None, None, 2, 0, 1, P, 64, False, None, 0, False, None) == status
    assert fa.fa_kv_read_q4(c, rows(), rows(), 2, 1, False, None) == status
    if "table" not in str(bad) and "seq_len" not in bad:
        assert fa.fa_copy_pages_q4(c, P, P, None, 1, None) == status


@cuda_toolkit
def test_bad_forwards(lib):
    def fwd(c=None, q=None, o=None, B=2, Hq=4, T=1, ws=P, size=BIG):
        return fa.fa_fwd_paged_q4(q or rows(), c or cache4(), o or rows(), P, B, Hq, T, True, NAN, False, ws, size, None)
    assert fwd(B=-1) == BAD and fwd(Hq=-2) == BAD and fwd(T=-1) == BAD
    assert fwd(Hq=3) == BAD                                     # no multiple of the key heads
    assert fwd(q=rows(ptr=None)) == BAD and fwd(o=rows(stride_n=0), T=2) == BAD and fwd(q=rows(stride_h=12)) == BAD
    assert fwd(ws=None) == BAD and fwd(ws=P + 8) == BAD and fwd(size=16) == BAD
    assert fwd(B=0) == fa.FA_OK and fwd(T=0) == fa.FA_OK and fwd(Hq=0) == fa.FA_OK


@cuda_toolkit
def test_bad_turns(lib):
    def append(c=None, k=None, q=None, qo=None, Hq=4, T=1, freq=P, rot=64, pos=None, offset=0):
        return fa.fa_kv_append_q4(c or cache4(), k or rows(), rows(), q, qo, 2, Hq, T, freq, rot, False, pos, offset, False, None)

    def rotary(q=None, qo=None, k=None, ko=None, B=2, Hq=4, Hkv=2, T=1, D=64, freq=P, rot=64, pos=None, offset=0):
        return fa.fa_rotary(q or rows(), qo or rows(), k or rows(ptr=2 * P), ko or rows(ptr=2 * P), B, Hq, Hkv, T, D,
                            freq, rot, False, pos, offset, False, False, None)
    for call in (append, rotary):
        assert call(rot=66) == BAD and call(rot=-2) == BAD and call(rot=7) == BAD and call(freq=None) == BAD
        assert call(offset=-1) == BAD and call(offset=(1 << 40) + 1) == BAD
        for bad in (dict(n=None), dict(n=P + 2), dict(axes=0), dict(pair_axis=P + 1), dict(stride_b=-1)):
            assert call(pos=positions(**bad)) == BAD
        assert call(T=0) == fa.FA_OK
    assert append(k=rows(ptr=P + 8)) == BAD and append(q=rows(), qo=rows()) == BAD       # the queries over the keys
    assert append(q=rows(ptr=2 * P), qo=rows(ptr=2 * P, stride_h=128)) == BAD
    assert rotary(D=60) == UNSUPPORTED and rotary(D=264) == UNSUPPORTED and rotary(D=0) == BAD
    assert rotary(q=rows(stride_n=60)) == BAD and rotary(qo=rows(stride_h=0)) == BAD
    assert rotary(qo=rows(ptr=2 * P)) == BAD and rotary(ko=rows(ptr=P)) == BAD
    assert rotary(qo=rows(ptr=3 * P), ko=rows(ptr=3 * P)) == BAD
    assert rotary(Hq=0, Hkv=0) == fa.FA_OK


BAD_TABLES = [dict(B=-1), dict(table_width=-1), dict(num_pages=-1), dict(page_size=0), dict(table=None), dict(seq_len=None),
              dict(refs=None), dict(table=P + 1), dict(seq_len=P + 2), dict(refs=P + 3), dict(table_stride=3),
              dict(table_width=1 << 30, table_stride=1 << 30)]


@cuda_toolkit
@pytest.mark.parametrize("bad", BAD_TABLES)
def test_bad_tables(lib, bad):
    t = table(**bad)
    assert fa.fa_pages_workspace_bytes(t, 4) == 0
    assert fa.fa_kv_grow(t, P, P, P, BIG, None) == BAD
    assert fa.fa_kv_free(t, P, 1, None) == BAD
    assert fa.fa_kv_fork(t, P, P, 1, P, P, P, BIG, None) == BAD
    assert fa.fa_kv_compact(t, P, P, P, P, P, BIG, None) == BAD


@cuda_toolkit
def test_bad_page_calls(lib):
    t = table()
    need = fa.fa_pages_workspace_bytes(t, 4)
    assert need > 0
    for ws, size in ((None, BIG), (P + 8, BIG), (P, need - 1)):
        assert fa.fa_kv_grow(t, P, P, ws, fa.fa_pages_workspace_bytes(t, 0) - 1 if size < BIG else size, None) == BAD
        assert fa.fa_kv_fork(t, P, P, 4, P, P, ws, size, None) == BAD
        assert fa.fa_kv_compact(t, P, P, P, P, ws, fa.fa_pages_workspace_bytes(t, 0) - 1 if size < BIG else size, None) == BAD
    assert fa.fa_kv_grow(t, None, P, P, BIG, None) == BAD and fa.fa_kv_grow(t, P, P + 1, P, BIG, None) == BAD
    assert fa.fa_kv_free(t, None, 1, None) == BAD and fa.fa_kv_free(t, P, -1, None) == BAD
    assert fa.fa_kv_free(t, None, 0, None) == fa.FA_OK and fa.fa_kv_grow(table(B=0), None, None, None, 0, None) == fa.FA_OK
    assert fa.fa_kv_fork(t, P, None, 1, P, P, P, BIG, None) == BAD and fa.fa_kv_fork(t, P, P, -1, P, P, P, BIG, None) == BAD
    assert fa.fa_kv_fork(t, None, None, 0, None, None, None, 0, None) == fa.FA_OK
    assert fa.fa_kv_compact(t, P, P, P, None, P, BIG, None) == BAD
    assert fa.fa_copy_pages_q4(cache4(), None, P, None, 1, None) == BAD
    assert fa.fa_copy_pages_q4(cache4(), P, P, P + 2, 1, None) == BAD
    assert fa.fa_copy_pages_q4(cache4(), P, P, None, -1, None) == BAD
    assert fa.fa_copy_pages_q4(cache4(), None, None, None, 0, None) == fa.FA_OK


@cuda_toolkit
def test_counts_that_32_bits_do_not_hold_a_block_further(lib):
    most = 2 ** 31 - 1025
    assert fa.fa_pages_workspace_bytes(table(num_pages=most), most) > 0
    for pages in (most + 1, 2 ** 31 - 1):
        t = table(num_pages=pages)
        assert fa.fa_pages_workspace_bytes(t, 0) == 0 and fa.fa_kv_grow(t, P, P, P, 2 ** 40, None) == BAD
        assert fa.fa_kv_compact(t, P, P, P, P, P, 2 ** 40, None) == BAD
    for n in (most + 1, 2 ** 31 - 1):
        assert fa.fa_pages_workspace_bytes(table(), n) == 0 and fa.fa_kv_free(table(), P, n, None) == BAD
        assert fa.fa_kv_fork(table(), P, P, n, P, P, P, 2 ** 40, None) == BAD
        assert fa.fa_copy_pages_q4(cache4(), P, P, None, n, None) == BAD


def test_the_references_format():
    """Every number of the format is itself, and halfway goes to the even one."""
    s = ref.scales()
    assert float(s[-1]) == 10240 and float(s[1]) == 2.0 ** -17 and bool((s[1:] > s[:-1]).all())
    for b in (1, 7, 8, 100, 226):
        row = torch.tensor(ref.U + [-x for x in ref.U], dtype=torch.float64) * s[b]
        data, code = ref.pack(row)
        assert int(code[0]) == b and torch.equal(ref.unpack(data, code), row)
    halfway = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 6] + [0] * 7, dtype=torch.float64)
    assert ref.values(halfway).tolist()[:9] == [0, 1, 1, 2, 2, 4, 4, -4, 6]
    assert ref.values(torch.full((16,), 70000.0, dtype=torch.float64))[0] == 61440


def test_the_references_pages():
    """Counts are what the tables say after any calls, and no page is used by two that
    write to it."""
    rng = random.Random(3)
    for _ in range(50):
        page, B, width, N = rng.choice([1, 3, 16]), rng.randint(1, 6), rng.randint(1, 5), rng.randint(1, 25)
        x = ref.Pages(torch.full((B, width), -1), torch.zeros(B, dtype=torch.int32), torch.zeros(N, dtype=torch.int32), page)
        for _ in range(20):
            how = rng.choice(["grow", "grow", "free", "fork", "compact"])
            if how == "grow":
                x.grow([rng.choice([0, 1, page, -2, 2 * page + 1]) for _ in range(B)])
            elif how == "free":
                x.free([rng.randint(-1, B) for _ in range(rng.randint(0, 3))])
            elif how == "fork":
                n = rng.randint(0, 3)
                x.fork([rng.randint(-1, B) for _ in range(n)], [rng.randint(-1, B) for _ in range(n)])
            else:
                x.compact()
                assert all((n > 0) == (p < sum(m > 0 for m in x.refs)) for p, n in enumerate(x.refs))
            uses, tails = [0] * N, []
            for b in range(B):
                n = x.length(b)
                for e in range(x.have(n)):
                    uses[x.table[b][e]] += 1
                if n % page:
                    tails.append(x.table[b][n // page])
            assert uses == x.refs
            assert all(uses[p] == 1 for p in tails)
