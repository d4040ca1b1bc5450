"""kv_append() with q_out=q: the queries are turned in place, in every pairing."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
from test_paged_abi import append, rows
from test_paged_gpu import BF16, F16, Pool


def test_queries_over_other_rows_are_refused():
    """(no GPU needed) An output at an input's address is that input's rows."""
    fa.build()
    bad = fa.FA_ERR_INVALID_ARG
    assert append(q=rows(), qo=rows(stride_b=8 * 64)) == bad
    assert append(q=rows(stride_h=128), qo=rows(), T=2) == bad
    p = rows().ptr
    assert append(k=rows(ptr=p + 32), q=rows(ptr=p + 64), qo=rows(ptr=p + 32)) == bad     # over K
    assert append(k=rows(ptr=p + 32), q=rows(ptr=p + 64), qo=rows()) == bad               # over V


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 64, True), (40, 40, False), (96, 18, False),
                                               (80, 72, False), (256, 40, False), (8, 6, False), (128, 120, False),
                                               (64, 0, False), (256, 250, False)])
@pytest.mark.parametrize("slices", [False, True])
def test_in_place_equals_out_of_place(D, rot, interleaved, dtype, slices):
    fa.build()
    B, Hq, Hkv, T = 3, 21, 2, 5
    pool = Pool([300, 4, 0], Hkv, D, 16, dtype, seed=D + rot)
    freq = (1000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float().cuda() if rot else None
    qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=pool.g).to(dtype).cuda()
    q, k, v = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], dim=2))
    if not slices:
        q = q.contiguous()
    one, two = pool.gpu(), pool.gpu()
    want = fa.kv_append(one, k, v, q=q, inv_freq=freq, interleaved=interleaved, position_offset=77)
    kept = k.clone(), v.clone()
    for _ in range(20):
        x = qkv.clone() if slices else None
        y = x[:, :, :Hq].transpose(1, 2) if slices else q.clone()
        got = fa.kv_append(two, k, v, q=y, inv_freq=freq, interleaved=interleaved, position_offset=77, q_out=y)
        assert got is y and torch.equal(got, want)
        if slices:
            assert torch.equal(x[:, :, Hq:], qkv[:, :, Hq:])
    assert torch.equal(k, kept[0]) and torch.equal(v, kept[1])
    for a, b in ((one.k_cache, two.k_cache), (one.v_cache, two.v_cache)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
