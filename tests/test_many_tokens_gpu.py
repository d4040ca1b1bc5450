"""rotary() and kv_append() where tokens are many and have little (a warp each): the same
results as for few tokens (a CTA each), which other tests hold against 64 bits."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
from test_rotary_gpu import check, turned

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
SHAPES = [  # Hq, Hkv, D, rot, interleaved; the three ways that pairs lie
    (1, 1, 8, 8, True), (3, 1, 64, 64, False), (2, 2, 80, 40, False), (5, 1, 128, 22, True), (1, 2, 256, 256, False),
    (2, 1, 72, 72, False), (1, 1, 256, 70, False)]


def tokens(D):
    """Of each of three sequences: enough for a warp each; the last CTA has one or three."""
    return 1667 if D < 100 else 3333


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


@pytest.mark.parametrize("Hq,Hkv,D,rot,interleaved", SHAPES)
def test_rotary(Hq, Hkv, D, rot, interleaved):
    g = torch.Generator().manual_seed(D)
    B, T, dtype = 3, tokens(D), BF16 if D % 16 else F16
    q, k = (torch.randn((B, T, H, D), generator=g).to(dtype).cuda().transpose(1, 2).requires_grad_() for H in (Hq, Hkv))
    freq = 10000.0 ** (-torch.arange(rot // 2) / (rot / 2))
    pos = torch.randint(-1000, 1 << 20, (3, B, T), generator=g, dtype=torch.int32)
    axis = torch.randint(0, 3, (rot // 2,), generator=g, dtype=torch.int32)
    out = fa.rotary(q, freq.cuda(), pos.cuda(), k=k, pair_axis=axis.cuda(), interleaved=interleaved)
    upstream = [torch.randn(x.shape, generator=g).to(dtype).cuda() for x in out]
    grads = torch.autograd.grad(out, (q, k), upstream)
    for x, y, d, grad in zip((q, k), out, upstream, grads):
        check(y.detach(), *turned(x.detach(), pos, axis, freq, interleaved), dtype)
        check(grad, *turned(d, pos, axis, freq, interleaved, back=True), dtype)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("Hq,Hkv,D,rot,interleaved", SHAPES)
def test_append(Hq, Hkv, D, rot, interleaved, bits):
    """In place, with sequences shorter than the call, and pages and a table's end that
    are not there, against calls of one sequence's piece each."""
    g = torch.Generator().manual_seed(D + 1)
    B, T, page, dtype = 3, tokens(D), 16, F16 if D % 16 else BF16
    lens = [T, 900, 5000]
    pages, width = 700, 310                                                # 4960 places of the third
    table = torch.full((B, width), -1, dtype=torch.int32)
    order, at = torch.randperm(pages, generator=g).to(torch.int32), 0
    for b, n in enumerate(lens):
        need = min(-(-n // page), width)
        table[b, :need] = order[at:at + need]
        at += need
    table[2, 300:303] = torch.tensor([-1, pages, 1 << 30])
    table, n = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    q, k, v = (torch.randn((B, T, H, D), generator=g).to(dtype).cuda().transpose(1, 2) for H in (Hq, Hkv, Hkv))
    freq = (10000.0 ** (-torch.arange(rot // 2) / (rot / 2))).cuda()

    def cache_of(table, n, pools=None):
        if pools is None and bits == 16:
            pools = [torch.full((pages, Hkv, page, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        elif pools is None:
            P = 64 if D <= 64 else 128 if D <= 128 else 256
            pools = [torch.full((pages, Hkv, page, P // e), 7, dtype=torch.uint8, device="cuda") for e in (2, 2, 16, 16)]
        cache = fa.PagedKV(*pools, table, n) if bits == 16 else fa.PagedKV4(*pools, table, n, D=D, dtype=dtype)
        return cache, pools

    cache, pools = cache_of(table, n)
    mine = q.clone(memory_format=torch.preserve_format)
    out = fa.kv_append(cache, k, v, q=mine, q_out=mine, inv_freq=freq, interleaved=interleaved, position_offset=3)
    _, other = cache_of(table, n)
    want = torch.empty_like(q)
    for b in range(B):
        for first in range(0, T, 400):
            last = min(first + 400, T)
            part, _ = cache_of(table[b:b + 1], n[b:b + 1] - (T - last), other)
            fa.kv_append(part, k[b:b + 1, :, first:last], v[b:b + 1, :, first:last], q=q[b:b + 1, :, first:last],
                         q_out=want[b:b + 1, :, first:last], inv_freq=freq, interleaved=interleaved, position_offset=3)
    assert out.data_ptr() == mine.data_ptr() and torch.equal(out, want)
    assert not out[1, :, :T - 900].any() and out[1, :, T - 900:].any()
    for a, b in zip(pools, other):
        assert torch.equal(a, b)
    if bits == 16:                                                         # and a rotary() of the same places
        text = (n[:, None] - T + torch.arange(T, device="cuda")).to(torch.int32)
        a, _ = fa.rotary(q, freq, text, k=k, interleaved=interleaved, position_offset=3)
        assert torch.equal(a[0], out[0]) and torch.equal(a[2], out[2])
