"""rotary() and kv_append()'s positions on the GPU against 64 bits, and its gradients."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import paged_reference

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def turned(x, pos, axis, freq, interleaved, offset=0, back=False):
    """x [B, H, T, D] by pos [axes, B, T] in 64 bits, and sum |x| of each pair; pairs of no
    axis do not turn."""
    x = x.double().cpu().clone()
    half = freq.numel()
    i = torch.arange(half)
    on = (axis >= 0) & (axis < pos.shape[0])
    n = pos.double()[axis.clamp(0, pos.shape[0] - 1).long()].permute(1, 2, 0) + offset
    angle = torch.where(on, n * freq.double(), 0)[:, None] * (-1 if back else 1)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., first].clone(), x[..., second].clone()
    size = torch.zeros_like(x)
    size[..., first] = size[..., second] = a.abs() + b.abs()
    x[..., first], x[..., second] = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
    return x, size


def check(got, want, size, dtype):
    """The angle's fp32 form, its sine and cosine and the products are off by 2^-20 of
    |x| + |y| (2^-22.3 + 2^-22 + 3 2^-24), and the result is rounded once."""
    u, off = paged_reference.HALF_STEP[dtype], 2.0 ** -20 * size
    assert bool(((got.double().cpu() - want).abs() <= off + u * (want.abs() + off) + 2.0 ** -25).all())


CASES = [  # B, T, Hq, Hkv, D, rot, axes, interleaved
    (1, 1, 1, 1, 8, 8, 1, False), (2, 37, 4, 2, 128, 128, 3, False), (3, 5, 2, 0, 64, 40, 2, True),
    (1, 130, 3, 3, 80, 22, 4, False), (2, 9, 1, 5, 256, 256, 3, True), (1, 3, 7, 2, 96, 96, 2, False), (1, 2, 1, 1, 248, 6, 1, True)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,axes,interleaved", CASES)
def test_forward_and_gradient(B, T, Hq, Hkv, D, rot, axes, interleaved, dtype):
    g = torch.Generator().manual_seed(D + T)
    qkv = torch.randn((B, T, Hq + Hkv, D), generator=g).to(dtype).cuda().requires_grad_()
    q, k = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv], dim=2))
    freq = (10000.0 ** (-torch.arange(rot // 2) / (rot / 2))) * torch.where(torch.arange(rot // 2) % 3 == 1, -1, 1)
    pos = torch.randint(-1000, 1 << 20, (axes, B, T), generator=g, dtype=torch.int32)
    axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    axis[-1:] = axes if rot > 2 and axes > 1 else 0                   # no axis: does not turn
    args = dict(pair_axis=axis.cuda() if axes > 1 else None, interleaved=interleaved)
    axis = axis if axes > 1 else torch.zeros_like(axis)
    p = pos.cuda() if axes > 1 else pos[0].cuda()
    r = fa.rotary(q, freq.cuda(), p, k=k if Hkv else None, **args)
    got = r if Hkv else (r,)
    upstream = [torch.randn(x.shape, generator=g).to(dtype).cuda() for x in got]
    (grad,) = torch.autograd.grad(got, qkv, [x.transpose(2, 3).contiguous().transpose(2, 3) for x in upstream])
    for x, y, d, i in zip((q, k), got, upstream, (0, Hq)):
        check(y, *turned(x.detach(), pos, axis, freq, interleaved), dtype)
        want, size = turned(d, pos, axis, freq, interleaved, back=True)
        check(grad[:, :, i:i + x.shape[1]].transpose(1, 2), want, size, dtype)


def test_gradient_against_differences():
    """The operation is linear: a difference quotient over any step is exact but for the
    roundings of the two outputs, half a step of each."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn((1, 2, 3, 16), generator=g).to(F16).cuda().requires_grad_()
    freq, pos = torch.rand(8, generator=g).cuda(), torch.randint(0, 50, (1, 3), generator=g, dtype=torch.int32).cuda()
    w = torch.randn(x.shape, generator=g).to(F16).cuda()
    (grad,) = torch.autograd.grad(fa.rotary(x, freq, pos), x, w)
    base = fa.rotary(x.detach(), freq, pos).double()
    for at in range(0, x.numel(), 5):
        y = x.detach().clone()
        step = 4.0
        y.view(-1)[at] += step
        moved = float(y.view(-1)[at].double() - x.detach().view(-1)[at].double())
        out = fa.rotary(y, freq, pos).double()
        quotient = float((w.double() * (out - base)).sum()) / moved
        change = out != base
        slack = float((w.double().abs() * (out.abs() + base.abs()) * change).sum()) * 2.0 ** -11 * 1.01 / moved + 2.0 ** -10
        got = float(grad.view(-1)[at])
        assert abs(quotient - got) <= slack + 2.0 ** -11 * abs(got)


def test_text_positions_one_of_two_gradients_and_twice():
    g = torch.Generator().manual_seed(4)
    q = torch.randn((2, 3, 6, 32), generator=g).to(BF16).cuda().requires_grad_()
    k = torch.randn((2, 1, 6, 32), generator=g).to(BF16).cuda().requires_grad_()
    freq = torch.rand(16, generator=g)
    a, b = fa.rotary(q, freq.cuda(), k=k, position_offset=5)
    where, axis = torch.arange(6).expand(1, 2, 6), torch.zeros(16, dtype=torch.long)
    check(a.detach(), *turned(q.detach(), where, axis, freq, False, 5), BF16)
    grad_q, grad_k = torch.autograd.grad(b.sum(), (q, k), allow_unused=True, retain_graph=True)
    assert grad_q is None
    check(grad_k, *turned(torch.ones(k.shape), where, axis, freq, False, 5, True), BF16)
    # the gradient is linear in the upstream gradient: its own gradient turns forward
    up = torch.ones_like(a).requires_grad_()
    (grad,) = torch.autograd.grad(a, q, up, create_graph=True)
    (twice,) = torch.autograd.grad(grad, up, torch.ones_like(grad))
    check(twice, *turned(torch.ones(q.shape), where, axis, freq, False, 5), BF16)


def test_broadcast_inputs_and_positions():
    """A head that is expanded gets the sum of its copies' gradients."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn((1, 1, 4, 64), generator=g).to(F16).cuda().requires_grad_()
    freq = torch.rand(32, generator=g)
    pos = torch.randint(0, 99, (2, 1, 4), generator=g, dtype=torch.int32)
    axis = torch.randint(0, 2, (32,), generator=g, dtype=torch.int32)
    out = fa.rotary(x.expand(3, 5, 4, 64), freq.cuda(), pos.cuda().expand(2, 3, 4), pair_axis=axis.cuda())
    want, size = turned(x.detach(), pos, axis, freq, False)
    check(out.detach(), want.expand(3, 5, 4, 64), size.expand(3, 5, 4, 64), F16)
    (grad,) = torch.autograd.grad(out, x, torch.ones_like(out))
    one, size = turned(torch.ones(x.shape), pos, axis, freq, False, back=True)
    # 15 equal numbers, each rounded once, added with at most 15 roundings of their sum
    assert bool(((grad.double().cpu() - 15 * one).abs() <= 15 * 16 * 2.0 ** -11 * (one.abs() + 2.0 ** -20 * size) + 15 * 2.0 ** -20 * size).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_and_rotary_agree(interleaved):
    """kv_append() with positions turns queries and keys to the bit as rotary() does, and
    without them as before."""
    g = torch.Generator().manual_seed(8)
    B, T, D, page, lens = 2, 5, 72, 8, [9, 5]
    q, k = torch.randn((B, 4, T, D), generator=g).to(BF16).cuda(), torch.randn((B, 2, T, D), generator=g).to(BF16).cuda()
    freq = torch.rand(36, generator=g).cuda()
    pool = torch.zeros((8, 2, page, D), dtype=BF16, device="cuda")
    table = torch.arange(8, dtype=torch.int32).view(2, 4).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    cache = fa.PagedKV(pool, pool.clone(), table, n)
    pos = torch.randint(0, 1 << 30, (3, B, T), generator=g, dtype=torch.int32).cuda()
    axis = torch.randint(0, 3, (36,), generator=g, dtype=torch.int32).cuda()
    out = fa.kv_append(cache, k, k, q=q, inv_freq=freq, interleaved=interleaved, position_offset=3, positions=pos, pair_axis=axis)
    a, b = fa.rotary(q, freq, pos, k=k, pair_axis=axis, interleaved=interleaved, position_offset=3)
    assert torch.equal(out, a) and torch.equal(fa.kv_read(cache, T)[0], b) and torch.equal(fa.kv_read(cache, T)[1], k)
    text = (n[:, None] - T + torch.arange(T, device="cuda")).to(torch.int32)
    plain = fa.kv_append(cache, k, k, q=q, inv_freq=freq, interleaved=interleaved)
    given = fa.kv_append(cache, k, k, q=q, inv_freq=freq, interleaved=interleaved, positions=text)
    assert torch.equal(plain, given)


def test_training_step_and_graph():
    """attention() over rotated queries and keys: gradients against 64-bit autograd, and
    forward and backward captured into a graph."""
    g = torch.Generator().manual_seed(9)
    B, H, N, D = 1, 2, 96, 64
    x = [torch.randn((B, H, N, D), generator=g).to(BF16).cuda() for _ in range(4)]
    freq, axis = torch.rand(32, generator=g), torch.arange(32, dtype=torch.int32) % 3
    pos = torch.randint(0, 40, (3, B, N), generator=g, dtype=torch.int32)
    f, p, a = freq.cuda(), pos.cuda(), axis.cuda()
    leaves = [y.clone().requires_grad_() for y in x[:3]]

    def step():
        q, k = fa.rotary(leaves[0], f, p, k=leaves[1], pair_axis=a)
        return torch.autograd.grad(fa.attention(q, k, leaves[2]), leaves, x[3])

    first = [y.clone() for y in step()]
    torch.cuda.synchronize()
    wide = [y.double().cpu().requires_grad_() for y in x[:3]]
    angle = (pos.double()[axis.long()].permute(1, 2, 0) * freq.double())[:, None]

    def turn(y):
        u, w = y[..., :32], y[..., 32:]
        return torch.cat([u * angle.cos() - w * angle.sin(), w * angle.cos() + u * angle.sin()], -1)

    s = turn(wide[0]) @ turn(wide[1]).transpose(2, 3) / 8
    s = s.masked_fill(~torch.ones(N, N, dtype=torch.bool).tril(), -torch.inf)
    want = torch.autograd.grad(s.softmax(-1) @ wide[2], wide, x[3].double().cpu())
    for got, w in zip(first, want):
        # bf16 q, k, P and dS: a few half steps of the largest, as the backward's own tests allow
        assert float((got.double().cpu() - w).abs().max()) <= 2e-2 * float(w.abs().max())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    # (dQ is summed in an order that may differ)
    assert torch.equal(got[2], first[2]) and float((got[0] - first[0]).abs().max()) <= 2e-2 * float(first[0].abs().max())


def test_refusals():
    q, f = torch.zeros((1, 2, 3, 64), dtype=BF16, device="cuda"), torch.ones(32, device="cuda")
    pos = torch.zeros((2, 1, 3), dtype=torch.int32, device="cuda")
    pair = torch.zeros(32, dtype=torch.int32, device="cuda")
    for args, kw in (((q.float(), f), {}), ((q.cpu(), f), {}), ((q[0], f), {}), ((q, f.double()), {}), ((q, f, pos), {}),
                     ((q, f, pos[:, :, :2]), dict(pair_axis=pair)), ((q, f, pos), dict(pair_axis=pair[:3])),
                     ((q, f), dict(pair_axis=pair)), ((q, f), dict(k=q.half())), ((q, f), dict(k=q[:, :, :2])), ((q, f.cpu()), {})):
        with pytest.raises(ValueError):
            fa.rotary(*args, **kw)
    with pytest.raises(fa.FAError):
        fa.rotary(q, torch.ones(33, device="cuda"))
    with pytest.raises(fa.FAError):
        fa.rotary(q[..., :60], f[:8])
    with pytest.raises(fa.FAError):
        fa.rotary(q, f, position_offset=-1)
    with pytest.raises(TypeError):
        fa.rotary(q, 1.0)
    assert fa.rotary(q[:, :, :0], f).shape == (1, 2, 0, 64)
