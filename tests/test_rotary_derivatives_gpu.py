"""Derivatives of rotary() in forward mode, alone and over a gradient.  The operation is
linear: a tangent turns as its tensor does, to the bit."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def made(dtype, interleaved):
    g = torch.Generator().manual_seed(1)
    q, tq, k, tk = (torch.randn((2, H, 5, 48), generator=g).to(dtype).cuda() for H in (3, 3, 1, 1))
    freq = torch.rand(20, generator=g).cuda()
    how = dict(positions=torch.randint(-9, 99, (2, 2, 5), generator=g, dtype=torch.int32).cuda(),
               pair_axis=torch.randint(0, 2, (20,), generator=g, dtype=torch.int32).cuda(), interleaved=interleaved,
               position_offset=3)
    return q, tq, k, tk, freq, how


def back(x, freq, how):
    """Turned back: the angles of -freq are those of freq with the other sign."""
    return fa.rotary(x, -freq, **how)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("leaf", [False, True])
@pytest.mark.parametrize("which", ["q", "k", "both", "q alone"])
def test_tangents_turn(which, leaf, interleaved, dtype):
    q, tq, k, tk, freq, how = made(dtype, interleaved)
    want = fa.rotary(q, freq, k=k, **how)
    want_t = fa.rotary(tq, freq, k=tk, **how)
    if leaf:
        q.requires_grad_(), k.requires_grad_()
    with fwd.dual_level():
        x = q if which == "k" else fwd.make_dual(q, tq)
        y = k if which in ("q", "q alone") else fwd.make_dual(k, tk)
        got = (fa.rotary(x, freq, **how),) if which == "q alone" else fa.rotary(x, freq, k=y, **how)
        for i, r in enumerate(got):
            a, t = fwd.unpack_dual(r)
            assert torch.equal(a, want[i]) and a.requires_grad == leaf
            if which == ("k", "q")[i]:
                assert t is None or not t.any()
            else:
                assert t is not None and torch.equal(t, want_t[i])


def test_tangents_without_gradients_and_on_another_stream():
    q, tq, k, tk, freq, how = made(BF16, False)
    want = fa.rotary(tq, freq, **how)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with fwd.dual_level():
        with torch.no_grad():
            assert torch.equal(fwd.unpack_dual(fa.rotary(fwd.make_dual(q, tq), freq, **how)).tangent, want)
        r = fa.rotary(fwd.make_dual(q, tq), freq, stream=side, **how)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(fwd.unpack_dual(r).tangent, want)


@pytest.mark.parametrize("create_graph", [False, True])
def test_forward_mode_over_a_gradient(create_graph):
    """The gradient turns back, and so does the tangent of the gradient behind it."""
    q, tq, k, tk, freq, how = made(BF16, False)
    q.requires_grad_(), k.requires_grad_()
    up, tup = torch.randn_like(q), torch.randn_like(q)
    a, b = fa.rotary(q, freq, k=k, **how)
    with fwd.dual_level():
        dq, dk = torch.autograd.grad((a, b), (q, k), (fwd.make_dual(up, tup), torch.ones_like(b)), create_graph=create_graph)
        value, tangent = fwd.unpack_dual(dq)
        assert torch.equal(value, back(up, freq, how)) and tangent is not None and torch.equal(tangent, back(tup, freq, how))
        assert torch.equal(fwd.unpack_dual(dk).primal, back(torch.ones_like(b), freq, how))


def test_the_gradient_of_a_tangent():
    """Tangents that require grad are part of the graph."""
    q, tq, k, tk, freq, how = made(F16, True)
    q.requires_grad_(), tq.requires_grad_()
    with fwd.dual_level():
        r = fwd.unpack_dual(fa.rotary(fwd.make_dual(q, tq), freq, **how))
        up = torch.randn_like(q)
        gq, gt = torch.autograd.grad((r.primal, r.tangent), (q, tq), (up, 2 * up))
    assert torch.equal(gq, back(up, freq, how)) and torch.equal(gt, back(2 * up, freq, how))


def test_tangents_that_have_no_memory():
    """Zeros that torch keeps without memory turn into zeros."""
    q, _, k, tk, freq, how = made(BF16, False)
    want = fa.rotary(tk, freq, **how)
    with fwd.dual_level():
        zeros = torch._efficientzerotensor(q.shape, dtype=q.dtype, device=q.device)
        a, b = fa.rotary(fwd.make_dual(q, zeros), freq, k=fwd.make_dual(k, tk), **how)
        t = fwd.unpack_dual(a).tangent
        assert (t is None or not t.any()) and torch.equal(fwd.unpack_dual(b).tangent, want)
