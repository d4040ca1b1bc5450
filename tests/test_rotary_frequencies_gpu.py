"""rotary() gives its frequencies no gradient, and says so."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


@pytest.mark.parametrize("leaf", [False, True])
def test_frequencies_that_ask_for_a_gradient_are_refused(leaf):
    q = torch.randn((1, 2, 3, 16), device="cuda").half().requires_grad_(leaf)
    freq = torch.rand(8, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="inv_freq"):
        fa.rotary(q, freq)
    with pytest.raises(ValueError, match="inv_freq"):
        fa.rotary(q, 2 * freq, k=q)
    want = fa.rotary(q, freq.detach())
    with torch.no_grad():                           # nobody asks
        assert torch.equal(fa.rotary(q, freq), want)
    with fwd.dual_level(), pytest.raises(ValueError, match="inv_freq"):
        fa.rotary(q, fwd.make_dual(freq.detach(), torch.ones(8, device="cuda")))
