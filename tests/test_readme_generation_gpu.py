"""The generation steps that README.md shows, run as they stand there."""
import os
import textwrap

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def step_with(call):
    """The last kv_append() in front of `call`, and `call`, out of README.md's
    indented lines."""
    with open(os.path.join(ROOT, "README.md")) as f:
        lines = [x for x in f.read().splitlines() if x.startswith("    ") and "#" not in x.split("fa.")[0]]
    at = next(i for i, x in enumerate(lines) if call in x and "fa." in x)
    append = max(i for i in range(at + 1) if "fa.kv_append(" in lines[i])
    return textwrap.dedent("\n".join(lines[append:at + 1]))


def test_steps_are_found():
    """(no GPU needed)"""
    for call in ("forward_paged(", "forward_shared_prefix("):
        code = step_with(call)
        compile(code, "README.md", "exec")
        assert "kv_append(" in code and "fa." + call in code


@pytest.mark.gpu
@pytest.mark.parametrize("length", [0, 48])
def test_a_step_equals_the_whole_sequence(length):
    """A prompt's keys, then one token by the README's lines; the answer is that
    of the same text in one table without a prefix."""
    fa.build()
    B, Hkv, group, D, page, n = 2, 2, 2, 64, 16, 37
    g = torch.Generator().manual_seed(5)
    text_k, text_v = (torch.randn((B, Hkv, length + n + 1, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    for x in (text_k, text_v):
        x[1, :, :length] = x[0, :, :length]
    text_q = torch.randn((B, Hkv * group, 1, D), generator=g).to(torch.bfloat16).cuda()
    inv_freq = (1000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()

    def pool():
        k_pool, v_pool = (torch.zeros((20, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return k_pool, v_pool, torch.randperm(20, generator=g).to(torch.int32).cuda()
    # the whole text, without a prefix
    k_pool, v_pool, order = pool()
    whole = fa.PagedKV(k_pool, v_pool, order.view(2, 10), torch.full((B,), length + n + 1, dtype=torch.int32, device="cuda"))
    want = fa.forward_paged(fa.kv_append(whole, text_k, text_v, q=text_q.expand(-1, -1, length + n + 1, -1),
                                         inv_freq=inv_freq)[:, :, -1:], whole)
    # as a program would come to that point
    k_pool, v_pool, order = pool()
    pages = order[:length // page].contiguous()
    if length:
        front = fa.PagedKV(k_pool, v_pool, pages[None], torch.tensor([length], dtype=torch.int32, device="cuda"))
        fa.kv_append(front, text_k[:1, :, :length], text_v[:1, :, :length], inv_freq=inv_freq)
    block_table, seq_len = order[6:14].view(2, 4).contiguous(), torch.full((B,), n, dtype=torch.int32, device="cuda")
    cache = fa.PagedKV(k_pool, v_pool, block_table, seq_len)
    fa.kv_append(cache, text_k[:, :, length:length + n], text_v[:, :, length:length + n], inv_freq=inv_freq,
                 position_offset=length)
    seq_len += 1
    names = {"fa": fa, "cache": cache, "k": text_k[:, :, -1:], "v": text_v[:, :, -1:], "q": text_q, "inv_freq": inv_freq,
             "pages": pages, "length": length}
    exec(step_with("forward_shared_prefix(" if length else "forward_paged("), names)       # noqa: S102
    torch.cuda.synchronize()
    # two bf16 roundings of a result in which |v| < 5, and the weights' 2^-16
    assert (names["o"].float() - want[0].float()).abs().max() <= 2 * 2.0 ** -8 * 5
    assert (names["lse"] - want[1]).abs().max() <= 1e-4
