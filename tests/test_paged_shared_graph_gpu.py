"""A generation step behind a shared prefix in a captured graph: seq_len += 1,
append, attend.  The row kernel and the merge read the step's queries and lengths
while the prefix kernel runs, at the same addresses in every replay."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("B,prefix,T", [(12, 700, 1), (40, 3000, 1), (12, 700, 3), (3, 200, 1)])
def test_a_shared_step_in_a_graph(B, prefix, T):
    fa.build()
    Hkv, group, D, page, n = 2, 4, 64, 16, 30
    g = torch.Generator().manual_seed(B)
    q, k, v = (torch.randn((n, B, h, T, D), generator=g).to(BF16).cuda() for h in (Hkv * group, Hkv, Hkv))
    freq = (1000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    first, own = -(-prefix // page), -(-n * T // page)
    order = torch.randperm(first + B * own, generator=g).to(torch.int32).cuda()
    pool = torch.randn((2, first + B * own, Hkv, page, D), generator=g).to(BF16).cuda()
    table = order[:first].contiguous()

    def new():
        both = pool.clone()
        return fa.PagedKV(both[0], both[1], order[first:].view(B, own), torch.zeros(B, dtype=torch.int32, device="cuda"))

    def step(cache, q, k, v):
        cache.seq_len += T
        x = fa.kv_append(cache, k, v, q=q, inv_freq=freq, position_offset=prefix)
        return fa.forward_shared_prefix(x, cache, table, prefix)
    eager = new()
    want = []
    for i in range(n):                              # each with everything before it done
        want.append(step(eager, q[i], k[i], v[i]))
        torch.cuda.synchronize()
    cache, x = new(), (q[0].clone(), k[0].clone(), v[0].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache, *x)
    for _ in range(8):
        cache.seq_len.zero_()
        got = []
        for i in range(n):                          # one behind the other, without a pause
            for a, b in zip(x, (q[i], k[i], v[i])):
                a.copy_(b)
            graph.replay()
            got.append((out[0].clone(), out[1].clone()))
        torch.cuda.synchronize()
        for i in range(n):
            assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1]), i
    assert fa.fa_device_status(None) == fa.FA_OK
