"""The page operators, appends and reads of two caches at once, on streams and host
threads of their own: the same as one after the other."""
import threading

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

pytestmark = pytest.mark.gpu
B, HKV, PAGE, D, WIDTH, STEPS = 6, 2, 16, 64, 20, 12


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def made(four, pages):
    table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    if four:
        pools = [torch.zeros((pages, HKV, PAGE, D // e), dtype=torch.uint8, device="cuda") for e in (2, 2, 16, 16)]
        return fa.PagedKV4(*pools, table, n), pools
    pools = [torch.zeros((pages, HKV, PAGE, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return fa.PagedKV(*pools, table, n), pools


def run(cache, refs, inputs, stream=None):
    """Rows grow and are appended to, 1 and 3 end and are forked from 0 and 2, and the pool
    is compacted, STEPS times."""
    ended, parents, seen = inputs["ended"], inputs["parents"], []
    for i in range(STEPS):
        seen.append(fa.kv_grow(cache, refs, inputs["tokens"][i], stream=stream))
        q = fa.kv_append(cache, inputs["k"][i], inputs["k"][i], q=inputs["q"][i], inv_freq=inputs["freq"], stream=stream)
        fa.kv_free(cache, refs, ended, stream=stream)
        seen.append(fa.kv_fork(cache, refs, parents, ended, stream=stream))
        seen.append(fa.kv_compact(cache, refs, stream=stream))
        seen.append(fa.forward_paged(q, cache, stream=stream)[0])
        seen.extend(fa.kv_read(cache, 7, stream=stream))
    return seen


def test_two_at_once():
    g = torch.Generator().manual_seed(5)
    sides = []
    for four, pages in ((True, 70000), (False, 90)):                       # (the first is listed in segments)
        T = 9
        sides.append((four, pages, dict(
            tokens=torch.full((STEPS, B), T, dtype=torch.int32).cuda(),
            k=torch.randn((STEPS, B, HKV, T, D), generator=g).to(torch.bfloat16).cuda(),
            q=torch.randn((STEPS, B, 4, T, D), generator=g).to(torch.bfloat16).cuda(),
            freq=torch.rand(D // 2, generator=g).cuda(),
            ended=torch.tensor([1, 3], dtype=torch.int32).cuda(), parents=torch.tensor([0, 2], dtype=torch.int32).cuda())))
    want = []
    for four, pages, inputs in sides:
        cache, pools = made(four, pages)
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        want.append((run(cache, refs, inputs), pools, refs, cache))
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def side(i, stream):
        try:
            four, pages, inputs = sides[i]
            got[i][1].extend(run(got[i][0], got[i][3], inputs, stream))
        except Exception as e:                                             # noqa: BLE001
            errors.append(e)

    for i, (four, pages, _) in enumerate(sides):
        cache, pools = made(four, pages)
        got[i] = (cache, [], pools, torch.zeros(pages, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=side, args=(i, torch.cuda.Stream())) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (seen, pools, refs, cache), (other, also, others, counts) in zip(want, got):
        assert torch.equal(refs, counts) and torch.equal(cache.block_table, other.block_table)
        assert torch.equal(cache.seq_len, other.seq_len) and len(seen) == len(also)
        for a, b in zip(seen, also):
            assert torch.equal(a, b)
        for a, b in zip(pools, others):
            assert torch.equal(a, b)
    assert int(want[0][3].seq_len.min()) > 0


def test_rotary_on_a_stream_of_its_own():
    g = torch.Generator().manual_seed(6)
    q = torch.randn((2, 3, 300, 64), generator=g).to(torch.bfloat16).cuda().requires_grad_()
    freq, up = torch.rand(32, generator=g).cuda(), torch.randn((2, 3, 300, 64), generator=g).to(torch.bfloat16).cuda()
    want = fa.rotary(q, freq)
    (grad,) = torch.autograd.grad(want, q, up)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = fa.rotary(q, freq, stream=s)
    (mine,) = torch.autograd.grad(out, q, up)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(grad, mine)
