"""Calls of the paged-cache operators at the edges of what they allow: many
sequences, far offsets, caches that share one tensor, several host threads, and
waits that run out.  Tolerances are those of tests/paged_reference.py."""
import json
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import paged_reference as ref
from test_paged_gpu import BF16, F16, Pool, run_paged

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()
    fa.load()


@pytest.mark.parametrize("B,T,Hkv,prefix,page", [(70, 1, 1, 0, 8), (700, 1, 1, 0, 8), (2100, 1, 1, 0, 5), (40, 33, 1, 0, 8),
                                                 (70, 1, 2, 300, 8), (700, 1, 1, 130, 16), (1100, 1, 1, 40, 7)])
def test_many_sequences(B, T, Hkv, prefix, page):
    """More sequences than lanes, and strips of sequences longer than a warp;
    most are short, some are empty, one is long."""
    lens = [(b * 7) % 4 for b in range(B)]
    lens[B // 2], lens[B - 1] = 150, 0
    pool = Pool(lens, Hkv, 64, page, BF16, seed=B, prefix=prefix)
    run_paged(pool, Hkv, T, prefix=prefix)


def test_only_empty_sequences():
    for prefix in (0, 40):
        pool = Pool([0] * 40, 1, 64, 8, BF16, seed=1, prefix=prefix)
        run_paged(pool, 4, 1, prefix=prefix)
        if prefix:                                  # every query sees the prefix, and nothing else
            run_paged(pool, 4, 1, causal=False, prefix=prefix)


@pytest.mark.parametrize("T,page", [(1, 16), (1, 12), (40, 16)])
def test_offsets_past_32_bits(T, page):
    """The sequence's pages lie past element 2^32 of the pool."""
    Hkv, D, n = 2, 128, 300
    per_page = Hkv * page * D
    pages = (1 << 32) // per_page + 64
    pool = Pool([n], Hkv, D, page, BF16, seed=7)
    q = pool.queries(8, T)
    small = pool.table.clone()
    k, v = (torch.empty((pages, Hkv, page, D), dtype=BF16, device="cuda") for _ in range(2))
    far = pages - 1 - torch.arange(pool.k.shape[0], dtype=torch.int64)          # page p of the small pool is far[p]
    k[far.cuda()], v[far.cuda()] = pool.k.cuda(), pool.v.cuda()
    used = -(-n // page)
    table = far[small[0, :used].long()][None].to(torch.int32)
    cache = fa.PagedKV(k, v, table.cuda(), pool.lens.cuda())
    o, lse = fa.forward_paged(q.cuda(), cache)
    torch.cuda.synchronize()
    want = ref.attention(q, pool.k, pool.v, small, pool.lens)
    ref.check_attention(o, lse, want, n, BF16)
    # and an append there
    x = torch.randn((1, Hkv, 1, D), generator=pool.g).to(BF16).cuda()
    fa.kv_append(cache, x, -x)
    at = (int(table[0, (n - 1) // page]), slice(None), (n - 1) % page)
    assert torch.equal(k[at], x[0, :, 0]) and torch.equal(v[at], -x[0, :, 0])


@pytest.mark.parametrize("T", [1, 3, 40])
def test_keys_and_values_of_one_tensor(T):
    """A pool [pages, 2, Hkv, slots, D] holds both; so does [pages, slots, 2, Hkv, D]."""
    pool = Pool([200, 45], 2, 64, 16, BF16, seed=31)
    q, _, o, lse = run_paged(pool, 8, T)
    both = torch.stack([pool.k, pool.v], dim=1).cuda()
    cache = fa.PagedKV(both[:, 0], both[:, 1], pool.table.cuda(), pool.lens.cuda())
    got = fa.forward_paged(q.cuda(), cache)
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    mixed = torch.stack([pool.k, pool.v], dim=1).permute(0, 3, 1, 2, 4).contiguous().cuda()
    cache = fa.PagedKV(mixed[:, :, 0].transpose(1, 2), mixed[:, :, 1].transpose(1, 2), pool.table.cuda(), pool.lens.cuda())
    got = fa.forward_paged(q.cuda(), cache)
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_one_page_one_head_and_shared_pages():
    # dimensions of one entry, whose strides nobody follows
    pool = Pool([13], 1, 64, 16, BF16, seed=32, spare=0)
    run_paged(pool, 3, 1)
    run_paged(pool, 3, 40)
    # sequences that share pages, whole or in part
    pool = Pool([100, 60], 2, 64, 16, BF16, seed=33)
    pool.table[1] = pool.table[0]
    run_paged(pool, 4, 1)
    run_paged(pool, 4, 40)


@pytest.mark.parametrize("D,T,group,dtype", [(64, 1, 2, F16), (128, 40, 4, BF16)])
def test_wide_values(D, T, group, dtype):
    """Queries that score hundreds apart within a row, in both directions."""
    pool = Pool([400], 1, D, 16, dtype, seed=34)
    q = pool.queries(group, T) * 30
    run_paged(pool, group, T, q=q)


def test_two_threads_on_the_default_stream():
    """They share the workspace that the cache keeps."""
    pool = Pool([700, 33, 900], 2, 64, 16, BF16, seed=35, prefix=300)
    cache, table = pool.gpu(), pool.prefix_table.cuda()
    qs = [pool.queries(8, 1).cuda(), pool.queries(8, 1).cuda()]
    want = [(fa.forward_paged(x, cache), fa.forward_shared_prefix(x, cache, table, 300)) for x in qs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            for _ in range(200):
                a = fa.forward_paged(qs[i], cache)
                b = fa.forward_shared_prefix(qs[i], cache, table, 300)
                if not (torch.equal(a[0], want[i][0][0]) and torch.equal(b[0], want[i][1][0])
                        and torch.equal(a[1], want[i][0][1]) and torch.equal(b[1], want[i][1][1])):
                    wrong.append(i)
        except Exception as e:                      # noqa: BLE001 (a thread's exception would be lost)
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_streams_at_once():
    pool = Pool([1500, 333], 2, 128, 16, BF16, seed=36)
    cache = pool.gpu()
    qs = [pool.queries(8, 1).cuda(), pool.queries(8, 40).cuda()]
    want = [fa.forward_paged(x, cache) for x in qs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fa.forward_paged(qs[i], cache))
        got.append([fa.forward_paged(qs[0], cache)])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])
    assert all(torch.equal(x[0][0], want[0][0]) for x in got[2:])


def test_a_generation_step_in_a_graph():
    """seq_len += 1, append, attend, captured once and replayed."""
    B, Hkv, group, D, page, n = 3, 2, 4, 64, 16, 40
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn((n, B, h, 1, D), generator=g).to(BF16).cuda() for h in (Hkv * group, Hkv, Hkv))
    freq = (1000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()

    def new():
        kc, vc = (torch.full((B * 3, Hkv, page, D), math.nan, dtype=BF16, device="cuda") for _ in range(2))
        table = torch.arange(B * 3, dtype=torch.int32, device="cuda").view(3, B).t().contiguous()
        return fa.PagedKV(kc, vc, table, torch.zeros(B, dtype=torch.int32, device="cuda"))

    def step(cache, q, k, v):
        cache.seq_len += 1
        return fa.forward_paged(fa.kv_append(cache, k, v, q=q, inv_freq=freq), cache)
    eager = new()
    want = [step(eager, q[i], k[i], v[i]) for i in range(n)]
    cache, x = new(), (q[0].clone(), k[0].clone(), v[0].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache, *x)
    cache.seq_len.zero_()
    for i in range(n):
        for a, b in zip(x, (q[i], k[i], v[i])):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1]), i
    assert torch.equal(cache.k_cache.view(torch.int16), eager.k_cache.view(torch.int16))


def test_refusals_of_cuda_tensors():
    pool = Pool([10, 3], 2, 64, 16, BF16, seed=20, prefix=20)
    cache, table = pool.gpu(), pool.prefix_table.cuda()
    q = pool.queries(4, 1).cuda()
    kv = pool.queries(2, 1).cuda()

    def refused(text, fn, *args, error=ValueError, **kw):
        with pytest.raises(error, match=text):
            fn(*args, **kw)
    for bad in (q[:1], q[..., :32], q[0], q[:, :, :, :40].contiguous()):
        refused("q must have shape", fa.forward_paged, bad, cache)
    refused("dtype and device", fa.forward_paged, q.half(), cache)
    refused("dtype and device", fa.forward_paged, q.cpu(), cache)
    refused("multiple of the cache's key heads", fa.forward_paged, q[:, :3], cache)
    refused("must be a tensor", fa.forward_paged, None, cache, error=TypeError)
    refused("out must be a tensor like q", fa.forward_paged, q, cache, out=q.half())
    refused("contiguous last dimension", fa.forward_paged, q, cache, out=torch.empty((2, 4, 1, 65), dtype=BF16, device="cuda")[..., :64])
    refused("lse must be", fa.forward_paged, q, cache, lse=torch.empty((2, 4), device="cuda"))
    refused("workspace must be", fa.forward_paged, q, cache, workspace=torch.empty(10))
    with pytest.raises(fa.FAError) as e:
        fa.forward_paged(q, cache, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    refused("prefix_table must be", fa.forward_shared_prefix, q, cache, table.long(), 20)
    refused("prefix_len must lie", fa.forward_shared_prefix, q, cache, table, 33)
    refused("prefix_len must lie", fa.forward_shared_prefix, q, cache, table, -1)
    refused("k must have shape", fa.kv_append, cache, q, kv)
    refused("v must have shape", fa.kv_append, cache, kv, kv.expand(2, 2, 2, 64))
    refused("q must have shape", fa.kv_append, cache, kv, kv, q=q.expand(2, 4, 2, 64))
    refused("q_out needs q", fa.kv_append, cache, kv, kv, q_out=q)
    refused("inv_freq must be", fa.kv_append, cache, kv, kv, inv_freq=torch.ones(4))
    with pytest.raises(fa.FAError) as e:
        fa.kv_append(cache, kv, kv, inv_freq=torch.ones(33, device="cuda"))
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FAError):
        fa.kv_append(cache, kv, kv, position_offset=-1)


CHILD = r"""
import json, sys
sys.path.insert(0, sys.argv[2])
import torch
import exact_tiled_attention_23_gb300 as fa

T = int(sys.argv[1])
k = torch.randn((8192, 8, 16, 128), device="cuda", dtype=torch.bfloat16)
table = torch.randperm(8192, device="cuda").to(torch.int32).view(32, 256)
cache = fa.PagedKV(k, k.clone(), table, torch.full((32,), 4096, dtype=torch.int32, device="cuda"))
q = torch.randn((32, 32, T, 128), device="cuda", dtype=torch.bfloat16)
a, b = (torch.empty(1 << 29, device="cuda", dtype=torch.bfloat16) for _ in range(2))
torch.cuda.synchronize()
with torch.cuda.stream(torch.cuda.Stream()):
    for _ in range(60):
        b.copy_(a)
for _ in range(100):
    fa.forward_paged(q, cache)
torch.cuda.synchronize()
status = fa.fa_device_status(None)
total = torch.ones(1 << 20, device="cuda").sum().item()
print(json.dumps({"status": status, "sum": total, "after": fa.fa_device_status(None)}))
"""


@pytest.mark.parametrize("T", [1, 40], ids=["rows", "tensor_cores"])
def test_a_wait_that_runs_out_reports_a_timeout(T):
    """A budget of 0.2 us.  A probe of a barrier may itself be suspended for some
    microseconds, so what runs out is a wait well above that: 100 calls, whose
    copies (29 MB at once from device memory) compete with another stream's.
    The kernels end by themselves, and the context still runs work."""
    run = subprocess.run([sys.executable, "-c", CHILD, str(T), ROOT], env=dict(os.environ, FA_WAIT_LIMIT_MS="0.0002"),
                         capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-2000:]
    got = json.loads(run.stdout.strip().splitlines()[-1])
    assert got == {"status": fa.FA_ERR_TIMEOUT, "sum": float(1 << 20), "after": fa.FA_OK}


FIRST_IN_A_GRAPH = r"""
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import exact_tiled_attention_23_gb300 as fa
from test_paged_gpu import BF16, Pool

for T, width, prefix in ((1, None, 0), (1, None, 100), (1, 1300, 0), (40, None, 0), (40, None, 300)):
    pool = Pool([200, 30], 2, 64, 16, BF16, seed=51, prefix=prefix, width=width)
    cache, q, table = pool.gpu(), pool.queries(4, T).cuda(), pool.prefix_table.cuda()
    x = torch.randn((2, 2, 1, 64), device="cuda").to(BF16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fa.kv_append(cache, x, x)
        o, lse = fa.forward_shared_prefix(q, cache, table, prefix) if prefix else fa.forward_paged(q, cache)
    graph.replay()
    torch.cuda.synchronize()
    want = fa.forward_shared_prefix(q, cache, table, prefix) if prefix else fa.forward_paged(q, cache)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), (T, width, prefix)
assert fa.fa_device_status(None) == fa.FA_OK
print("same")
"""


def test_first_calls_of_a_process_can_be_captured():
    """What the library asks the driver for once per process may be asked during a capture."""
    run = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH, ROOT], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stderr[-2000:]
