"""Calls of few query rows: clusters of CTAs that share a tile, where the table
allows few keys, and the same calls behind a table so wide that their keys are
cut as one line.  Tolerances are those of tests/paged_reference.py."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
from test_paged_gpu import BF16, CASES, F16, SHARED, Pool, run_paged

pytestmark = pytest.mark.gpu

FEW = [c for c in CASES if c[2] * c[3] <= 8 and c[4] <= 128]
FEW_SHARED = [c for c in SHARED if c[3] * c[4] <= 8 and c[5] <= 128]


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()
    fa.load()


def wide(page):
    """Entries of a table that allows more keys than teams take."""
    return 20000 // page


@pytest.mark.parametrize("lens,Hkv,group,T,D,page,dtype", FEW)
@pytest.mark.parametrize("causal", [True, False])
def test_wide_tables_match_64_bits(lens, Hkv, group, T, D, page, dtype, causal):
    pool = Pool(lens, Hkv, D, page, dtype, seed=len(lens) * 100 + T + D, width=wide(page))
    run_paged(pool, Hkv * group, T, causal)


@pytest.mark.parametrize("prefix,lens,Hkv,group,T,D,page,dtype", FEW_SHARED)
@pytest.mark.parametrize("causal", [True, False])
def test_wide_tables_behind_a_prefix_match_64_bits(prefix, lens, Hkv, group, T, D, page, dtype, causal):
    pool = Pool(lens, Hkv, D, page, dtype, seed=prefix, prefix=prefix, width=wide(page))
    run_paged(pool, Hkv * group, T, causal, prefix=prefix)


# Clusters of 8, 4, 2 and 1 CTAs, the last number of tiles that a GPU of 152 SMs
# takes and the first that it does not.
@pytest.mark.parametrize("B", [1, 15, 16, 36, 37, 76, 77, 152, 153])
@pytest.mark.parametrize("D,page,dtype,prefix", [(64, 16, BF16, 0), (128, 24, F16, 0), (128, 5, BF16, 0), (64, 8, F16, 90)])
def test_teams_of_every_size(B, D, page, dtype, prefix):
    lens = [(b * 7) % 4 for b in range(B)]
    lens[B // 2], lens[-1] = 700, 0
    lens[0] = 333
    pool = Pool(lens, 1, D, page, dtype, seed=B, prefix=prefix)
    run_paged(pool, 2, 1, prefix=prefix)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 1023, 1024, 1025, 4000, 8191, 8192, 8193])
def test_lengths_around_a_teams_chunks(n):
    """64 warps of 16 keys a chunk, up to eight chunks each; 8193 are a line."""
    pool = Pool([n], 1, 128, 16, BF16, seed=n)
    run_paged(pool, 4, 1)


@pytest.mark.parametrize("D", [8, 24, 56, 64, 72, 88, 120, 128])
@pytest.mark.parametrize("n", [40, 900])
def test_teams_of_odd_head_sizes(D, n):
    """Four columns go to the team's CTAs in turn."""
    pool = Pool([n, 3], 1, D, 8, BF16, seed=D)
    run_paged(pool, 8, 1)
    run_paged(pool, 2, 3)


@pytest.mark.parametrize("prefix", [1, 31, 32, 33, 1000])
def test_teams_behind_a_prefix(prefix):
    """No own keys at all, own keys behind a chunk that the prefix leaves half
    empty, more query tokens than the sequence has."""
    pool = Pool([0, 1, 2, 33, 200], 2, 64, 16, BF16, seed=prefix, prefix=prefix)
    for T in (1, 3):
        for causal in (True, False):
            run_paged(pool, 4, T, causal, prefix=prefix)


def test_pages_outside_the_pool_are_hidden_from_teams():
    pool = Pool([200, 64, 30], 2, 64, 16, BF16, seed=41, prefix=100)
    pool.table[0, 3], pool.table[0, 5], pool.table[1, :] = -1, 1 << 30, 10000
    pool.prefix_table[2] = -5
    run_paged(pool, 4, 1)
    run_paged(pool, 4, 1, prefix=100)
    pool.prefix_table[:] = 1 << 30                  # the second sequence sees nothing
    run_paged(pool, 4, 1, prefix=100)


def test_teams_write_rows_only():
    """The output between the rows, and the LSE behind the last, stay as they were."""
    pool = Pool([200, 0, 77], 2, 64, 16, F16, seed=42)
    q, cache, o, lse = run_paged(pool, 6, 2)
    out = torch.full((3, 6, 2, 128), 7.0, dtype=F16, device="cuda")
    row = torch.full((3 * 6 * 2 + 50,), 7.0, device="cuda")
    fa.forward_paged(q.cuda(), cache, out=out[..., :64], lse=row[:36].view(3, 6, 2))
    assert torch.equal(out[..., :64], o) and (out[..., 64:] == 7).all()
    assert torch.equal(row[:36].view(3, 6, 2), lse) and (row[36:] == 7).all()


@pytest.mark.parametrize("prefix", [0, 200])
def test_teams_in_graphs_follow_lengths(prefix):
    """A step in a graph: kv_append, then the attention, with lengths that grow."""
    pool = Pool([300, 300, 300], 2, 64, 16, BF16, seed=43, prefix=prefix)
    cache, want_cache = pool.gpu(), pool.gpu()
    x = [torch.randn((3, 2, 1, 64), generator=pool.g).to(BF16).cuda() for _ in range(2)]
    q = pool.queries(4, 1).cuda()
    pt = pool.prefix_table.cuda()

    def step(c):
        fa.kv_append(c, *x)
        return fa.forward_shared_prefix(q, c, pt, prefix) if prefix else fa.forward_paged(q, c)

    for c in (cache, want_cache):
        c.seq_len.copy_(torch.tensor([1, 20, 150], dtype=torch.int32))
    step(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(cache)
    for lens in ([1, 20, 150], [2, 0, 151], [299, 300, 16], [300, 17, 1]):
        for c in (cache, want_cache):
            c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        want = step(want_cache)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("D,T", [(64, 1), (256, 1), (64, 40)])
def test_tables_without_pages(D, T):
    """Sequences that own no pages at all: nothing to see but a prefix."""
    pool = Pool([0, 0], 2, D, 16, BF16, seed=44, prefix=70)
    cache = fa.PagedKV(pool.k.cuda(), pool.v.cuda(), torch.empty((2, 0), dtype=torch.int32, device="cuda"),
                       torch.tensor([0, 5], dtype=torch.int32, device="cuda"))       # 5 counts as 0
    q = pool.queries(4, T).cuda()
    o, lse = fa.forward_paged(q, cache, causal=False)
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = fa.forward_shared_prefix(q, cache, pool.prefix_table.cuda(), 70)
    assert (o == 0).all() and torch.isneginf(lse).all()
    got = fa.forward_shared_prefix(q, cache, pool.prefix_table.cuda(), 70, causal=False)
    torch.cuda.synchronize()
    want = run_paged(pool, 4, T, causal=False, prefix=70, q=q.cpu())
    assert torch.equal(got[0], want[2]) and torch.equal(got[1], want[3])
