"""The page operators on the GPU against their steps in Python, and a run of all of them
beside the attention that reads the pages."""
import random

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import four_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def pools(four, pages, Hkv, page, D, g, slots_first=False):
    """Pools of a 16-bit cache, or of a 4-bit one with its scales, with random bytes."""
    P = ref.padded(D)
    made = []
    for n in ((P // 2, P // 2, P // 16, P // 16) if four else (D, D)):
        shape = (pages, page, Hkv, n) if slots_first else (pages, Hkv, page, n)
        x = torch.randint(0, 200, shape, generator=g, dtype=torch.uint8)
        x = x.cuda() if four else x.to(torch.float16).cuda()
        made.append(x.transpose(1, 2) if slots_first else x)
    return made


def cache_of(four, data, table, seq_len, D):
    return fa.PagedKV4(*data, table, seq_len, D=D) if four else fa.PagedKV(*data, table, seq_len)


def same(cache, refs, x):
    assert cache.block_table.tolist() == x.table and cache.seq_len.tolist() == x.seq_len and refs.tolist() == x.refs


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_calls_in_any_order(four, seed):
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    page, B, width = rng.choice([1, 3, 16]), rng.randint(1, 40), rng.randint(1, 9)
    N, Hkv, D = rng.randint(1, 2 * B * width), rng.choice([1, 3]), rng.choice([8, 64, 128, 256])
    table = torch.full((B, width + 3), -1, dtype=torch.int32).cuda()[:, :width]      # rows further apart
    data = pools(four, N, Hkv, page, D, g, slots_first=seed % 3 == 0)
    cache = cache_of(four, data, table, ints([0] * B), D)
    refs = ints([0] * N)
    x = ref.Pages(table, cache.seq_len, refs, page)
    held = [d.cpu().clone() for d in data]
    for _ in range(30):
        how = rng.choice(["grow", "grow", "free", "fork", "compact", "copy"])
        if how == "grow":
            tokens = [rng.choice([0, 1, page, -2, 2 * page + 1, 1 << 30, 2 ** 31 - 1] if rng.random() < 0.2 else [0, 1, page + 1]) for _ in range(B)]
            assert fa.kv_grow(cache, refs, ints(tokens)).tolist() == x.grow(tokens)
        elif how == "free":
            rows = [rng.randint(-1, B) for _ in range(rng.randint(0, B))]
            assert fa.kv_free(cache, refs, ints(rows)) is None
            x.free(rows)
        elif how == "fork":
            n = rng.randint(0, B)
            parent, child = ([rng.randint(-1, B) for _ in range(n)] for _ in range(2))
            src, taken = x.fork(parent, child)
            assert fa.kv_fork(cache, refs, ints(parent), ints(child)).tolist() == taken
            for h in held:
                for a, b in zip(src, taken):
                    if a >= 0:
                        h[b] = h[a]
        elif how == "compact":
            moved, move = x.compact()
            assert fa.kv_compact(cache, refs).tolist() == moved
            for h in held:
                for a, b in move.items():
                    h[b] = h[a]
        else:
            order = list(range(N))
            rng.shuffle(order)
            n = N // 2
            src, dst = order[:n] + [-1, N], order[n:2 * n] + [0, 0]
            count = rng.choice([None, rng.randint(0, n + 9)])
            fa.copy_pages(cache, ints(src), ints(dst), None if count is None else ints([count]))
            for h in held:
                for a, b in list(zip(src, dst))[:count]:
                    if 0 <= a < N:
                        h[b] = h[a]
        same(cache, refs, x)
        for d, h in zip(data, held):
            assert torch.equal(d.cpu(), h)


@pytest.mark.parametrize("N", [65536, 65537, 200001, 3000000])
def test_pools_that_one_cta_does_not_list(N):
    """Against plain torch, on pools that are listed in segments."""
    g = torch.Generator().manual_seed(N)
    page, B, width = 2, 1500, 40
    have = torch.randint(0, width + 1, (B,), generator=g)
    n = (have * page - torch.randint(0, 2, (B,), generator=g)).clamp_min(0)
    order = torch.randperm(N, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += int(have[b])
    refs = torch.zeros(N, dtype=torch.int32)
    refs[order[:at].long()] = 1
    data = [torch.zeros((N, 1, page, 8), dtype=torch.float16, device="cuda") for _ in range(2)]
    data[0][:, 0, 0, 0] = torch.arange(N, device="cuda") % 2048
    cache = cache_of(False, data, table.cuda(), n.to(torch.int32).cuda(), 8)
    x, counts = ref.Pages(table, cache.seq_len, refs, page), refs.cuda()
    tokens = torch.randint(0, 9, (B,), generator=g).tolist()
    assert fa.kv_grow(cache, counts, ints(tokens)).tolist() == x.grow(tokens)
    same(cache, counts, x)
    rows = list(range(0, B, 3))
    fa.kv_free(cache, counts, ints(rows))
    x.free(rows)
    parent = [r + 1 for r in rows if r + 1 < B]
    src, taken = x.fork(parent, rows[:len(parent)])
    assert fa.kv_fork(cache, counts, ints(parent), ints(rows[:len(parent)])).tolist() == taken
    same(cache, counts, x)
    before = data[0][:, 0, 0, 0].cpu().tolist()
    moved, move = x.compact()
    assert fa.kv_compact(cache, counts).tolist() == moved
    same(cache, counts, x)
    after = data[0][:, 0, 0, 0].cpu().tolist()
    assert all(after[b] == before[a] for a, b in move.items())


def test_counts_that_the_caller_added_and_layers():
    """A prefix's pages stay when its sequences go, every layer's pools are copied, and
    tables of the caller's own are mapped by what kv_compact() returns."""
    g = torch.Generator().manual_seed(0)
    table, n, refs = torch.full((3, 4), -1, dtype=torch.int32).cuda(), ints([0, 0, 0]), ints([0] * 12)
    layers = [cache_of(four, pools(four, 12, 2, 8, 64, g), table, n, 64) for four in (False, True, False)]
    fa.kv_grow(layers, refs, ints([12, 0, 0]))
    prefix = table[0, :2].clone()
    refs[prefix.long()] += 1
    taken = fa.kv_fork(layers, refs, ints([0]), ints([2]))
    assert taken.tolist() == [2] and table[2].tolist() == [0, 2, -1, -1] and refs[:4].tolist() == [3, 2, 1, 0]
    for c in layers:
        assert torch.equal(c.k_cache[2], c.k_cache[1]) and torch.equal(c.v_cache[2], c.v_cache[1])
    fa.kv_free(layers, refs, ints([0]))
    assert refs[:3].tolist() == [2, 1, 1]
    kept = [c.k_cache[2].clone() for c in layers]
    refs[1] = 0                                     # page 1 is given up: a hole
    moved = fa.kv_compact(layers, refs)
    assert moved.tolist() == [0, -1, 1] + [-1] * 9 and table[2].tolist() == [0, 1, -1, -1]
    assert all(torch.equal(c.k_cache[1], x) for c, x in zip(layers, kept))


def test_generation_with_all_operators():
    """Sequences that are admitted, grow, fork, end and are compacted, in both kinds of
    cache: what is read back is what each sequence was given, and its attention is that
    of a fresh cache with the same tokens."""
    rng, g = random.Random(1), torch.Generator().manual_seed(1)
    B, Hkv, Hq, D, page, width, N = 6, 2, 8, 64, 8, 16, 60
    for four in (False, True):
        table, n, refs = torch.full((B, width), -1, dtype=torch.int32).cuda(), ints([0] * B), ints([0] * N)
        data = pools(four, N, Hkv, page, D, g)
        cache = fa.PagedKV4(*data, table, n, dtype=torch.float16) if four else fa.PagedKV(*data, table, n)
        tokens = [[] for _ in range(B)]
        for step in range(40):
            grow = [rng.choice([0, 1, 1, 5]) if rng.random() < 0.9 else 20 for _ in range(B)]
            taken = fa.kv_grow(cache, refs, ints(grow)).tolist()
            T = max(grow)
            new = torch.randn((B, Hkv, T, D), generator=g).to(torch.float16)
            grown = [t if got != -2 else 0 for t, got in zip(grow, taken)]
            for b, t in enumerate(grown):           # rows that took fewer write again what they have
                old = tokens[b][max(0, len(tokens[b]) - (T - t)):]
                if old and t < T:
                    new[b, :, T - t - len(old):T - t] = torch.stack(old, 1)
                tokens[b] += [new[b, :, i] for i in range(T - t, T)]
            if T:
                # (a page that two rows share is written by both, with the same tokens)
                fa.kv_append(cache, new.cuda(), -new.cuda())
            if step % 5 == 3:
                rows = [rng.randrange(B)]
                fa.kv_free(cache, refs, ints(rows))
                tokens[rows[0]] = []
                parent = rng.choice([b for b in range(B) if b != rows[0]])
                if fa.kv_fork(cache, refs, ints([parent]), ints(rows)).tolist()[0] != -2:
                    tokens[rows[0]] = list(tokens[parent])
            if step % 7 == 6:
                fa.kv_compact(cache, refs)
                assert not bool(refs[int((refs > 0).sum()):].any())
            assert n.tolist() == [len(t) for t in tokens]
            most = max(1, *(len(t) for t in tokens))
            k, v = fa.kv_read(cache, most)
            want = torch.zeros((B, Hkv, most, D), dtype=torch.float64)
            for b, t in enumerate(tokens):
                if t:
                    x = torch.stack(t, 1).double()
                    want[b, :, most - len(t):] = ref.values(x) if four else x
            assert torch.equal(k.cpu().double(), want) and torch.equal(v.cpu().double(), -want)
            if step % 10 == 9:
                q = torch.randn((B, Hq, 1, D), generator=g).to(torch.float16).cuda()
                o, lse = fa.forward_paged(q, cache)
                fresh = torch.zeros((B, Hkv, most, D), dtype=torch.float16, device="cuda")
                for b, t in enumerate(tokens):
                    if t:
                        fresh[b, :, :len(t)] = k[b, :, most - len(t):]
                plain = fa.PagedKV(fresh, -fresh, torch.arange(B, dtype=torch.int32).cuda()[:, None], n)
                o2, lse2 = fa.forward_paged(q, plain)
                # weights good to 2^-22 in both, 2^-20 of an exponent, and O rounded once
                a = fa.forward_paged(q, fa.PagedKV(fresh, fresh.abs(), plain.block_table, n))[0].double()
                assert bool(((o.double() - o2.double()).abs() <= 2.0 ** -10 * o2.double().abs() + 2.0 ** -15 * a + 2.0 ** -24).all())
                assert torch.equal(torch.isneginf(lse), torch.isneginf(lse2))


def test_operators_in_a_graph():
    g = torch.Generator().manual_seed(2)
    table, n, refs = torch.full((4, 6), -1, dtype=torch.int32).cuda(), ints([0] * 4), ints([0] * 20)
    cache = cache_of(True, pools(True, 20, 1, 4, 64, g), table, n, 64)
    tokens, rows, parent, child = ints([9, 0, 3, 0]), ints([0]), ints([2]), ints([3])

    def step():
        fa.kv_free(cache, refs, child)
        fa.kv_grow(cache, refs, tokens)
        taken = fa.kv_fork(cache, refs, parent, child)
        fa.kv_free(cache, refs, rows)
        return taken, fa.kv_compact(cache, refs)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taken, moved = step()
    x = ref.Pages(table, n, refs, 4)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        x.free([3])
        x.grow([9, 0, 3, 0])
        _, want = x.fork([2], [3])
        x.free([0])
        to, _ = x.compact()
        assert taken.tolist() == want and moved.tolist() == to
        same(cache, refs, x)


def test_refusals():
    g = torch.Generator().manual_seed(3)
    table, n, refs = torch.full((2, 4), -1, dtype=torch.int32).cuda(), ints([0, 0]), ints([0] * 5)
    cache = cache_of(False, pools(False, 5, 1, 4, 64, g), table, n, 64)
    other = cache_of(False, pools(False, 5, 1, 4, 64, g), table.clone(), n, 64)
    fewer = cache_of(False, pools(False, 4, 1, 4, 64, g), table, n, 64)
    for bad in (refs[:4], refs.long(), refs.cpu(), torch.zeros(10, dtype=torch.int32).cuda()[::2]):
        with pytest.raises(ValueError):
            fa.kv_grow(cache, bad, ints([1, 1]))
    with pytest.raises(ValueError):
        fa.kv_grow(cache, refs, ints([1]))
    with pytest.raises(ValueError):
        fa.kv_fork(cache, refs, ints([0]), ints([1, 1]))
    with pytest.raises(ValueError):
        fa.kv_free(cache, refs, torch.zeros((1, 1), dtype=torch.int32).cuda())
    with pytest.raises(ValueError):
        fa.copy_pages(cache, ints([0, 1]), ints([2]))
    for layers in ([], [cache, other], [cache, fewer]):
        with pytest.raises(ValueError):
            fa.kv_compact(layers, refs)
    with pytest.raises(TypeError):
        fa.kv_free(cache, refs, [0])
    assert fa.kv_grow(cache, refs, ints([0, 0])).tolist() == [0, 0] and refs.tolist() == [0] * 5
    fa.kv_free(cache, refs, ints([]))
    assert fa.kv_fork(cache, refs, ints([]), ints([])).numel() == 0
    fa.copy_pages(cache, ints([]), ints([]))
