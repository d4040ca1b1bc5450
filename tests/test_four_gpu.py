"""The 4-bit cache on the GPU against 64-bit references: append, read, attention."""
import math

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import four_reference as ref
import paged_reference

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def empty_pools(pages, Hkv, page, D, slots_first=False, pad=0):
    """Zeroed pools and scales; slots_first: [pages, slots, heads, bytes] in memory; pad:
    bytes between rows."""
    P = ref.padded(D)
    made = []
    for n in (P // 2, P // 2, P // 16, P // 16):
        extra = pad if n == P // 2 else pad * (P // 16)
        shape = (pages, page, Hkv, n + extra) if slots_first else (pages, Hkv, page, n + extra)
        x = torch.zeros(shape, dtype=torch.uint8, device="cuda")[..., :n]
        made.append(x.transpose(1, 2) if slots_first else x)
    return made


def filled(pages, Hkv, page, D, g, scale=1.0, **kw):
    """Pools with random rows, and what they stand for in 64 bits (on the CPU)."""
    pools = empty_pools(pages, Hkv, page, D, **kw)
    held = []
    for i in range(2):
        x = torch.randn((pages, Hkv, page, D), generator=g, dtype=torch.float64) * scale
        data, code = ref.pack(torch.nn.functional.pad(x, (0, ref.padded(D) - D)))
        pools[i].copy_(data)
        pools[2 + i].copy_(code)
        held.append(ref.unpack(data, code)[..., :D])
    return pools, held


def tables(lens, page, g, spare=2, width=None):
    need = [math.ceil(max(n, 0) / page) for n in lens]
    pages = sum(need) + spare
    order, at = torch.randperm(pages, generator=g).to(torch.int32), 0
    t = torch.full((len(lens), width or max(1, *need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, pages


def make(lens, Hkv, page, D, dtype, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    t, pages = tables(lens, page, g)
    pools, held = filled(pages, Hkv, page, D, g, **kw)
    cache = fa.PagedKV4(*pools, t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), D=D, dtype=dtype)
    return cache, held, t, g


# ---------------------------------------------------------------- append, read
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,page,T,lens,kw", [
    (64, 16, 1, [1, 16, 17, 0], {}), (128, 8, 5, [5, 3, 40, -1], dict(slots_first=True)),
    (40, 24, 30, [30, 70, 12], {}), (96, 1, 3, [2, 9], {}), (256, 100, 17, [120, 16], dict(pad=16)), (8, 5, 2, [2, 7], {})])
def test_append_without_rotation_is_exact(dtype, D, page, T, lens, kw):
    """Bytes and scales are those of the 64-bit reference: dividing 16-bit numbers by 6 or
    a scale in fp32 meets no border that 64 bits do not (11 bits against borders of 8)."""
    g = torch.Generator().manual_seed(D + T)
    t, pages = tables(lens, page, g, width=max(1, *(math.ceil(n / page) for n in lens)) + 1)
    pools = empty_pools(pages, 2, page, D, **kw)
    cache = fa.PagedKV4(*pools, t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), D=D, dtype=dtype)
    # groups of very different sizes, zeros, halfway cases and the largest numbers among them
    k, v = (torch.randn((len(lens), 2, T, D), generator=g) * 2.0 ** torch.randint(-22, 14, (len(lens), 2, T, D // 8), generator=g).repeat_interleave(8, -1)
            for _ in range(2))
    k[0, 0, 0, :8] = torch.tensor([6, 0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5])
    v[0, 0, 0] = 0
    v[0, 1, -1, 0] = 65504 if dtype == F16 else 3e38
    k, v = k.to(dtype), v.to(dtype)
    before = [x.clone() for x in pools]
    assert fa.kv_append(cache, k.cuda().transpose(1, 2).contiguous().transpose(1, 2), v.cuda()) is None
    want = [x.cpu().clone() for x in before]
    P = ref.padded(D)
    rk, rv = (torch.zeros((len(lens), 2, T, D), dtype=torch.float64) for _ in range(2))
    for x, data, scale, read in ((k, want[0], want[2], rk), (v, want[1], want[3], rv)):
        rows, codes = ref.pack(torch.nn.functional.pad(x.double(), (0, P - D)))
        for b, n in enumerate(lens):
            for i in range(max(0, T - max(n, 0)), T):
                at = n - T + i
                p, s = int(t[b, at // page]), at % page
                data[p, :, s], scale[p, :, s] = rows[b, :, i], codes[b, :, i]
                read[b, :, i] = ref.unpack(rows[b, :, i], codes[b, :, i])[..., :D]
    for i in (2, 3):
        assert torch.equal(pools[i].cpu(), want[i])
    for i in (0, 1):                                # (a zero may have a sign)
        assert torch.equal(ref.unpack(pools[i].cpu(), pools[2 + i].cpu()), ref.unpack(want[i], want[2 + i]))
    got_k, got_v = fa.kv_read(cache, T)
    assert got_k.dtype == dtype and torch.equal(got_k.cpu().double(), rk) and torch.equal(got_v.cpu().double(), rv)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,axes", [(128, 128, 0), (64, 40, 3), (80, 80, 2), (96, 22, 1), (256, 128, 0)])
def test_append_with_rotation(dtype, interleaved, D, rot, axes):
    """A turned element is off by 2^-20 (|x| + |y|) in fp32; rounding is monotone, so a
    scale lies between those of the group's largest less and plus that, and a value
    between the roundings of the element less and plus that."""
    B, T, Hq, Hkv, page, lens = 3, 9, 4, 2, 16, [9, 4, 100]
    g = torch.Generator().manual_seed(rot + axes)
    t, pages = tables(lens, page, g)
    cache = fa.PagedKV4(*empty_pools(pages, Hkv, page, D), t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), D=D, dtype=dtype)
    q, k, v = (torch.randn((B, H, T, D), generator=g).to(dtype) for H in (Hq, Hkv, Hkv))
    freq = 10000.0 ** (-torch.arange(rot // 2) / (rot / 2))
    pos = pair = None
    at = torch.tensor(lens)[:, None] - T + torch.arange(T)
    where = at[None].expand(1, B, T)
    axis = torch.zeros(rot // 2, dtype=torch.long)
    if axes:
        pos = torch.randint(-50, 100000, (axes, B, T), generator=g, dtype=torch.int32)
        axis = torch.randint(0, axes, (rot // 2,), generator=g)
        pair, where = axis.to(torch.int32), pos
    out = fa.kv_append(cache, k.cuda(), v.cuda(), q=q.cuda(), inv_freq=freq.cuda(), interleaved=interleaved,
                       position_offset=7, positions=pos if pos is None else pos.cuda(), pair_axis=pair if pair is None else pair.cuda())
    half = rot // 2
    i = torch.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    angle = (where.double()[axis].permute(1, 2, 0) + 7)[:, None] * freq.double()

    def turned(x):
        x = x.double().clone()
        off = torch.zeros_like(x)
        a, b = x[..., first].clone(), x[..., second].clone()
        x[..., first], x[..., second] = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
        off[..., first] = off[..., second] = 2.0 ** -20 * (a.abs() + b.abs())
        return x, off

    live = (at >= 0)[:, None, :, None]
    want, off = turned(q)
    u = paged_reference.HALF_STEP[dtype]
    assert bool(((out.cpu().double() - torch.where(live, want, 0)).abs() <= off + u * (want.abs() + off) + 2.0 ** -25).all())
    assert not out.cpu()[~live.expand_as(out)].any()
    want, off = (torch.nn.functional.pad(x, (0, ref.padded(D) - D)) for x in turned(k))
    g16 = lambda x: x.unflatten(-1, (-1, 16))                                                  # noqa: E731
    lo, hi = ref.scale_of((g16(want.abs() - off).amax(-1)).clamp_min(0)), ref.scale_of(g16(want.abs() + off).amax(-1))
    got = fa.kv_read(cache, T)
    for b, n in enumerate(lens):
        for j in range(max(0, T - n), T):
            p, s = int(t[b, (n - T + j) // page]), (n - T + j) % page
            code = cache.k_scales[p, :, s].cpu().long()
            assert bool(((lo[b, :, j] <= code) & (code <= hi[b, :, j])).all())
            value = ref.unpack(cache.k_cache[p, :, s].cpu(), code)
            low, high = (ref.values(want[b, :, j] + e * off[b, :, j], code) for e in (-1, 1))
            assert bool(((low <= value) & (value <= high)).all())
            assert torch.equal(got[0][b, :, j].cpu().double(), value[..., :D])
            assert torch.equal(got[1][b, :, j].cpu().double(), ref.values(torch.nn.functional.pad(v[b, :, j].double(), (0, ref.padded(D) - D)))[..., :D])


def test_read_of_a_16_bit_cache_and_missing_pages():
    g = torch.Generator().manual_seed(1)
    pool = torch.randn((6, 3, 4, 24), generator=g).to(BF16)
    table = torch.tensor([[0, 5, -1], [9, 2, 1], [3, 3, 3]], dtype=torch.int32)
    cache = fa.PagedKV(pool.cuda(), -pool.cuda(), table.cuda(), torch.tensor([11, 8, 2], dtype=torch.int32).cuda())
    k, v = fa.kv_read(cache, 7)
    for b, n in enumerate([11, 8, 2]):
        for i in range(7):
            at = n - 7 + i
            p = int(table[b, at // 4]) if at >= 0 else -1
            want = pool[p, :, at % 4] if 0 <= p < 6 else torch.zeros(3, 24, dtype=BF16)
            assert torch.equal(k[b, :, i].cpu(), want) and torch.equal(v[b, :, i].cpu(), -want)
    k, v = fa.kv_read(cache, 0)
    assert k.shape == (3, 3, 0, 24)


def test_elements_that_are_not_finite_stay_within_their_group():
    cache, _, t, g = make([1], 1, 16, 64, F16)
    x = torch.ones((1, 1, 1, 64), dtype=F16)
    x[..., 3], x[..., 20] = float("nan"), float("inf")
    fa.kv_append(cache, x.cuda(), x.cuda())
    k, _ = fa.kv_read(cache, 1)
    # (1 / 6 rounds to a scale of 1.375 / 8, and 1 is held as 6 of those)
    ones = ref.values(torch.ones(64, dtype=torch.float64))
    assert float(ones[0]) == 1.03125
    assert k.isfinite().all() and torch.equal(k[0, 0, 0, 32:].cpu().double(), ones[32:])
    assert torch.equal(k[0, 0, 0, :3].cpu().double(), ones[:3])


# ------------------------------------------------------------------ attention
def attention(cache, held, t, lens, Hq, T, dtype, g, causal=True, scale=None, q_scale=1.0):
    B, Hkv, D = len(lens), cache.Hkv, cache.D
    q = (torch.randn((B, Hq, T, D), generator=g) * q_scale).to(dtype)
    o, lse = fa.forward_paged(q.cuda().transpose(1, 2).contiguous().transpose(1, 2), cache, causal=causal, scale=scale)
    assert fa.fa_device_status(None) == fa.FA_OK
    want = paged_reference.attention(q, *held, t, lens, causal=causal, scale=scale)
    return o, lse, want


CASES = [
    # lens, Hq, Hkv, T, D, page, causal
    ([1], 1, 1, 1, 64, 16, True), ([1000], 8, 2, 1, 128, 16, True), ([0, 5, 300, 77], 8, 2, 1, 128, 32, True),
    ([33, 64, 65, 1], 4, 4, 1, 64, 64, True), ([200, 31], 14, 2, 1, 256, 16, True), ([200, 31], 2, 1, 3, 256, 100, False),
    ([40, 500, 3], 12, 4, 5, 128, 24, True), ([40, 500, 3], 12, 4, 5, 96, 8, False), ([90, 10], 4, 1, 4, 40, 1, True),
    ([130, 129], 16, 2, 3, 128, 128, True), ([130, 129], 16, 2, 3, 64, 10, True), ([70], 3, 1, 11, 80, 16, True),
    ([200, 2], 32, 1, 1, 128, 16, True), ([60], 1, 1, 60, 256, 16, True), ([60, 0], 8, 1, 9, 128, 12, True),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page,causal", CASES)
def test_row_kernel(lens, Hq, Hkv, T, D, page, causal, dtype):
    cache, held, t, g = make(lens, Hkv, page, D, dtype, seed=len(lens) + D)
    o, lse, want = attention(cache, held, t, lens, Hq, T, dtype, g, causal)
    if Hq // Hkv * T > 32 and D <= 128 and page % 8 == 0:      # 33 rows: the tensor cores' errors, as documented
        paged_reference.check_attention(o, lse, want, max(lens), dtype)
    else:
        ref.check_rows(o, lse, want, max(lens), dtype, D)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page", [
    ([150, 40], 4, 2, 40, 128, 16), ([600], 4, 1, 130, 64, 64), ([0, 33, 257], 3, 1, 33, 96, 8), ([129], 40, 1, 1, 128, 128)])
def test_many_rows_on_the_tensor_cores(lens, Hq, Hkv, T, D, page, dtype):
    cache, held, t, g = make(lens, Hkv, page, D, dtype, seed=T)
    o, lse, want = attention(cache, held, t, lens, Hq, T, dtype, g)
    paged_reference.check_attention(o, lse, want, max(lens), dtype)


@pytest.mark.parametrize("T", [1, 40])
def test_pages_that_are_not_there_hide_their_keys(T):
    lens, page = [100, 70, 50], 16
    cache, held, t, g = make(lens, 2, page, 128, BF16)
    t[0, 2], t[1, 4], t[2] = -1, 1 << 30, -1                   # in the middle, the last, all
    cache.block_table.copy_(t)
    o, lse, want = attention(cache, held, t, lens, 4, T, BF16, g)
    (ref.check_rows(o, lse, want, 100, BF16, 128) if T == 1 else paged_reference.check_attention(o, lse, want, 100, BF16))
    assert torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("T", [1, 40])
def test_what_lies_behind_a_sequence_does_not_matter(T):
    """Bytes that are no number of the format, behind the last key and in free pages."""
    lens, page = [37, 16, 50], 16
    cache, held, t, g = make(lens, 1, page, 64, F16)
    q = torch.randn((3, 4, T, 64), generator=g).to(F16).cuda()
    o, lse = fa.forward_paged(q, cache)
    used = torch.zeros(cache.k_cache.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(n):
            used[t[b, i // page], i % page] = True
    for x in (cache.k_cache, cache.v_cache, cache.k_scales, cache.v_scales):
        x[:, 0][~used.cuda()] = 255
    o2, lse2 = fa.forward_paged(q, cache)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_strided_pools_lengths_past_the_table_and_far_scales(dtype):
    lens, page = [48, 30], 16
    for kw in (dict(slots_first=True), dict(pad=16)):
        cache, held, t, g = make(lens, 3, page, 128, dtype, **kw)
        cache.seq_len.copy_(torch.tensor([1000, 30]))          # clamped to the row's 48
        o, lse, want = attention(cache, held, t, [1000, 30], 6, 1, dtype, g, scale=0.3)
        ref.check_rows(o, lse, want, 48, dtype, 128)


@pytest.mark.parametrize("k_scale,q_scale", [(2.0 ** -13, 2.0 ** 13), (2.0 ** 11, 2.0 ** -11), (200.0, 1.0), (1.0, 2.0 ** -100)])
def test_small_and_large_numbers(k_scale, q_scale):
    """Queries whose bits do not fit an IEEE half as they are, and attention that one key
    takes alone."""
    lens = [300, 64]
    g = torch.Generator().manual_seed(7)
    t, pages = tables(lens, 16, g)
    pools, held = filled(pages, 1, 16, 128, g, scale=k_scale)
    cache = fa.PagedKV4(*pools, t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    o, lse, want = attention(cache, held, t, lens, 8, 1, BF16, g, q_scale=q_scale)
    ref.check_rows(o, lse, want, 300, BF16, 128)


def test_not_a_number_among_the_queries_reaches_its_rows_only():
    cache, held, t, g = make([50], 1, 16, 64, BF16)
    q = torch.randn((1, 4, 1, 64), generator=g).to(BF16).cuda()
    good, _ = fa.forward_paged(q, cache)
    q[0, 2, 0, 5] = float("nan")
    o, _ = fa.forward_paged(q, cache)
    assert o[0, 2].isnan().all() and torch.equal(o[0, [0, 1, 3]], good[0, [0, 1, 3]])


def test_many_sequences_and_long_ones():
    """Tiles that pieces of the line cut, states that the merge joins, against the 16-bit
    operator over the same numbers (exact in both), which has its own tests."""
    g = torch.Generator().manual_seed(3)
    for B, top, Hkv, Hq, D, page, T, dtype in ((64, 700, 2, 8, 128, 32, 1, BF16), (3, 20000, 1, 8, 64, 64, 1, F16),
                                               (300, 90, 1, 2, 128, 16, 4, F16), (2, 9000, 4, 48, 128, 16, 1, BF16)):
        lens = [int(x) for x in torch.randint(0, top, (B,), generator=g)]
        cache, held, t, _ = make(lens, Hkv, page, D, dtype, seed=B)
        wide = fa.PagedKV(held[0].to(dtype).cuda(), held[1].to(dtype).cuda(), cache.block_table, cache.seq_len)
        q = torch.randn((B, Hq, T, D), generator=g).to(dtype).cuda()
        o, lse = fa.forward_paged(q, cache)
        o2, lse2 = fa.forward_paged(q, wide)
        # both are within half a step of the exact answer, and a weight's error of sum p |v|
        a = fa.forward_paged(q, fa.PagedKV(wide.k_cache, wide.v_cache.abs(), cache.block_table, cache.seq_len))[0].double()
        u, w = paged_reference.HALF_STEP[dtype], 2.0 ** -22 if dtype == F16 else 2.0 ** -11
        bound = 2.02 * u * torch.maximum(o.double().abs(), o2.double().abs()) + 2 * (w + 2.0 ** -15) * a * (1 + 2 * u) + 2.0 ** -24
        assert bool(((o.double() - o2.double()).abs() <= bound).all())
        empty = torch.isneginf(lse2)
        assert torch.equal(torch.isneginf(lse), empty) and bool(((lse - lse2)[~empty].abs() < 1e-4).all())


def test_offsets_past_32_bits():
    """A pool of 9 GB, whose last page is used."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    g = torch.Generator().manual_seed(5)
    pages, Hkv, page, D = 600000, 2, 256, 64
    k = torch.zeros((pages, Hkv, page, 32), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((pages, Hkv, page, 4), dtype=torch.uint8, device="cuda")
    x = torch.randn((1, Hkv, 20, D), generator=g).to(BF16)
    cache = fa.PagedKV4(k, k, ks, ks, torch.tensor([[pages - 1]], dtype=torch.int32).cuda(), torch.tensor([20], dtype=torch.int32).cuda())
    fa.kv_append(cache, x.cuda(), x.cuda())
    got, _ = fa.kv_read(cache, 20)
    held = ref.values(x.double())
    assert torch.equal(got.cpu().double(), held)
    for T in (1, 20):
        q = torch.randn((1, 4, T, D), generator=g).to(BF16)
        o, lse = fa.forward_paged(q.cuda(), cache)
        want = paged_reference.attention(q, held, held, torch.zeros((1, 1), dtype=torch.int32), [20])
        # (held is [1, Hkv, 20, D]: one page of 20 slots)
        (ref.check_rows(o, lse, want, 20, BF16, D) if T == 1 else paged_reference.check_attention(o, lse, want, 20, BF16))
    fa.copy_pages(cache, torch.tensor([pages - 1], dtype=torch.int32).cuda(), torch.tensor([pages - 2], dtype=torch.int32).cuda())
    assert torch.equal(k[pages - 1], k[pages - 2]) and not k[pages - 3].any()


# ------------------------------------------------------- streams, graphs, refusals
def test_a_step_in_a_graph_and_on_another_stream():
    lens = [20, 0, 75]
    cache, held, t, g = make(lens, 2, 16, 128, BF16)
    cache.seq_len.sub_(torch.tensor([1, 0, 1], dtype=torch.int32).cuda())
    start = [x.clone() for x in (cache.k_cache, cache.v_cache, cache.k_scales, cache.v_scales, cache.seq_len)]
    q, k, v = (torch.randn((3, H, 1, 128), generator=g).to(BF16).cuda() for H in (8, 2, 2))
    freq = (10000.0 ** (-torch.arange(64) / 64)).cuda()
    one = torch.tensor([1, 0, 1], dtype=torch.int32).cuda()

    def step():
        cache.seq_len.add_(one)
        return fa.forward_paged(fa.kv_append(cache, k, v, q=q, inv_freq=freq), cache)

    def reset():
        for x, y in zip((cache.k_cache, cache.v_cache, cache.k_scales, cache.v_scales, cache.seq_len), start):
            x.copy_(y)

    want = [x.clone() for x in step()]
    state = [x.clone() for x in (cache.k_cache, cache.k_scales)]
    side = torch.cuda.Stream()
    reset()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    reset()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(state[0], cache.k_cache) and torch.equal(state[1], cache.k_scales)


def test_refusals():
    g = torch.Generator().manual_seed(1)
    t, n = torch.zeros((1, 2), dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    k, v, ks, vs = empty_pools(4, 2, 16, 128)
    for bad in (dict(D=64), dict(D=129), dict(D=0), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            fa.PagedKV4(k, v, ks, vs, t, n, **bad)
    for args in ((k.short(), v, ks, vs), (k, v, ks[..., :4], vs[..., :4]), (k, v[:2], ks, vs), (k, v, ks, vs.cpu()), (k[..., :48], v[..., :48], ks, vs)):
        with pytest.raises(ValueError):
            fa.PagedKV4(*args, t, n)
    cache = fa.PagedKV4(k, v, ks, vs, t, n)
    q, x = torch.randn((1, 4, 1, 128), generator=g).to(BF16).cuda(), torch.randn((1, 2, 1, 128), generator=g).to(BF16).cuda()
    with pytest.raises(ValueError):
        fa.forward_shared_prefix(q, cache, t[0], 16)
    with pytest.raises(ValueError):
        fa.forward_paged(q.half(), cache)
    with pytest.raises(ValueError):
        fa.forward_paged(q[:, :3], cache)
    with pytest.raises(fa.FAError):
        fa.forward_paged(q, cache, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    freq, pos = torch.ones(64).cuda(), torch.zeros((2, 1, 1), dtype=torch.int32).cuda()
    pair = torch.zeros(64, dtype=torch.int32).cuda()
    for bad in (dict(positions=pos), dict(positions=pos.long(), pair_axis=pair), dict(positions=pos[:, :, 0], pair_axis=pair),
                dict(pair_axis=pair), dict(positions=pos, pair_axis=pair[:32]), dict(positions=pos.cpu(), pair_axis=pair)):
        with pytest.raises(ValueError):
            fa.kv_append(cache, x, x, inv_freq=freq, **bad)
    with pytest.raises(AttributeError):
        cache.k_scales = ks.clone()
    with pytest.raises(ValueError):
        fa.kv_read(cache, -1)
    ks.data = ks.clone()
    with pytest.raises(ValueError):
        fa.kv_read(cache, 1)


def test_tables_without_pages_and_an_empty_batch():
    pools = empty_pools(4, 2, 16, 128)
    for B, W, T in ((2, 0, 1), (2, 0, 40), (2, 0, 300), (0, 3, 1)):
        table = torch.zeros((B, W), dtype=torch.int32, device="cuda")
        cache = fa.PagedKV4(*pools, table, torch.full((B,), 5, dtype=torch.int32, device="cuda"))
        q = torch.ones((B, 4, T, 128), dtype=BF16, device="cuda")
        o, lse = fa.forward_paged(q, cache)
        assert o.shape == q.shape and not o.any() and bool(torch.isneginf(lse).all())
        x = torch.ones((B, 2, T, 128), dtype=BF16, device="cuda")
        fa.kv_append(cache, x, x)
        assert not pools[0].any()
        k, v = fa.kv_read(cache, 3)
        assert k.shape == (B, 2, 3, 128) and not k.any()
