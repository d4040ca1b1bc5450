"""The paged-cache operators against plain 64-bit implementations.

Tolerances are derived in tests/paged_reference.py.  Slots that no sequence
owns are filled with NaN, so that a read of one shows.
"""
import math

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import paged_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()
    fa.load()


class Pool:
    """A pool with shuffled pages whose unowned slots hold NaN, on the CPU and the GPU."""

    def __init__(self, lens, Hkv, D, page, dtype, seed, prefix=0, slots_first=False, spare=2, width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        first = -(-prefix // page)
        self.page, self.Hkv, self.D, self.dtype = page, Hkv, D, dtype
        pages = first + sum(need) + spare
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), width or max(1, max(need, default=1))), -7, dtype=torch.int32)
        self.k = torch.full((pages, Hkv, page, D), math.nan, dtype=dtype)
        self.v = self.k.clone()
        at = first
        self.prefix_table = order[:first].clone()
        rows = [(self.prefix_table, prefix)]
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            rows.append((self.table[b], lens[b]))
            at += n
        for table, n in rows:
            for i in range(0, n, page):
                m = min(page, n - i)
                for c in (self.k, self.v):
                    c[int(table[i // page]), :, :m] = torch.randn((Hkv, m, D), generator=g).to(dtype)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.g = g
        self.slots_first = slots_first

    def gpu(self):
        def put(c):
            # [pages, slots, Hkv, D] in memory, seen as [pages, Hkv, slots, D]
            return c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.slots_first else c.cuda()
        return fa.PagedKV(put(self.k), put(self.v), self.table.cuda(), self.lens.cuda())

    def queries(self, Hq, T):
        return torch.randn((len(self.lens), Hq, T, self.D), generator=self.g).to(self.dtype)


def run_paged(pool, Hq, T, causal=True, scale=None, prefix=0, q=None):
    q = pool.queries(Hq, T) if q is None else q
    cache = pool.gpu()
    if prefix:
        o, lse = fa.forward_shared_prefix(q.cuda(), cache, pool.prefix_table.cuda(), prefix, causal=causal, scale=scale)
    else:
        o, lse = fa.forward_paged(q.cuda(), cache, causal=causal, scale=scale)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    want = ref.attention(q, pool.k, pool.v, pool.table, pool.lens, causal, scale, pool.prefix_table, prefix)
    ref.check_attention(o, lse, want, prefix + int(max(pool.lens.max(), 0)), pool.dtype)
    return q, cache, o, lse


CASES = [
    # lens, Hkv, group, T, D, page, dtype
    ([1], 1, 1, 1, 64, 16, BF16),
    ([0], 2, 2, 1, 128, 16, BF16),
    ([0, 5, 0, 130, 64, 0], 2, 4, 1, 128, 16, BF16),
    ([63, 64, 65, 127, 128, 129], 1, 8, 1, 64, 8, F16),
    ([1000], 2, 4, 1, 128, 16, BF16),
    ([300, 7], 1, 3, 1, 40, 24, BF16),
    ([257, 1, 100], 2, 7, 1, 80, 1, F16),
    ([333], 1, 1, 1, 8, 7, BF16),
    ([200, 77], 2, 5, 1, 96, 100, BF16),
    ([500, 31], 2, 2, 1, 256, 16, BF16),
    ([150], 1, 16, 1, 256, 64, F16),
    # several query tokens: more than the sequence has, tiles of 16, 32 and more rows
    ([3, 0, 40], 2, 4, 5, 64, 16, BF16),
    ([100, 2], 1, 8, 4, 128, 8, F16),
    ([90], 2, 3, 33, 128, 12, BF16),
    ([200, 65], 1, 2, 65, 64, 100, F16),
    ([130], 1, 4, 20, 256, 16, BF16),
    # more rows than the row kernel takes, pages that copy tiles
    ([300, 40, 0], 2, 4, 40, 128, 16, BF16),
    ([520], 1, 8, 129, 64, 64, BF16),
    ([400, 399], 1, 3, 100, 128, 24, F16),
    ([1030], 1, 1, 300, 96, 128, BF16),
    ([700], 1, 5, 64, 40, 8, F16),
    ([129, 640], 2, 1, 128, 64, 256, BF16),
]


@pytest.mark.parametrize("lens,Hkv,group,T,D,page,dtype", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_paged_matches_64_bits(lens, Hkv, group, T, D, page, dtype, causal):
    pool = Pool(lens, Hkv, D, page, dtype, seed=len(lens) * 1000 + T + D)
    run_paged(pool, Hkv * group, T, causal)


@pytest.mark.parametrize("lens,Hkv,group,T,D,page,dtype", [CASES[2], CASES[8], CASES[12], CASES[16]])
def test_slots_before_heads(lens, Hkv, group, T, D, page, dtype):
    pool = Pool(lens, Hkv, D, page, dtype, seed=5, slots_first=True)
    run_paged(pool, Hkv * group, T)


SHARED = [
    # prefix, lens, Hkv, group, T, D, page, dtype
    (1, [1, 1], 1, 1, 1, 64, 16, BF16),
    (100, [1, 0, 50], 2, 4, 1, 128, 16, BF16),
    (64, [20, 3, 1, 64], 1, 8, 2, 64, 8, F16),
    (333, [70, 9], 2, 2, 3, 96, 24, BF16),
    (129, [5] * 9, 1, 7, 1, 40, 7, F16),
    (200, [17, 2, 90], 1, 4, 4, 256, 16, BF16),
    # many stacked rows
    (700, [30, 1, 0, 8, 12, 100, 64, 65, 3, 2], 2, 8, 1, 128, 16, BF16),
    (515, [33] * 20, 1, 4, 2, 64, 64, F16),
    (260, [40] * 7, 1, 3, 13, 128, 8, BF16),
    (257, [50, 60], 2, 4, 40, 128, 32, F16),
]


@pytest.mark.parametrize("prefix,lens,Hkv,group,T,D,page,dtype", SHARED)
@pytest.mark.parametrize("causal", [True, False])
def test_shared_prefix_matches_64_bits(prefix, lens, Hkv, group, T, D, page, dtype, causal):
    pool = Pool(lens, Hkv, D, page, dtype, seed=prefix, prefix=prefix)
    run_paged(pool, Hkv * group, T, causal, prefix=prefix)


def test_scale_argument():
    pool = Pool([100, 31], 2, 64, 16, BF16, seed=3)
    run_paged(pool, 4, 1, scale=0.37)
    pool = Pool([300], 1, 64, 16, BF16, seed=4)
    run_paged(pool, 4, 40, scale=0.37)


@pytest.mark.parametrize("T", [1, 40])
def test_pages_outside_the_pool_are_hidden(T):
    pool = Pool([600, 200], 2, 64, 16, BF16, seed=9)
    pool.table[0, 3] = -1
    pool.table[0, 8:17] = 1 << 30
    pool.table[1, :] = pool.k.shape[0]              # the whole sequence
    run_paged(pool, 8, T)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_lengths_are_clamped(T):
    pool = Pool([48, 48], 1, 64, 16, BF16, seed=10)
    pool.lens = torch.tensor([1 << 30, -5], dtype=torch.int32)
    run_paged(pool, 2, T)


@pytest.mark.parametrize("T", [1, 40])
def test_large_and_one_hot_scores(T):
    """Scores of hundreds, one key dominant late in the row."""
    pool = Pool([700], 1, 64, 16, BF16, seed=11)
    q = pool.queries(4, T) * 8
    i = 690 - T
    pool.k[int(pool.table[0, i // 16]), 0, i % 16] = q[0, 0, 0] * 2
    run_paged(pool, 4, T, q=q)


@pytest.mark.parametrize("T,prefix", [(1, 0), (40, 0), (1, 100), (40, 100)])
def test_strided_tensors_and_output_bounds(T, prefix):
    pool = Pool([90, 45], 2, 64, 16, BF16, seed=12, prefix=prefix)
    B, Hq, D = 2, 8, 64
    wide = torch.randn((B, T, Hq + 3, D + 8), generator=pool.g).to(BF16)
    q = wide[:, :, 1:1 + Hq, :D].transpose(1, 2)
    cache, table = pool.gpu(), pool.prefix_table.cuda()
    args = (table, prefix) if prefix else ()
    fn = fa.forward_shared_prefix if prefix else fa.forward_paged
    want = fn(q.contiguous().cuda(), cache, *args)
    buf = torch.full((B, T, Hq + 2, D + 8), 7.0, dtype=BF16, device="cuda")
    out = buf[:, :, 1:1 + Hq, :D].transpose(1, 2)
    got = fn(wide.cuda()[:, :, 1:1 + Hq, :D].transpose(1, 2), cache, *args, out=out)
    assert got[0] is out
    assert torch.equal(out, want[0]) and torch.equal(got[1], want[1])
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[:, :, 1:1 + Hq, :D] = False
    assert (buf[keep] == 7).all()
    # an odd stride is read through a copy; a broadcast query too
    odd = torch.randn((B, Hq, T, D + 1), generator=pool.g).to(BF16).cuda()[..., :D]
    assert torch.equal(fn(odd, cache, *args)[0], fn(odd.contiguous(), cache, *args)[0])
    one = torch.randn((1, 1, T, D), generator=pool.g).to(BF16).cuda().expand(B, Hq, T, D)
    assert torch.equal(fn(one, cache, *args)[0], fn(one.contiguous(), cache, *args)[0])
    # without the LSE
    assert torch.equal(fn(q.cuda(), cache, *args, return_lse=False), want[0])


@pytest.mark.parametrize("T,prefix", [(1, 0), (40, 0), (1, 500)])
def test_repeats_are_bit_identical_and_ignore_the_workspace(T, prefix):
    pool = Pool([900, 1, 300, 64], 2, 128, 16, BF16, seed=13, prefix=prefix)
    q, cache, o, lse = run_paged(pool, 8, T, prefix=prefix)
    args = (pool.prefix_table.cuda(), prefix) if prefix else ()
    fn = fa.forward_shared_prefix if prefix else fa.forward_paged
    need = fa.fa_fwd_shared_prefix_workspace_bytes(cache.c, prefix, 4, 8, T)
    for fill in (0, 255):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        again = fn(q.cuda(), cache, *args, workspace=ws[:need])
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
        assert (ws[need:] == fill).all()


def test_another_stream():
    pool = Pool([500, 333], 2, 64, 16, BF16, seed=14)
    q, cache, o, lse = run_paged(pool, 4, 1)
    side = torch.cuda.Stream()
    qg = q.cuda()
    side.wait_stream(torch.cuda.current_stream())
    a = fa.forward_paged(qg, cache, stream=side)
    b = fa.forward_paged(qg.expand(2, 4, 1, 64), cache, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a[0], o) and torch.equal(b[0], o) and torch.equal(a[1], lse)


@pytest.mark.parametrize("T,prefix", [(1, 0), (40, 0), (1, 300)])
def test_captured_graphs_follow_lengths_and_share_a_workspace(T, prefix):
    """A replay reads seq_len and the table as they are then; two graphs may
    share a workspace when their replays are ordered."""
    pool = Pool([200, 200], 2, 64, 16, BF16, seed=15, prefix=prefix)
    cache = pool.gpu()
    q = pool.queries(4, T)
    qs = [q.cuda(), (q * 0.5).cuda()]
    args = (pool.prefix_table.cuda(), prefix) if prefix else ()
    fn = fa.forward_shared_prefix if prefix else fa.forward_paged
    ws = torch.empty(fa.fa_fwd_shared_prefix_workspace_bytes(cache.c, prefix, 2, 4, T), dtype=torch.uint8, device="cuda")
    fn(qs[0], cache, *args, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fn(x, cache, *args, workspace=ws))
    for lens in ([200, 200], [33, 0], [1, 199]):
        cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, (o, lse) in zip(qs, outs):
            want = fn(x, cache, *args)
            torch.cuda.synchronize()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------- append
def run_append(lens, Hq, Hkv, T, D, page, dtype, rot, interleaved, offset=0, slots_first=False, with_q=True, seed=1):
    pool = Pool(lens, Hkv, D, page, dtype, seed=seed, slots_first=slots_first)
    cache = pool.gpu()
    B = len(lens)
    qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=pool.g).to(dtype)
    q, k, v = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], dim=2))
    dev = qkv.cuda()
    qd, kd, vd = (x.transpose(1, 2) for x in dev.split([Hq, Hkv, Hkv], dim=2))
    freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float() if rot else None
    out = fa.kv_append(cache, kd, vd, q=qd if with_q else None, inv_freq=freq.cuda() if rot else None,
                       interleaved=interleaved, position_offset=offset)
    torch.cuda.synchronize()
    u = ref.HALF_STEP[dtype]
    freq = torch.zeros(0) if freq is None else freq

    def near(got, x, pos):
        """Half a step of the result, and 2^-21 of the pair for cos, sin and
        their products in fp32 (fp16: results below its normal range, 2^-25)."""
        want = ref.rotated(x, pos, freq, interleaved)
        pair = x.double().abs().amax() * 2
        off = (got.double().cpu() - want).abs()
        assert (off <= u * want.abs() + 2.0 ** -21 * pair + 2.0 ** -25).all(), off.max()
        assert torch.equal(got.cpu()[..., rot:], x[..., rot:])

    want_k, want_v = pool.k.clone(), pool.v.clone()
    got_k, got_v = cache.k_cache.cpu(), cache.v_cache.cpu()
    for b, n in enumerate(ref.lengths(lens, pool.table.shape[1], page)):
        t = min(T, n)
        if with_q:
            assert (out[b, :, :T - t] == 0).all()
        if t == 0:
            continue
        pos = torch.arange(n - t, n)
        if with_q:
            near(out[b, :, T - t:], q[b, :, T - t:], pos + offset)
        for i in range(t):
            j = n - t + i
            at = (int(pool.table[b, j // page]), slice(None), j % page)
            near(got_k[at][:, None], k[b, :, T - t + i][:, None], pos[i:i + 1] + offset)
            want_k[at], want_v[at] = got_k[at], v[b, :, T - t + i]
    # every value as given, every other slot as it was
    for got, want in ((got_k, want_k), (got_v, want_v)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    if not with_q:
        assert out is None


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page,rot,interleaved", [
    ([1], 1, 1, 1, 64, 16, 64, False),
    ([1000, 17, 0], 8, 2, 1, 128, 16, 128, False),
    ([40, 3, 0, 9], 4, 4, 9, 64, 8, 32, True),
    ([70], 3, 1, 70, 80, 24, 80, False),
    ([33, 5], 2, 2, 4, 40, 7, 40, False),       # pairs that split 16-byte units
    ([33, 5], 2, 2, 4, 40, 1, 20, True),
    ([33], 2, 1, 4, 96, 16, 18, False),
    ([20, 21], 2, 1, 3, 256, 100, 256, False),
    ([20], 2, 1, 2, 64, 16, 0, False),
    ([20], 2, 1, 2, 8, 16, 2, False),
])
def test_append_matches_64_bits(lens, Hq, Hkv, T, D, page, dtype, rot, interleaved):
    run_append(lens, Hq, Hkv, T, D, page, dtype, rot, interleaved)


def test_append_layouts_offsets_and_no_queries():
    run_append([50, 6], 4, 2, 8, 64, 16, BF16, 64, False, offset=977, slots_first=True)
    run_append([50, 6], 4, 2, 8, 64, 16, F16, 64, True, with_q=False)


@pytest.mark.parametrize("offset", [0, 131071, (1 << 31) + 12345, 1 << 40])
def test_append_far_positions(offset):
    """The angle of a far position against exact arithmetic: n * f is a
    rational number, reduced with a 200-bit value of 2 pi."""
    from fractions import Fraction
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    D, n = 64, offset + 4
    freq = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float()
    freq[5], freq[6], freq[7] = -0.75, 0.0, 65536.0
    pool = Pool([5], 1, D, 16, F16, seed=2)
    cache = pool.gpu()
    ones = torch.zeros((1, 1, 1, D), dtype=F16)
    ones[..., :32] = 1                              # (1, 0) turns into (cos, sin)
    out = fa.kv_append(cache, ones.cuda(), ones.cuda(), q=ones.cuda(), inv_freq=freq.cuda(), position_offset=offset)
    got = out.cpu().double()[0, 0, 0]
    for p in range(32):
        x = Fraction(float(freq[p])) * n
        x = float(x - two_pi * round(x / two_pi))
        # the fraction of a turn is good to n f 2^-61 + n 2^-64, its fp32 form to 2^-22 radians
        off = 2.0 ** -20 + 7 * n * (abs(float(freq[p])) * 2.0 ** -61 + 2.0 ** -64) + 2.0 ** -11
        assert abs(float(got[p]) - math.cos(x)) <= off and abs(float(got[32 + p]) - math.sin(x)) <= off, (p, n)


def test_append_outside_the_pool_is_dropped():
    pool = Pool([40, 20], 2, 64, 16, BF16, seed=6)
    pool.table[0, 2] = -1
    pool.table[1, 1] = pool.k.shape[0]
    cache = pool.gpu()
    x = torch.randn((2, 2, 10, 64), generator=pool.g).to(BF16).cuda()
    q = fa.kv_append(cache, x, x, q=x)
    torch.cuda.synchronize()
    assert torch.equal(q, x)
    got = cache.k_cache.cpu()
    want = pool.k.clone()
    for b, n in ((0, 40), (1, 20)):
        for i in range(10):
            j = n - 10 + i
            p = int(pool.table[b, j // 16])
            if 0 <= p < pool.k.shape[0]:
                want[p, :, j % 16] = x[b, :, i].cpu()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# --------------------------------------------------------------- run together
@pytest.mark.parametrize("D,Hkv,group,prefix", [(64, 2, 2, 0), (128, 1, 4, 0), (64, 2, 4, 37), (128, 2, 2, 150)])
def test_generation_equals_the_forward_pass(D, Hkv, group, prefix):
    """A prompt in two pieces, then tokens one by one, behind an optional
    shared prefix: append and attend, step by step, and compare with fa_fwd on
    the whole rotated sequence."""
    B, page, n = 2, 16, 150
    Hq = Hkv * group
    g = torch.Generator().manual_seed(D + prefix)
    q, k, v = (torch.randn((B, h, prefix + n, D), generator=g).to(BF16).cuda() for h in (Hq, Hkv, Hkv))
    k[1:, :, :prefix], v[1:, :, :prefix] = k[:1, :, :prefix], v[:1, :, :prefix]
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    pages = -(-prefix // page) + B * -(-n // page)
    order = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    kc, vc = (torch.full((pages, Hkv, page, D), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    first = -(-prefix // page)
    prefix_table = order[:first].contiguous()
    if prefix:
        front = fa.PagedKV(kc, vc, prefix_table[None], torch.tensor([prefix], dtype=torch.int32, device="cuda"))
        fa.kv_append(front, k[:1, :, :prefix], v[:1, :, :prefix], inv_freq=freq)
    cache = fa.PagedKV(kc, vc, order[first:].view(B, -1), torch.zeros(B, dtype=torch.int32, device="cuda"))
    outs, rotated, at = [], [], 0
    for t in [70, 50] + [1] * 25 + [3, 2]:
        cache.seq_len += t
        piece = slice(prefix + at, prefix + at + t)
        x = fa.kv_append(cache, k[:, :, piece], v[:, :, piece], q=q[:, :, piece], inv_freq=freq, position_offset=prefix)
        rotated.append(x)
        outs.append(fa.forward_shared_prefix(x, cache, prefix_table, prefix) if prefix else fa.forward_paged(x, cache))
        at += t
    assert at == n
    got = torch.cat([o for o, _ in outs], dim=2)
    got_lse = torch.cat([x for _, x in outs], dim=2)
    # the cache's own keys, row by row, as fa_fwd takes them
    def rows(c):
        own = c[cache.block_table.long()].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :n]
        pre = c[prefix_table.long()].transpose(0, 1).reshape(1, Hkv, -1, D)[:, :, :prefix].expand(B, -1, -1, -1)
        return torch.cat([pre, own], dim=2).repeat_interleave(group, dim=1)
    full_q = torch.cat([torch.zeros((B, Hq, prefix, D), dtype=BF16, device="cuda"), torch.cat(rotated, dim=2)], dim=2)
    o, lse = fa.forward(full_q, rows(kc), rows(vc), causal=True)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    # two bf16 roundings of a result, and of weights in (0, 1] times |v| < 5
    assert (got.float() - o[:, :, prefix:].float()).abs().max() <= 2e-2
    assert (got_lse - lse[:, :, prefix:]).abs().max() <= 1e-4
    # fa_fwd's own 64-bit comparison holds for the same rows
    table = torch.cat([prefix_table.expand(B, -1), cache.block_table], dim=1) if prefix % page == 0 else None
    if table is not None and prefix:
        whole = fa.PagedKV(kc, vc, table.contiguous(), torch.full((B,), prefix + n, dtype=torch.int32, device="cuda"))
        assert (fa.forward_paged(full_q[:, :, -1:], whole)[0].float() - got[:, :, -1:].float()).abs().max() <= 2e-2


def test_empty_calls():
    pool = Pool([10, 3], 2, 64, 16, BF16, seed=20)
    cache = pool.gpu()
    q = torch.empty((2, 4, 0, 64), dtype=BF16, device="cuda")
    o, lse = fa.forward_paged(q, cache)
    assert o.shape == q.shape and lse.shape == (2, 4, 0)
    kv = torch.empty((2, 2, 0, 64), dtype=BF16, device="cuda")
    assert fa.kv_append(cache, kv, kv, q=q).shape == q.shape
    # a table of no pages: every query sees nothing
    none = fa.PagedKV(cache.k_cache, cache.v_cache, torch.empty((2, 0), dtype=torch.int32, device="cuda"), cache.seq_len)
    o, lse = fa.forward_paged(pool.queries(4, 1).cuda(), none)
    assert (o == 0).all() and torch.isneginf(lse).all()
