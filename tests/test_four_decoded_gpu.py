"""The 4-bit cache where more than 512 query rows share a key, so that the keys are decoded
into pages of the workspace first: what those pages do not get, behind a sequence's last
key and where a page is not there, may hold anything."""
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


def made(lens, Hkv, page, D, dtype, seed):
    """A cache with random rows, and what they stand for."""
    g = torch.Generator().manual_seed(seed)
    need = [math.ceil(max(n, 0) / page) for n in lens]
    pages, at = sum(need) + 2, 0
    order, table = torch.randperm(pages, generator=g).to(torch.int32), torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    data, held = [], []
    for _ in range(2):
        x = torch.randn((pages, Hkv, page, D), generator=g, dtype=torch.float64)
        rows, code = ref.pack(torch.nn.functional.pad(x, (0, ref.padded(D) - D)))
        data.append((rows, code))
        held.append(ref.unpack(rows, code)[..., :D])
    pools = [data[0][0], data[1][0], data[0][1], data[1][1]]
    cache = fa.PagedKV4(*(x.cuda() for x in pools), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), D=D, dtype=dtype)
    return cache, held, table, g


def forward(q, cache, causal, fill):
    """Over a workspace full of a byte (255: not numbers in either type)."""
    workspace = torch.full((cache.workspace_bytes(q.shape[1], q.shape[2]),), fill, dtype=torch.uint8, device="cuda")
    o, lse = fa.forward_paged(q, cache, causal=causal, workspace=workspace)
    assert fa.fa_device_status(None) == fa.FA_OK
    return o, lse


CASES = [  # lengths that end inside a page, inside 8 rows, on both, and none at all
    ([37, 16, 150, 0], 4, 1, 130, 64, 16, True), ([61, 301, 8], 5, 1, 103, 128, 24, True), ([129, 5], 12, 2, 86, 40, 8, False),
    ([250, 127], 4, 1, 129, 128, 128, True)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page,causal", CASES)
def test_what_the_workspace_held_does_not_matter(lens, Hq, Hkv, T, D, page, causal, dtype):
    assert T * Hq // Hkv > 512
    cache, held, table, g = made(lens, Hkv, page, D, dtype, seed=T)
    q = torch.randn((len(lens), Hq, T, D), generator=g).to(dtype)
    o, lse = forward(q.cuda(), cache, causal, 255)
    paged_reference.check_attention(o, lse, paged_reference.attention(q, *held, table, lens, causal=causal), max(lens), dtype)
    o2, lse2 = forward(q.cuda(), cache, causal, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # bytes that are no number of the format, behind the last key and in free pages
    used = torch.zeros(cache.k_cache.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(n):
            used[table[b, i // page], i % page] = True
    for x in (cache.k_cache, cache.v_cache, cache.k_scales, cache.v_scales):
        x.transpose(1, 2)[~used.cuda()] = 255
    o2, lse2 = forward(q.cuda(), cache, causal, 255)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page", [8, 48])
def test_pages_that_are_not_there_hide_their_keys(page, dtype):
    lens = [200, 150, 97, 140]
    cache, held, table, g = made(lens, 2, page, 128, dtype, seed=page)
    table[0, 1], table[1, (150 - 1) // page], table[2], table[3, 0] = -1, 1 << 30, -1, cache.k_cache.shape[0]
    cache.block_table.copy_(table)
    q = torch.randn((4, 8, 131, 128), generator=g).to(dtype)
    o, lse = forward(q.cuda(), cache, True, 255)
    paged_reference.check_attention(o, lse, paged_reference.attention(q, *held, table, lens), max(lens), dtype)
    assert torch.isneginf(lse[2]).all()


def test_groups_of_sequences_reuse_the_pages():
    """Sequences whose keys are decoded after others' find those in the workspace."""
    lens, page = [40, 3, 70, 0, 55], 16
    g = torch.Generator().manual_seed(0)
    cache, held, table, _ = made(lens, 1, page, 128, BF16, seed=0)
    # rows of the table that take 128 MB each as 16-bit pages: two sequences at a time
    width = (128 << 20) // (page * 128 * 4)
    wide = torch.full((len(lens), width), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    long = fa.PagedKV4(cache.k_cache, cache.v_cache, cache.k_scales, cache.v_scales, wide.cuda(), cache.seq_len)
    assert long.workspace_bytes(4, 130) > 256 << 20
    q = torch.randn((len(lens), 4, 130, 128), generator=g).to(BF16).cuda()
    o, lse = forward(q, cache, True, 255)
    o2, lse2 = forward(q, long, True, 255)
    want = paged_reference.attention(q.cpu(), *held, table, lens)
    for x, y in ((o, lse), (o2, lse2)):
        paged_reference.check_attention(x, y, want, max(lens), BF16)
