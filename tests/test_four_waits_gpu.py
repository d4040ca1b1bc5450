"""Waits of the 4-bit cache's kernels that run out end the kernel with a status, and the
CUDA context stays usable; workspaces of exactly the size that is asked for."""
import json
import os
import subprocess
import sys

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import four_reference as ref
import paged_reference

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16

CHILD = r"""
import json, sys
sys.path.insert(0, sys.argv[2])
import torch
import exact_tiled_attention_23_gb300 as fa

T, keys, B = int(sys.argv[1]), 16384, 32
pages = B * keys // 32
k, v = (torch.zeros((pages, 8, 32, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
ks, vs = (torch.zeros((pages, 8, 32, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
table = torch.randperm(pages, device="cuda").to(torch.int32).view(B, -1)
cache = fa.PagedKV4(k, v, ks, vs, table, torch.full((B,), keys, dtype=torch.int32, device="cuda"))
q = torch.ones((B, 32, T, 128), dtype=torch.bfloat16, device="cuda")
a, b = (torch.empty(1 << 29, device="cuda", dtype=torch.bfloat16) for _ in range(2))
torch.cuda.synchronize()
with torch.cuda.stream(torch.cuda.Stream()):
    for _ in range(60):
        b.copy_(a)
for _ in range(5):
    fa.forward_paged(q, cache)
torch.cuda.synchronize()
status = fa.fa_device_status(None)
detail = fa.fa_last_error_detail()
total = torch.ones(1 << 20, device="cuda").sum().item()
print(json.dumps({"status": status, "detail": detail, "sum": total, "status_after": fa.fa_device_status(None)}))
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


@pytest.mark.parametrize("T", [40], ids=["tensor_cores"])
def test_a_wait_that_runs_out_reports_a_timeout(T):
    """The budget is 0.2 us.  A probe of a barrier may itself be suspended for some
    microseconds, so what runs out is a wait well above that, for a tile of queries or
    products while another stream's copies compete.  (The row kernel's copies are too
    small for it: a hundred calls of one token did not.)"""
    env = dict(os.environ, FA_WAIT_LIMIT_MS="0.0002")
    run = subprocess.run([sys.executable, "-c", CHILD, str(T), ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-2000:]
    result = json.loads(run.stdout.strip().splitlines()[-1])
    assert result["status"] == fa.FA_ERR_TIMEOUT and result["detail"] & 1, result
    assert result["sum"] == float(1 << 20) and result["status_after"] == 0, result


def cache_of(lens, Hkv, page, D, width, seed):
    """A PagedKV4 whose table rows are `width` entries long, and what it holds."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    x = torch.randn((2, pages, Hkv, page, D), generator=g, dtype=torch.float64)
    packed = [ref.pack(torch.nn.functional.pad(y, (0, ref.padded(D) - D))) for y in x]
    held = [ref.unpack(*y)[..., :D] for y in packed]
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    cache = fa.PagedKV4(packed[0][0].cuda(), packed[1][0].cuda(), packed[0][1].cuda(), packed[1][1].cuda(), table.cuda(),
                        torch.tensor(lens, dtype=torch.int32).cuda(), D=D)
    return cache, held, table, g


@pytest.mark.parametrize("T,width", [(1, 4), (1, 2000), (3, 40), (20, 40), (150, 40), (150, 6000)])
def test_the_workspace_is_as_large_as_asked_for(T, width):
    """Small and large calls, decoded by themselves or first (150 tokens of 4 heads; behind
    rows of 6000 pages a few sequences at a time): nothing is written behind the
    workspace, and the answer is right."""
    lens = [30, 0, 50, 64, 3]
    cache, held, table, g = cache_of(lens, 2, 16, 128, width, T)
    q = torch.randn((len(lens), 8, T, 128), generator=g).to(BF16)
    need = cache.workspace_bytes(8, T)
    assert need > 0
    if (T, width) == (150, 6000):
        assert need < 5 * 6000 * 16 * 2 * 128 * 4            # not all sequences' rows at once
    space = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    o, lse = fa.forward_paged(q.cuda(), cache, workspace=space[:need])
    assert bool((space[need:] == 171).all())
    want = paged_reference.attention(q, *held, table, lens)
    if 4 * T > 32:
        paged_reference.check_attention(o, lse, want, max(lens), BF16)
    else:
        ref.check_rows(o, lse, want, max(lens), BF16, 128)
    assert fa.fa_device_status(None) == fa.FA_OK
    with pytest.raises(fa.FAError):
        fa.forward_paged(q.cuda(), cache, workspace=space[:need - 1])
