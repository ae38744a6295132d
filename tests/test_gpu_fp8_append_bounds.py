"""kv_append_fp8 under the widest bounds it takes."""
import numpy as np
import pytest
import torch

from paged_kv_cache_189_gb300 import pkv
from test_gpu_fp8_append import Cache

pytestmark = pytest.mark.gpu

WIDEST = 0x7fffff00  # the largest key bound


@pytest.mark.parametrize("rows_bound", [2 ** 31 - 1, 2 ** 30 + 77])
@pytest.mark.parametrize("kv,real", [([1000, 33, 0], [40, 33, 0]), ([31, 5, 2050], [1, 9, 3])])
def test_both_bounds_near_their_largest(rows_bound, kv, real):
    """More pages after a sequence's first one than 2^31 positions hold: the
    positions past it must not wrap.  (A table as wide as the bound: 268 MB a
    sequence, its entries past the last key -1.)"""
    H, D, pages = 1, 64, 70
    c = Cache(pages, H, D, seed=11)
    g = np.random.default_rng(12)
    table = torch.full((len(kv), WIDEST // 32), -1, dtype=torch.int32, device="cuda")
    used = g.permutation(pages).astype(np.int32)
    at, host = 0, np.full((len(kv), 70), -1, dtype=np.int32)
    for b, k in enumerate(kv):
        n = (k + 31) // 32
        host[b, :n] = used[at:at + n]
        at += n
    assert at <= pages
    table[:, :70] = torch.from_numpy(host).cuda()
    indptr = np.concatenate([[0], np.cumsum(real)])
    src = [torch.from_numpy(g.standard_normal((int(indptr[-1]), H, D))).to(torch.bfloat16) for _ in "kv"]
    pkv.kv_append_fp8(src[0].cuda(), src[1].cuda(), table, torch.tensor(kv, dtype=torch.int32, device="cuda"),
                      torch.tensor(indptr, dtype=torch.int32, device="cuda"), c.pools[0], c.pools[1],
                      c.dev_scales[0], c.dev_scales[1], max_q_rows=rows_bound, max_kv_len=WIDEST)
    torch.cuda.synchronize()
    c.append(src, host, kv, real, indptr, WIDEST, float(torch.finfo(torch.bfloat16).max))
    c.same()
