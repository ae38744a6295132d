"""One workspace of paged_attention_latent, sized once for the largest step,
serves the smaller steps that a draining server makes."""
import numpy as np
import pytest
import torch

from latent_testutil import Case, L, compare
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,H,keys,steps", [
    (128, 16, 1024, [128, 64, 7, 1]),       # one to a CTA, then shares and a join
    (70, 128, 512, [70, 30, 2]),            # pairs
    (20, 65, 3000, [20, 1])])
def test_sized_for_the_largest_step(most, H, keys, steps):
    ws = torch.full((pkv.paged_attention_latent_workspace_size(most, 1, H, keys),), 255, dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    for n in steps:
        kv = [int(x) for x in np.random.default_rng(n).integers(keys // 2, keys + 1, n)]
        c = Case(kv, [1] * n, [1] * n, H, seed=n)
        T = c.q_full.shape[0]
        table = np.full((n, keys // 32 + 1), 1 << 29, dtype=np.int32)
        table[:, :c.table.shape[1]] = c.table[:, :table.shape[1]]
        out = torch.full((T, H, L), 7.0, dtype=torch.float32, device="cuda")
        lse = torch.full((T, H), 9.0, device="cuda")
        pkv.paged_attention_latent(c.q_full.cuda(), c.pool.cuda(), i32(table), i32(kv), i32(c.indptr), out, lse=lse,
                                   max_q_rows=1, max_kv_len=keys, scale=c.scale, workspace=ws)
        want, wl, tol_o, tol_l = c.expected()
        compare(out.cpu(), lse.cpu(), want, wl, tol_o, tol_l, torch.float32)
