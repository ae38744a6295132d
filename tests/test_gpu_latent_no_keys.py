"""paged_attention_latent before anything is cached: max_kv_len 0, tables
without columns, pools without pages, no workspace."""
import pytest
import torch

from latent_testutil import L, P, R
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("flags", [pkv.PKV_FLAG_SIMT_ONLY, 0])
@pytest.mark.parametrize("pages,width", [(0, 0), (3, 2), (3, 0), (0, 2)])
@pytest.mark.parametrize("B,rows,H", [(1, 1, 1), (2, 3, 16), (300, 1, 100)])
def test_no_cached_prefix(B, rows, H, pages, width, flags):
    T = B * rows + 2
    q = torch.full((T, H, L + R), float("nan"), dtype=torch.bfloat16, device=DEV)
    pool = torch.full((pages, P, L + R), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    qi = torch.arange(0, B * rows + 1, rows, dtype=torch.int32, device=DEV)
    kv = torch.zeros(B, dtype=torch.int32, device=DEV)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((T, H, L), 7.0, dtype=dtype, device=DEV)
        lse, err = torch.full((T, H), 9.0, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        pkv.paged_attention_latent(q, pool, table, kv, qi, out, lse=lse, max_q_rows=rows, max_kv_len=0, scale=0.1,
                                   flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
        assert int(err) == 0
        assert (out[:-2] == 0).all() and torch.isneginf(lse[:-2]).all()
        assert (out[-2:] == 7).all() and (lse[-2:] == 9).all()
