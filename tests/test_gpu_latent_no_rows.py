"""A step in which no sequence has a query row: nothing to do, not an error."""
import pytest
import torch

from latent_testutil import L, NOPE, P, R, V
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("flags", [pkv.PKV_FLAG_SIMT_ONLY, 0])
@pytest.mark.parametrize("most", [0, 1, 4])
def test_no_rows(most, flags):
    H, n = 16, 70
    bf = dict(dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    lens, lse = torch.full((2,), n, dtype=torch.int32, device=DEV), torch.empty(0, H, device=DEV)
    table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(256, pkv.paged_attention_latent_workspace_size(2, max(most, 1), H, n)), dtype=torch.uint8, device=DEV)
    pkv.paged_attention_latent(torch.zeros(0, H, L + R, **bf), torch.zeros(1, P, L + R, **bf), table, lens, zero,
                               torch.empty(0, H, L, **bf), lse=lse, max_q_rows=most, max_kv_len=n, scale=0.1, workspace=ws,
                               flags=flags)
    pkv.ragged_attention_latent(torch.zeros(0, H, NOPE + R, **bf), torch.zeros(n, H, NOPE, **bf), torch.zeros(n, R, **bf),
                                torch.zeros(n, H, V, **bf), zero, zero, torch.empty(0, H, V, **bf), lse=lse, max_q_rows=most,
                                max_kv_len=n, scale=0.1, flags=flags)
    torch.cuda.synchronize()
