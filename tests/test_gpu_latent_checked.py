"""Checked mode reports lengths beyond the bounds of sequences that have no
query row in the call, in either kernel of either form."""
import pytest
import torch

from latent_testutil import L, NOPE, P, R, V
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("flags", [pkv.PKV_FLAG_SIMT_ONLY, 0])
@pytest.mark.parametrize("kv,bad", [([40, 33], False), ([40, 65], True), ([40, -1], True), ([65, 33], True)])
@pytest.mark.parametrize("H", [16, 128])
def test_absorbed(kv, bad, H, flags):
    q = torch.zeros(1, H, L + R, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(4, P, L + R, dtype=torch.bfloat16, device=DEV)
    out, err = torch.empty(1, H, L, device=DEV), i32([0])
    ws = torch.empty(max(256, pkv.paged_attention_latent_workspace_size(2, 1, H, 64)), dtype=torch.uint8, device=DEV)
    pkv.paged_attention_latent(q, pool, i32([[0, 1], [2, 3]]), i32(kv), i32([0, 1, 1]), out, max_q_rows=1, max_kv_len=64,
                               scale=0.1, workspace=ws, flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
    assert int(err) == (pkv.PKV_ERRBIT_LEN if bad else 0)


@pytest.mark.parametrize("flags", [pkv.PKV_FLAG_SIMT_ONLY, 0])
@pytest.mark.parametrize("ends,bad", [([0, 40, 90], False), ([0, 40, 105], True), ([0, 40, 39], True), ([0, 65, 70], True)])
def test_expanded(ends, bad, flags):
    H, n = 2, 110
    bf = dict(dtype=torch.bfloat16, device=DEV)
    out, err = torch.empty(1, H, V, device=DEV), i32([0])
    pkv.ragged_attention_latent(torch.zeros(1, H, NOPE + R, **bf), torch.zeros(n, H, NOPE, **bf), torch.zeros(n, R, **bf),
                                torch.zeros(n, H, V, **bf), i32([0, 1, 1]), i32(ends), out, max_q_rows=1, max_kv_len=64, scale=0.1,
                                flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
    assert int(err) == (pkv.PKV_ERRBIT_LEN if bad else 0)
