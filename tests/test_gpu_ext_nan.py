"""A NaN score makes its own row NaN, output and LSE, and no other, whichever
kernel runs and however its keys are split."""
import numpy as np
import pytest
import torch

from ext_testutil import P, Case, call, check
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


def states_bytes(c):
    """Workspace beyond the pages an 8-bit call expands: partial states of split keys."""
    size = pkv.paged_attention_fp8_workspace_size if c.fp8 else pkv.paged_attention_window_workspace_size
    n = size(len(c.kv), c.max_rows(), c.Hq, c.Hkv, c.D, c.max_kv(), c.window, c.sinks)
    if c.fp8 and c.max_rows() * c.Hq // c.Hkv > 80:
        n -= 2 * (len(c.kv) * ((c.max_kv() + P - 1) // P) * P * c.Hkv * c.D * 2)
    return n


def outputs(c, t, flags=0):
    out = torch.empty(sum(c.rows), c.Hq, c.D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(sum(c.rows), c.Hq, device="cuda")
    call(c, t, out, lse, flags=flags)
    torch.cuda.synchronize()
    return out, lse


def hold(c, out, lse, ref, nan):
    """NaN exactly where `nan` [rows, heads] says; the rest as the definition has it."""
    nan = torch.from_numpy(nan).cuda()
    assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()
    out[nan] = torch.from_numpy(ref[0]).to(out)[nan]
    lse[nan] = torch.from_numpy(ref[1]).to(lse)[nan]
    check(c, out, lse, ref)


def case(fp8, new, seed):
    kv = [5200, 6100]
    return Case(kv, [new, new], [new, new], 8, 2, 128, fp8, window=0 if fp8 else 5000, sinks=0 if fp8 else 4, seed=seed)


@pytest.mark.parametrize("flags", [0, pkv.PKV_FLAG_SIMT_ONLY])
@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("fp8", [True, False])
def test_nan_query_over_split_keys(fp8, new, flags):
    """Every split's state of the row is NaN."""
    c = case(fp8, new, 50)
    if flags == 0:
        assert states_bytes(c) > 0, "the keys are not split"
    ref = c.reference()
    t = c.on("cuda")
    nan = np.zeros((2 * new, 8), dtype=bool)
    for r, h in ((0, 3), (2 * new - 1, 6)):
        t["q"][r, h, 5] = float("nan")
        nan[r, h] = True
    hold(c, *outputs(c, t, flags), ref, nan)


@pytest.mark.parametrize("flags", [0, pkv.PKV_FLAG_SIMT_ONLY])
@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("fp8", [True, False])
def test_nan_key_over_split_keys(fp8, new, flags):
    """One split's state of the row is NaN: one key of one head, which the last
    rows of a windowed sequence no longer see."""
    c = case(fp8, new, 51)
    ref = c.reference()
    t = c.on("cuda")
    j = 6100 - new - 4999 + new // 2 if not fp8 else 3000  # the window of row new / 2 starts there
    page, slot = int(c.table[1, j // P]), j % P
    t["k_pool"].view(torch.uint8 if fp8 else torch.int16)[page, slot, 1, 7] = 0x7f if fp8 else 0x7fc0
    nan = np.zeros((2 * new, 8), dtype=bool)
    for i in range(new):
        nan[new + i, 4:] = j in c.row_keys(1, i)
    assert nan.any()
    hold(c, *outputs(c, t, flags), ref, nan)
