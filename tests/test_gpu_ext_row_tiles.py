"""The few-row kernel's cut line of keys (planner, pieces, partial states, join)
in all its forms: row tiles of 8 and 16, heads of 64 and 128, both pools, few
long units and more units than CTAs; and the tile kernel with split keys."""
import pytest
import torch

from ext_testutil import Case, call, check
from paged_kv_cache_189_gb300 import pkv
from test_gpu_ext_attention import ragged
from test_gpu_ext_nan import states_bytes

pytestmark = pytest.mark.gpu


def pairs(c):
    return c.max_rows() * c.Hq // c.Hkv


def hold(c, repeats=2):
    """Against the definition, and the same bits every time."""
    t, ref = c.on("cuda"), c.reference()
    first = None
    for _ in range(repeats):
        out = torch.full((sum(c.rows), c.Hq, c.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((sum(c.rows), c.Hq), float("nan"), device="cuda")
        call(c, t, out, lse)
        torch.cuda.synchronize()
        if first is None:
            check(c, out, lse, ref)
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def make(fp8, batch, new, kv, Hq, Hkv, D, window, pad, seed):
    lens, real, rows = ragged(seed, batch, new, kv, pad)
    lens[0], real[0], rows[0] = kv[1], new[1], new[1] + pad  # the largest there is
    return Case(lens, real, rows, Hq, Hkv, D, fp8, window=window, sinks=9 if window else 0, seed=seed)


@pytest.mark.parametrize("fp8,new,pad,Hq,Hkv,D,window", [
    (False, (1, 1), 0, 8, 2, 128, 3000), (False, (1, 1), 0, 8, 1, 64, 3000),      # 4 and 8 pairs: tiles of 8
    (False, (3, 4), 0, 8, 2, 128, 3000), (False, (2, 3), 1, 8, 2, 64, 3000),      # 16: tiles of 16
    (False, (9, 13), 2, 2, 2, 128, 3000), (False, (1, 1), 0, 32, 2, 64, 4000),    # 15 of one head, 16 heads
    (True, (1, 1), 0, 8, 2, 128, 0), (True, (1, 1), 0, 16, 2, 64, 0),
    (True, (3, 4), 0, 8, 2, 64, 0), (True, (2, 3), 1, 8, 2, 128, 4000),
    (True, (5, 12), 2, 8, 2, 128, 0), (True, (17, 20), 0, 8, 2, 128, 0), (True, (17, 20), 0, 8, 2, 64, 4000),
    (True, (6, 10), 0, 48, 6, 64, 0), (True, (40, 80), 0, 2, 2, 128, 0)])
def test_few_long_units(fp8, new, pad, Hq, Hkv, D, window):
    c = make(fp8, 5, new, (3300, 6000), Hq, Hkv, D, window, pad, 80)
    assert pairs(c) <= (80 if fp8 else 16) and states_bytes(c) > 0  # the few-row kernel, its keys cut
    hold(c)


@pytest.mark.parametrize("fp8,new,Hq,Hkv,D,window", [
    (False, (2, 4), 8, 2, 128, 1500), (False, (2, 4), 8, 2, 64, 2500), (False, (1, 1), 8, 2, 64, 2500),
    (True, (2, 4), 8, 2, 64, 0), (True, (2, 4), 8, 2, 128, 2500), (True, (17, 20), 4, 1, 128, 0)])
def test_more_units_than_ctas_by_ticket(fp8, new, Hq, Hkv, D, window):
    """Part of the keys is taken by ticket: the same bits whoever takes which."""
    batch = 240 if new[1] < 17 else 64
    c = make(fp8, batch, new, (1, 3600), Hq, Hkv, D, window, 0, 81)
    assert pairs(c) <= (80 if fp8 else 16) and states_bytes(c) > 0
    hold(c, 4)


@pytest.mark.parametrize("fp8,new,pad,window", [(True, (20, 22), 2, 0), (True, (60, 90), 3, 3000),
                                                (False, (4, 5), 2, 3000), (False, (60, 90), 3, 5000)])
def test_tile_kernel_with_split_keys(fp8, new, pad, window):
    c = make(fp8, 3, new, (4000, 7000), 8, 2, 128, window, pad, 82)
    assert pairs(c) > (80 if fp8 else 16)
    t = c.on("cuda")
    if not (fp8 and window):  # (of an 8-bit window the pages counted here are not all expanded)
        assert states_bytes(c) > 0
    hold(c)
