"""Calls over a part of a packed batch: the query ranges start behind rows of
other sequences, which are left as they were."""
import pytest
import torch

from ext_testutil import Case, call, check
from paged_kv_cache_189_gb300 import pkv
from test_gpu_ext_nan import states_bytes

pytestmark = pytest.mark.gpu


def moved(c, before):
    """The case's tensors with `before` rows of others in front of the queries."""
    t = c.on("cuda")
    front = torch.randn(before, c.Hq, c.D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    t["q"] = torch.cat([front, t["q"]])
    t["q_indptr"] = t["q_indptr"] + before
    out = torch.full((before + sum(c.rows), c.Hq, c.D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((before + sum(c.rows), c.Hq), 9.0, device="cuda")
    return t, out, lse


def hold(c, out, lse, before):
    assert (out[:before] == 9).all() and (lse[:before] == 9).all()
    check(c, out[before:], lse[before:])


@pytest.mark.parametrize("flags", [0, pkv.PKV_FLAG_SIMT_ONLY])
@pytest.mark.parametrize("before", [1, 1000])
@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("fp8", [True, False])
def test_rows_behind_others(fp8, new, before, flags):
    c = Case([5200, 6100], [new, new], [new, new], 8, 2, 128, fp8, window=0 if fp8 else 5000, sinks=0 if fp8 else 4,
             seed=60)
    if flags == 0:
        assert states_bytes(c) > 0, "the keys are not split"
    t, out, lse = moved(c, before)
    call(c, t, out, lse, flags=flags)
    torch.cuda.synchronize()
    hold(c, out, lse, before)


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("new", [5, 60, 300])
def test_rows_behind_others_without_a_window(new, splits):
    """The tile kernels of paged_attention: the same states, the same join."""
    kv = [5200, 6100]
    c = Case(kv, [new, new], [new, new], 8, 2, 128, False, window=max(kv), seed=61)
    t, out, lse = moved(c, 777)
    n = pkv.paged_attention_workspace_size(2, new, 8, 2, 128, max(kv), splits)
    assert (n > 0) == (splits > 1)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    pkv.paged_attention(t["q"], t["k_pool"], t["v_pool"], t["table"], t["kv_lens"], t["q_indptr"], out,
                        q_real=t["q_real"], lse=lse, max_q_rows=new, max_kv_len=max(kv), num_splits=splits,
                        workspace=ws)
    torch.cuda.synchronize()
    hold(c, out, lse, 777)


@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("before", [1, 1000])
def test_decode_rows_behind_others(before, Hq, Hkv, D, splits):
    """The decode kernel of paged_attention, its keys split or not."""
    kv = [5200, 6100, 33]
    c = Case(kv, [1] * 3, [1] * 3, Hq, Hkv, D, False, window=max(kv), seed=62)
    t, out, lse = moved(c, before)
    ws = torch.full((pkv.paged_attention_workspace_size(3, 1, Hq, Hkv, D, max(kv), splits),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    for _ in range(2):  # the split counts are left as they were found
        out.fill_(9)
        lse.fill_(9)
        pkv.paged_attention(t["q"], t["k_pool"], t["v_pool"], t["table"], t["kv_lens"], t["q_indptr"], out,
                            q_real=t["q_real"], lse=lse, max_q_rows=1, max_kv_len=max(kv), num_splits=splits,
                            workspace=ws)
        torch.cuda.synchronize()
        hold(c, out, lse, before)
