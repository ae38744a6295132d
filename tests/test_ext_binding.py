"""What the binding refuses of the tensors given to kv_append_fp8,
paged_attention_fp8 and paged_attention_window, and what it takes of them, on
the host: nothing reaches a GPU."""
import pytest
import torch

from paged_kv_cache_189_gb300 import pkv

H, D, N = 8, 64, 6


@pytest.mark.parametrize("scales,stride", [
    (torch.ones(N, H), H),
    (torch.ones(N, H + 3)[:, :H], H + 3),             # rows further apart
    (torch.ones(2 * N, H)[::2], 2 * H),
    (torch.ones(N, 1), 1),                            # one head
    (torch.ones(N, 3)[:, :1], 3),
    (torch.ones(N, H)[3:4], H),                       # one page: its stride is not used
    (torch.ones(1, H).as_strided((1, H), (0, 1)), H),
    (torch.ones(1, 1).as_strided((1, 1), (0, 0)), 1),
    (torch.ones(0, H), H)])
def test_scale_strides(scales, stride):
    assert pkv._scales(scales, scales, *scales.shape) == stride


@pytest.mark.parametrize("scales", [
    torch.ones(1, H).expand(N, H),                    # one scale a head, for all pages: 8 floats of storage
    torch.ones(1, 1).expand(N, 1),                    # one scale
    torch.ones(N + H).as_strided((N, H), (1, 1)),     # overlapping rows
    torch.ones(N * H).as_strided((N, H), (H - 1, 1)),
    torch.ones(N, 1).expand(N, H),                    # one scale a page: no unit head stride
    torch.ones(H, N).t()])
def test_scales_that_reach_past_their_storage(scales):
    """Pages that share a stride below the heads would have the kernels read,
    and the append write, past the tensor."""
    with pytest.raises(ValueError):
        pkv._scales(scales, scales, *scales.shape)


def args(op, **kw):
    """A call whose tensors fit but for `kw`, and for not being on a GPU."""
    pool = torch.zeros(N, 32, H, D, dtype=torch.bfloat16 if op == "window" else torch.uint8)
    one = torch.ones(1, dtype=torch.int32)
    a = dict(block_table=torch.zeros(1, 1, dtype=torch.int32), kv_lens=one, q_indptr=torch.tensor([0, 1]).int(),
             k_pool=pool, v_pool=pool, max_q_rows=1, max_kv_len=1)
    if op != "window":
        a.update(k_scale=torch.ones(N, H), v_scale=torch.ones(N, H))
    if op == "append":
        a.update(k_src=torch.zeros(1, H, D), v_src=torch.zeros(1, H, D))
    else:
        a.update(q=torch.zeros(1, 2 * H, D, dtype=torch.bfloat16), out=torch.zeros(1, 2 * H, D))
    if op == "window":
        a.update(window=4)
    a.update(kw)
    return a


CALL = {"append": pkv.kv_append_fp8, "fp8": pkv.paged_attention_fp8, "window": pkv.paged_attention_window}


@pytest.mark.parametrize("op", CALL)
def test_tensors_that_fit(op):
    """The calls below are refused for what they change: this one only for its device."""
    with pytest.raises(ValueError, match="CUDA device"):
        CALL[op](**args(op))


@pytest.mark.parametrize("dtype", [torch.float64, torch.int32, torch.uint8])
@pytest.mark.parametrize("op", ["fp8", "window"])
def test_output_types(op, dtype):
    with pytest.raises(ValueError, match="out must be"):
        CALL[op](**args(op, out=torch.zeros(1, 2 * H, D).to(dtype)))


@pytest.mark.parametrize("mask", ["Causal", "", None, 1])
def test_mask_names(mask):
    with pytest.raises(ValueError, match="one of none, causal, block_causal"):
        CALL["fp8"](**args("fp8", mask=mask))


@pytest.mark.parametrize("op", ["fp8", "window"])
def test_workspaces_that_reach_past_their_storage(op):
    """An expanded tensor counts more bytes than it has."""
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            CALL[op](**args(op, workspace=ws))


@pytest.mark.parametrize("op", CALL)
@pytest.mark.parametrize("err", [torch.zeros(1, dtype=torch.uint8), torch.zeros(1), torch.zeros(0, dtype=torch.int32)])
def test_error_flags(op, err):
    with pytest.raises(ValueError, match="err"):
        CALL[op](**args(op, err=err))
