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
