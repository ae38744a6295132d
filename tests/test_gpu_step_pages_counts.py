"""assign_step_pages at the largest page count that it takes: a loop's counter
comes within one step of 2^31."""
import pytest
import torch

from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


def test_as_many_pages_given_back_as_counts_hold():
    """4096 sequences of 2^19 pages each have ended; the stack takes 2^31 - 256 pages and the rest is dropped."""
    batch, width, cap = 4096, 1 << 19, (1 << 31) - 256
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 20 GB of device memory")
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(batch * width, **i32).view(batch, width)
    stack = torch.full((cap,), -1, **i32)
    kv, new = torch.full((batch,), 32 * width, **i32), torch.full((batch,), -1, **i32)
    lens, free, err = torch.full((batch,), 77, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    qi = torch.full((batch + 1,), 77, **i32)
    slots, positions = (torch.full((3,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    pkv.assign_step_pages(new, kv, free, stack, table, kv_lens_out=lens, num_free_out=free, q_indptr=qi, slots=slots,
                          positions=positions, err=err)
    assert int(free) == cap and int(err) == pkv.PKV_ERRBIT_PAGE and not lens.any() and not qi.any()
    assert slots.tolist() == [-1] * 3 and positions.tolist() == [0] * 3
    for a in range(0, cap, 1 << 28):
        n = min(1 << 28, cap - a)
        assert torch.equal(stack[a:a + n], torch.arange(a, a + n, **i32))
    assert torch.equal(table.view(-1)[-1000:], torch.arange(batch * width - 1000, batch * width, **i32))
