"""assign_step_pages without sequences: an empty step, whatever an earlier one left."""
import pytest
import torch

from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def empty_step(stack, free, in_place=False, stream=None):
    n = i32([free])
    out = n if in_place else i32([77])
    qi, err = i32([5, 6]), i32([0])
    slots, positions = (torch.full((9,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    none, table = i32([]), torch.empty(0, 4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pkv.assign_step_pages(none, none, n, stack, table, kv_lens_out=none, num_free_out=out, q_indptr=qi, slots=slots,
                          positions=positions, err=err, stream=stream)
    torch.cuda.synchronize()
    assert slots.tolist() == [-1] * 9 and positions.tolist() == [0] * 9 and qi.tolist() == [0, 6]
    return int(out), int(err)


@pytest.mark.parametrize("in_place", [False, True])
def test_outputs_of_an_empty_batch(in_place):
    stack = i32([3, 4, 5, 9])
    assert empty_step(stack, 3, in_place=in_place) == (3, 0)
    assert empty_step(stack, 7, in_place=in_place) == (4, pkv.PKV_ERRBIT_PAGE)
    assert empty_step(stack, -2, in_place=in_place) == (0, pkv.PKV_ERRBIT_PAGE)
    assert empty_step(i32([]), 0, in_place=in_place) == (0, 0)
    assert stack.tolist() == [3, 4, 5, 9]


def test_on_other_streams():
    s = torch.cuda.Stream()
    assert empty_step(i32([3]), 1, stream=s) == (1, 0)
    assert empty_step(i32([3]), 1, stream=s.cuda_stream) == (1, 0)


def test_default_stream_by_its_number():
    """Stream 0 is the default stream, in order with what runs there."""
    none, n, out, qi, table = i32([]), i32([2]), i32([77]), i32([5]), torch.empty(0, 4, dtype=torch.int32, device="cuda")
    stack = i32([3, 4, 5])
    slots, positions = (torch.zeros(9, dtype=torch.int64, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.default_stream()):
        torch.cuda._sleep(50_000_000)
        slots.fill_(77)
    pkv.assign_step_pages(none, none, n, stack, table, kv_lens_out=none, num_free_out=out, q_indptr=qi, slots=slots,
                          positions=positions, stream=0)
    torch.cuda.synchronize()
    assert slots.tolist() == [-1] * 9 and int(out) == 2


def test_captured():
    none, n, qi = i32([]), i32([2]), i32([5])
    slots, positions = (torch.full((3,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    out, err, stack, table = i32([77]), i32([0]), i32([3, 4, 5]), torch.empty(0, 4, dtype=torch.int32, device="cuda")

    def step():
        pkv.assign_step_pages(none, none, n, stack, table, kv_lens_out=none, num_free_out=out, q_indptr=qi, slots=slots,
                              positions=positions, err=err)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    n.fill_(1)
    slots.fill_(77)
    graph.replay()
    torch.cuda.synchronize()
    assert slots.tolist() == [-1] * 3 and int(out) == 1 and int(err) == 0 and qi.tolist() == [0]


def test_rows_of_an_earlier_step_stay():
    """The append behind an empty step writes nothing."""
    pool = torch.zeros(2, 32, 576, dtype=torch.bfloat16, device="cuda")
    table, stack, kv, n, qi = i32([[-1, -1]]), i32([0, 1]), i32([0]), i32([2]), i32([0, 0])
    slots, positions = (torch.zeros(8, dtype=torch.int64, device="cuda") for _ in range(2))
    ang = torch.zeros(64, 64, device="cuda")
    ang[:, :32] = 1.0
    rows = torch.ones(8, 576, dtype=torch.bfloat16, device="cuda")
    pkv.assign_step_pages(i32([8]), kv, n, stack, table, kv_lens_out=kv, num_free_out=n, q_indptr=qi, slots=slots,
                          positions=positions)
    pkv.kv_append_latent(rows, positions, ang, slots, pool)
    assert int(pool.sum()) == 8 * 576
    none = i32([])
    pkv.assign_step_pages(none, none, n, stack, table, kv_lens_out=none, num_free_out=n, q_indptr=qi, slots=slots,
                          positions=positions)
    pkv.kv_append_latent(rows * 5, positions, ang, slots, pool)
    assert int(pool.sum()) == 8 * 576 and int(n) == 1
