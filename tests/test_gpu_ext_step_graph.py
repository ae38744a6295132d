"""A decode step as a program captures it: append to the 8-bit cache, then
attend over it, in one graph, replayed while the sequences grow."""
import numpy as np
import pytest
import torch

from ext_testutil import P, Case, check
from paged_kv_cache_189_gb300 import pkv
from test_gpu_fp8_append import TOP, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 4, 30])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1900, 5)])
@pytest.mark.parametrize("lens", [[40, 7, 200], [2970, 31, 3200]])  # whole units; the cut line, split tiles
def test_append_and_attend_in_one_graph(lens, window, sinks, new):
    Hq, Hkv, D, B, steps, bound = 8, 2, 128, 3, 5, lens[2] + 200
    g = np.random.default_rng(90)
    width = (bound + P - 1) // P
    c = Cache(B * width, Hkv, D, seed=91)
    table = g.permutation(B * width).reshape(B, width).astype(np.int32)
    kv, real = list(lens), [new] * B
    dev = dict(table=i32(table), kv=i32(kv), indptr=i32(np.arange(B + 1) * new))
    src = [torch.zeros(B * new, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    q = torch.zeros(B * new, Hq, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(B * new, Hq, device="cuda")
    n = pkv.paged_attention_fp8_workspace_size(B, new, Hq, Hkv, D, bound, window, sinks)
    assert (n > 0) == (lens[2] > 1000 or new > 20)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")

    def step():
        pkv.kv_append_fp8(src[0], src[1], dev["table"], dev["kv"], dev["indptr"], c.pools[0], c.pools[1],
                          c.dev_scales[0], c.dev_scales[1], max_q_rows=new, max_kv_len=bound)
        pkv.paged_attention_fp8(q, c.pools[0], c.pools[1], c.dev_scales[0], c.dev_scales[1], dev["table"], dev["kv"],
                                dev["indptr"], out, lse=lse, max_q_rows=new, max_kv_len=bound, window=window,
                                num_sinks=sinks, workspace=ws)

    dev["kv"].zero_()  # nothing is written or seen while the kernels load
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in range(steps):
        kv = [k + new for k in kv]
        for x in src:
            x.copy_(torch.from_numpy(g.standard_normal(tuple(x.shape)) * 2.0 ** (s % 3)))
        case = Case(kv, real, real, Hq, Hkv, D, True, window=window, sinks=sinks, seed=92 + s)
        q.copy_(case.q_full)
        dev["kv"].copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.append([x.cpu() for x in src], table, kv, real, np.arange(B + 1) * new, bound, TOP[torch.bfloat16])
        case.table = table[:, :case.table.shape[1]]
        case.num_pages = B * width
        case.k64, case.v64 = (c.codes[w] * c.scales[w][:, None, :, None] for w in range(2))
        check(case, out, lse)
    c.same()
