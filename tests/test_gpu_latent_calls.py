"""Calls of the latent operators that their documentation allows beside the
usual ones: tensors broadcast along an axis, rows ahead of the first sequence,
replayed graphs of the expanded form and of the append, other streams, bounds
far above the lengths, pages that sequences share, NaN in rows that pad."""
import numpy as np
import pytest
import torch

from latent_testutil import Case, L, NOPE, P, R, Ragged, V, attend, compare
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIMT = pkv.PKV_FLAG_SIMT_ONLY


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def expanded(q, k, pe, v, qi, ki, **kw):
    out = torch.full((q.shape[0], q.shape[1], V), 7.0, device=DEV)
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    rows, keys = (max(1, int((x[1:] - x[:-1]).max())) for x in (qi, ki))
    pkv.ragged_attention_latent(q, k, pe, v, qi, ki, out, lse=lse, max_q_rows=rows, max_kv_len=keys, scale=0.07, **kw)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("T,n", [(20, 150), (200, 300)])
def test_expanded_form_of_broadcast_tensors(T, n, flags):
    """Axes of stride 0 give what copies give, bit for bit."""
    H = 4
    g = torch.Generator().manual_seed(T)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    full = [bf(T, H, NOPE + R), bf(n, H, NOPE), bf(n, R), bf(n, H, V)]
    qi, ki = i32([0, T]), i32([0, n])
    for which, axis in ((0, 0), (0, 1), (1, 0), (1, 1), (2, 0), (3, 0), (3, 1)):
        x = list(full)
        x[which] = x[which].narrow(axis, 0, 1).expand(x[which].shape)
        got = expanded(*x, qi, ki, flags=flags)
        want = expanded(*[t.contiguous() for t in x], qi, ki, flags=flags)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (which, axis)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("first", [1, 2])
def test_expanded_form_of_the_last_sequences(first, flags):
    """Index tensors that begin in the middle of q and of the keys."""
    c = Ragged([130, 40, 200], [200, 70, 260], 2, seed=first)
    c.q_lens, c.kv, c.qi, c.ki = c.q_lens[first:], c.kv[first:], c.qi[first:], c.ki[first:]
    c.check(flags)


def test_expanded_form_replayed():
    """A captured call whose lengths change between replays, on a stream of its own."""
    c = Ragged([300, 257], [400, 300], 3, seed=5)
    both = c.both.to(DEV)
    q, pe = c.q_full.to(DEV), c.k_pe.to(DEV)
    qi, ki = i32(c.qi), i32(c.ki)
    out = torch.full((q.shape[0], 3, V), 7.0, device=DEV)
    lse = torch.full((q.shape[0], 3), 9.0, device=DEV)
    err = i32([0])

    def step(stream=None):
        pkv.ragged_attention_latent(q, both[..., :NOPE], pe, both[..., NOPE:], qi, ki, out, lse=lse, max_q_rows=300,
                                    max_kv_len=400, scale=c.scale, flags=pkv.PKV_FLAG_CHECKED, err=err, stream=stream)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for ql, kv in (([300, 257], [400, 300]), ([1, 200], [1, 390]), ([0, 130], [300, 129]), ([40, 0], [0, 0])):
        c.q_lens, c.kv = ql, kv
        c.qi, c.ki = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (ql, kv))
        qi.copy_(i32(c.qi))
        ki.copy_(i32(c.ki))
        want, wl, tol_o, tol_l = c.expected()
        for run in (graph.replay, lambda: step(torch.cuda.Stream()), lambda: step(torch.cuda.Stream().cuda_stream)):
            out.fill_(7.0)
            lse.fill_(9.0)
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert int(err) == 0
            compare(out.cpu(), lse.cpu(), want, wl, tol_o, tol_l, torch.float32)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H", [16, 5, 128])
def test_absorbed_form_of_broadcast_queries(H, flags):
    c = Case([300, 90], [3, 1], [3, 1], H, seed=H)
    for axis in (0, 1):
        x = Case([300, 90], [3, 1], [3, 1], H, seed=H)
        x.q_full = c.q_full.narrow(axis, 0, 1).expand(c.q_full.shape).contiguous()
        want = x.run(flags=flags)
        stored = x.q_full
        x.q_full = _Broadcast(stored, axis)
        got = x.run(flags=flags)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), axis


class _Broadcast:
    """Moves to the GPU as one row (or head) expanded along its axis."""

    def __init__(self, t, axis):
        self.t, self.axis, self.shape = t, axis, t.shape

    def to(self, dev):
        return self.t.narrow(self.axis, 0, 1).to(dev).expand(self.t.shape)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H", [16, 128])
def test_absorbed_form_under_wide_bounds(H, flags):
    """Bounds of a server's largest step, a batch that is the first part of its tables, no LSE."""
    c = Case([300, 1, 70], [1, 2, 1], [1, 4, 1], H, seed=H)
    width, rows = 300, 40
    table = np.full((9, width), 1 << 29, dtype=np.int32)
    table[:3, :c.table.shape[1]] = c.table
    out = torch.full((c.q_full.shape[0], H, L), 7.0, dtype=torch.float32, device=DEV)
    ws = torch.empty(max(256, pkv.paged_attention_latent_workspace_size(9, rows, H, width * P)), dtype=torch.uint8, device=DEV)
    pkv.paged_attention_latent(c.q_full.to(DEV), c.pool.to(DEV), i32(table), i32(c.kv + [1 << 20] * 6),
                               i32(list(c.indptr) + [1 << 20] * 6), out, q_real=i32(c.real + [5] * 6), batch=3, max_q_rows=rows,
                               max_kv_len=width * P, scale=c.scale, workspace=ws, flags=flags)
    want, wl, tol_o, tol_l = c.expected()
    compare(out.cpu(), torch.from_numpy(wl), want, wl, tol_o, tol_l, torch.float32)


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_pages_that_sequences_share(flags):
    """A shared prefix: the same pages in several rows of the table, and twice in one."""
    c = Case([128, 128, 100], [1, 1, 1], [1, 1, 1], 16, seed=1)
    c.table[1, :2] = c.table[0, :2]
    c.table[2, 1] = c.table[2, 0]
    c.check(flags=flags)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H", [16, 24, 128])
def test_nan_in_rows_that_pad(H, flags):
    """Queries behind a sequence's real rows hold anything; their outputs are zeros."""
    c = Case([300, 70], [1, 2], [4, 9], H, seed=H)
    for b in range(2):
        c.q_full[c.indptr[b] + c.real[b]:c.indptr[b + 1]] = float("nan")
    got, gl, err = c.run(flags=flags)
    assert err == 0
    clean = Case([300, 70], [1, 2], [4, 9], H, seed=H)
    want, wl, tol_o, tol_l = clean.expected()
    compare(got, gl, want, wl, tol_o, tol_l, torch.bfloat16)


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_lengths_and_ranges_below_zero(flags):
    """Taken as empty, and reported in checked mode."""
    c = Case([100, 70], [1, 1], [1, 1], 16, seed=2)
    want = c.run(flags=flags)[0]
    out = torch.full_like(want, 7.0).to(DEV)
    ws = torch.empty(max(256, pkv.paged_attention_latent_workspace_size(2, 1, 16, 100)), dtype=torch.uint8, device=DEV)
    err = i32([0])
    pkv.paged_attention_latent(c.q_full.to(DEV), c.pool.to(DEV), i32(c.table), i32([100, -70]), i32(c.indptr), out, max_q_rows=1,
                               max_kv_len=100, scale=c.scale, workspace=ws, flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
    assert int(err) == pkv.PKV_ERRBIT_LEN
    assert torch.equal(out[0].cpu(), want[0]) and (out[1] == 0).all() and (out[2:] == 7).all()


def test_append_of_one_row_into_pages_apart():
    """A source of stride 0, pages further apart than their slots, a captured call, another stream."""
    T, pages, pad = 40, 4, 72
    g = torch.Generator().manual_seed(7)
    row = torch.randn(1, L + R, generator=g).to(torch.bfloat16).to(DEV)
    big = torch.full((pages, P * (L + R) + pad), 3.0, dtype=torch.bfloat16, device=DEV)
    pool = big.as_strided((pages, P, L + R), (big.stride(0), L + R, 1))
    slots = torch.randperm(pages * P, generator=g)[:T].to(DEV)
    pos = torch.zeros(T, dtype=torch.int64, device=DEV)
    ang = torch.zeros(1, R, device=DEV)
    ang[:, :R // 2] = 1.0
    q = torch.randn(1, 1, R, generator=g).to(torch.bfloat16).to(DEV).expand(T, 3, R)
    heads = torch.zeros(3, T, R, dtype=torch.bfloat16, device=DEV)     # heads ahead of tokens
    torch.cuda.synchronize()

    def step(stream=None):
        pkv.kv_append_latent(row.expand(T, L + R), pos, ang, slots, pool, q_pe=q, q_out=heads.transpose(0, 1), stream=stream)

    def check():
        torch.cuda.synchronize()
        want = torch.full((pages * P, L + R), 3.0, dtype=torch.bfloat16, device=DEV)
        want[slots] = row
        assert torch.equal(pool.reshape(-1, L + R), want) and (big[:, P * (L + R):] == 3).all()
        assert torch.equal(heads, q.transpose(0, 1))
        pool.fill_(3.0)
        heads.zero_()
        torch.cuda.synchronize()
    step(torch.cuda.Stream())
    check()
    step(torch.cuda.Stream().cuda_stream)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    slots.copy_(torch.randperm(pages * P, generator=g)[:T])
    graph.replay()
    check()


def test_one_key_one_row_one_head():
    c = Case([1], [1], [1], 1, seed=3)
    c.check()
    Ragged([1], [1], 1, seed=3).check()
    q, k = c.q_full[0].double().numpy(), c.pool[c.table[0, 0], :1].double().numpy()
    assert np.allclose(attend(q, k, k[:, :L], c.scale)[0], k[:, :L])   # the only key's value
