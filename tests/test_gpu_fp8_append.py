"""GPU tests of kv_append_fp8 against a plain 64-bit implementation, bit for
bit, and of a decode loop that appends and attends over the 8-bit cache."""
import numpy as np
import pytest
import torch

from ext_testutil import P, Case, check, codes_of, e4m3_grid, scale_for
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


class Cache:
    """The 8-bit cache in float64 (codes and scales) and on the device."""

    def __init__(self, pages, Hkv, D, seed=0, page_pad=0, scale_pad=0):
        g = np.random.default_rng(seed)
        self.codes = [e4m3_grid(g.standard_normal((pages, P, Hkv, D)) * 100) for _ in "kv"]
        self.scales = [np.exp2(g.integers(-12, -4, size=(pages, Hkv))).astype(np.float64) for _ in "kv"]
        row = P * Hkv * D
        self.pools, self.dev_scales = [], []
        for c, s in zip(self.codes, self.scales):
            room = torch.zeros(pages, row + page_pad, dtype=torch.uint8, device="cuda")
            room[:, :row] = codes_of(c).view(torch.uint8).flatten(1).cuda()
            self.pools.append(room[:, :row].unflatten(1, (P, Hkv, D)).view(torch.float8_e4m3fn))
            sroom = torch.zeros(pages, Hkv + scale_pad, device="cuda")
            sroom[:, :Hkv] = torch.from_numpy(s).float().cuda()
            self.dev_scales.append(sroom[:, :Hkv])

    def append(self, src, table, kv, real, indptr, max_kv, top):
        """The definition, page by page."""
        for w in range(2):
            x64 = np.clip(src[w].double().numpy(), -top, top)
            for b in range(len(kv)):
                n = min(kv[b], max_kv)
                first = kv[b] - real[b]
                for p in range(max(first, 0) // P, (max(n, 0) + P - 1) // P):
                    lo, hi = max(first, p * P, 0), min(n, (p + 1) * P)
                    if hi <= lo or real[b] <= 0:
                        continue
                    ph = table[b, p]
                    if ph < 0:
                        continue
                    kept = max(0, first - p * P)
                    x = x64[indptr[b] + lo - first:indptr[b] + hi - first]
                    for h in range(x.shape[1]):
                        fin = abs(x[:, h][~np.isnan(x[:, h])])
                        need = scale_for(float(fin.max()) if fin.size else 0.0)
                        had = self.scales[w][ph, h] if kept else 0.0
                        s = max(had, need)
                        d = s if s > 0 else 1.0
                        if kept and s != had:
                            self.codes[w][ph, :kept, h] = e4m3_grid(self.codes[w][ph, :kept, h] * had / d)
                        y = x[:, h] / d if s > 0 else x[:, h] * 0
                        self.codes[w][ph, lo - p * P:hi - p * P, h] = e4m3_grid(y)
                        self.scales[w][ph, h] = s

    def same(self):
        for w in range(2):
            got = self.pools[w].float().cpu().numpy()
            assert np.array_equal(got, self.codes[w].astype(np.float32), equal_nan=True), "codes"
            assert np.array_equal(self.dev_scales[w].cpu().double().numpy(), self.scales[w]), "scales"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def append(c, src, table, kv, real, rows, *, max_kv=None, q_real=True, **kw):
    indptr = np.concatenate([[0], np.cumsum(rows)])
    pkv.kv_append_fp8(src[0].cuda() if not src[0].is_cuda else src[0], src[1].cuda() if not src[1].is_cuda else src[1],
                      i32(table), i32(kv), i32(indptr), c.pools[0], c.pools[1], c.dev_scales[0], c.dev_scales[1],
                      q_real=i32(real) if q_real else None, max_q_rows=max(max(rows), 1),
                      max_kv_len=max_kv or max(max(kv), 1), **kw)
    torch.cuda.synchronize()
    return indptr


TOP = {torch.bfloat16: float(torch.finfo(torch.bfloat16).max), torch.float16: 65504.0,
       torch.float32: float(torch.finfo(torch.float32).max)}


def tables(g, batch, width, pages):
    return g.permutation(pages)[:batch * width].reshape(batch, width).astype(np.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("Hkv,D", [(2, 64), (8, 128), (1, 128), (3, 64)])
@pytest.mark.parametrize("new,size", [(1, 3.0), (1, 1e-4), (2, 1.0), (31, 1.0), (32, 2.0), (33, 1.0), (100, 50.0)])
def test_append(dtype, Hkv, D, new, size):
    """Starts at every kind of slot; sizes below and above what the pages hold."""
    g = np.random.default_rng(new)
    starts = [0, 1, 31, 32, 40, 63]
    kv = [s + new for s in starts]
    real, rows = [new] * 6, [new + (b % 3) for b in range(6)]
    width = max(kv) // P + 1
    c = Cache(6 * width + 3, Hkv, D, seed=1, page_pad=32, scale_pad=3)
    table = tables(g, 6, width, 6 * width + 3)
    wide = torch.from_numpy(g.standard_normal((sum(rows), Hkv * 3, D)) * size).to(dtype).cuda()
    src = [wide[:, Hkv:2 * Hkv], wide[:, 2 * Hkv:]]
    indptr = append(c, src, table, kv, real, rows)
    c.append([x.cpu() for x in src], table, kv, real, indptr, max(kv), TOP[dtype])
    c.same()
    append(c, src, table, kv, real, rows)  # the same call again writes the same
    c.same()


def test_special_values():
    """Zeros, infinities, NaN, subnormals, and amax on and next to 448 * 2^e."""
    rows = torch.zeros(12, 1, 64)
    rows[1, 0, 3] = 448.0
    rows[2, 0, 3] = 448.0 * 2 ** -20
    rows[3, 0, 3] = 450.0
    rows[4, 0, 5] = float("inf")
    rows[5, 0, 5] = float("-inf")
    rows[6, 0, 0] = float("nan")
    rows[7, 0, 0], rows[7, 0, 1] = float("nan"), 2.0
    rows[8, 0, :] = 1e-39
    rows[9, 0, 7] = -3.3e38
    rows[10, 0, :] = torch.linspace(-1, 1, 64)
    for dtype in (torch.bfloat16, torch.float32):
        x = rows.to(dtype)
        g = np.random.default_rng(0)
        c = Cache(30, 1, 64, seed=2)
        table = tables(g, 12, 2, 30)
        kv, ones = [1 + 32 * (b % 2) for b in range(12)], [1] * 12
        indptr = append(c, [x, x.clone()], table, kv, ones, ones)
        c.append([x, x], table, kv, ones, indptr, max(kv), TOP[dtype])
        c.same()
        # and into the middle of pages that hold tokens
        kv = [k + 9 for k in kv]
        indptr = append(c, [x, x.clone()], table, kv, ones, ones)
        c.append([x, x], table, kv, ones, indptr, max(kv), TOP[dtype])
        c.same()


def test_empty_and_bounds():
    """Sequences without rows, padding rows, no keys, more rows than keys, keys
    past the host bound, freed pages: skipped, everything else kept."""
    g = np.random.default_rng(3)
    c = Cache(40, 2, 64, seed=3)
    table = tables(g, 6, 6, 40)
    table[5, 1] = -1
    kv, real, rows = [0, 50, 3, 70, 150, 60], [0, 0, 5, 4, 20, 30], [2, 0, 5, 9, 20, 30]
    src = [torch.from_numpy(g.standard_normal((sum(rows), 2, 64))).to(torch.bfloat16) for _ in "kv"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    indptr = append(c, src, table, kv, real, rows, max_kv=140, checked=True, err=err)
    c.append(src, table, kv, real, indptr, 140, TOP[torch.bfloat16])
    c.same()
    assert err.item() == pkv.PKV_ERRBIT_LEN | pkv.PKV_ERRBIT_PAGE
    pkv.kv_append_fp8(src[0].cuda(), src[1].cuda(), i32(table)[:0], i32(kv)[:0], i32([0]), c.pools[0], c.pools[1],
                      c.dev_scales[0], c.dev_scales[1], max_q_rows=1, max_kv_len=32)
    c.same()


@pytest.mark.parametrize("bound", [2 ** 31 - 1, 2 ** 31 - 31, 1000])
def test_row_bound_far_above_the_rows(bound):
    c = Cache(6, 2, 64, seed=9)
    g = torch.Generator().manual_seed(10)
    src = [torch.randn(41, 2, 64, generator=g).bfloat16() for _ in "kv"]
    table, kv, real = np.array([[4, 1, 2], [0, 5, 3]]), [70, 7], [36, 5]
    pkv.kv_append_fp8(src[0].cuda(), src[1].cuda(), i32(table), i32(kv), i32([0, 36, 41]), c.pools[0], c.pools[1],
                      c.dev_scales[0], c.dev_scales[1], max_q_rows=bound, max_kv_len=96)
    torch.cuda.synchronize()
    c.append(src, table, kv, real, [0, 36, 41], 96, torch.finfo(torch.bfloat16).max)
    c.same()


@pytest.mark.parametrize("bad", [10 ** 6, -3])
def test_bad_page_is_skipped(bad):
    c = Cache(8, 2, 64, seed=4)
    x = [torch.ones(2, 2, 64, dtype=torch.bfloat16) for _ in "kv"]
    table = np.array([[1], [bad]], dtype=np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    indptr = append(c, x, table, [7, 7], [1, 1], [1, 1], checked=True, err=err)
    table[1, 0] = -1
    c.append(x, table, [7, 7], [1, 1], indptr, 32, TOP[torch.bfloat16])
    c.same()
    assert err.item() == pkv.PKV_ERRBIT_PAGE


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_prompt_then_decode(window, sinks):
    """A prompt chunk, then tokens one by one: appended, then attended, with the
    same index tensors; the attention is held against the codes the definition
    gives."""
    Hq, Hkv, D, B, steps = 8, 2, 128, 3, 40
    g = np.random.default_rng(5)
    prompt = [17, 70, 33]
    width = 4
    c = Cache(B * width, Hkv, D, seed=6)
    table = tables(g, B, width, B * width)
    kv = list(prompt)

    def step(real):
        indptr = np.concatenate([[0], np.cumsum(real)])
        src = [torch.from_numpy(g.standard_normal((sum(real), Hkv, D))).to(torch.bfloat16) for _ in "kv"]
        append(c, src, table, kv, real, real)
        c.append(src, table, kv, real, indptr, width * P, TOP[torch.bfloat16])
        case = Case([k for k in kv], list(real), list(real), Hq, Hkv, D, True, window=window, sinks=sinks,
                    seed=len(kv))
        case.table = np.full_like(case.table, -1)
        case.table = table[:, :case.table.shape[1]]
        case.num_pages = B * width
        case.k64 = c.codes[0] * c.scales[0][:, None, :, None]
        case.v64 = c.codes[1] * c.scales[1][:, None, :, None]
        out = torch.empty(sum(real), Hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(sum(real), Hq, device="cuda")
        n = pkv.paged_attention_fp8_workspace_size(B, max(real), Hq, Hkv, D, max(kv), window, sinks)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        pkv.paged_attention_fp8(case.q_full.cuda(), c.pools[0], c.pools[1], c.dev_scales[0], c.dev_scales[1],
                                i32(table), i32(kv), i32(indptr), out, lse=lse, max_q_rows=max(real),
                                max_kv_len=max(kv), window=window, num_sinks=sinks, workspace=ws)
        torch.cuda.synchronize()
        check(case, out, lse)

    step(prompt)
    for n in range(steps):
        kv = [k + 1 for k in kv]
        if n % 8 == 0 or n in (14, 15, 16):
            step([1] * B)
        else:
            src = [torch.from_numpy(g.standard_normal((B, Hkv, D)) * (1 + n)).to(torch.bfloat16) for _ in "kv"]
            append(c, src, table, kv, [1] * B, [1] * B)
            c.append(src, table, kv, [1] * B, np.arange(B + 1), width * P, TOP[torch.bfloat16])
    c.same()


def test_append_in_a_graph():
    """Captured with one length, replayed with the next."""
    c = Cache(6, 2, 64, seed=7)
    g = np.random.default_rng(8)
    table, kv, indptr = i32([[0, 1, 2], [3, 4, 5]]), i32([10, 20]), i32([0, 1, 2])
    src = [torch.from_numpy(g.standard_normal((2, 2, 64))).to(torch.bfloat16).cuda() for _ in "kv"]
    args = (src[0], src[1], table, kv, indptr, c.pools[0], c.pools[1], c.dev_scales[0], c.dev_scales[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_append_fp8(*args, max_q_rows=1, max_kv_len=96)
    for n in range(25):
        for x in src:
            x.copy_(torch.from_numpy(g.standard_normal((2, 2, 64)) * 2.0 ** (n % 5)).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        c.append([x.cpu() for x in src], table.cpu().numpy(), kv.tolist(), [1, 1], [0, 1, 2], 96, TOP[torch.bfloat16])
        kv += 1
    c.same()


def test_fork_of_a_partly_filled_page():
    """Two samples of one prompt: the whole page shared, the partly filled one
    copied (slots and scales), then each appends its own tokens."""
    H, D = 2, 64
    c = Cache(8, H, D, seed=9)
    g = np.random.default_rng(10)
    top = TOP[torch.bfloat16]
    prompt = [torch.from_numpy(g.standard_normal((45, H, D))).to(torch.bfloat16) for _ in "kv"]
    table = np.array([[3, 5]], dtype=np.int32)
    indptr = append(c, prompt, table, [45], [45], [45])
    c.append(prompt, table, [45], [45], indptr, 64, top)
    # page 5 -> 6: the pools' bytes as 2-byte elements
    pools = [p.view(torch.uint8).view(torch.bfloat16) for p in c.pools]
    slots = torch.arange(32, dtype=torch.int64, device="cuda")
    pkv.copy_kv_slots(pools[0], pools[1], 5 * 32 + slots, 6 * 32 + slots)
    for w in range(2):
        c.dev_scales[w][6] = c.dev_scales[w][5]
        c.codes[w][6], c.scales[w][6] = c.codes[w][5], c.scales[w][5]
    fork = np.array([[3, 5], [3, 6]], dtype=np.int32)
    for n in range(4):
        src = [torch.from_numpy(g.standard_normal((2, H, D)) * 10 ** n).to(torch.bfloat16) for _ in "kv"]
        indptr = append(c, src, fork, [46 + n] * 2, [1, 1], [1, 1], max_kv=64)
        c.append(src, fork, [46 + n] * 2, [1, 1], indptr, 64, top)
    c.same()
