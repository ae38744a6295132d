"""GPU parity of paged_attention_fp8 and paged_attention_window against a plain
64-bit implementation: types, head layouts, lengths from no key to long rows,
odd sizes, strides, masks that leave a row empty, and both the chosen kernel
and the generic one."""
import numpy as np
import pytest
import torch

from ext_testutil import Case, call, check, run
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
FLAGS = [0, pkv.PKV_FLAG_SIMT_ONLY]
HEADS = [(4, 2, 64), (32, 8, 128), (8, 8, 128), (8, 1, 64), (16, 1, 128), (6, 2, 128), (24, 1, 64)]


def ragged(seed, batch, new, kv, pad=0):
    g = np.random.default_rng(seed)
    real = g.integers(new[0], new[1], size=batch, endpoint=True).tolist()
    lens = [max(int(k), r) for k, r in zip(g.integers(kv[0], kv[1], size=batch, endpoint=True), real)]
    rows = [r + (int(g.integers(0, pad, endpoint=True)) if pad else 0) for r in real]
    return lens, real, rows


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("fp8,window,sinks", [(True, 0, 0), (True, 50, 4), (False, 50, 4), (False, 1, 0)])
def test_decode(Hq, Hkv, D, fp8, window, sinks, flags):
    kv, real, rows = ragged(1, 5, (1, 1), (1, 400))
    kv[0], kv[1], kv[2] = 1, 32, 33
    c = Case(kv, real, rows, Hq, Hkv, D, fp8, window=window, sinks=sinks, seed=2)
    check(c, *run(c, flags=flags))


@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("kv", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 1000, 2049])
@pytest.mark.parametrize("fp8", [True, False])
def test_lengths(kv, fp8, flags):
    c = Case([kv], [1], [1], 4, 1, 128, fp8, window=0 if fp8 else 4096, seed=kv)
    check(c, *run(c, flags=flags))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (31, 0), (32, 0), (33, 5), (64, 32), (64, 33), (100, 64),
                                          (7, 200), (300, 4), (4096, 16)])
@pytest.mark.parametrize("fp8", [True, False])
def test_window_edges(window, sinks, fp8):
    """Windows and sinks that end inside, at and past pages; sinks that reach into the window."""
    kv = [1, 5, 32, 64, 90, 200, 333, 334, 335]
    c = Case(kv, [1] * 9, [1] * 9, 8, 2, 128, fp8, window=window, sinks=sinks, seed=window + sinks)
    check(c, *run(c))


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fp8", [True, False])
def test_long_rows(fp8, out_dtype):
    """Few long rows: the keys are split between blocks and joined."""
    c = Case([9001, 20000, 77], [1, 1, 1], [1, 1, 1], 8, 2, 128, fp8, window=0 if fp8 else 15000, sinks=0, seed=5)
    check(c, *run(c, out_dtype=out_dtype))


@pytest.mark.parametrize("fp8,window", [(True, 0), (True, 700), (False, 700)])
def test_ragged_batch(fp8, window):
    """A batch of very different lengths, some of them empty."""
    kv, real, rows = ragged(3, 70, (1, 1), (1, 3000))
    kv[3], real[3] = 0, 0          # a padding row alone
    kv[10] = 1
    rows[20], real[20] = 0, 0      # a sequence without rows
    c = Case(kv, real, rows, 8, 2, 64, fp8, window=window, sinks=3 if window else 0, seed=4)
    check(c, *run(c))


# ------------------------------------------------------------------ several rows
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (32, 8, 128), (6, 2, 128), (16, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("fp8,mask,cb,window,sinks", [
    (True, "causal", 0, 0, 0), (True, "none", 0, 0, 0), (True, "block_causal", 3, 0, 0),
    (True, "causal", 0, 40, 5), (False, "causal", 0, 40, 5), (False, "causal", 0, 2, 0)])
@pytest.mark.parametrize("new", [(2, 4), (5, 9), (12, 40)])
def test_rows(Hq, Hkv, D, fp8, mask, cb, window, sinks, new, flags):
    kv, real, rows = ragged(6, 4, new, (1, 300), pad=3)
    c = Case(kv, real, rows, Hq, Hkv, D, fp8, mask, cb, window, sinks, seed=7)
    check(c, *run(c, flags=flags))


@pytest.mark.parametrize("fp8,mask,cb,window,sinks", [
    (True, "causal", 0, 0, 0), (True, "none", 0, 0, 0), (True, "block_causal", 100, 0, 0),
    (True, "causal", 0, 130, 5), (False, "causal", 0, 130, 5), (False, "causal", 0, 1000, 140),
    (False, "causal", 0, 5, 0), (False, "causal", 0, 129, 129)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 1, 64), (2, 2, 128), (6, 2, 64)])
def test_chunk(Hq, Hkv, D, fp8, mask, cb, window, sinks):
    """Prompt chunks over several key tiles, ragged, with padding rows."""
    kv, real, rows = ragged(8, 3, (130, 300), (300, 900), pad=5)
    kv[0] = real[0]  # a chunk that starts its sequence
    c = Case(kv, real, rows, Hq, Hkv, D, fp8, mask, cb, window, sinks, seed=9)
    check(c, *run(c))


@pytest.mark.parametrize("new", [1, 3, 100])
@pytest.mark.parametrize("fp8", [True, False])
def test_more_rows_than_keys(new, fp8):
    """q_real above kv_len: the first positions fall below key 0 and see nothing."""
    c = Case([max(1, new // 2), 40], [new, new], [new, new + 2], 8, 2, 128, fp8, window=0 if fp8 else 16,
             sinks=0 if fp8 else 2, seed=11)
    check(c, *run(c))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("new", [(1, 1), (3, 6), (70, 90)])
def test_strides(fp8, new):
    """Pages further apart than a page, queries sliced out of a wider tensor."""
    kv, real, rows = ragged(12, 3, new, (100, 300))
    c = Case(kv, real, rows, 8, 2, 128, fp8, window=0 if fp8 else 60, seed=13, slot_pad=64, q_pad=5)
    check(c, *run(c))


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("new", [(1, 1), (4, 4), (80, 80)])
def test_any_scale(new):
    """Scales that are not powers of two (written by another quantiser).  The
    tile kernel's bf16 expansion rounds such values once more: 2^-8 of k and v."""
    kv, real, rows = ragged(14, 3, new, (100, 300))
    c = Case(kv, real, rows, 8, 2, 128, True, seed=15, pow2=False)
    out, lse = run(c)
    if new[0] * 4 > 64:
        O, L, A, S = c.reference()
        got = out.double().cpu().numpy()
        # k rounded: scores off by 2^-8 of S, weights by twice that; v rounded: 2^-8 of A
        tol = (2 * 2.0 ** -8 * (1 + S) + 2.0 ** -8)[..., None] * A + 2.0 ** -8 * abs(O) + 2.0 ** -20
        assert (abs(got - O) <= tol).all()
    else:
        check(c, out, lse)


@pytest.mark.parametrize("kexp,vexp", [(0, -60), (0, 60), (-40, 0)])
@pytest.mark.parametrize("rows", [1, 3])
def test_far_scales(kexp, vexp, rows):
    """V magnitudes down to 2^-89 and up to 2^82, pages that differ by many powers of two."""
    c = Case([500, 200], [rows] * 2, [rows] * 2, 8, 2, 128, True, seed=16)
    g = np.random.default_rng(17)
    for name, e in (("k_scale", kexp), ("v_scale", vexp)):
        s = getattr(c, name)
        spread = g.integers(-20, 20, size=s.shape) if name == "v_scale" else np.zeros(s.shape)
        f = torch.from_numpy(np.exp2(e + spread)).float()
        s *= f
        arr = c.k64 if name == "k_scale" else c.v64
        arr *= f.double().numpy()[:, None, :, None]
    check(c, *run(c, out_dtype=torch.float32))


def test_zero_scale():
    """A page whose V is all zero has scale 0 and takes its share of the weight."""
    c = Case([200], [1], [1], 4, 1, 128, True, seed=18)
    c.v_scale[c.table[0, 2]] = 0
    c.v64[c.table[0, 2]] = 0
    check(c, *run(c))


# ------------------------------------------------------------------ checked mode, streams, graphs
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("new", [1, 3, 90])
@pytest.mark.parametrize("fp8", [True, False])
def test_checked(fp8, new, flags):
    c = Case([200, 300], [new, new], [new, new], 8, 2, 128, fp8, window=0 if fp8 else 64, seed=19)
    t = c.on("cuda")
    out = torch.zeros(sum(c.rows), 8, 128, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = c.reference()
    lse = torch.zeros(sum(c.rows), 8, device="cuda")
    call(c, t, out, lse, flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
    assert err.item() == 0
    check(c, out, lse, ref)
    # a page outside the pool is reported and not read
    for bad in (c.num_pages, -7, 2 ** 30):
        t["table"][1, (c.kv[1] - 1) // 32] = bad
        err.zero_()
        call(c, t, out, lse, flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
        assert err.item() == pkv.PKV_ERRBIT_PAGE
        O, L, A, S = ref
        r = c.rows[0]
        check_rows = slice(0, r)  # the first sequence is as before
        assert np.allclose(out.double().cpu().numpy()[check_rows], O[check_rows], atol=0.05)
    t = c.on("cuda")
    err.zero_()
    call(c, t, out, lse, flags=flags | pkv.PKV_FLAG_CHECKED, err=err, max_kv_len=256)
    assert err.item() & pkv.PKV_ERRBIT_LEN


@pytest.mark.parametrize("new", [1, 4, 90])
@pytest.mark.parametrize("fp8", [True, False])
def test_graph_and_streams(fp8, new):
    """Captured once, replayed with other lengths, and two calls at once on two
    streams with a workspace each."""
    big = Case([700, 650], [new, new], [new, new], 8, 2, 128, fp8, window=0 if fp8 else 100, sinks=0 if fp8 else 3,
               seed=20)
    small = Case([new + 3, 500], [new, new], [new, new], 8, 2, 128, fp8, window=big.window, sinks=big.sinks, seed=21)
    t = big.on("cuda")
    # room for either case's pool
    pages = max(big.num_pages, small.num_pages)
    for n in ("k_pool", "v_pool") + (("k_scale", "v_scale") if fp8 else ()):
        room = torch.zeros((pages,) + tuple(t[n].shape[1:]), dtype=torch.float32).to(t[n].dtype).cuda()
        room[:big.num_pages].copy_(t[n])
        t[n] = room
    out = torch.empty(2 * new, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2 * new, 8, device="cuda")
    ws = call(big, t, out, lse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(big, t, out, lse, workspace=ws, stream=torch.cuda.current_stream())
    out.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    check(big, out, lse)
    u = small.on("cuda")
    for n in ("k_pool", "v_pool") + (("k_scale", "v_scale") if fp8 else ()):
        t[n][:small.num_pages].copy_(u[n])
    for n in ("q", "kv_lens"):
        t[n].copy_(u[n])
    t["table"].fill_(-1)
    t["table"][:, :u["table"].shape[1]].copy_(u["table"])
    g.replay()
    torch.cuda.synchronize()
    check(small, out, lse)
    # two calls at once
    a, b = big.on("cuda"), small.on("cuda")
    oa, ob = torch.empty_like(out), torch.empty_like(out)
    la, lb = torch.empty_like(lse), torch.empty_like(lse)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    wa = wb = None
    for _ in range(5):
        wa = call(big, a, oa, la, workspace=wa, stream=sa)
        wb = call(small, b, ob, lb, workspace=wb, stream=sb)
    torch.cuda.synchronize()
    check(big, oa, la)
    check(small, ob, lb)


def test_same_bits_every_time():
    c = Case([5000, 300, 9000], [1] * 3, [1] * 3, 8, 2, 128, True, seed=22)
    a, la = run(c)
    for _ in range(3):
        b, lb = run(c)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_rows_behind_the_last_sequence_are_left():
    c = Case([100, 50], [2, 2], [2, 2], 4, 2, 64, True, seed=23)
    t = c.on("cuda")
    out = torch.full((4 + 3, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4 + 3, 4), 9.0, device="cuda")
    t["q"] = torch.cat([t["q"], t["q"][:3]])
    call(c, t, out, lse)
    torch.cuda.synchronize()
    assert (out[4:] == 9).all() and (lse[4:] == 9).all()
    check(c, out[:4], lse[:4])


def test_window_without_reach_is_causal():
    """A window as long as the sequence gives what paged_attention gives."""
    c = Case([300, 77, 150], [1] * 3, [1] * 3, 8, 2, 128, False, window=300, seed=24)
    out, lse = run(c)
    t = c.on("cuda")
    ref, rl = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(max(pkv.paged_attention_workspace_size(3, 1, 8, 2, 128, 300), 1), dtype=torch.uint8,
                     device="cuda")
    pkv.paged_attention(t["q"], t["k_pool"], t["v_pool"], t["table"], t["kv_lens"], t["q_indptr"], ref,
                        q_real=t["q_real"], lse=rl, max_q_rows=1, max_kv_len=300, workspace=ws)
    check(c, out, lse)
    check(c, ref, rl)


# ------------------------------------------------------------------ the cut line of keys
@pytest.mark.parametrize("fp8,window,new,D,Hkv", [
    (True, 0, (1, 1), 128, 2), (False, 1800, (1, 1), 128, 2), (True, 0, (2, 6), 128, 2), (True, 2500, (1, 1), 64, 3)])
def test_more_units_than_ctas(fp8, window, new, D, Hkv):
    """Enough (sequence, head) units that part of the keys is taken by ticket;
    the same bits whoever takes which."""
    kv, real, rows = ragged(30, 170, new, (1, 3600), pad=1 if new[1] > 1 else 0)
    kv[5], real[5], rows[5] = 0, 0, 1
    real[6] = rows[6] = 0
    kv[7] = 3600
    c = Case(kv, real, rows, 4 * Hkv, Hkv, D, fp8, window=window, sinks=5 if window else 0, seed=31)
    ref = c.reference()
    t = c.on("cuda")
    out = torch.empty(sum(rows), c.Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(sum(rows), c.Hq, device="cuda")
    wide = torch.full((len(kv), 200), -1, dtype=torch.int32, device="cuda")
    wide[:, :t["table"].shape[1]] = t["table"]
    t["table"] = wide
    call(c, t, out, lse, max_kv_len=6400)
    torch.cuda.synchronize()
    check(c, out, lse, ref)
    for _ in range(3):
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        call(c, t, o2, l2, max_kv_len=6400)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def call_bounds(c, max_kv_len):
    """A call whose table is as wide as a larger host bound asks for."""
    t = c.on("cuda")
    wide = torch.full((len(c.kv), (max_kv_len + 31) // 32), -1, dtype=torch.int32, device="cuda")
    wide[:, :t["table"].shape[1]] = t["table"]
    t["table"] = wide
    out = torch.empty(sum(c.rows), c.Hq, c.D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(sum(c.rows), c.Hq, device="cuda")
    call(c, t, out, lse, max_kv_len=max_kv_len)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("batch,kv", [(300, (1, 900)), (2100, (1, 120))])
def test_large_batches(batch, kv):
    """More sequences than a CTA, and than the planner's shared memory, looks through."""
    lens, real, rows = ragged(32, batch, (1, 1), kv)
    c = Case(lens, real, rows, 4, 1, 128, True, seed=33)
    check(c, *call_bounds(c, 4000))


@pytest.mark.parametrize("fp8,new", [(True, (5, 12)), (False, (1, 3)), (True, (17, 20))])
def test_several_row_tiles(fp8, new):
    """Row tiles of 8 and 16 on long rows, few and many of them."""
    kv, real, rows = ragged(34, 6, new, (2000, 5000), pad=2)
    c = Case(kv, real, rows, 8, 2, 128, fp8, window=0 if fp8 else 3000, sinks=0 if fp8 else 9, seed=35)
    check(c, *run(c))


def test_large_group():
    """More query heads a K/V head than the tile kernel takes."""
    c = Case([300, 40], [3, 2], [3, 4], 160, 2, 128, True, seed=36)
    check(c, *run(c))
    c = Case([300, 140], [40, 30], [40, 30], 80, 1, 64, False, window=50, sinks=2, seed=37)
    check(c, *run(c))


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("fp8", [True, False])
def test_extreme_bounds(new, fp8):
    """The largest window and sink counts, rows below key 0, an empty cache."""
    c = Case([max(1, new - 2), 50], [new, new], [new, new], 8, 2, 128, fp8, window=2 ** 31 - 1, sinks=2 ** 31 - 1,
             seed=38)
    check(c, *run(c))
    c = Case([70, 50], [new, new], [new, new], 8, 2, 128, fp8, window=1, sinks=2 ** 31 - 1, seed=39)
    check(c, *run(c))
    c = Case([0, 0], [new, 0], [new, 2], 8, 2, 128, fp8, window=0 if fp8 else 4, seed=40)
    t = c.on("cuda")
    out, lse = (torch.full(s, 5.0, dtype=d, device="cuda") for s, d in
                (((new + 2, 8, 128), torch.bfloat16), ((new + 2, 8), torch.float32)))
    kw = dict(q_real=t["q_real"], lse=lse, max_q_rows=max(c.rows), max_kv_len=0, window=c.window)
    if fp8:
        pkv.paged_attention_fp8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], t["table"], t["kv_lens"],
                                t["q_indptr"], out, **kw)
    else:
        pkv.paged_attention_window(t["q"], t["k_pool"], t["v_pool"], t["table"], t["kv_lens"], t["q_indptr"], out, **kw)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kv", [100, 6000])
def test_wait_that_runs_out(kv):
    """The failure path: consumers give up on a barrier nothing completes, the
    error bit is set, every warp winds down, and the next call is unharmed."""
    c = Case([kv, 20], [1, 1], [1, 1], 8, 2, 128, True, seed=41)
    t = c.on("cuda")
    out = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = call(c, t, out, lse, flags=pkv.PKV_FLAG_TEST_WAIT_TIMEOUT, err=err)
    torch.cuda.synchronize()
    assert err.item() == pkv.PKV_ERRBIT_TIMEOUT
    err.zero_()
    call(c, t, out, lse, err=err, workspace=ws)
    torch.cuda.synchronize()
    assert err.item() == 0
    check(c, out, lse)
    with pytest.raises(pkv.PkvError):  # the tile kernel has no such hook
        big = Case([kv], [50], [50], 8, 2, 128, True, seed=42)
        call(big, big.on("cuda"), torch.zeros(50, 8, 128, dtype=torch.bfloat16, device="cuda"),
             torch.zeros(50, 8, device="cuda"), flags=pkv.PKV_FLAG_TEST_WAIT_TIMEOUT, err=err)


def test_nan_scores_stay_in_their_rows():
    """NaN in one sequence's query shows in its rows only."""
    for new in (1, 3, 60):
        c = Case([200, 300], [new, new], [new, new], 8, 2, 128, True, seed=43)
        ref = c.reference()
        t = c.on("cuda")
        t["q"][0, 3, 5] = float("nan")
        out = torch.empty(2 * new, 8, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(2 * new, 8, device="cuda")
        call(c, t, out, lse)
        torch.cuda.synchronize()
        assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
        out[0, 3] = torch.from_numpy(ref[0][0, 3]).to(out)
        lse[0, 3] = float(ref[1][0, 3])
        check(c, out, lse, ref)
