"""paged_attention_latent against a plain 64-bit implementation: head counts on
both sides of every column tile, lengths on both sides of pages and key tiles,
one token to chunks, empty rows, strides, and values that must not be read."""
import numpy as np
import pytest
import torch

from latent_testutil import Case, compare
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
SIMT = pkv.PKV_FLAG_SIMT_ONLY


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H", [1, 5, 16, 17, 32, 33, 64, 65, 100, 128, 130])
def test_heads_one_token(H, flags):
    Case([37, 100, 1, 64], [1] * 4, [1] * 4, H, seed=H).check(flags=flags)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("kv", [1, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 191, 192, 193, 1000])
def test_lengths(kv, flags):
    Case([kv, 70, kv], [1] * 3, [1] * 3, 16, seed=kv).check(flags=flags, out_dtype=torch.float32)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H,real,rows", [(16, [4, 3, 4], [4, 4, 4]), (3, [7, 1, 12], [9, 1, 12]), (16, [20, 9, 1], [21, 9, 8]),
                                         (128, [2, 3, 1], [2, 3, 1]), (5, [40, 13, 2], [40, 20, 2])])
def test_several_rows(H, real, rows, flags):
    Case([50, 200, 333], real, rows, H, seed=H).check(flags=flags)
    Case([50, 200, 333], real, rows, H, mask="none", seed=H + 1).check(flags=flags, out_dtype=torch.float32)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_rows_that_see_nothing(H, flags):
    """Sequences without keys or rows, more new rows than keys, padding rows."""
    c = Case([0, 3, 65, 0, 1], [1, 5, 0, 0, 1], [1, 7, 2, 0, 3], H, seed=H)
    c.check(flags=flags)
    out, lse, _ = c.run(flags=flags)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()            # no key
    assert (out[1:3] == 0).all() and torch.isneginf(lse[1:3]).all()        # rows ahead of the first key
    assert (out[-2:] == 7).all() and (lse[-2:] == 9).all()                 # rows behind the last sequence


@pytest.mark.parametrize("H", [16, 24, 64, 128])
@pytest.mark.parametrize("growing,key_size", [(True, 1.0), (False, 12.0), (False, 0.01)])
def test_score_ranges(H, growing, key_size):
    Case([700, 90, 300], [1, 2, 1], [1, 2, 1], H, growing=growing, key_size=key_size, seed=3).check()


@pytest.mark.parametrize("H,real", [(256, [1, 1]), (192, [1, 2]), (8, [8, 16]), (4, [16, 5]), (2, [8, 3]), (64, [3, 1])])
def test_whole_rows_of_heads(H, real):
    """Head counts that divide a CTA's columns or are a multiple of them: queries as
    boxes for full column groups, piece by piece for the last."""
    Case([90, 200], real, real, H, seed=H, q_pad=1).check()
    Case([90, 200], real, [r + 1 for r in real], H, seed=H + 1, lead=2).check(out_dtype=torch.float32)


def test_padded_batch():
    """Far more padding rows than real ones: zeros, however many."""
    c = Case([40, 0, 300, 65], [2, 0, 1, 0], [150, 90, 200, 130], 16, seed=13)
    c.check()


@pytest.mark.parametrize("H", [16, 128])
def test_long_sequence_shared_out(H):
    """One sequence over all SMs, and long beside short ones."""
    Case([9000], [1], [1], H, seed=1).check(out_dtype=torch.float32)
    Case([5000, 1, 2500, 33], [1] * 4, [1] * 4, H, seed=2).check()


def test_many_sequences():
    g = np.random.default_rng(0)
    kv = [int(x) for x in g.integers(0, 200, 300)]
    Case(kv, [1] * 300, [1] * 300, 8, seed=4).check()


@pytest.mark.parametrize("B,H", [(100, 16), (152, 3), (70, 128), (60, 64)])
def test_short_units_one_to_a_cluster(B, H):
    """As many short units as run at once, of uneven lengths, some empty."""
    g = np.random.default_rng(B)
    kv = [int(x) if x > 40 else 0 for x in g.integers(0, 400, B)]
    Case(kv, [1] * B, [1] * B, H, seed=B).check()


@pytest.mark.parametrize("H", [16, 128])
def test_chunk_over_context(H):
    Case([300, 700], [100, 41], [100, 50], H, seed=5).check()


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_strides_and_leading_rows(flags):
    Case([37, 100], [1, 3], [1, 3], 16, page_pad=72, q_pad=5, lead=3, seed=6).check(flags=flags)
    Case([37, 100], [1, 3], [1, 3], 100, page_pad=8, q_pad=2, lead=3, seed=6).check(flags=flags)


@pytest.mark.parametrize("H", [16, 33, 64, 128])
def test_same_bits_every_time(H):
    c = Case([900, 40, 2100], [1, 4, 1], [1, 4, 1], H, seed=8)
    a, la, _ = c.run()
    for _ in range(3):
        b, lb, _ = c.run()
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H", [16, 128])
def test_nan_stays_in_its_row(H, flags):
    """NaN in one query row makes that row's output and LSE NaN, no other's."""
    c = Case([300, 500], [2, 1], [2, 1], H, seed=9)
    clean, cl, _ = c.run(flags=flags)
    c.q_full[1, 3, 100] = float("nan")
    got, gl, _ = c.run(flags=flags)
    assert torch.isnan(got[1, 3]).all() and torch.isnan(gl[1, 3])
    got[1, 3], gl[1, 3] = clean[1, 3], cl[1, 3]
    assert torch.equal(got, clean) and torch.equal(gl, cl)


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_pages_out_of_range_read_as_zeros(flags):
    c = Case([100, 70], [1, 1], [1, 1], 16, seed=10)
    for bad in (-1, c.num_pages, 1 << 30):
        c.table[0, 1] = bad
        got, gl, err = c.run(flags=flags)
        assert err == pkv.PKV_ERRBIT_PAGE
        assert c.run(flags=flags, checked=False)[2] == 0
        z = Case([100, 70], [1, 1], [1, 1], 16, seed=10)
        z.pool[z.table[0, 1]] = 0
        want, wl, tol_o, tol_l = z.expected()
        compare(got, gl, want, wl, tol_o, tol_l, torch.bfloat16)


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_lengths_beyond_the_bounds_are_reported(flags):
    c = Case([100, 70], [1, 1], [1, 1], 16, seed=11)
    want = c.run(flags=flags)[0]
    kv = [100, 170]  # the second is past the bound of 100 keys
    i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    out = torch.empty_like(want).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(256, pkv.paged_attention_latent_workspace_size(2, 1, 16, 100)), dtype=torch.uint8, device="cuda")
    pkv.paged_attention_latent(c.q_full.cuda(), c.pool.cuda(), i32(c.table), i32(kv), i32(c.indptr), out,
                               max_q_rows=1, max_kv_len=100, scale=c.scale, workspace=ws,
                               flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
    assert int(err) & pkv.PKV_ERRBIT_LEN
    assert torch.equal(out[0].cpu(), want[0])


def test_other_stream():
    c = Case([300, 500], [1, 1], [1, 1], 16, seed=12)
    want, wl, _ = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gl, _ = c.run()
    assert torch.equal(got, want) and torch.equal(gl, wl)

