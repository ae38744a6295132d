"""ragged_attention_latent against a plain 64-bit implementation: prompts and
continued prompts of every small length, tile borders, rows that see nothing,
strides, and neighbours' keys that must not be read."""
import pytest
import torch

from latent_testutil import NOPE, Ragged
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
SIMT = pkv.PKV_FLAG_SIMT_ONLY


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("q_lens,kv", [([1, 2, 3], [1, 2, 3]), ([9, 40], [37, 100]), ([127, 128, 129], [127, 128, 129]),
                                       ([1, 64, 65], [300, 64, 200]), ([255, 256, 257], [255, 300, 257])])
@pytest.mark.parametrize("mask", ["causal", "none"])
def test_lengths(q_lens, kv, mask, flags):
    Ragged(q_lens, kv, 3, mask=mask, seed=len(q_lens) + kv[0]).check(flags)


@pytest.mark.parametrize("flags", [SIMT, 0])
@pytest.mark.parametrize("H", [1, 2, 5, 16])
def test_heads_and_types(H, flags):
    Ragged([33, 70], [60, 70], H, seed=H, q_pad=3).check(flags, torch.float32)
    Ragged([33, 70], [60, 70], H, seed=H, fused=False).check(flags)


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_rows_that_see_nothing(flags):
    """Empty sequences, queries without keys, more rows than keys."""
    c = Ragged([3, 0, 200, 5, 0], [0, 4, 130, 2, 0], 2, seed=1)
    c.check(flags)
    out, lse, _ = c.run(flags)
    assert (out[:3] == 0).all() and torch.isneginf(lse[:3]).all()
    assert (out[3:73] == 0).all() and torch.isneginf(lse[3:73]).all()   # 70 rows ahead of the first key
    assert (out[-1] == 7).all() and (lse[-1] == 9).all()                # behind the last sequence


@pytest.mark.parametrize("growing,key_size", [(True, 1.0), (False, 6.0), (False, 0.01)])
def test_score_ranges(growing, key_size):
    Ragged([300, 40], [400, 500], 2, growing=growing, key_size=key_size, seed=2).check()


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_no_keys_at_all(flags):
    c = Ragged([3, 2], [0, 0], 4, seed=3)
    k = torch.empty(0, 4, NOPE, dtype=torch.bfloat16, device="cuda")
    out = torch.full((5, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.ragged_attention_latent(c.q_full.cuda()[:5], k, k[:, 0, :64], k, torch.as_tensor(c.qi).cuda(),
                                torch.as_tensor(c.ki).cuda(), out, max_q_rows=3, max_kv_len=0, scale=1.0, flags=flags)
    assert (out == 0).all()


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_nan_stays_in_its_row(flags):
    c = Ragged([130, 20], [200, 20], 3, seed=4)
    clean, cl, _ = c.run(flags)
    c.q_full[77, 1, 5] = float("nan")
    got, gl, _ = c.run(flags)
    assert torch.isnan(got[77, 1]).all() and torch.isnan(gl[77, 1])
    got[77, 1], gl[77, 1] = clean[77, 1], cl[77, 1]
    assert torch.equal(got, clean) and torch.equal(gl, cl)


@pytest.mark.parametrize("flags", [SIMT, 0])
def test_lengths_beyond_the_bounds_are_reported(flags):
    c = Ragged([10, 30], [10, 90], 2, seed=5)
    want = c.run(flags)[0]
    out = torch.full_like(want, 7.0).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    both = c.both.cuda()
    pkv.ragged_attention_latent(c.q_full.cuda(), both[..., :NOPE], c.k_pe.cuda(), both[..., NOPE:],
                                torch.as_tensor(c.qi).cuda(), torch.as_tensor(c.ki).cuda(), out, max_q_rows=20,
                                max_kv_len=90, scale=c.scale, flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
    assert int(err) == pkv.PKV_ERRBIT_LEN
    assert torch.equal(out[:10].cpu(), want[:10]) and (out[30:] == 7).all()


@pytest.mark.parametrize("mask", ["causal", "none"])
def test_more_key_tiles_than_the_ring_repeats_after(mask):
    """The ring's order of blocks repeats every eight key tiles."""
    Ragged([300, 20], [2300, 1100], 2, mask=mask, seed=7).check()


def test_more_pairs_than_run_at_once():
    Ragged([300, 257, 10, 280, 300, 260], [300, 400, 30, 280, 500, 260], 16, seed=8).check()


def test_same_bits_every_time():
    c = Ragged([300, 256], [700, 256], 4, seed=6)
    a, la, _ = c.run()
    for _ in range(3):
        b, lb, _ = c.run()
        assert torch.equal(a, b) and torch.equal(la, lb)
