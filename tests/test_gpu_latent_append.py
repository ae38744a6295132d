"""kv_append_latent against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from latent_testutil import BF16_STEP, L, P, R
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
MAX_POS = 300


def angles():
    a = np.arange(MAX_POS)[:, None] * 10000.0 ** (-np.arange(R // 2) / (R // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


def rotated(x, cs, interleaved):
    """(value, sum of the magnitudes of its two products)."""
    x, cs = x.double(), cs.double()
    c, s = cs[..., :R // 2], cs[..., R // 2:]
    out, mag = torch.empty_like(x), torch.empty_like(x)
    ia = torch.arange(R // 2) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else R // 2)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, mag


def close(got, want, mag):
    """One rounding to bf16 of a value that f32 arithmetic (a few operations on
    terms of size `mag`: 4 * 2^-24 for products and sum; the norm: a sum of 512
    squares over a warp, 16 in a chain and 5 levels, a square root and a
    division, within 2^-19) gives."""
    tol = BF16_STEP * want.abs() + 2.0 ** -18 * mag + 2.0 ** -133
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), bad.nonzero()[:4]


def run_case(T, H, interleaved=False, norm=True, size=1.0, seed=0, in_place=False, slots=None, positions=None, checked=True):
    g = torch.Generator().manual_seed(seed)
    num_pages = T // P + 3
    proj = (torch.randn(T, 40 + L + R + 8, generator=g) * size).to(torch.bfloat16).cuda()
    src = proj[:, 40:40 + L + R]
    w = torch.randn(L, generator=g).to(torch.bfloat16).cuda() if norm else None
    pool = torch.full((num_pages, P, L + R), 3.0, dtype=torch.bfloat16, device="cuda")
    if slots is None:
        slots = torch.randperm(num_pages * P, generator=g)[:T]
        slots[::5] = -1
    if positions is None:
        positions = torch.randint(0, MAX_POS, (T,), generator=g)
    q = torch.randn(T, H, 128 + R, generator=g).to(torch.bfloat16).cuda()
    before = q.clone()
    q_rows = q if in_place else torch.full((T, H, L + R), 5.0, dtype=torch.bfloat16, device="cuda")
    q_out = q[..., 128:] if in_place else q_rows[..., L:]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv_append_latent(src, positions.cuda(), angles().cuda(), slots.cuda(), pool, norm_weight=w, eps=1e-5,
                         q_pe=q[..., 128:] if H else None, q_out=q_out if H else None, interleaved=interleaved,
                         checked=checked, err=err)
    cs = angles()[positions.clamp(0, MAX_POS - 1)]
    x = src.cpu().double()
    want = torch.full((num_pages * P, L + R), 3.0, dtype=torch.float64)
    mag = torch.zeros_like(want)
    lat = x[:, :L]
    if norm:
        lat = lat / torch.sqrt(lat.square().mean(1, keepdim=True) + 1e-5) * w.cpu().double()
    pe, pe_mag = rotated(x[:, L:], cs, interleaved)
    ok = (slots >= 0) & (slots < num_pages * P)
    want[slots[ok]] = torch.cat([lat, pe], 1)[ok]
    mag[slots[ok]] = torch.cat([lat.abs(), pe_mag], 1)[ok]
    close(pool.cpu().view(-1, L + R), want, mag)
    if not norm:
        assert torch.equal(pool.cpu().view(-1, L + R)[slots[ok]][:, :L], src.cpu()[ok][:, :L])
    if H:
        qw, qm = rotated(before.cpu()[..., 128:], cs[:, None], interleaved)
        close(q_out.cpu(), qw, qm)
        if in_place:
            assert torch.equal(q[..., :128], before[..., :128])
        else:
            assert (q_rows[..., :L] == 5).all()
    return int(err)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 16), (2, 1), (7, 3), (33, 8), (100, 33), (5, 128), (9, 0)])
def test_against_plain(T, H, interleaved):
    assert run_case(T, H, interleaved, seed=T) == 0


@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_sizes_and_no_norm(size):
    run_case(20, 4, size=size, seed=1)
    run_case(20, 4, size=size, norm=False, seed=2)


def test_in_place_queries():
    run_case(20, 4, in_place=True, seed=3)
    run_case(20, 4, in_place=True, interleaved=True, seed=3)


def test_zero_rows_keep_zero():
    """A row of zeros has no size to divide by: eps keeps it zero."""
    pool = torch.full((1, P, L + R), 3.0, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(1, dtype=torch.int64, device="cuda")
    pkv.kv_append_latent(torch.zeros(1, L + R, dtype=torch.bfloat16, device="cuda"), z, angles().cuda(), z, pool,
                         norm_weight=torch.ones(L, dtype=torch.bfloat16, device="cuda"))
    assert (pool[0, 0] == 0).all() and (pool[0, 1:] == 3).all()


def test_bad_slots_and_positions():
    slots, positions = torch.tensor([0, 5, 4 * P, 1 << 40, -3]), torch.tensor([0, 1, 2, 3, 4])
    assert run_case(5, 2, slots=slots, positions=positions) == pkv.PKV_ERRBIT_SLOT
    assert run_case(5, 2, slots=slots, positions=positions, checked=False) == 0
    slots, positions = torch.tensor([0, 5, 7]), torch.tensor([-1, MAX_POS, 3])
    assert run_case(3, 2, slots=slots, positions=positions) == pkv.PKV_ERRBIT_LEN


def test_no_tokens():
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    pool = torch.ones(1, P, L + R, dtype=torch.bfloat16, device="cuda")
    pkv.kv_append_latent(torch.empty(0, L + R, dtype=torch.bfloat16, device="cuda"), e, angles().cuda(), e, pool)
    assert (pool == 1).all()
