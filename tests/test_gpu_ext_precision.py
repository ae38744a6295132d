"""How many bits the softmax weights keep on their way into the P.V product.

The few-row kernel over 8-bit pools rounds weight x V scale once to f16, the
generic kernel nothing; the general tolerance of the other tests allows bf16
weights everywhere, this one tells f16 from bf16.

With u = 2^-11 (half a step of f16), D dimensions, S the largest sum of
|q_d k_d| of a row, n its keys, A = sum_j w_j |v_j|, all relative:
 * a score sums D products in f32 and takes three factors: (D + 3) 2^-24 S;
   a weight is off by twice that (its own and the sum's), and by 2^-20 for its
   exponential, the sum's and the factors that join states;
 * f16: u relative, or half the subnormal step 2^-25; the largest w of a state is
   2^6 at least, so 2^-31 of it (and of the row's) for each key;
 * a matrix step adds 16 products to a sum: 16 * 2^-24 for aligning them, and the
   sum cut at 2^-22; a warp makes n / 64 steps at most (16 keys a step, 4 warps);
 * the output's own rounding."""
import math

import numpy as np
import pytest
import torch

from ext_testutil import P, Case, e4m3_grid, run
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


def bounds(c, weight):
    """O, LSE, the tolerance of every output element, of every row and head's
    norm, and of every LSE; weight: half a step of the rounded weights, or 0."""
    O, L, A, S = c.reference()
    total, G = sum(c.rows), c.Hq // c.Hkv
    sub, B, steps = np.zeros_like(O), np.zeros_like(O), np.zeros((total, 1))
    q = c.q_full[:, :c.Hq].double().numpy()
    scale = c.v_scale.double().numpy()
    for b in range(len(c.kv)):
        for i in range(c.rows[b]):
            j = c.row_keys(b, i)
            if not len(j):
                continue
            r = c.indptr[b] + i
            ph = c.table[b, j // P]
            K, V, vs = c.k64[ph, j % P], c.v64[ph, j % P], scale[ph]
            s = np.einsum("hgd,khd->hgk", q[r].reshape(c.Hkv, G, c.D) / math.sqrt(c.D), K)
            w = np.exp(s - L[r].reshape(c.Hkv, G, 1))
            top = (w * vs.T[:, None, :]).max(-1)                                   # [Hkv, G]
            code = np.where(vs > 0, 1 / np.where(vs > 0, vs, 1), 0)[..., None] * abs(V)
            sub[r] = np.einsum("hg,hd->hgd", top, code.sum(0)).reshape(c.Hq, c.D) * 2.0 ** -31
            B[r] = np.sqrt(np.einsum("hgk,khd->hgd", w ** 2, V ** 2)).reshape(c.Hq, c.D)
            steps[r] = len(j) / 64 + 1
    es = (c.D + 3) * 2.0 ** -24 * S
    rest = 2 * es + 2 * 2.0 ** -20 + steps * 2.0 ** -22
    if not weight:
        sub = sub * 0
        rest = 2 * es + 2.0 ** -20 + 64 * steps * 2.0 ** -23  # key after key in f32
    tol = (weight + rest)[..., None] * A + sub
    # independent roundings add up as their squares; twice that for their spread
    norm = 2 * weight * np.linalg.norm(B, axis=-1) + rest * np.linalg.norm(A, axis=-1) + np.linalg.norm(sub, axis=-1)
    return O, L, tol, norm, es + 2.0 ** -18 + 2.0 ** -22 * abs(np.where(np.isneginf(L), 0, L))


def hold(c, out, lse, weight):
    O, L, tol, norm, tl = bounds(c, weight)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    u = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    none = np.isneginf(L)
    assert (got[none] == 0).all() and np.isneginf(gl[none]).all()
    err = abs(got - O)
    assert (err <= tol + u * abs(O)).all(), np.max(err - tol - u * abs(O))
    rows = np.linalg.norm(err, axis=-1) - norm - u * np.linalg.norm(O, axis=-1)
    assert (rows <= 0).all(), rows.max()
    assert (abs(np.where(none, 0, gl) - np.where(none, 0, L)) <= tl).all()


CASES = [  # kv, new rows, padding rows, Hq, Hkv, D, window
    ([40, 300, 257], 1, 0, 32, 8, 128, 0), ([40, 300, 257], 1, 0, 8, 1, 64, 0), ([250, 300], 4, 1, 8, 2, 128, 0),
    ([250, 300], 3, 0, 16, 2, 64, 0), ([400, 900], 1, 0, 8, 2, 128, 200), ([9000, 700], 1, 0, 8, 2, 128, 0),
    ([9000, 700], 4, 0, 8, 2, 128, 0), ([9000, 700], 3, 1, 8, 2, 64, 0), ([9000, 700], 20, 0, 8, 2, 128, 0)]


def few_rows(kv, new, pad, Hq, Hkv, D, window):
    # small scores: their own error does not hide the weights'
    return Case(kv, [new] * len(kv), [new + pad] * len(kv), Hq, Hkv, D, True, window=window, sinks=3 if window else 0,
                seed=70, key_size=0.05)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_weights_keep_eleven_bits(case, out_dtype):
    c = few_rows(*case)
    assert c.max_rows() * c.Hq // c.Hkv <= 80  # the few-row kernel's
    hold(c, *run(c, out_dtype=out_dtype), 2.0 ** -11)


@pytest.mark.parametrize("case", CASES[:5])
def test_generic_kernel_rounds_no_weight(case):
    c = few_rows(*case)
    hold(c, *run(c, out_dtype=torch.float32, flags=pkv.PKV_FLAG_SIMT_ONLY), 0)


def pointed(n, octaves, top, D=128):
    """One key far above n - 1 others, whose weights are 2^-octaves of its; V is
    1, and `top` for the one."""
    c = Case([n], [1], [1], 4, 1, D, True, seed=71)
    k, v = np.zeros_like(c.k64), np.ones_like(c.v64)
    at = c.table[0, n // 3 // P], n // 3 % P
    k[at][0, 0] = 1.0
    v[at] = top
    c.k_pool, c.v_pool = (torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn) for x in (k, v))
    c.k_scale, c.v_scale = torch.ones_like(c.k_scale), torch.ones_like(c.v_scale)
    c.k64, c.v64 = k, v
    c.q_full = torch.zeros_like(c.q_full)
    c.q_full[..., 0] = octaves * math.log(2) * math.sqrt(D)
    return c


@pytest.mark.parametrize("top", [1.0, 0.0])
@pytest.mark.parametrize("octaves", [13, 18, 22, 25.3, 27])
@pytest.mark.parametrize("n", [1500, 60000])
def test_many_small_weights(n, octaves, top):
    """Weights far below the largest one's add up, and count by themselves where
    its V is 0."""
    c = pointed(n, octaves, top)
    out, lse = run(c, out_dtype=torch.float32)
    hold(c, out, lse, 2.0 ** -11)


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("e", [-80, -40, 40, 80, 90])
def test_v_scales_of_the_whole_range(e, rows):
    c = Case([500, 9000], [rows] * 2, [rows] * 2, 8, 2, 128, True, seed=72, key_size=0.05)
    c.v_scale = torch.from_numpy(np.exp2(np.random.default_rng(73).integers(-3, 1, size=c.v_scale.shape) + e)).float()
    if e < 0:
        c.v_scale *= 8
    codes = e4m3_grid(c.v_pool.double().numpy())
    c.v64 = codes * c.v_scale.double().numpy()[:, None, :, None]
    out, lse = run(c, out_dtype=torch.float32)
    hold(c, out, lse, 2.0 ** -11)
