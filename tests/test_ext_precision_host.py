"""The tolerance that holds the few-row kernel over 8-bit pools to weights of 11
bits: on the host, the definition with weights of 11 bits is inside it, with
weights of 8 bits (bf16's) outside."""
import math

import numpy as np
import pytest

from ext_testutil import P
from test_gpu_ext_precision import CASES, bounds, few_rows


def rounded(c, bits):
    """What the definition gives with weight x scale rounded to so many bits."""
    O = np.zeros((sum(c.rows), c.Hq, c.D))
    _, L, _, _ = c.reference()
    G = c.Hq // c.Hkv
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
            w = np.exp(s - L[r].reshape(c.Hkv, G, 1)) * vs.T[:, None, :]
            step = np.exp2(np.floor(np.log2(w)) - bits + 1)
            O[r] = np.einsum("hgk,khd->hgd", np.round(w / step) * step, V / vs[..., None]).reshape(c.Hq, c.D)
    return O


@pytest.mark.parametrize("case", CASES)
def test_the_tolerance_tells_eleven_bits_from_eight(case):
    c = few_rows(*case)
    O, L, tol, norm, _ = bounds(c, 2.0 ** -11)
    err = {bits: rounded(c, bits) - O for bits in (11, 8)}
    assert (abs(err[11]) <= tol).all() and (np.linalg.norm(err[11], axis=-1) <= norm).all()
    # (in longer rows the bound on their sums' own error hides the weights')
    short = np.array([0 < len(c.row_keys(b, i)) <= 1000 for b in range(len(c.kv)) for i in range(c.rows[b])])
    assert short.any() and (np.linalg.norm(err[8], axis=-1) > norm)[short].mean() > 0.9
