"""V scales far from 1, in all pages alike."""
import numpy as np
import pytest
import torch

from ext_testutil import Case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("e", [-126, -110, -95, 93, 98, 110, 118])
def test_v_scales_beyond_the_range(e, rows):
    """Too small: what is lost is far below any output; too large: infinite, not
    small.  The LSE is right with either."""
    c = Case([500, 300], [rows] * 2, [rows] * 2, 8, 2, 128, True, seed=74)
    c.v_scale = torch.full_like(c.v_scale, 2.0 ** e)
    c.v64 = np.nan_to_num(c.v_pool.double().numpy()) * 2.0 ** e
    out, lse = run(c, out_dtype=torch.float32)
    O, L, A, S = c.reference()
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    es = c.D * 2.0 ** -24 * S
    assert (abs(gl - L) <= es + 2.0 ** -18 + 2.0 ** -22 * abs(L)).all()
    tol = (2 * 2.0 ** -8 + 2 * es + 2.0 ** -20)[..., None] * A + 2.0 ** -24 * abs(O) + max(c.kv) * 2.0 ** -102
    assert ((abs(got - O) <= tol) | ((e > 90) & ~np.isfinite(got))).all()
