"""Sizes at the edges of what paged_attention_fp8 and paged_attention_window
take, on the host: nothing here reaches a GPU."""
import pytest

from paged_kv_cache_189_gb300 import pkv
from test_ext_host import L, attend  # noqa: F401  (L is a fixture)

INVALID, UNSUPPORTED = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("mq", [1, 200])
@pytest.mark.parametrize("flags", [0, pkv.PKV_FLAG_SIMT_ONLY])
@pytest.mark.parametrize("fp8", [True, False])
def test_a_pool_without_pages(L, fp8, flags, mq):  # noqa: F811
    """A look-up that fails reads the page behind the pool's last, which the
    copies fill with zeros: of no pages there is no such page."""
    assert attend(L, fp8, pages=0, mq=mq, flags=flags) == INVALID
    assert "without pages" in pkv.last_error()


@pytest.mark.parametrize("flags", [0, pkv.PKV_FLAG_SIMT_ONLY])
@pytest.mark.parametrize("kw", [dict(mq=2 ** 31 - 1), dict(mq=2 ** 31 - 255), dict(mk=2 ** 31 - 1, bts=2 ** 27)])
@pytest.mark.parametrize("fp8", [True, False])
def test_bounds_that_leave_32_bits(L, fp8, kw, flags):  # noqa: F811
    """Rows and keys rounded up to tiles have to stay in 32 bits."""
    assert attend(L, fp8, **kw, flags=flags) == UNSUPPORTED
    assert "2^31 - 256" in pkv.last_error()
    size = pkv.paged_attention_fp8_workspace_size if fp8 else pkv.paged_attention_window_workspace_size
    assert size(2, kw.get("mq", 1), 32, 8, 128, kw.get("mk", 100), 0 if fp8 else 50, 0, flags) == 0
