"""kv_append_latent refuses query outputs whose rows overlap: CTAs would write
the same elements in no order."""
import pytest

from paged_kv_cache_189_gb300 import build as pkv_build
from paged_kv_cache_189_gb300 import pkv
from test_latent_host import APP, APP_D, BAD, call

WIDE = 1 << 20


@pytest.fixture(scope="module")
def entry():
    pkv_build.build()
    return pkv.lib().kv_append_latent


# page_size is checked ahead of the strides, the missing error flag of checked mode behind them
@pytest.mark.parametrize("T,h,ots,ohs,overlap", [
    (4, 16, 1024, 64, False), (4, 16, 64, 256, False), (4, 16, 9216, 576, False), (4, 16, 576, 4 * 576, False),
    (4, 16, 64, 64, True),        # (token, head + 1) is (token + 1, head)
    (4, 16, 1016, 64, True),      # the last head ends in the next token
    (4, 16, 128, 64, True), (4, 16, 64, 248, True), (4, 16, 72, 136, True), (4, 16, 0, 64, True), (4, 16, 1024, 56, True),
    (1, 16, 0, 64, False), (1, 16, 0, 56, True), (4, 1, 64, 0, False), (4, 1, 56, 0, True), (1, 1, 0, 0, False),
    (3, 9, WIDE, WIDE // 16, False), (3, 19, WIDE, WIDE // 16, True), (2 ** 14, 16, 2 ** 61, 2 ** 57, False),
    (2, 2, 2 ** 61, 2 ** 61, True)])
def test_rows_of_the_output(entry, T, h, ots, ohs, overlap):
    status = call(entry, APP, APP_D, T=T, h=h, ots=ots, ohs=ohs, qts=ots, qhs=ohs, flags=pkv.PKV_FLAG_CHECKED, err=None)
    assert status == BAD
    assert ("overlap" in pkv.last_error()) == overlap, pkv.last_error()
