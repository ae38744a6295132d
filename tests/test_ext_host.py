"""Refusals of the 8-bit cache's and the windowed attention's entry points, on
the host: nothing here reaches a GPU."""
import ctypes

import pytest
import torch

from paged_kv_cache_189_gb300 import build as pkv_build
from paged_kv_cache_189_gb300 import pkv

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1002)
INVALID, UNSUPPORTED, WORKSPACE = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


def append(L, **kw):
    a = dict(k=FAKE, v=FAKE, dt=0, ts=8 * 128, hs=128, bt=FAKE, bts=4, kl=FAKE, qi=FAKE, qr=None, batch=2, mq=1,
             mk=100, hkv=8, d=128, kp=FAKE, vp=FAKE, pages=10, ps=32, pstride=32 * 8 * 128, ks=FAKE, vs=FAKE,
             ss=8, flags=0, err=None)
    a.update(kw)
    return L.kv_append_fp8(*[a[n] for n in ("k", "v", "dt", "ts", "hs", "bt", "bts", "kl", "qi", "qr", "batch",
                                            "mq", "mk", "hkv", "d", "kp", "vp", "pages", "ps", "pstride", "ks",
                                            "vs", "ss", "flags", "err")], None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=7), INVALID), (dict(batch=-1), INVALID), (dict(k=None), INVALID), (dict(ks=None), INVALID),
    (dict(ps=16), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(pstride=100), INVALID),
    (dict(pstride=32 * 8 * 128 + 8), INVALID), (dict(ss=7), INVALID), (dict(k=ODD), INVALID), (dict(ts=1001), INVALID),
    (dict(hs=-128), INVALID), (dict(kp=ODD), INVALID), (dict(vs=ODD), INVALID), (dict(mk=129), INVALID),
    (dict(batch=70000), UNSUPPORTED), (dict(flags=pkv.PKV_FLAG_CHECKED), INVALID),
    (dict(batch=0), pkv.PKV_OK), (dict(mq=0), pkv.PKV_OK), (dict(mk=0), pkv.PKV_OK)])
def test_append_refusals(L, kw, want):
    assert append(L, **kw) == want
    assert (pkv.last_error() == "") == (want == pkv.PKV_OK)


def attend(L, fp8, **kw):
    a = dict(q=FAKE, qts=32 * 128, qhs=128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, ss=8, pages=10, ps=32,
             pstride=32 * 8 * 128, bt=FAKE, bts=4, kl=FAKE, qi=FAKE, qr=None, batch=2, mq=1, mk=100, hq=32, hkv=8,
             d=128, mask=1, cb=0, window=0 if fp8 else 50, sinks=0, scale=0.0, out=FAKE, odt=0, lse=None, ws=None,
             wsb=0, flags=pkv.PKV_FLAG_SIMT_ONLY, err=None)
    a.update(kw)
    names = ("q", "qts", "qhs", "k", "v", "ks", "vs", "ss", "pages", "ps", "pstride", "bt", "bts", "kl", "qi", "qr",
             "batch", "mq", "mk", "hq", "hkv", "d", "mask", "cb", "window", "sinks", "scale", "out", "odt", "lse",
             "ws", "wsb", "flags", "err")
    if not fp8:
        names = [n for n in names if n not in ("ks", "vs", "ss", "mask", "cb")]
    return (L.paged_attention_fp8 if fp8 else L.paged_attention_window)(*[a[n] for n in names], None)


COMMON = [
    (dict(q=None), INVALID), (dict(bt=None), INVALID), (dict(out=None), INVALID), (dict(hq=30), INVALID),
    (dict(batch=-1), INVALID), (dict(sinks=-1), INVALID), (dict(ps=64), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(odt=pkv.PKV_F16), UNSUPPORTED), (dict(batch=70000), UNSUPPORTED), (dict(pstride=1000), INVALID),
    (dict(pstride=32 * 8 * 128 + 4), INVALID), (dict(q=ODD), INVALID), (dict(k=ODD), INVALID), (dict(qts=4), INVALID),
    (dict(out=ODD), INVALID), (dict(bts=3), INVALID), (dict(flags=pkv.PKV_FLAG_CHECKED), INVALID),
    (dict(flags=pkv.PKV_FLAG_TEST_WAIT_TIMEOUT), INVALID),
    (dict(flags=pkv.PKV_FLAG_STREAM_K), UNSUPPORTED), (dict(batch=0), pkv.PKV_OK), (dict(mq=0), pkv.PKV_OK)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(ks=None), INVALID), (dict(ss=7), INVALID), (dict(vs=ODD), INVALID), (dict(mask=5), INVALID),
    (dict(mask=2), INVALID), (dict(window=-1), INVALID), (dict(sinks=4), INVALID),
    (dict(mask=0, window=9), UNSUPPORTED), (dict(mask=2, cb=4, window=9), UNSUPPORTED)])
def test_fp8_refusals(L, kw, want):
    assert attend(L, True, **kw) == want
    assert (pkv.last_error() == "") == (want == pkv.PKV_OK)


@pytest.mark.parametrize("kw,want", COMMON + [(dict(window=0), INVALID), (dict(window=-5), INVALID)])
def test_window_refusals(L, kw, want):
    assert attend(L, False, **kw) == want
    assert (pkv.last_error() == "") == (want == pkv.PKV_OK)


@pytest.mark.parametrize("fp8", [True, False])
def test_workspaces(L, fp8):
    """A workspace where the call needs one: none for a short cache, partial
    states for a long one, the expanded pages of an 8-bit prompt chunk."""
    def size(batch, rows, kv, window=0 if fp8 else 10 ** 6, heads=(32, 8), D=128, flags=0):
        f = pkv.paged_attention_fp8_workspace_size if fp8 else pkv.paged_attention_window_workspace_size
        return f(batch, rows, *heads, D, kv, window, 0, flags)
    assert size(2, 1, 100) == 0 and size(0, 1, 100) == 0 and size(2, 1, 0) == 0
    assert size(2, 1, 10 ** 5, flags=pkv.PKV_FLAG_SIMT_ONLY) == 0
    long = size(2, 1, 10 ** 5)
    assert long > 0 and size(200, 1, 10 ** 5) > long
    chunk = size(4, 2048, 8192)
    if fp8:
        assert chunk >= 2 * 4 * 8192 * 8 * 128 * 2
        assert size(4, 2048, 8192, window=1000) < chunk  # only the window's pages are expanded
    kw = dict(flags=0, mk=8192, bts=256, ws=FAKE, wsb=1 << 40)
    if fp8:
        assert attend(L, fp8, mq=200, mk=8192, bts=256, flags=0, ws=None) == WORKSPACE
    assert attend(L, fp8, **{**kw, "ws": ctypes.c_void_p(0x1010)}, mq=1, window=0 if fp8 else 8192) == WORKSPACE  # misaligned
    assert attend(L, fp8, **{**kw, "wsb": 100}, mq=1, window=0 if fp8 else 8192) == WORKSPACE                    # too small


def test_binding_refusals(L):
    """The binding names what does not fit before it hands out a pointer."""
    D, H, n = 64, 2, 3
    kp = torch.zeros(n, 32, H, D, dtype=torch.uint8).view(torch.float8_e4m3fn)
    vp, sc = kp.clone(), torch.ones(n, H)
    q = torch.zeros(1, 4, D, dtype=torch.bfloat16)
    bt, one, qi = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.tensor([0, 1]).int()
    out = torch.empty_like(q)

    def fp8(**kw):
        a = dict(q=q, k_pool=kp, v_pool=vp, k_scale=sc, v_scale=sc, block_table=bt, kv_lens=one, q_indptr=qi, out=out,
                 max_q_rows=1, max_kv_len=1)
        a.update(kw)
        pkv.paged_attention_fp8(**a)

    for kw in (dict(k_pool=kp.float(), v_pool=vp.float()), dict(k_scale=sc.double()), dict(v_scale=sc[:2]),
               dict(q=q.float()), dict(q=q[..., :32]), dict(out=out[:, :2]), dict(block_table=bt.long()),
               dict(kv_lens=one.long()), dict(q_indptr=qi[:1]), dict(lse=torch.empty(1, 4, dtype=torch.float64)),
               dict(q_real=one.float()), dict(v_pool=vp[:2]), dict()):  # the last: tensors that are not on a GPU
        with pytest.raises(ValueError):
            fp8(**kw)
    x = torch.zeros(1, H, D, dtype=torch.bfloat16)
    for kw in (dict(k_src=x.double(), v_src=x.double()), dict(v_src=x.float()), dict(k_src=x[:, :1]), dict()):
        a = dict(k_src=x, v_src=x, block_table=bt, kv_lens=one, q_indptr=qi, k_pool=kp, v_pool=vp, k_scale=sc,
                 v_scale=sc, max_q_rows=1, max_kv_len=1)
        a.update(kw)
        with pytest.raises(ValueError):
            pkv.kv_append_fp8(**a)
    kb = torch.zeros(n, 32, H, D, dtype=torch.bfloat16)
    for kw in (dict(k_pool=kb.half(), v_pool=kb.half()), dict(q=q.float()), dict()):
        a = dict(q=q, k_pool=kb, v_pool=kb, block_table=bt, kv_lens=one, q_indptr=qi, out=out, window=4, max_q_rows=1,
                 max_kv_len=1)
        a.update(kw)
        with pytest.raises(ValueError):
            pkv.paged_attention_window(**a)
