"""Host checks of the latent entry points and of assign_step_pages: bad
arguments are refused before anything is enqueued, empty calls are accepted."""
import ctypes

import pytest
import torch

from paged_kv_cache_189_gb300 import build as pkv_build
from paged_kv_cache_189_gb300 import pkv

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1002)
BAD, UNS, WS = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


def call(fn, names, defaults, **kw):
    assert set(kw) <= set(defaults)
    a = dict(defaults, **kw)
    return fn(*[a[n] for n in names.split()])


ATTN = "q qts qhs pool pages ps pst bt bts kl qi qr batch mq mk h ld rd mask scale out odt lse ws wsb flags err stream"
ATTN_D = dict(q=FAKE, qts=16 * 576, qhs=576, pool=FAKE, pages=10, ps=32, pst=32 * 576, bt=FAKE, bts=4, kl=FAKE, qi=FAKE,
              qr=None, batch=2, mq=1, mk=100, h=16, ld=512, rd=64, mask=1, scale=0.1, out=FAKE, odt=0, lse=None, ws=None,
              wsb=0, flags=0, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(mk=-1), BAD), (dict(ps=16), UNS), (dict(ld=256), UNS), (dict(rd=32), UNS), (dict(q=None), BAD),
    (dict(pool=None), BAD), (dict(bt=None), BAD), (dict(out=None), BAD), (dict(mask=2), UNS), (dict(mask=7), BAD),
    (dict(odt=1), UNS), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
    (dict(pages=0), BAD), (dict(pst=32 * 576 - 8), BAD), (dict(pst=32 * 576 + 4), BAD), (dict(q=ODD), BAD), (dict(pool=ODD), BAD),
    (dict(out=ODD), BAD), (dict(qts=12), BAD), (dict(qhs=-8), BAD), (dict(bts=3), BAD), (dict(flags=1), BAD), (dict(flags=4), UNS),
    (dict(flags=0x10), UNS), (dict(mk=2 ** 31 - 1, bts=2 ** 27), UNS), (dict(mq=2 ** 31 - 1), UNS), (dict(batch=70000), UNS),
    (dict(batch=60000, mk=2 ** 27, bts=2 ** 22), UNS), (dict(ws=FAKE, wsb=100), WS), (dict(), WS), (dict(ws=ODD, wsb=1 << 30), WS),
    (dict(kl=ODD), BAD), (dict(batch=0), 0), (dict(mq=0), 0), (dict(h=0), 0)])
def test_attention(L, kw, status):
    assert call(L.paged_attention_latent, ATTN, ATTN_D, **kw) == status


RAG = "q qts qhs k kts khs pe pes v vts vhs n qi ki batch mq mk h nd rd vd mask scale out odt lse flags err stream"
RAG_D = dict(q=FAKE, qts=16 * 192, qhs=192, k=FAKE, kts=16 * 256, khs=256, pe=FAKE, pes=64, v=FAKE, vts=16 * 256, vhs=256,
             n=50, qi=FAKE, ki=FAKE, batch=2, mq=9, mk=30, h=16, nd=128, rd=64, vd=128, mask=1, scale=0.1, out=FAKE, odt=0,
             lse=None, flags=0, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(n=-1), BAD), (dict(nd=64), UNS), (dict(rd=128), UNS), (dict(vd=64), UNS), (dict(q=None), BAD),
    (dict(k=None), BAD), (dict(pe=None), BAD), (dict(v=None), BAD), (dict(ki=None), BAD), (dict(out=None), BAD), (dict(mask=2), UNS),
    (dict(mask=9), BAD), (dict(odt=1), UNS), (dict(scale=0.0), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
    (dict(k=ODD), BAD), (dict(kts=12), BAD), (dict(vhs=-8), BAD), (dict(pes=4), BAD), (dict(flags=1), BAD), (dict(flags=8), UNS),
    (dict(batch=70000), UNS), (dict(h=70000), UNS), (dict(mk=2 ** 31 - 1), UNS), (dict(n=2 ** 33), UNS), (dict(mq=2 ** 28), UNS),
    (dict(kts=1 << 40), UNS), (dict(qi=ODD), BAD), (dict(batch=0), 0), (dict(mq=0), 0), (dict(h=0), 0)])
def test_ragged(L, kw, status):
    assert call(L.ragged_attention_latent, RAG, RAG_D, **kw) == status


APP = "src ss T w eps pos cs mp il slots pool pages ps pst ld rd q qts qhs o ots ohs h flags err stream"
APP_D = dict(src=FAKE, ss=576, T=4, w=FAKE, eps=1e-6, pos=FAKE, cs=FAKE, mp=10, il=0, slots=FAKE, pool=FAKE, pages=2, ps=32,
             pst=32 * 576, ld=512, rd=64, q=FAKE, qts=1024, qhs=64, o=FAKE, ots=1024, ohs=64, h=16, flags=0, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(ld=256), UNS), (dict(rd=32), UNS), (dict(ps=64), UNS), (dict(src=None), BAD), (dict(slots=None), BAD),
    (dict(pool=None), BAD), (dict(cs=None), BAD), (dict(pos=None), BAD), (dict(q=None), BAD), (dict(o=None), BAD), (dict(mp=0), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD), (dict(pst=32), BAD), (dict(src=ODD), BAD), (dict(w=ODD), BAD),
    (dict(ss=12), BAD), (dict(qts=12), BAD), (dict(ohs=-8), BAD), (dict(ohs=0), BAD), (dict(ots=8), BAD), (dict(qhs=128), BAD),
    (dict(h=70000), UNS), (dict(T=2 ** 31), UNS), (dict(T=2 ** 28), UNS), (dict(flags=1), BAD), (dict(T=0), 0)])
def test_append(L, kw, status):
    assert call(L.kv_append_latent, APP, APP_D, **kw) == status


PAG = "new kv nf fp cap bt bts batch mt ps ko fo qi slots pos err stream"
PAG_D = dict(new=FAKE, kv=FAKE, nf=FAKE, fp=FAKE, cap=10, bt=FAKE, bts=4, batch=2, mt=5, ps=32, ko=FAKE, fo=FAKE, qi=FAKE,
             slots=FAKE, pos=FAKE, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(mt=-1), BAD), (dict(cap=-1), BAD), (dict(bts=-1), BAD), (dict(new=None), BAD), (dict(fp=None), BAD),
    (dict(bt=None), BAD), (dict(ko=None), BAD), (dict(fo=None), BAD), (dict(qi=None), BAD), (dict(slots=None), BAD), (dict(pos=None), BAD),
    (dict(ps=16), UNS), (dict(batch=4097), UNS), (dict(mt=2 ** 30 + 1), UNS), (dict(cap=2 ** 32), UNS), (dict(bts=2 ** 27), UNS),
    (dict(new=ctypes.c_void_p(0x1001)), BAD), (dict(slots=ctypes.c_void_p(0x1004)), BAD), (dict(batch=0), 0)])
def test_step_pages(L, kw, status):
    assert call(L.assign_step_pages, PAG, PAG_D, **kw) == status


def test_workspace_sizes(L):
    size = pkv.paged_attention_latent_workspace_size
    assert size(0, 1, 16, 100) == 0 and size(2, 1, 16, 100, flags=pkv.PKV_FLAG_SIMT_ONLY) == 0
    assert size(2, 2 ** 30, 16, 100) == 0       # more columns than a call takes
    assert size(60000, 1, 16, 2 ** 27) == 0     # more key tiles
    # a partial state of a first and a last segment for every cluster, 16 columns of 512 f32 and their LSEs
    assert 152 * 2 * 16 * 513 * 4 <= size(64, 1, 16, 8192) <= 152 * 2 * 16 * 513 * 4 + 8192
    assert size(2, 1, 16, 60) < size(2, 1, 16, 6000)
    assert L.paged_attention_latent_workspace_size(2, 1, 16, 100, 256, 64, 0) == 0


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_tensors():
    """Wrong types, shapes, strides and devices raise ValueError before a pointer is handed out."""
    i32 = lambda n: cpu(n, dtype=torch.int32)  # noqa: E731
    i64 = lambda n: cpu(n, dtype=torch.int64)  # noqa: E731
    q, pool, bt = cpu(2, 4, 576), cpu(3, 32, 576), cpu(2, 4, dtype=torch.int32)
    kw = dict(max_q_rows=1, max_kv_len=100, scale=1.0)

    def attn(q=q, pool=pool, bt=bt, kl=i32(2), qi=i32(3), out=cpu(2, 4, 512), **more):
        pkv.paged_attention_latent(q, pool, bt, kl, qi, out, **dict(kw, **more))
    for bad in (dict(q=q.float()), dict(q=cpu(2, 4, 512)), dict(q=cpu(2, 576, 4).transpose(1, 2)), dict(pool=pool.float()),
                dict(pool=cpu(3, 32, 512)), dict(pool=cpu(3, 64, 576)[:, ::2]), dict(out=cpu(2, 4, 576)),
                dict(out=cpu(2, 8, 512)[:, ::2]), dict(lse=cpu(2, 4)), dict(kl=i64(2)), dict(qi=i32(2)), dict(bt=i32(8)),
                dict(bt=cpu(2, 3, dtype=torch.int32)), dict(mask="windowed"), dict(workspace=cpu(8, 8)[:, ::2]), dict(err=i64(1)),
                dict()):  # the last: CPU tensors
        with pytest.raises(ValueError):
            attn(**bad)

    def ragged(q=cpu(5, 4, 192), k=cpu(6, 4, 128), pe=cpu(6, 64), v=cpu(6, 4, 128), qi=i32(2), ki=i32(2), out=cpu(5, 4, 128), **more):
        pkv.ragged_attention_latent(q, k, pe, v, qi, ki, out, **dict(kw, **more))
    for bad in (dict(q=cpu(5, 4, 128)), dict(k=cpu(6, 3, 128)), dict(v=cpu(5, 4, 128)), dict(pe=cpu(6, 128)), dict(k=cpu(6, 4, 128).float()),
                dict(qi=i64(2)), dict(ki=i32(1)), dict(out=cpu(5, 4, 192)), dict(mask="x"), dict()):
        with pytest.raises(ValueError):
            ragged(**bad)

    def append(src=cpu(3, 576), pos=i64(3), cs=cpu(9, 64, dtype=torch.float32), slots=i64(3), pool=pool, **more):
        pkv.kv_append_latent(src, pos, cs, slots, pool, **more)
    for bad in (dict(src=cpu(3, 512)), dict(src=cpu(576, 3).t()), dict(pos=i32(3)), dict(slots=i64(2)), dict(cs=cpu(9, 64)),
                dict(cs=cpu(9, 32, dtype=torch.float32)), dict(norm_weight=cpu(511)), dict(norm_weight=cpu(512).float()),
                dict(q_pe=cpu(3, 2, 64)), dict(q_pe=cpu(3, 2, 64), q_out=cpu(3, 3, 64)), dict(q_pe=cpu(2, 2, 64), q_out=cpu(2, 2, 64)),
                dict()):
        with pytest.raises(ValueError):
            append(**bad)

    def step(new=i32(2), kv=i32(2), nf=i32(1), fp=i32(9), bt=bt, ko=i32(2), fo=i32(1), qi=i32(3), slots=i64(4), pos=i64(4), **more):
        pkv.assign_step_pages(new, kv, nf, fp, bt, kv_lens_out=ko, num_free_out=fo, q_indptr=qi, slots=slots, positions=pos, **more)
    for bad in (dict(new=i64(2)), dict(kv=i32(1)), dict(nf=i32(0)), dict(fp=i64(9)), dict(bt=cpu(2, 8, dtype=torch.int32)[:, ::2]),
                dict(bt=cpu(1, 4, dtype=torch.int32)), dict(ko=i32(1)), dict(qi=i32(2)), dict(slots=i32(4)), dict(pos=i64(3)),
                dict(err=i64(1)), dict()):
        with pytest.raises(ValueError):
            step(**bad)
