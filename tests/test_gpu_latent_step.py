"""The latent operators as a serving step uses them: page tables and slot map,
append, attention, in one captured graph that is replayed while sequences grow,
finish and start; a prompt's expanded attention joined with its cached prefix;
calls on two streams at once; caches whose offsets pass 32 bits."""
import math

import numpy as np
import pytest
import torch

from latent_testutil import BF16_STEP, L, NOPE, P, R, V, attend, compare
from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(192)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("H", [16, 128])
def test_captured_step_while_sequences_grow(H):
    """Every replay: new_lens asks for one to three tokens a sequence, one ends
    and starts again.  The oracle keeps each sequence's rows in a list."""
    B, T, pages, width, steps = 5, 16, 40, 9, 9
    g = torch.Generator().manual_seed(H)
    pool = torch.full((pages, P, L + R), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    kv, new, num_free = i32([0] * B), i32([0] * B), i32([pages])
    free = i32(list(range(pages)) + [-1] * 4)
    qi = i32([0] * (B + 1))
    slots, positions = (torch.zeros(T, dtype=torch.int64, device=DEV) for _ in range(2))
    a = np.arange(400)[:, None] * 10000.0 ** (-np.arange(R // 2) / (R // 2))
    cos_sin = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float().to(DEV)
    src, w = torch.zeros(T, L + R, dtype=torch.bfloat16, device=DEV), torch.ones(L, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(T, H, 128 + R, dtype=torch.bfloat16, device=DEV)
    rows = torch.zeros(T, H, L + R, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(T, H, L, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, H, device=DEV)
    err = i32([0])
    ws = torch.empty(pkv.paged_attention_latent_workspace_size(B, T, H, width * P), dtype=torch.uint8, device=DEV)

    def step():
        pkv.assign_step_pages(new, kv, num_free, free, table, kv_lens_out=kv, num_free_out=num_free, q_indptr=qi,
                              slots=slots, positions=positions, err=err)
        pkv.kv_append_latent(src, positions, cos_sin, slots, pool, norm_weight=w, q_pe=q[..., 128:], q_out=rows[..., L:],
                             checked=True, err=err)
        pkv.paged_attention_latent(rows, pool, table, kv, qi, out, lse=lse, max_q_rows=T, max_kv_len=width * P, scale=SCALE,
                                   workspace=ws, flags=pkv.PKV_FLAG_CHECKED, err=err)
    step()  # nothing asked for: nothing done
    torch.cuda.synchronize()
    assert kv.tolist() == [0] * B and int(num_free) == pages
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [0] * B
    for n in range(steps):
        ask = [1 + (n + b) % 3 for b in range(B)] if n else [70, 33, 1, 0, 64]
        T_now = sum(ask)
        if n == 4:
            ask[0] = -1
            T_now = sum(x for x in ask if x > 0)
        if n == 0:  # prompts do not fit the captured step's 16 tokens: refused, and asked for in pieces
            new.copy_(i32(ask))
            graph.replay()
            torch.cuda.synchronize()
            assert int(err) == pkv.PKV_ERRBIT_LEN and kv.tolist() == [0] * B and qi.tolist() == [0] * (B + 1)
            err.zero_()
            for part in range(14):
                new.copy_(i32([5 if b != 2 else 1 for b in range(3)] + [0, 5]))
                src.copy_(torch.randn(T, L + R, generator=g))
                graph.replay()
                held = [h + x for h, x in zip(held, [5, 5, 1, 0, 5])]
            torch.cuda.synchronize()
            assert int(err) == 0 and kv.tolist() == held
            continue
        new.copy_(i32(ask))
        src.copy_(torch.randn(T, L + R, generator=g))
        q.copy_(torch.randn(T, H, 128 + R, generator=g))
        rows[..., :L].copy_(torch.randn(T, H, L, generator=g))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        held = [0 if x < 0 else h + x for h, x in zip(held, ask)]
        assert int(err) == 0 and kv.tolist() == held
        ends = np.cumsum([max(x, 0) for x in ask])
        assert qi.tolist() == [0] + ends.tolist()
        used = [table[b, :(held[b] + P - 1) // P].tolist() for b in range(B)]
        flat = sum(used, [])
        assert len(set(flat)) == len(flat) == pages - int(num_free)     # every page has one owner
        want, wl = np.full((T, H, L), 7.0), np.zeros((T, H))
        to, tl = np.zeros_like(want), np.zeros_like(wl)
        p64, r64 = pool.double().cpu().numpy(), rows.double().cpu().numpy()
        for b in range(B):
            j = np.arange(held[b])
            c = p64[np.array(used[b], dtype=int)[j // P], j % P] if held[b] else np.zeros((0, L + R))
            real = max(ask[b], 0)
            for i in range(real):
                r, k = ends[b] - real + i, held[b] - real + i + 1
                want[r], wl[r], to[r], tl[r] = attend(r64[r], c[:k], c[:k, :L], SCALE)
        lse[T_now:] = 0
        compare(out.cpu(), lse.cpu(), want, wl, to, tl, torch.bfloat16)


def test_prompt_joined_with_its_cached_prefix():
    """Absorbed attention over the cached prefix, expanded over the new tokens;
    values projected, the two states merged: attention over all of them."""
    H, prefix, n = 4, 150, 70
    g = torch.Generator().manual_seed(0)
    lat = torch.randn(prefix + n, L, generator=g).to(torch.bfloat16)
    pe = torch.randn(prefix + n, R, generator=g).to(torch.bfloat16)
    wk, wv = (torch.randn(H, L, d, generator=g, dtype=torch.float64) / math.sqrt(L) for d in (NOPE, V))
    q = torch.randn(n, H, NOPE + R, generator=g).to(torch.bfloat16)
    pages = (prefix + P - 1) // P
    pool = torch.zeros(pages, P, L + R, dtype=torch.bfloat16)
    pool.view(-1, L + R)[:prefix] = torch.cat([lat, pe], 1)[:prefix]
    # the per-head keys and values of the new tokens, and the absorbed queries, rounded as a model rounds them
    k = torch.einsum("kc,hcd->khd", lat[prefix:].double(), wk).to(torch.bfloat16)
    v = torch.einsum("kc,hcd->khd", lat[prefix:].double(), wv).to(torch.bfloat16)
    qa = torch.cat([torch.einsum("qhd,hcd->qhc", q[..., :NOPE].double(), wk).to(torch.bfloat16), q[..., NOPE:]], -1)
    oa = torch.empty(n, H, L, dtype=torch.float32, device=DEV)
    la, lb, lm = (torch.empty(n, H, device=DEV) for _ in range(3))
    ob, om = (torch.empty(n, H, V, dtype=torch.float32, device=DEV) for _ in range(2))
    ws = torch.empty(pkv.paged_attention_latent_workspace_size(1, n, H, prefix), dtype=torch.uint8, device=DEV)
    pkv.paged_attention_latent(qa.to(DEV), pool.to(DEV), i32([list(range(pages))]), i32([prefix]), i32([0, n]), oa, lse=la,
                               max_q_rows=n, max_kv_len=prefix, mask="none", scale=SCALE, workspace=ws)
    pkv.ragged_attention_latent(q.to(DEV), k.to(DEV), pe[prefix:].to(DEV), v.to(DEV), i32([0, n]), i32([0, n]), ob, lse=lb,
                                max_q_rows=n, max_kv_len=n, scale=SCALE)
    ov = torch.einsum("qhc,hcd->qhd", oa.double(), wv.to(DEV)).float().contiguous()  # (einsum's result may be permuted)
    pkv.merge_attn_states(ov, la, ob, lb, om, lm)
    # the definition over all keys, each part's scores and values as that part has them
    want = torch.empty(n, H, V, dtype=torch.float64)
    for i in range(n):
        cached = torch.cat([lat, pe], 1)[:prefix].double()
        s0 = torch.einsum("hc,kc->hk", qa[i].double(), cached) * SCALE
        key = torch.cat([k.double(), pe[prefix:].double()[:, None].expand(-1, H, -1)], -1)[:i + 1]
        s1 = torch.einsum("hd,khd->hk", q[i].double(), key) * SCALE
        w = torch.softmax(torch.cat([s0, s1], 1), 1)
        v0 = torch.einsum("kc,hcd->hkd", lat[:prefix].double(), wv)
        want[i] = torch.einsum("hk,hkd->hd", w, torch.cat([v0, v[:i + 1].double().transpose(0, 1)], 1))
    # weights off by 2^-8 each (and their sums): both parts' values through it, at most 2 * 2^-8 of
    # the weighted magnitudes; values have size ~1, so sum w |v| <= their largest
    top = max(float(v.abs().max()), float(torch.einsum("kc,hcd->khd", lat[:prefix].double(), wv).abs().max()))
    assert (om.double().cpu() - want).abs().max() <= 2.1 * BF16_STEP * top
    assert torch.isfinite(lm).all()


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace."""
    from latent_testutil import Case
    cases = [Case([900, 40, 2100], [1, 1, 1], [1, 1, 1], 16, seed=1), Case([700, 300], [1, 2], [1, 2], 128, seed=2)]
    want = [c.run()[:2] for c in cases]
    states = []
    for c in cases:
        dev = [t.to(DEV) for t in (c.q_full, c.pool)] + [i32(x.tolist() if hasattr(x, "tolist") else x)
                                                        for x in (c.table, c.kv, c.indptr, c.real)]
        n = pkv.paged_attention_latent_workspace_size(len(c.kv), max(c.rows), c.H, max(c.kv))
        out = torch.full((c.q_full.shape[0], c.H, L), 7.0, dtype=torch.bfloat16, device=DEV)
        states.append((c, dev, torch.empty(n, dtype=torch.uint8, device=DEV), out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for c, (q, pool, bt, kl, qi, qr), ws, out, s in states:
            pkv.paged_attention_latent(q, pool, bt, kl, qi, out, q_real=qr, max_q_rows=max(c.rows), max_kv_len=max(c.kv),
                                       scale=c.scale, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (c, _, _, out, _), (o, _) in zip(states, want):
        assert torch.equal(out.cpu(), o)


def test_offsets_past_32_bits():
    """Pages whose first element lies past 2^31, slots past 2^22 pages' tokens."""
    pages = (1 << 31) // (P * (L + R)) + 40
    pool = torch.empty(pages, P, L + R, dtype=torch.bfloat16, device=DEV)
    pool[-40:] = float("nan")
    T, H = 45, 16
    g = torch.Generator().manual_seed(3)
    src = torch.randn(T, L + R, generator=g).to(torch.bfloat16).to(DEV)
    first = pages - 3
    table = i32([[first, first + 2]])
    j = torch.arange(T)
    slots = (torch.tensor([first, first + 2])[j // P] * P + j % P).to(DEV)
    ang = torch.zeros(T, R, device=DEV)
    ang[:, :R // 2] = 1.0     # no rotation
    pkv.kv_append_latent(src, j.to(DEV), ang, slots, pool)
    assert torch.equal(pool.view(-1, L + R)[slots], src)
    q = torch.randn(1, H, L + R, generator=g).to(torch.bfloat16)
    for flags in (0, pkv.PKV_FLAG_SIMT_ONLY):
        out, lse = torch.empty(1, H, L, dtype=torch.float32, device=DEV), torch.empty(1, H, device=DEV)
        ws = torch.empty(max(256, pkv.paged_attention_latent_workspace_size(1, 1, H, T)), dtype=torch.uint8, device=DEV)
        pkv.paged_attention_latent(q.to(DEV), pool, table, i32([T]), i32([0, 1]), out, lse=lse, max_q_rows=1, max_kv_len=T,
                                   scale=SCALE, workspace=ws, flags=flags)
        c = src.double().cpu().numpy()
        want, wl, to, tl = attend(q[0].double().numpy(), c, c[:, :L], SCALE)
        compare(out.cpu(), lse.cpu(), want[None], wl[None], to[None], tl[None], torch.float32)


def test_expanded_offsets_past_32_bits():
    """Token strides that put the last keys past 2^31 elements."""
    H, n, stride = 2, 300, 1 << 23
    g = torch.Generator().manual_seed(4)
    big = torch.empty((n - 1) * stride + H * (NOPE + V), dtype=torch.bfloat16, device=DEV)
    both = big.as_strided((n, H, NOPE + V), (stride, NOPE + V, 1))
    x = torch.randn(n, H, NOPE + V, generator=g).to(torch.bfloat16)
    both.copy_(x)
    pe = torch.randn(n, R, generator=g).to(torch.bfloat16)
    q = torch.randn(20, H, NOPE + R, generator=g).to(torch.bfloat16)
    out, lse = torch.empty(20, H, V, dtype=torch.float32, device=DEV), torch.empty(20, H, device=DEV)
    pkv.ragged_attention_latent(q.to(DEV), both[..., :NOPE], pe.to(DEV), both[..., NOPE:], i32([0, 20]), i32([0, n]), out,
                                lse=lse, max_q_rows=20, max_kv_len=n, scale=SCALE)
    key = np.concatenate([x[..., :NOPE].double().numpy(), np.broadcast_to(pe.double().numpy()[:, None], (n, H, R))], -1)
    for i in range(20):
        k = n - 20 + i + 1
        want, wl, to, tl = attend(q[i].double().numpy(), key[:k], x[:k, :, NOPE:].double().numpy(), SCALE)
        compare(out[i:i + 1].cpu(), lse[i:i + 1].cpu(), want[None], wl[None], to[None], tl[None], torch.float32)
