"""Cases and plain 64-bit implementations for the latent cache and for
attention over expanded keys.  What a call must not read holds values that
would show: NaN in the slots past a sequence's last key and in free pages,
entries far out of range in the table past the last page a row sees."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

from paged_kv_cache_189_gb300 import pkv

P = 32
L, R = 512, 64
NOPE, V = 128, 128
BF16_STEP = 2.0 ** -8       # a rounding to bf16 is off by half a unit in 8 bits, relative to the value
F32_SUM = 2.0 ** -23        # a term of an f32 sum, truncated rather than rounded


def pages(n):
    return (n + P - 1) // P


@dataclass
class Case:
    kv: list
    real: list
    rows: list
    H: int
    mask: str = "causal"
    seed: int = 0
    key_size: float = 1.0
    growing: bool = False    # scores rise along the keys: the running maximum moves again and again
    page_pad: int = 0        # elements between pages
    q_pad: int = 0           # heads between the rows of the tensor the queries are sliced from
    lead: int = 0            # query rows ahead of the first sequence's
    scale: float = 1.0 / math.sqrt(192)

    def __post_init__(self):
        g = np.random.default_rng(self.seed)
        B = len(self.kv)
        width = max(max(pages(k) for k in self.kv), 1)
        held = sum(pages(k) for k in self.kv)
        self.num_pages = held + 3
        order = list(g.permutation(self.num_pages))
        table = np.full((B, width + 1), 1 << 29, dtype=np.int32)
        pool = torch.full((self.num_pages, P, L + R), float("nan"), dtype=torch.bfloat16)
        for b, k in enumerate(self.kv):
            for p in range(pages(k)):
                page = int(order.pop())
                table[b, p] = page
                n = min(P, k - p * P)
                x = g.standard_normal((n, L + R)) * self.key_size
                if self.growing:
                    x[:, :8] += 0.04 * (p * P + np.arange(n))[:, None]
                pool[page, :n] = torch.from_numpy(x).to(torch.bfloat16)
        self.table, self.pool = table, pool
        total = self.lead + sum(self.rows) + 2   # two rows behind the last sequence
        q = g.standard_normal((total, self.H + self.q_pad, L + R))
        if self.growing:
            q[..., :8] = np.abs(q[..., :8]) + 1.0
        self.q_full = torch.from_numpy(q).to(torch.bfloat16)
        self.indptr = (self.lead + np.concatenate([[0], np.cumsum(self.rows)])).astype(np.int32)

    def run(self, flags=0, out_dtype=torch.bfloat16, checked=True, stream=None):
        """out, lse (filled with 7 and 9 beforehand) and the error bits."""
        dev = "cuda"
        q = self.q_full.to(dev)[:, self.q_pad // 2:self.q_pad // 2 + self.H]
        if self.page_pad:
            big = torch.zeros(self.num_pages, P * (L + R) + self.page_pad, dtype=torch.bfloat16, device=dev)
            big[:, :P * (L + R)] = self.pool.to(dev).flatten(1)
            pool = big.as_strided((self.num_pages, P, L + R), (big.stride(0), L + R, 1))
        else:
            pool = self.pool.to(dev)
        T = self.q_full.shape[0]
        out = torch.full((T, self.H, L), 7.0, dtype=out_dtype, device=dev)
        lse = torch.full((T, self.H), 9.0, dtype=torch.float32, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        mq, mk = max(self.rows), max(self.kv)
        ws = None
        if not flags & pkv.PKV_FLAG_SIMT_ONLY:
            n = pkv.paged_attention_latent_workspace_size(len(self.kv), mq, self.H, mk)
            ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device=dev)
        i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).to(dev)  # noqa: E731
        pkv.paged_attention_latent(q, pool, i32(self.table), i32(self.kv), i32(self.indptr), out, q_real=i32(self.real),
                                   lse=lse, max_q_rows=mq, max_kv_len=mk, mask=self.mask, scale=self.scale,
                                   workspace=ws, flags=flags | (pkv.PKV_FLAG_CHECKED if checked else 0), err=err,
                                   stream=stream)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu(), int(err)

    def expected(self):
        """out, lse, and what each may be off by (see :func:`bounds`)."""
        T = self.q_full.shape[0]
        out, lse = np.full((T, self.H, L), 7.0), np.full((T, self.H), 9.0)
        tol_o, tol_l = np.zeros_like(out), np.zeros_like(lse)
        q_all = self.q_full[:, self.q_pad // 2:self.q_pad // 2 + self.H].double().numpy()
        pool = self.pool.double().numpy()
        for b, (kv, real, rows) in enumerate(zip(self.kv, self.real, self.rows)):
            j = np.arange(kv)
            c = pool[self.table[b, j // P], j % P]
            for i in range(rows):
                r = self.indptr[b] + i
                n = 0 if i >= real else kv if self.mask == "none" else max(0, kv - real + i + 1)
                out[r], lse[r], tol_o[r], tol_l[r] = attend(q_all[r], c[:n], c[:n, :L], self.scale)
        return out, lse, tol_o, tol_l

    def check(self, out_dtype=torch.bfloat16, **kw):
        got, gl, err = self.run(out_dtype=out_dtype, **kw)
        assert err == 0
        want, wl, tol_o, tol_l = self.expected()
        compare(got, gl, want, wl, tol_o, tol_l, out_dtype)


def attend(q, k, v, scale):
    """One query row [H, d] over keys [n, d] (or [n, H, d]) and values, in 64
    bits, with the errors of 32-bit sums and of weights rounded to bf16.

    A score is a sum of d products: off by ds = d * 2^-23 * sum |q k| scale at
    most, as are the sum of the weights and the LSE (d * 2^-23: the terms kept
    in f32, each addition truncated).  The weights the values meet are rounded:
    w (1 + e), |e| <= 2^-8, and so is their sum, so out is off by
    sum w |e| |v - out| / sum w <= (2^-8 + 2 ds) (sum w |v| + |out|), and by the
    f32 sum over n keys, n 2^-23 sum w |v| at most, with n no more than the terms
    added one after the other (keys of a tile, then tiles: n / 16 + 16)."""
    H, n = q.shape[0], k.shape[0]
    dv = v.shape[-1]
    if n == 0:
        return np.zeros((H, dv)), np.full(H, -np.inf), np.zeros((H, dv)), np.zeros(H)
    kh = k if k.ndim == 3 else np.broadcast_to(k[:, None], (n, H, k.shape[-1]))
    vh = v if v.ndim == 3 else np.broadcast_to(v[:, None], (n, H, dv))
    s = np.einsum("hd,nhd->hn", q, kh) * scale
    ds = (np.einsum("hd,nhd->hn", np.abs(q), np.abs(kh)) * scale).max(1) * q.shape[-1] * F32_SUM
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    tot = w.sum(1)
    w /= tot[:, None]
    o = np.einsum("hn,nhd->hd", w, vh)
    a = np.einsum("hn,nhd->hd", w, np.abs(vh))
    lse = m[:, 0] + np.log(tot)
    chain = (n / 16 + 16) * F32_SUM
    tol_o = (1.01 * BF16_STEP + 2 * ds[:, None] + chain) * (a + np.abs(o))
    # the LSE: the scores', the sum's, ex2's and lg2's (2^-21 of a value near 1 each), the last rounding
    tol_l = ds + chain + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)
    return o, lse, tol_o, tol_l


def compare(got, gl, want, wl, tol_o, tol_l, out_dtype):
    got, gl = got.double().numpy(), gl.double().numpy()
    step = BF16_STEP if out_dtype == torch.bfloat16 else 2.0 ** -24
    bad = np.abs(got - want) > tol_o * (1 + step) + step * np.abs(want)
    bad |= ~np.isfinite(got)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), float(np.abs(got - want).max()))
    same = (gl == wl) | (np.abs(gl - np.where(np.isinf(wl), 0, wl)) <= tol_l)
    assert same.all(), (np.argwhere(~same)[:4].tolist(), gl[~same][:4], wl[~same][:4])


@dataclass
class Ragged:
    q_lens: list
    kv: list
    H: int
    mask: str = "causal"
    seed: int = 0
    key_size: float = 1.0
    growing: bool = False
    fused: bool = True      # K and V side by side in one tensor
    q_pad: int = 0
    scale: float = 1.0 / math.sqrt(192)

    def __post_init__(self):
        g = np.random.default_rng(self.seed)
        bf = lambda *s: torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16)  # noqa: E731
        T, K = sum(self.q_lens) + 1, sum(self.kv) + 2
        self.q_full = bf(T, self.H + self.q_pad, NOPE + R)
        both = bf(K, self.H, NOPE + V) * self.key_size
        if self.growing:
            q = self.q_full[..., :8].abs() + 1
            self.q_full[..., :8] = q
            both[..., :8] += 0.05 * torch.arange(K)[:, None, None].to(torch.bfloat16)
        self.both, self.k_pe = both, bf(K, R)
        # rows behind the last sequence's keys are read by nobody
        self.both[sum(self.kv):] = float("nan")
        self.k_pe[sum(self.kv):] = float("nan")
        self.qi = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        self.ki = np.concatenate([[0], np.cumsum(self.kv)]).astype(np.int32)

    def run(self, flags=0, out_dtype=torch.bfloat16):
        dev = "cuda"
        q = self.q_full.to(dev)[:, self.q_pad // 2:self.q_pad // 2 + self.H]
        both, pe = self.both.to(dev), self.k_pe.to(dev)
        k, v = both[..., :NOPE], both[..., NOPE:]
        if not self.fused:
            k, v = k.contiguous(), v.transpose(0, 1).contiguous().transpose(0, 1)
        T = q.shape[0]
        out = torch.full((T, self.H, V), 7.0, dtype=out_dtype, device=dev)
        lse = torch.full((T, self.H), 9.0, dtype=torch.float32, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        i32 = lambda x: torch.as_tensor(x).to(dev)  # noqa: E731
        pkv.ragged_attention_latent(q, k, pe, v, i32(self.qi), i32(self.ki), out, lse=lse, max_q_rows=max(self.q_lens),
                                    max_kv_len=max(self.kv), mask=self.mask, scale=self.scale,
                                    flags=flags | pkv.PKV_FLAG_CHECKED, err=err)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu(), int(err)

    def expected(self):
        T = self.q_full.shape[0]
        out, lse = np.full((T, self.H, V), 7.0), np.full((T, self.H), 9.0)
        tol_o, tol_l = np.zeros_like(out), np.zeros_like(lse)
        q_all = self.q_full[:, self.q_pad // 2:self.q_pad // 2 + self.H].double().numpy()
        pe = np.broadcast_to(self.k_pe.double().numpy()[:, None], (self.k_pe.shape[0], self.H, R))
        both = self.both.double().numpy()
        key = np.concatenate([both[..., :NOPE], pe], -1)
        for b, (ql, kv) in enumerate(zip(self.q_lens, self.kv)):
            for i in range(ql):
                n = kv if self.mask == "none" else max(0, kv - ql + i + 1)
                r, k0 = self.qi[b] + i, self.ki[b]
                out[r], lse[r], tol_o[r], tol_l[r] = attend(q_all[r], key[k0:k0 + n], both[k0:k0 + n, :, NOPE:],
                                                            self.scale)
        return out, lse, tol_o, tol_l

    def check(self, flags=0, out_dtype=torch.bfloat16):
        got, gl, err = self.run(flags, out_dtype)
        assert err == 0
        want, wl, tol_o, tol_l = self.expected()
        compare(got, gl, want, wl, tol_o, tol_l, out_dtype)
