"""Cases and a plain 64-bit implementation for the 8-bit cache and for windowed
attention.  Everything a call must not read holds values that would show: NaN
codes and NaN scales in free pages, NaN in the slots past a sequence's last
key, -1 in block-table entries of pages that no row sees."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

from paged_kv_cache_189_gb300 import pkv

P = 32


def e4m3_grid(x):
    """The nearest e4m3 value (ties to even, saturating at 448) of float64 values; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(x)
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        return np.where(np.isnan(x), x, np.clip(np.round(x / step) * step, -448.0, 448.0))


def scale_for(amax):
    """2^e, the smallest e >= -126 with amax <= 448 * 2^e; 0 for 0."""
    if not amax > 0:
        return 0.0
    e = math.frexp(amax / 448.0)[1]            # amax / 448 in [2^(e-1), 2^e)
    if amax <= 448.0 * math.ldexp(1.0, e - 1):
        e -= 1
    return math.ldexp(1.0, max(e, -126))


def codes_of(values):
    """float8_e4m3fn tensor of values that are on the grid."""
    return torch.from_numpy(np.asarray(values, dtype=np.float32)).to(torch.float8_e4m3fn)


@dataclass
class Case:
    kv: list
    real: list
    rows: list
    Hq: int
    Hkv: int
    D: int
    fp8: bool
    mask: str = "causal"
    cb: int = 0
    window: int = 0
    sinks: int = 0
    seed: int = 0
    pow2: bool = True       # scales are powers of two
    slot_pad: int = 0       # extra elements between pages
    q_pad: int = 0          # extra query heads in the tensor the queries are sliced from
    key_size: float = 1.0

    def __post_init__(self):
        g = np.random.default_rng(self.seed)
        B = len(self.kv)
        width = max(max((k + P - 1) // P for k in self.kv), 1)
        seen = [self.seen_keys(b) for b in range(B)]
        held = [(b, p) for b in range(B) for p in range(width)
                if seen[b].size and (seen[b] // P == p).any()]
        self.num_pages = len(held) + 3
        order = g.permutation(self.num_pages)
        table = np.full((B, width), -1, dtype=np.int32)
        for (b, p), at in zip(held, order):
            table[b, p] = at
        self.table = table
        shape = (self.num_pages, P, self.Hkv, self.D)
        k = g.standard_normal(shape) * np.exp(0.5 * g.standard_normal((self.Hkv, self.D))) * self.key_size
        v = g.standard_normal(shape)
        # slots that hold a key of some sequence and are seen by one of its rows
        used = np.zeros((self.num_pages, P), dtype=bool)
        for b in range(B):
            if seen[b].size:
                used[table[b, seen[b] // P], seen[b] % P] = True
        self.k_scale = self.v_scale = None
        if self.fp8:
            sc = [np.exp2(g.integers(-9, 3, size=(self.num_pages, self.Hkv))) *
                  (1.0 if self.pow2 else g.uniform(1, 2, size=(self.num_pages, self.Hkv))) for _ in "kv"]
            sc = [s.astype(np.float32) for s in sc]
            kc, vc = [e4m3_grid(x / s[:, None, :, None].astype(np.float64)) for x, s in zip((k, v), sc)]
            self.k64 = kc * sc[0][:, None, :, None].astype(np.float64)
            self.v64 = vc * sc[1][:, None, :, None].astype(np.float64)
            kc[~used], vc[~used] = np.nan, np.nan
            free = ~used.any(1)
            for s in sc:
                s[free] = np.nan
            self.k_pool, self.v_pool = codes_of(kc), codes_of(vc)
            self.k_scale, self.v_scale = torch.from_numpy(sc[0]), torch.from_numpy(sc[1])
        else:
            self.k_pool = torch.from_numpy(k).to(torch.bfloat16)
            self.v_pool = torch.from_numpy(v).to(torch.bfloat16)
            self.k64, self.v64 = self.k_pool.double().numpy(), self.v_pool.double().numpy()
            self.k_pool[torch.from_numpy(~used)] = float("nan")
            self.v_pool[torch.from_numpy(~used)] = float("nan")
        if self.slot_pad:
            def padded(pool):
                raw = pool.contiguous().view(torch.uint8 if self.fp8 else torch.int16).flatten(1)
                big = torch.zeros(raw.shape[0], raw.shape[1] + self.slot_pad, dtype=raw.dtype)
                big[:, :raw.shape[1]] = raw
                return big
            self.k_pool, self.v_pool = padded(self.k_pool), padded(self.v_pool)
        total = sum(self.rows)
        self.q_full = torch.from_numpy(g.standard_normal((total, self.Hq + self.q_pad, self.D))).to(torch.bfloat16)
        self.indptr = np.concatenate([[0], np.cumsum(self.rows)]).astype(np.int32)

    def limits(self, b, i):
        """(first window key, end) of row i of sequence b."""
        kv, real = self.kv[b], self.real[b]
        if i >= real:
            return 0, 0
        first = kv - real
        end = kv if self.mask == "none" else first + i + 1
        if self.mask == "block_causal":
            end = first + min(real, (i // self.cb + 1) * self.cb)
        lo = max(0, first + i - self.window + 1) if self.window else 0
        return lo, max(0, min(end, kv))

    def row_keys(self, b, i):
        lo, end = self.limits(b, i)
        j = np.arange(end)
        return j[(j >= lo) | (j < self.sinks)]

    def seen_keys(self, b):
        m = np.zeros(max(self.kv[b], 0), dtype=bool)
        for i in range(self.real[b]):
            m[self.row_keys(b, i)] = True
        return np.nonzero(m)[0]

    def on(self, dev):
        """Device tensors of the case."""
        kp, vp = self.k_pool.to(dev), self.v_pool.to(dev)
        if self.slot_pad:
            n = P * self.Hkv * self.D

            def strided(x):
                y = x.view(torch.float8_e4m3fn if self.fp8 else torch.bfloat16)
                return y[:, :n].unflatten(1, (P, self.Hkv, self.D))
            kp, vp = strided(kp), strided(vp)
        t = dict(k_pool=kp, v_pool=vp, q=self.q_full.to(dev)[:, :self.Hq],
                 table=torch.from_numpy(self.table).to(dev),
                 kv_lens=torch.tensor(self.kv, dtype=torch.int32, device=dev),
                 q_real=torch.tensor(self.real, dtype=torch.int32, device=dev),
                 q_indptr=torch.from_numpy(self.indptr).to(dev))
        if self.fp8:
            t["k_scale"], t["v_scale"] = self.k_scale.to(dev), self.v_scale.to(dev)
        return t

    def max_rows(self):
        return max(self.rows)

    def max_kv(self):
        return max(max(self.kv), 1)

    def reference(self):
        """out, lse, and for the tolerances: the weights' product with |v|, and
        the largest sum over d of |q_d k_d| * scale of a row's keys."""
        total, G = sum(self.rows), self.Hq // self.Hkv
        O = np.zeros((total, self.Hq, self.D))
        A = np.zeros_like(O)
        L = np.full((total, self.Hq), -np.inf)
        S = np.zeros((total, self.Hq))
        q = self.q_full[:, :self.Hq].double().numpy()
        for b in range(len(self.kv)):
            for i in range(self.rows[b]):
                j = self.row_keys(b, i)
                if not len(j):
                    continue
                r = self.indptr[b] + i
                ph = self.table[b, j // P]
                K, V = self.k64[ph, j % P], self.v64[ph, j % P]            # [keys, Hkv, D]
                qr = q[r].reshape(self.Hkv, G, self.D) / math.sqrt(self.D)
                s = np.einsum("hgd,khd->hgk", qr, K)
                S[r] = np.einsum("hgd,khd->hgk", abs(qr), abs(K)).max(-1).reshape(-1)
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                l = e.sum(-1, keepdims=True)
                L[r] = (m + np.log(l))[..., 0].reshape(-1)
                O[r] = np.einsum("hgk,khd->hgd", e / l, V).reshape(self.Hq, self.D)
                A[r] = np.einsum("hgk,khd->hgd", e / l, abs(V)).reshape(self.Hq, self.D)
        return O, L, A, S


def call(case, t, out, lse, *, flags=0, err=None, workspace=None, stream=None, max_q_rows=None, max_kv_len=None):
    mq, mk = max_q_rows or case.max_rows(), max_kv_len or case.max_kv()
    size = pkv.paged_attention_fp8_workspace_size if case.fp8 else pkv.paged_attention_window_workspace_size
    n = size(len(case.kv), mq, case.Hq, case.Hkv, case.D, mk, case.window, case.sinks, flags)
    if workspace is None and n:
        workspace = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # needs no clearing
    common = dict(q_real=t["q_real"], lse=lse, max_q_rows=mq, max_kv_len=mk, window=case.window,
                  num_sinks=case.sinks, workspace=workspace, flags=flags, err=err, stream=stream)
    if case.fp8:
        pkv.paged_attention_fp8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], t["table"],
                                t["kv_lens"], t["q_indptr"], out, mask=case.mask, causal_block=case.cb, **common)
    else:
        pkv.paged_attention_window(t["q"], t["k_pool"], t["v_pool"], t["table"], t["kv_lens"], t["q_indptr"],
                                   out, **common)
    return workspace


def run(case, out_dtype=torch.bfloat16, flags=0, **kw):
    t = case.on("cuda")
    total = sum(case.rows)
    out = torch.full((total, case.Hq, case.D), float("nan"), dtype=out_dtype, device="cuda")
    lse = torch.full((total, case.Hq), float("nan"), dtype=torch.float32, device="cuda")
    call(case, t, out, lse, flags=flags, **kw)
    torch.cuda.synchronize()
    return out, lse


def check(case, out, lse, ref=None):
    """Tolerances, from the roundings on the way (u = half a step, relative):
    a score is an f32 sum of D products, off by at most D 2^-24 of the sum of
    their magnitudes, so a weight is off by twice that (its own and the sum's)
    plus its exponential's 2^-21; the weights are rounded once, to bf16 (2^-8)
    at the coarsest, in the numerator and, as a sum of rounded or exact weights,
    in the denominator; the output is rounded to its type."""
    O, L, A, S = ref or case.reference()
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    none = np.isneginf(L)
    assert (got[none] == 0).all(), "rows without a key must be zero"
    assert np.isneginf(gl[none]).all(), "rows without a key must have LSE -inf"
    assert np.isfinite(got).all()
    es = case.D * 2.0 ** -24 * S
    u_out = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    tol = (2 * 2.0 ** -8 + 2 * es + 2.0 ** -20)[..., None] * A + u_out * abs(O)
    bad = abs(got - O) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.max(abs(got - O) - tol):.3e}"
    # the weights' roundings are independent: their mean is far below the bound
    if (~none).any():
        rel = np.linalg.norm((got - O)[~none]) / max(np.linalg.norm(O[~none]), 1e-30)
        assert rel < 2.0 ** -7, rel
    tl = es + 2.0 ** -18 + 2.0 ** -22 * abs(np.where(none, 0, L))
    badl = abs(np.where(none, 0, gl) - np.where(none, 0, L)) > tl
    badl &= ~none
    assert not badl.any(), f"{badl.sum()} LSEs off, worst {np.max((abs(gl - L) - tl)[~none]):.3e}"
