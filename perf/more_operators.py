"""Cases of the latent K/V cache (one vector a token, shared by all heads) and of
what a serving step needs around it: block tables and slot maps built on the
GPU from request lengths, the append that normalises, rotates and writes the
latent rows, attention over the paged latent rows themselves (absorbed form),
and attention over keys and values expanded from them (prompts).

``run`` makes the library's calls where ``own`` is true and computes the same
operators in elementary torch operations where it is false.  ``exact`` gives
the definitions in 64 bits (integers for the tables), sequence by sequence."""
import math
import random

import torch

own = False

PAGE = 32
LATENT = 512   # shared latent vector of a token: all heads' keys and values
ROPE = 64      # its rotary part, keys only
NOPE = 128     # per-head part of an expanded query or key
VALUE = 128    # per-head expanded value
EPS = 1e-6
MAX_POSITION = 1 << 15
DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _case(name, op, batch, heads, new_lo, new_hi, kv_lo, kv_hi, pad=0, mask="causal", finished=0, scarce=False,
          interleaved=False):
    c = dict(op=op, batch=batch, heads=heads, new_lo=new_lo, new_hi=new_hi, kv_lo=kv_lo, kv_hi=kv_hi, pad=pad,
             mask=mask, finished=finished, scarce=scarce, interleaved=interleaved)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # the tables of one decode step of a full serving batch: nothing but latency
        _case("tables_step", "tables", 64, 1, 1, 1, 512, 8192),
        # a large mixed step: prompt chunks beside decoding sequences, some finished, too few free pages for all
        _case("tables_mixed", "tables", 768, 1, 1, 256, 0, 8192, pad=500, finished=40, scarce=True),
        # one decode step of a serving batch: one latent row a sequence, rotary parts of its query heads
        _case("latent_append_step", "append", 64, 16, 1, 1, 513, 8193),
        # prompt chunks of four sequences, ragged, starting inside a page
        _case("latent_append_chunk", "append", 4, 32, 1800, 2048, 2100, 8192, pad=7, interleaved=True),
        # decode of two short sequences
        _case("latent_tiny", "absorbed", 2, 16, 1, 1, 37, 100),
        # decode of a serving batch whose heads are shared out over several GPUs: bound by the cache's bytes
        _case("latent_decode", "absorbed", 64, 16, 1, 1, 513, 8193),
        # decode of a serving batch with all heads on this GPU: bytes and matrix rate close to each other
        _case("latent_decode_wide", "absorbed", 64, 128, 1, 1, 513, 8193),
        # speculative verification: four tokens of each sequence at once
        _case("latent_verify", "absorbed", 64, 16, 4, 4, 516, 8196),
        # a few very long conversations: the key axis is the only parallelism
        _case("latent_long", "absorbed", 3, 16, 1, 1, 60000, 131072),
        # short prompt chunks on top of a long cached context, where expanding the context would cost more
        _case("latent_chunk", "absorbed", 4, 16, 150, 256, 4096, 8192, pad=5),
        # two short prompts
        _case("expanded_tiny", "expanded", 2, 16, 9, 40, 37, 100),
        # prompts of four sequences, continued ones: the largest piece of work here
        _case("expanded_prompt", "expanded", 4, 32, 1500, 2048, 2048, 4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "absorbed", "absorbed", "absorbed", "expanded"])
    if op == "tables":
        batch = _log_int(rng, 1, 1000)
        new_hi = rng.choice([1, _log_int(rng, 2, 256)])
        return _case(None, op, batch, 1, 1, new_hi, 0, _log_int(rng, 16, 8192), pad=rng.choice([0, rng.randint(1, 600)]),
                     finished=rng.randint(0, max(0, batch // 8)), scarce=rng.random() < 0.4)
    if op == "append":
        new_hi = rng.choice([1, _log_int(rng, 2, 2048)])
        batch = rng.randint(1, 4) if new_hi > 64 else _log_int(rng, 1, 64)
        return _case(None, op, batch, rng.choice([1, 3, 8, 16, 32]), max(1, new_hi // 2), new_hi, new_hi,
                     new_hi + _log_int(rng, 1, 6000), pad=rng.choice([0, rng.randint(1, 9)]),
                     interleaved=rng.random() < 0.5)
    if op == "absorbed":
        rows = rng.choice(["one", "one", "few", "chunk"])
        heads = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 128])
        mask = "none" if rng.random() < 0.2 else "causal"
        if rows == "chunk":
            batch, new_hi = rng.randint(1, 4), _log_int(rng, 13, 200)
            heads = min(heads, 16)
        else:
            batch, new_hi = _log_int(rng, 1, 64), 1 if rows == "one" else rng.randint(2, 12)
            heads = heads if rows == "one" else min(heads, 16)
        new_lo = max(1, new_hi // 2)
        kv_hi = new_hi + _log_int(rng, 8, 8000)
        return _case(None, op, batch, heads, new_lo, new_hi, max(new_hi, _log_int(rng, 1, kv_hi)), kv_hi,
                     pad=rng.choice([0, 0, rng.randint(1, 9)]), mask=mask)
    batch, new_hi = rng.randint(1, 2), _log_int(rng, 2, 2048)
    kv_hi = new_hi + rng.choice([0, _log_int(rng, 1, 2048)])
    return _case(None, op, batch, rng.choice([1, 3, 8, 16, 24]), max(1, new_hi // 2), new_hi, new_hi, kv_hi,
                 mask="none" if rng.random() < 0.3 else "causal")


def _lengths(case):
    """Keys, real new rows and query rows (padding included) of each sequence:
    part of the case, the same for every seed."""
    r = random.Random("/".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))
    n = case["batch"]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(n)]
    if case["op"] == "tables":
        # kv: keys before the step; most sequences of a mixed step decode one token
        if case["new_hi"] > 1:
            new = [q if r.random() < 0.25 else 1 for q in new]
        for b in r.sample(range(n), case["finished"]):
            new[b] = -1
        return kv, new, new
    kv = [max(k, q) for k, q in zip(kv, new)]
    rows = [q + (r.randint(0, case["pad"]) if case["pad"] else 0) for q in new]
    return kv, new, rows


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _tables_needs(case):
    """Pages each sequence asks for, pages the finished ones give back, free pages before the step."""
    kv, new, _ = _lengths(case)
    need = [_pages(k + q) - _pages(k) if q > 0 else 0 for k, q in zip(kv, new)]
    back = sum(_pages(k) for k, q in zip(kv, new) if q < 0)
    total = sum(need)
    free = max(0, int(0.8 * total) - back) if case["scarce"] else total + 64
    return need, back, free


def work(case):
    kv, new, rows = _lengths(case)
    heads = case["heads"]
    if case["op"] == "tables":
        need, back, _ = _tables_needs(case)
        tokens = sum(q for q in new if q > 0) + case["pad"]
        return {"bytes": 16 * tokens + 8 * sum(need) + 8 * back + 16 * case["batch"], "flops": 4 * tokens}
    if case["op"] == "append":
        t, row = sum(rows), LATENT + ROPE
        real = sum(new)
        return {"bytes": 4 * real * row + t * (4 * heads * ROPE + 4 * ROPE + 16) + 2 * LATENT,
                "flops": real * (4 * LATENT + 3 * ROPE) + 3 * t * heads * ROPE}
    pairs = sum(k * q if case["mask"] == "none" else q * (k - q) + q * (q + 1) // 2 for k, q in zip(kv, new))
    if case["op"] == "absorbed":
        state = sum(new) * heads * (LATENT + ROPE) * 2 + sum(rows) * heads * (LATENT * 2 + 4)
        return {"bytes": sum(kv) * (LATENT + ROPE) * 2 + 4 * sum(_pages(k) for k in kv) + state,
                "flops": 2 * pairs * heads * (2 * LATENT + ROPE)}
    keys = sum(kv) * (heads * (NOPE + VALUE) + ROPE) * 2
    return {"bytes": keys + sum(new) * heads * ((NOPE + ROPE + VALUE) * 2 + 4),
            "flops": 2 * pairs * heads * (NOPE + ROPE + VALUE)}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _indptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _angles(g):
    """cos and sin of every position and pair, in 64 bits, rounded once to 32."""
    inv = 10000.0 ** (-torch.arange(ROPE // 2, device=DEV, dtype=torch.float64) / (ROPE // 2))
    a = torch.arange(MAX_POSITION, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    kv, new, rows = _lengths(case)
    batch, heads = case["batch"], case["heads"]
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    r = random.Random(int(seed))

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale

    s = dict(case=case, kv=kv, new=new, rows=rows)
    if case["op"] == "tables":
        need, back, free = _tables_needs(case)
        held = [_pages(k) for k in kv]
        pages = list(range(sum(held) + free))
        r.shuffle(pages)
        width = max(h + n for h, n in zip(held, need)) + 1
        table = [[-1] * width for _ in range(batch)]
        for b in range(batch):
            table[b][:held[b]] = [pages.pop() for _ in range(held[b])]
        tokens = max(1, sum(q for q in new if q > 0) + case["pad"])
        s.update(table=_int32(table), new_lens=_int32(new), kv_lens=_int32(kv), num_free=_int32([free]),
                 free_pages=_int32(pages + [-1] * (back + 1)), kv_out=torch.zeros(batch, dtype=torch.int32, device=DEV),
                 free_out=torch.zeros(1, dtype=torch.int32, device=DEV),
                 q_indptr=torch.zeros(batch + 1, dtype=torch.int32, device=DEV),
                 slots=torch.zeros(tokens, dtype=torch.int64, device=DEV),
                 positions=torch.zeros(tokens, dtype=torch.int64, device=DEV))
        return s
    indptr = _indptr(rows)
    total = indptr[-1]
    if case["op"] == "expanded":
        # K and V of the heads as one projection of the latent rows gives them, side by side
        kvi = _indptr(kv)
        both = (normal(kvi[-1], heads, NOPE + VALUE) * torch.exp(0.3 * normal(heads, NOPE + VALUE))).to(torch.bfloat16)
        tq = _indptr(new)
        s.update(q=normal(tq[-1], heads, NOPE + ROPE).to(torch.bfloat16), k=both[..., :NOPE], v=both[..., NOPE:],
                 k_pe=normal(kvi[-1], ROPE).to(torch.bfloat16), q_indptr=_int32(tq), kv_indptr=_int32(kvi),
                 out=torch.empty(tq[-1], heads, VALUE, dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty(tq[-1], heads, dtype=torch.float32, device=DEV))
        return s
    # pages: every sequence's own, in a random order
    held = sum(_pages(k) for k in kv)
    order = list(range(held + max(1, held // 10)))
    r.shuffle(order)
    num_pages, width = len(order), max(_pages(k) for k in kv)
    table = [[order.pop() for _ in range(_pages(k))] for k in kv]
    gain = torch.exp(0.3 * normal(LATENT + ROPE))
    pool = (normal(num_pages, PAGE, LATENT + ROPE) * gain).to(torch.bfloat16)
    if case["op"] == "append":
        slots, positions = [-1] * total, [0] * total
        for b in range(batch):
            for i in range(new[b]):
                p = kv[b] - new[b] + i
                slots[indptr[b] + i] = table[b][p // PAGE] * PAGE + p % PAGE
                positions[indptr[b] + i] = p
        # the latent rows are the last columns of the projection that also gives the queries' inputs
        proj = normal(total, 192 + LATENT + ROPE).to(torch.bfloat16)
        q = normal(total, heads, NOPE + ROPE).to(torch.bfloat16)
        s.update(pool=pool, src=proj[:, 192:], q_pe=q[..., NOPE:], weight=gain[:LATENT].to(torch.bfloat16),
                 q_rows=torch.zeros(total, heads, LATENT + ROPE, dtype=torch.bfloat16, device=DEV), cos_sin=_angles(g),
                 slots=torch.tensor(slots, dtype=torch.int64, device=DEV),
                 positions=torch.tensor(positions, dtype=torch.int64, device=DEV))
        return s
    s.update(pool=pool, q=normal(total, heads, LATENT + ROPE).to(torch.bfloat16),
             table=_int32([t + [-1] * (width - len(t)) for t in table]), kv_lens=_int32(kv), q_real=_int32(new),
             q_indptr=_int32(indptr), workspace={},
             out=torch.empty(total, heads, LATENT, dtype=torch.bfloat16, device=DEV),
             lse=torch.empty(total, heads, dtype=torch.float32, device=DEV))
    return s


# the softmax scale of a model with NOPE + ROPE wide per-head queries, in either form
SCALE = 1.0 / math.sqrt(NOPE + ROPE)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "absorbed": _own_absorbed,
                "expanded": _own_expanded}[op](s)
    return {"tables": _plain_tables, "append": _plain_append, "absorbed": _plain_absorbed,
            "expanded": _plain_expanded}[op](s)


_TABLE_OUTPUTS = ("table", "free_pages", "kv_out", "free_out", "q_indptr", "slots", "positions")


def _own_tables(s):
    from paged_kv_cache_189_gb300 import pkv
    pkv.assign_step_pages(s["new_lens"], s["kv_lens"], s["num_free"], s["free_pages"], s["table"],
                          kv_lens_out=s["kv_out"], num_free_out=s["free_out"], q_indptr=s["q_indptr"],
                          slots=s["slots"], positions=s["positions"])
    return {n: s[n] for n in _TABLE_OUTPUTS}


def _own_append(s):
    from paged_kv_cache_189_gb300 import pkv
    pkv.kv_append_latent(s["src"], s["positions"], s["cos_sin"], s["slots"], s["pool"], norm_weight=s["weight"],
                         eps=EPS, q_pe=s["q_pe"], q_out=s["q_rows"][..., LATENT:],
                         interleaved=s["case"]["interleaved"])
    return {"pool": s["pool"], "q": s["q_rows"]}


def _own_absorbed(s):
    from paged_kv_cache_189_gb300 import pkv
    c, max_rows, max_kv = s["case"], max(s["rows"]), max(s["kv"])
    if "bytes" not in s["workspace"]:  # a program keeps its workspace from step to step
        size = pkv.paged_attention_latent_workspace_size(c["batch"], max_rows, c["heads"], max_kv)
        s["workspace"]["bytes"] = torch.empty(max(256, size), dtype=torch.uint8, device=DEV)
    pkv.paged_attention_latent(s["q"], s["pool"], s["table"], s["kv_lens"], s["q_indptr"], s["out"],
                               q_real=s["q_real"], lse=s["lse"], max_q_rows=max_rows, max_kv_len=max_kv,
                               mask=c["mask"], scale=SCALE, workspace=s["workspace"]["bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_expanded(s):
    from paged_kv_cache_189_gb300 import pkv
    pkv.ragged_attention_latent(s["q"], s["k"], s["k_pe"], s["v"], s["q_indptr"], s["kv_indptr"], s["out"],
                                lse=s["lse"], max_q_rows=max(s["new"]), max_kv_len=max(s["kv"]),
                                mask=s["case"]["mask"], scale=SCALE)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tables(s):
    """Every sequence's request against running sums; finished sequences' pages
    go on top of the free pages first, then pages are taken from the top."""
    new, kv, free = s["new_lens"].long(), s["kv_lens"].long(), s["num_free"].long()
    table, stack = s["table"], s["free_pages"]
    batch, width, tokens = new.numel(), table.shape[1], s["slots"].numel()
    held = (kv + PAGE - 1) // PAGE
    back = torch.where(new < 0, held, torch.zeros_like(held))
    back_end = torch.cumsum(back, 0)
    col = torch.arange(width, device=DEV)
    row, at = torch.nonzero(col < back[:, None], as_tuple=True)
    stack[free + (back_end - back)[row] + at] = table[row, at]
    top = free + back_end[-1]
    ask = new.clamp(min=0)
    need = torch.where(ask > 0, (kv + ask + PAGE - 1) // PAGE - held, torch.zeros_like(held))
    need_end = torch.cumsum(need, 0)
    fits = (torch.cumsum(ask, 0) <= tokens) & (held + need <= width) & ((need == 0) | (need_end <= top))
    # pages are numbered by the requests' running sum, so a refused request leaves its own on the stack's side
    take = torch.where(fits, need, torch.zeros_like(need))
    take_end = torch.cumsum(take, 0)
    row, at = torch.nonzero(col < take[:, None], as_tuple=True)
    page = stack[top - 1 - (take_end - take)[row] - at]
    table[row, held[row] + at] = page
    granted = torch.where(fits, ask, torch.zeros_like(ask))
    ends = torch.cumsum(granted, 0)
    s["q_indptr"].zero_()
    s["q_indptr"][1:] = ends.int()
    s["kv_out"].copy_(torch.where(new < 0, torch.zeros_like(kv), kv + granted).int())
    s["free_out"].copy_((top - take_end[-1]).int().view(1))
    t = torch.arange(tokens, device=DEV)
    seq = torch.searchsorted(ends, t, right=True)
    live = t < ends[-1]
    seq = seq.clamp(max=batch - 1)
    pos = torch.where(live, kv[seq] + t - (ends - granted)[seq], torch.zeros_like(t))
    page = table[seq, pos // PAGE].long()
    s["slots"].copy_(torch.where(live, page * PAGE + pos % PAGE, torch.full_like(t, -1)))
    s["positions"].copy_(pos)
    return {n: s[n] for n in _TABLE_OUTPUTS}


def _rotated(x, cos, sin, interleaved):
    """[..., ROPE] rotated by pairs (i, i + ROPE / 2), or (2 i, 2 i + 1) where interleaved."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    angle = s["cos_sin"][s["positions"].clamp(0, MAX_POSITION - 1)]
    cos, sin = angle[:, :ROPE // 2], angle[:, ROPE // 2:]
    x = s["src"].float()
    lat = x[:, :LATENT]
    lat = lat / torch.sqrt(lat.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    pe = _rotated(x[:, LATENT:], cos, sin, s["case"]["interleaved"])
    written = s["slots"] >= 0
    slot = s["slots"][written]
    s["pool"][slot // PAGE, slot % PAGE] = torch.cat([lat, pe], 1)[written].to(torch.bfloat16)
    q = _rotated(s["q_pe"].float(), cos[:, None], sin[:, None], s["case"]["interleaved"])
    s["q_rows"][..., LATENT:] = q.to(torch.bfloat16)
    return {"pool": s["pool"], "q": s["q_rows"]}


def _plain_absorbed(s):
    c = s["case"]
    heads, rows, batch, max_kv = c["heads"], max(s["rows"]), c["batch"], max(s["kv"])
    kv, real = s["kv_lens"].long(), s["q_real"].long()
    keys = torch.arange(max_kv, device=DEV)
    live = keys < kv[:, None]
    page = s["table"].gather(1, (keys // PAGE).expand(batch, -1)).long().clamp(min=0)
    lat = s["pool"][page, keys % PAGE].float().masked_fill_(~live[..., None], 0.0)   # [B, K, 576]
    start = s["q_indptr"][:-1].long()
    i = torch.arange(rows, device=DEV)
    q = s["q"][(start[:, None] + i).clamp(max=s["q"].shape[0] - 1)].float()           # [B, R, H, 576]
    scores = torch.matmul(q.view(batch, rows * heads, -1), lat.transpose(1, 2)) * SCALE
    scores = scores.view(batch, rows, heads, max_kv)
    seen = live[:, None] & (i[:, None] < real[:, None, None])
    if c["mask"] == "causal":
        seen = seen & (keys <= (kv - real)[:, None, None] + i[:, None])
    scores.masked_fill_(~seen[:, :, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    scores.sub_(top.masked_fill(top == float("-inf"), 0.0)).exp_()
    total = scores.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]
    o = torch.matmul(scores.view(batch, rows * heads, max_kv), lat[..., :LATENT]).view(batch, rows, heads, LATENT)
    o = o / total.clamp(min=1e-30)
    at = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(s["q_indptr"][1:].long(), at, right=True)
    return {"out": o[b, at - start[b]].to(torch.bfloat16), "lse": lse[b, at - start[b]]}


def _plain_expanded(s):
    out, lse = [], []
    a = k0 = 0
    for n, k in zip(s["new"], s["kv"]):
        q = s["q"][a:a + n].float().transpose(0, 1)                                   # [H, n, 192]
        pe = s["k_pe"][k0:k0 + k].float().expand(q.shape[0], -1, -1)
        key = torch.cat([s["k"][k0:k0 + k].float().transpose(0, 1), pe], 2)
        scores = torch.matmul(q, key.transpose(1, 2)) * SCALE
        if s["case"]["mask"] == "causal":
            i, j = torch.arange(n, device=DEV)[:, None], torch.arange(k, device=DEV)
            scores.masked_fill_(j > k - n + i, float("-inf"))
        top = scores.amax(-1, keepdim=True)
        scores.sub_(top).exp_()
        total = scores.sum(-1, keepdim=True)
        o = torch.matmul(scores, s["v"][k0:k0 + k].float().transpose(0, 1)) / total
        out.append(o.transpose(0, 1).to(torch.bfloat16))
        lse.append((top + total.log())[..., 0].t())
        a, k0 = a + n, k0 + k
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_tables(s):
    new, kv = s["new_lens"].tolist(), s["kv_lens"].tolist()
    table, stack, free = s["table"].tolist(), s["free_pages"].tolist(), s["num_free"].item()
    width, tokens = len(table[0]), s["slots"].numel()
    for b, q in enumerate(new):
        if q < 0:
            for p in table[b][:_pages(kv[b])]:
                stack[free] = p
                free += 1
    top, asked_pages, asked_tokens = free, 0, 0
    slots, positions, indptr, lens = [], [], [0], []
    for b, q in enumerate(new):
        length = 0 if q < 0 else kv[b]
        if q > 0:
            need = _pages(kv[b] + q) - _pages(kv[b])
            asked_pages, asked_tokens = asked_pages + need, asked_tokens + q
            if asked_tokens <= tokens and _pages(kv[b] + q) <= width and (need == 0 or asked_pages <= top):
                for i in range(need):
                    free -= 1
                    table[b][_pages(kv[b]) + i] = stack[free]
                for p in range(kv[b], kv[b] + q):
                    slots.append(table[b][p // PAGE] * PAGE + p % PAGE)
                    positions.append(p)
                length += q
        lens.append(length)
        indptr.append(len(slots))
    slots += [-1] * (tokens - len(slots))
    positions += [0] * (tokens - len(positions))
    long = dict(dtype=torch.int64, device=DEV)
    return {"table": _int32(table), "free_pages": _int32(stack), "kv_out": _int32(lens), "free_out": _int32([free]),
            "q_indptr": _int32(indptr), "slots": torch.tensor(slots, **long),
            "positions": torch.tensor(positions, **long)}


def _turned(x, angle, interleaved):
    """Pairs as complex numbers times cos + i sin."""
    turn = torch.complex(angle[..., :ROPE // 2], angle[..., ROPE // 2:])
    if interleaved:
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], ROPE // 2, 2).contiguous()) * turn).flatten(-2)
    z = torch.complex(x[..., :ROPE // 2].contiguous(), x[..., ROPE // 2:].contiguous()) * turn
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    kv, new, rows = _lengths(case)
    heads = case["heads"]
    if case["op"] == "tables":
        return _exact_tables(s)
    if case["op"] == "append":
        pool, q = s["pool"].double(), s["q_rows"].double()
        angle = s["cos_sin"].double()[s["positions"]]
        x = s["src"].double()
        rms = torch.linalg.vector_norm(x[:, :LATENT], dim=1, keepdim=True) / math.sqrt(LATENT)
        lat = x[:, :LATENT] * s["weight"].double() / torch.hypot(rms, torch.full_like(rms, math.sqrt(EPS)))
        row = torch.cat([lat, _turned(x[:, LATENT:], angle, case["interleaved"])], 1)
        flat = pool.view(-1, LATENT + ROPE)
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        flat[s["slots"][keep]] = row[keep]
        q[..., LATENT:] = _turned(s["q_pe"].double(), angle[:, None], case["interleaved"])
        return {"pool": pool, "q": q}
    paged = case["op"] == "absorbed"
    dv = LATENT if paged else VALUE
    out = torch.zeros(s["q"].shape[0], heads, dv, dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], float("-inf"), dtype=torch.float64, device=DEV)
    at = k0 = 0
    for b in range(case["batch"]):
        j = torch.arange(kv[b], device=DEV)
        if paged:
            lat = s["pool"][s["table"][b].long()[j // PAGE], j % PAGE].double()
        step = max(1, (1 << 26) // max(1, heads * kv[b]))
        for i0 in range(0, new[b], step):
            i1 = min(new[b], i0 + step)
            q = s["q"][at + i0:at + i1].double()
            if paged:
                sc = torch.einsum("rhd,kd->hrk", q, lat)
            else:
                sc = torch.einsum("rhd,khd->hrk", q[..., :NOPE], s["k"][k0:k0 + kv[b]].double())
                sc += torch.einsum("rhd,kd->hrk", q[..., NOPE:], s["k_pe"][k0:k0 + kv[b]].double())
            sc = sc / math.sqrt(NOPE + ROPE)
            if case["mask"] == "causal":
                p = (kv[b] - new[b] + torch.arange(i0, i1, device=DEV))[:, None]
                sc = torch.where(j <= p, sc, float("-inf"))
            l = torch.logsumexp(sc, -1)
            w = torch.exp(sc - l[..., None])
            if paged:
                out[at + i0:at + i1] = torch.einsum("hrk,kd->rhd", w, lat[:, :LATENT])
            else:
                out[at + i0:at + i1] = torch.einsum("hrk,khd->rhd", w, s["v"][k0:k0 + kv[b]].double())
            lse[at + i0:at + i1] = l.t()
        at += rows[b] if paged else new[b]
        k0 += kv[b]
    return {"out": out, "lse": lse}
