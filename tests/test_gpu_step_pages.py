"""assign_step_pages against its rules written out sequence by sequence."""
import random

import pytest
import torch

from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


def pages(n):
    return (n + 31) // 32


def plain(new, kv, free, stack, table, tokens):
    """The documented rules on Python lists; also the error bits."""
    table, stack, width, cap, err = [list(r) for r in table], list(stack), len(table[0]), len(stack), 0
    for b, q in enumerate(new):
        if q < 0:
            for p in table[b][:pages(kv[b])]:
                if free < cap:
                    stack[free] = p
                    free += 1
                else:
                    err |= pkv.PKV_ERRBIT_PAGE
    height, need_sum, token_sum = free, 0, 0
    slots, positions, indptr, lens = [], [], [0], []
    for b, q in enumerate(new):
        lens.append(0 if q < 0 else kv[b])
        if q > 0:
            need = pages(kv[b] + q) - pages(kv[b])
            need_sum, token_sum = need_sum + need, token_sum + q
            if token_sum > tokens or pages(kv[b] + q) > width:
                err |= pkv.PKV_ERRBIT_LEN
            elif need == 0 or need_sum <= height:
                for i in range(need):
                    free -= 1
                    table[b][pages(kv[b]) + i] = stack[free]
                for p in range(kv[b], kv[b] + q):
                    slots.append(table[b][p // 32] * 32 + p % 32)
                    positions.append(p)
                lens[b] += q
        indptr.append(len(slots))
    pad = tokens - len(slots)
    return table, stack, lens, free, indptr, slots + [-1] * pad, positions + [0] * pad, err


def make(rng, batch, kv_hi, new_hi, finished, free, spare=1, pad=0):
    kv = [rng.randint(0, kv_hi) for _ in range(batch)]
    new = [rng.choice([0, 1, rng.randint(1, new_hi)]) for _ in range(batch)]
    for b in rng.sample(range(batch), finished):
        new[b] = -1
    held = sum(pages(k) for k in kv)
    ids = list(range(held + free))
    rng.shuffle(ids)
    width = max(pages(k + max(q, 0)) for k, q in zip(kv, new)) + spare
    table = [[ids.pop() for _ in range(pages(k))] for k in kv]
    table = [t + [-7] * (width - len(t)) for t in table]
    stack = ids + [-9] * held
    return new, kv, free, stack, table, sum(q for q in new if q > 0) + pad


def check(new, kv, free, stack, table, tokens, in_place=False):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want = plain(new, kv, free, stack, table, tokens)
    t, s, nl, kl, nf = i32(table), i32(stack), i32(new), i32(kv), i32([free])
    ko, fo = (kl, nf) if in_place else (i32([77] * len(kv)), i32([77]))
    qi = i32([77] * (len(kv) + 1))
    slots, positions = (torch.full((tokens,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    err = i32([0])
    for _ in range(1 if in_place else 2):  # apart from its inputs a call can be repeated
        pkv.assign_step_pages(nl, kl, nf, s, t, kv_lens_out=ko, num_free_out=fo, q_indptr=qi, slots=slots,
                              positions=positions, err=err)
        got = (t.tolist(), s.tolist(), ko.tolist(), int(fo), qi.tolist(), slots.tolist(), positions.tolist(), int(err))
        for name, g, w in zip(("table", "stack", "kv", "free", "q_indptr", "slots", "positions", "err"), got, want):
            assert g == w, name


@pytest.mark.parametrize("batch", [1, 2, 31, 64, 257, 511, 512, 513, 1500, 4096])
@pytest.mark.parametrize("in_place", [False, True])
def test_random_batches(batch, in_place):
    rng = random.Random(batch)
    check(*make(rng, batch, 200, 40, batch // 7, 30 * batch, pad=rng.choice([0, 50])), in_place=in_place)


@pytest.mark.parametrize("seed", range(12))
def test_too_few_pages(seed):
    rng = random.Random(seed)
    batch = rng.choice([5, 60, 700])
    check(*make(rng, batch, 100, 70, rng.choice([0, batch // 4]), rng.randint(0, batch // 2)))


@pytest.mark.parametrize("batch", [3, 300])
def test_too_few_tokens_or_columns(batch):
    new, kv, free, stack, table, tokens = make(random.Random(1), batch, 100, 70, 1, 10 * batch)
    check(new, kv, free, stack, table, tokens // 2)
    check(new, kv, free, stack, table, 0)
    # a table too narrow for some requests
    width = len(table[0]) - 2
    fits = [b for b in range(batch) if pages(kv[b]) <= width]
    check([new[b] for b in fits], [kv[b] for b in fits], free, stack, [table[b][:width] for b in fits], tokens)


def test_prompts_of_many_pages():
    new, kv, free, stack, table, tokens = make(random.Random(2), 9, 500, 5000, 2, 2000, pad=7)
    check(new, kv, free, stack, table, tokens)


def test_no_free_pages_at_all():
    """An empty stack: only sequences with room in their last page go on."""
    check([1, 1, 5, -1], [31, 32, 20, 0], 0, [], [[3, -1], [4, -1], [5, -1], [-1, -1]], 9)


def test_stack_full_and_odd_counts():
    """Pages that do not fit the stack are dropped; counts outside it are clamped."""
    table = [[3, 4, 5], [6, 7, 8]]
    check([-1, 1], [96, 64], 1, [9, -1], table, 4)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for free, kv in ((5, 64), (-2, 64), (2, -4)):
        t, err, fo, ko, qi = i32(table), i32([0]), i32([0]), i32([0, 0]), i32([0, 0, 0])
        z = torch.zeros(4, dtype=torch.int64, device="cuda")
        pkv.assign_step_pages(i32([0, 1]), i32([10, kv]), i32([free]), i32([1, 2]), t, kv_lens_out=ko, num_free_out=fo,
                              q_indptr=qi, slots=z, positions=torch.zeros_like(z), err=err)
        assert int(err) == pkv.PKV_ERRBIT_PAGE
        height = min(max(free, 0), 2)
        granted = height > 0
        assert int(fo) == height - granted and qi.tolist() == [0, 0, int(granted)]
        assert ko.tolist() == [10, max(kv, 0) + granted]
