"""The slots and positions of assign_step_pages in the other caches' writes:
kv_scatter_slots and rope_write_kv_paged, with rows behind the step's last
token that must not be written."""
import pytest
import torch

from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
HKV, D = 2, 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("other_stream", [False, True])
def test_rows_land_where_the_tables_say(other_stream):
    """Two steps of three sequences: a prompt, one that grows over a page, one that waits and starts later."""
    pages, T = 12, 60
    g = torch.Generator().manual_seed(1)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    table, kv, n, qi = torch.full((3, 4), -1, dtype=torch.int32, device=DEV), i32([0, 0, 0]), i32([pages]), i32([0] * 4)
    stack = i32(list(range(pages)))
    slots, positions = (torch.zeros(T, dtype=torch.int64, device=DEV) for _ in range(2))
    ang = torch.zeros(128, D, device=DEV)
    ang[:, :D // 2] = (torch.arange(128, device=DEV) % 2 * 2.0 - 1)[:, None]   # turns by 0 or pi: a sign, exact
    pools = [torch.full((pages, 32, HKV, D), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    want = [p.clone() for p in pools]
    held = [0, 0, 0]
    stream = torch.cuda.Stream() if other_stream else torch.cuda.current_stream()
    for ask in ([40, 7, 0], [1, 30, 20]):
        k, v, q = bf(T, HKV, D), bf(T, HKV, D), bf(T, 4, D)
        new, before = i32(ask), q.clone()
        torch.cuda.synchronize()
        pkv.assign_step_pages(new, kv, n, stack, table, kv_lens_out=kv, num_free_out=n, q_indptr=qi, slots=slots,
                              positions=positions, stream=stream)
        pkv.kv_scatter_slots(k, v, slots, pools[0], pools[1], stream=stream)
        pkv.rope_write_kv_paged(q, k, v, positions, ang, slots, pools[2], pools[3], stream=stream)
        torch.cuda.synchronize()
        t = 0
        for b, x in enumerate(ask):
            for p in range(held[b], held[b] + x):
                page, off, sign = int(table[b, p // 32]), p % 32, 1.0 if p % 2 else -1.0
                want[0][page, off], want[1][page, off] = k[t], v[t]
                want[2][page, off], want[3][page, off] = k[t] * sign, v[t]
                assert torch.equal(q[t], before[t] * sign)
                t += 1
            held[b] += x
        assert kv.tolist() == held and qi.tolist()[-1] == t
        for got, w in zip(pools, want):
            assert torch.equal(got, w)
