"""A workspace of paged_attention_latent that is sized for the largest step
serves every smaller one: fewer sequences, rows, heads or keys never need more."""
import random

import pytest

from paged_kv_cache_189_gb300 import build as pkv_build
from paged_kv_cache_189_gb300 import pkv


@pytest.fixture(scope="module")
def size():
    pkv_build.build()
    return pkv.paged_attention_latent_workspace_size


def test_fewer_sequences(size):
    """128 short sequences go one to a CTA, 64 share the CTAs out and leave states to join."""
    sizes = [size(b, 1, 16, 1024) for b in range(1, 300)]
    assert sizes == sorted(sizes)
    # 64 sequences of 1024 keys: a first and a last state of 16 columns for each of 152 CTAs
    assert size(128, 1, 16, 1024) >= size(64, 1, 16, 1024) >= 152 * 2 * 16 * 513 * 4


@pytest.mark.parametrize("batch,keys", [(1, 64), (1, 8192), (3, 512), (64, 256), (64, 1024), (100, 8192), (152, 1024)])
def test_fewer_columns(size, batch, keys):
    """Across every column tile's border, by rows and by heads."""
    for counts in ([size(batch, 1, h, keys) for h in range(1, 300)], [size(batch, r, 1, keys) for r in range(1, 300)],
                   [size(batch, r, 16, keys) for r in range(1, 40)]):
        assert counts == sorted(counts)


@pytest.mark.parametrize("batch,heads", [(1, 16), (2, 128), (64, 16), (64, 65), (152, 64), (76, 128)])
def test_fewer_keys(size, batch, heads):
    sizes = [size(batch, 1, heads, k) for k in range(0, 3000, 13)]
    assert sizes == sorted(sizes)


def test_smaller_steps(size):
    rng = random.Random(0)
    for _ in range(3000):
        big = [rng.choice([1, rng.randint(1, 200)]), rng.choice([1, rng.randint(1, 64)]), rng.randint(1, 160),
               rng.choice([rng.randint(0, 1100), rng.randint(0, 20000)])]
        small = [rng.randint(min(1, x), x) for x in big]
        assert size(*small) <= size(*big), (small, big)
