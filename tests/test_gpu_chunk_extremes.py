"""Attention of chunks at the largest numbers of heads, of heads of a key head, and of sequences."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import chunk_ref  # noqa: E402
from test_gpu_chunk import TYPES, Held, normal, run  # noqa: E402


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,lens,counts", [
    (200, 1, 64, [90, 300], [3, 1]),                   # a tile of rows holds less than a token
    (129, 1, 128, [400], [5]),
    (4096, 1, 8, [70, 33], [2, 1]),
    (4096, 1024, 8, [40, 20], [1, 2]),
    (1024, 1024, 16, [33, 70], [1, 3]),
    (512, 2, 256, [140], [2]),
])
def test_heads(heads, kv_heads, dim, lens, counts, dtype):
    h = Held(dim + heads, 1, kv_heads, 16, dim, lens, TYPES[dtype])
    q = normal(7, sum(counts), heads, dim, dtype=TYPES[dtype])
    for window in (0, 20):
        chunk_ref.check(run(h, q, counts, window=window), *chunk_ref.chunk(q, h.k, h.v, counts, window=window))
    assert h.cache.errors() == 0


@pytest.mark.parametrize("n,heads,kv_heads", [(300, 4, 2), (4096, 2, 1)])
def test_sequences(n, heads, kv_heads):
    r = random.Random(n)
    lens = [r.choice([1, 5, 20, 70]) for _ in range(n)]
    lens[n - 2], lens[3] = 5000, 700
    counts = [r.choice([0, 1, min(m, 3), m if m < 10 else 1]) for m in lens]
    counts[n - 2], counts[3] = 150, 2
    h = Held(n, 1, kv_heads, 16, 64, lens, torch.bfloat16)
    for some in (counts, [min(c, 1) for c in counts]):  # in both kernels
        q = normal(7, sum(some), heads, 64, dtype=torch.bfloat16)
        chunk_ref.check(run(h, q, some), *chunk_ref.chunk(q, h.k, h.v, some))
    assert h.cache.errors() == 0
