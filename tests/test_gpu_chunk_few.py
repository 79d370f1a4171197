"""Attention of chunks of few rows (decoding steps, drafts) over a paged cache: scores capped, biased by distance and in a
window, against 64 bits (chunk_ref.py).  A call whose chunks have up to 32 rows (tokens times heads of a key head) on the
average goes to a kernel of its own, with 16 or 32 rows a block."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import chunk_ref  # noqa: E402
from test_gpu_chunk import DEV, TYPES, Held, normal, run  # noqa: E402

LENS = [300, 70, 1000, 64]
HEADS = [(4, 2, 64), (8, 2, 80), (8, 1, 128), (6, 2, 96), (4, 1, 256), (2, 1, 192), (16, 1, 128)]
COUNTS = [(1, 1, 1, 1), (3, 1, 5, 2), (8, 8, 8, 8), (2, 0, 9, 1)]


def rows_of(counts, heads, kv_heads):
    return -(-sum(counts) // len(counts)) * (heads // kv_heads)


FORMS = [(*h, c) for h in HEADS for c in COUNTS if rows_of(c, h[0], h[1]) <= 32]


def test_forms_reach_both_sizes_of_blocks():
    assert {-(-rows_of(c, h, g) // 16) for h, g, _, c in FORMS} == {1, 2}
    assert {d for _, _, d, _ in FORMS} >= {64, 80, 128, 256}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("cap,sloped,window", [(0.0, False, 0), (20.0, False, 0), (0.5, False, 0), (1024.0, False, 0),
                                               (0.0, True, 0), (0.0, True, 1), (0.0, False, 1),
                                               (0.0, False, 31), (0.0, False, 32), (0.0, False, 33), (0.0, False, 63),
                                               (0.0, False, 64), (0.0, False, 65), (3.0, False, 33),
                                               (30.0, True, 100), (30.0, True, 0), (0.0, False, (1 << 31) - 1)])
@pytest.mark.parametrize("heads,kv_heads,dim,counts", FORMS)
def test_scores(heads, kv_heads, dim, counts, cap, sloped, window, dtype):
    h = Held(dim + sum(counts), 1, kv_heads, 16, dim, LENS, TYPES[dtype])
    q = normal(7, sum(counts), heads, dim, dtype=TYPES[dtype], scale=4.0 if cap else 1.0)
    slopes = None
    if sloped:
        slopes = torch.tensor([2.0 ** (-8 * (i + 1) / heads) * (-0.01 if i == 1 else 1) for i in range(heads)],
                              dtype=torch.float32, device=DEV)
    out = run(h, q, list(counts), cap=cap, slopes=slopes, window=window)
    chunk_ref.check(out, *chunk_ref.chunk(q, h.k, h.v, counts, cap=cap, slopes=None if slopes is None else slopes.tolist(),
                                          window=window))
    assert h.cache.errors() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("count", [1, 5])
def test_large_pages_many_keys(count, dtype):
    """Keys that are shared out, places that lie inside large pages, a cap, a bias and a window that starts inside a page."""
    lens, heads, kv_heads, dim = [5000, 3210], 8, 2, 128
    counts = [count] * 2
    h = Held(dim + count, 1, kv_heads, 256, dim, lens, TYPES[dtype])
    q = normal(7, sum(counts), heads, dim, dtype=TYPES[dtype], scale=2.0)
    slopes = [2.0 ** -(i + 3) for i in range(heads)]
    out = run(h, q, counts, cap=15.0, slopes=torch.tensor(slopes, device=DEV), window=2777)
    chunk_ref.check(out, *chunk_ref.chunk(q, h.k, h.v, counts, cap=15.0, slopes=slopes, window=2777))
    assert h.cache.errors() == 0
