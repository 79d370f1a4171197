"""Decoding steps of many rows: one share a row, prefixes that only late rows hold, shares of the common keys that are longer
than one look-up of their pages."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import attn_ref  # noqa: E402
from test_gpu_attention import TYPES, check_decode, held_by, ints, make_cache, normal  # noqa: E402


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,rows", [(32, 32, 64, 33), (32, 16, 128, 70), (40, 2, 64, 300)])
def test_one_share_a_row(heads, kv_heads, dim, rows, dtype):
    """1024 tiles of queries and more."""
    assert rows * kv_heads * -(-(heads // kv_heads) // 16) >= 1024
    rnd = random.Random(rows)
    lens = [rnd.choice([0, 1, 15, 64, 130, 300]) for _ in range(rows)]
    lens[rows // 2] = 2500                             # one long row among them
    q = normal(4, rows, heads, dim, dtype=TYPES[dtype])
    check_decode(make_cache(61, dtype, kv_heads, dim, 16, lens), q)
    shared = 6
    lens = [0 if n == 0 else n if n < 64 else 16 * shared + n - 64 for n in lens]
    cache = make_cache(62, dtype, kv_heads, dim, 16, lens, shared=shared)
    for prefix in (shared, 0):
        check_decode(cache, q, prefix=prefix)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prefix_that_only_late_rows_hold(dtype):
    """More rows than one pass over the lengths takes, the first of which are too short."""
    shared = 20
    lens = [i % 17 for i in range(70)] + [16 * shared + i % 40 for i in range(30)] + [5] * 40 + [400]
    cache = make_cache(63, dtype, 2, 64, 16, lens, shared=shared)
    check_decode(cache, normal(4, len(lens), 8, 64, dtype=TYPES[dtype]), prefix=shared)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 64), (128, 32), (256, 48)])
def test_shares_of_many_tiles(dim, page, dtype):
    """512 rows of 64 heads leave two shares of the common keys, of 75 tiles each; also with a broken page in the second part of
    a share."""
    rows, heads = 512, 64
    shared = 9600 // page
    lens = [page * shared + i % 70 for i in range(rows)]
    cache = make_cache(64, dtype, 1, dim, page, lens, shared=shared, layers=1)
    q = normal(4, rows, heads, dim, dtype=TYPES[dtype])
    out = torch.full_like(q, float("nan"))
    some = [0, 1, 2, 69, 70, 255, 300, 510, 511]

    def check(drop=None):
        ks, vs = held_by(cache, 0)
        keep = [[j for j in range(lens[i]) if drop is None or j // page != drop] for i in some]
        ref = attn_ref.decode(q[some], [ks[i][k] for i, k in zip(some, keep)], [vs[i][k] for i, k in zip(some, keep)])
        attn_ref.check(out[some], *ref)
        assert torch.isfinite(out).all()

    pi.attn_decode(cache, 0, q, out, prefix=ints([shared]))
    assert cache.errors() == 0
    check()
    place = 4700 // page                               # tile 73 of the first share
    was = int(cache.table[0, place])
    cache.table[:, place] = cache.pages + 3
    pi.attn_decode(cache, 0, q, out, prefix=ints([shared]))
    assert cache.errors() == pi.PI_CACHE_EPAGE
    cache.table[:, place] = was
    check(place)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,rows,long", [(32, 32, 40, {7: 9000}), (16, 8, 140, {0: 1100, 70: 5000, 139: 6001}),
                                                      (2, 1, 1100, {5: 1025, 1099: 20000}), (32, 32, 40, {})])
def test_long_rows_among_many_short_ones(heads, kv_heads, rows, long, dtype):
    """Where the rows fill the card, the long ones are cut up all the same: those of several shares stand anywhere."""
    assert rows * kv_heads >= 1024
    lens = [long.get(i, 1 + i * 37 % 200) for i in range(rows)]
    cache = make_cache(65, dtype, kv_heads, 64, 64, lens, layers=2)
    q = normal(4, rows, heads, 64, dtype=TYPES[dtype])
    check_decode(cache, q)
    again = torch.empty_like(q)
    want = torch.empty_like(q)
    pi.attn_decode(cache, 1, q, want)
    for _ in range(3):
        pi.attn_decode(cache, 1, q, again)
        assert torch.equal(again, want)
