"""A prefix that the batch's slots do not have in common is reported, and one that they have is not."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
from test_gpu_attention import DEV, TYPES, check_decode, ints, make_cache, normal  # noqa: E402


def errors_of(cache, q, prefix, seqs=None):
    cache.words[1] = 0
    out = torch.empty_like(q)
    pi.attn_decode(cache, 0, q, out, prefix=ints([prefix]), seqs=None if seqs is None else ints(seqs))
    got = cache.errors()
    cache.words[1] = 0
    return got


@pytest.mark.parametrize("heads,rows", [(8, 5), (2, 90), (64, 600)])   # one share a row in the last
def test_prefix_that_a_slot_does_not_have(heads, rows):
    kv_heads = 2
    shared = 20
    lens = [16 * shared + 1 + i % 50 for i in range(rows)]
    cache = make_cache(31, "bf16", kv_heads, 64, 16, lens, shared=shared)
    q = normal(4, rows, heads, 64, dtype=TYPES["bf16"])
    assert errors_of(cache, q, shared) == 0
    for row in (0, 1, rows - 1):                       # another page at the last common place of one row
        was = int(cache.table[row, shared - 1])
        cache.table[row, shared - 1] = int(cache.table[row, shared])
        assert errors_of(cache, q, shared) == pi.PI_CACHE_EPREFIX, row
        assert errors_of(cache, q, shared - 1) == 0
        others = [i for i in range(rows) if i != row][:4]
        assert errors_of(cache, q[:4], shared, others) == 0
        assert errors_of(cache, q[:1], shared, [row]) == 0
        cache.table[row, shared - 1] = was
    # longer than what they have in common: those that hold so much differ, if there are two
    holders = sum(n >= 16 * (shared + 1) for n in lens)
    assert errors_of(cache, q, shared + 1) == (pi.PI_CACHE_EPREFIX if holders > 1 else 0)


def test_slots_too_short_for_the_prefix_and_empty_ones_do_not_count():
    lens = [40, 161, 0, 200, 15]
    cache = make_cache(11, "f16", 2, 64, 16, lens, shared=10)
    q = normal(4, len(lens), 8, 64, dtype=torch.float16)
    check_decode(cache, q, prefix=10)                  # no error, and the results are right
    cache.table[0, 0] = int(cache.table[4, 0])
    assert errors_of(cache, q, 10) == 0


def test_long_prefix():
    """More pages than a block has threads."""
    lens = [9000, 8500]
    cache = make_cache(32, "f16", 1, 64, 16, lens, shared=500, layers=1)
    q = normal(4, 2, 4, 64, dtype=torch.float16)
    assert errors_of(cache, q, 500) == 0
    for place in (0, 255, 256, 499):
        was = int(cache.table[1, place])
        cache.table[1, place] = int(cache.table[1, 501])
        assert errors_of(cache, q, 500) == pi.PI_CACHE_EPREFIX
        cache.table[1, place] = was
