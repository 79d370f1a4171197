"""Releases of a cache whose use counts or stack are broken: nothing changes but the error word, every time."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
from test_gpu_cache import Pair, ints, refused  # noqa: E402


@pytest.mark.parametrize("listed", [[0], [0, 1], [2, 1, 0], [0, 1, 2, 3]])
def test_a_page_that_is_held_more_often_than_counted(listed):
    p = Pair(1, 40, 1, 16, 8, 6, 8)
    p.extend_append([0, 3], [100, 70])
    p.m.fork([0, 0], [1, 2])
    p.c.fork(ints([0, 0]), ints([1, 2]))
    shared = int(p.c.table[0, 2])
    for count in range(len([s for s in listed if s != 3])):
        p.c.ref[shared] = count                        # one listed slot at least goes without
        for _ in range(5):
            refused(p, lambda: p.c.release(ints(listed)), pi.PI_CACHE_EPAGE)
    p.c.ref[shared] = 3
    p.m.release(listed)
    p.c.release(ints(listed))
    p.check()


@pytest.mark.parametrize("count", [0, -1, -(1 << 31)])
def test_a_count_that_cannot_be(count):
    p = Pair(1, 12, 1, 16, 8, 6, 8)
    p.extend_append([0, 1], [40, 17])
    page = int(p.c.table[0, 0])
    p.c.ref[page] = count
    refused(p, lambda: p.c.release(ints([1, 0])), pi.PI_CACHE_EPAGE)
    p.c.ref[page] = 1
    p.m.release([1, 0])
    p.c.release(ints([1, 0]))
    p.check()


def test_a_page_that_is_listed_twice_in_its_slot():
    p = Pair(1, 12, 1, 16, 8, 6, 8)
    p.extend_append([0, 1], [40, 17])
    was = int(p.c.table[0, 1])
    p.c.table[0, 1] = int(p.c.table[0, 0])
    refused(p, lambda: p.c.release(ints([0])), pi.PI_CACHE_EPAGE)
    p.c.table[0, 1] = was
    p.check()


def test_a_stack_without_room():
    """More pages would be free than there are."""
    p = Pair(1, 12, 1, 16, 8, 6, 8)
    p.extend_append([0, 1], [40, 17])
    p.c.words[0] = 10                                  # 7 are free, and the slots hold 5
    refused(p, lambda: p.c.release(ints([0])), pi.PI_CACHE_EPAGE)
    refused(p, lambda: p.c.release(ints([1, 0])), pi.PI_CACHE_EPAGE)
    p.c.words[0] = 7
    p.m.release([1, 0])
    p.c.release(ints([1, 0]))
    p.check()


def test_many_slots_that_share_pages():
    """More entries than a block has threads, each page held by many of the listed slots."""
    p = Pair(1, 700, 1, 16, 8, 60, 40)
    p.extend_append([0, 1], [600, 333])
    kids = list(range(2, 60))
    parents = [k % 2 for k in kids]
    p.m.fork(parents, kids)
    p.c.fork(ints(parents), ints(kids))
    p.check()
    for gone in (random.Random(1).sample(range(60), 40), list(range(60))):
        p.m.release(gone)
        p.c.release(ints(gone))
        p.check(pool=False)
    assert len(p.m.free) == 700
