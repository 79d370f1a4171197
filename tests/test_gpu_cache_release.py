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


@pytest.mark.parametrize("first,second", [(0, 1), (0, 5), (3, 4)])
def test_a_page_that_is_twice_on_the_stack(first, second):
    """It would go to two places: the call that needs both is refused."""
    p = Pair(1, 1300, 1, 16, 8, 6, 1200)
    p.extend_append([0], [30])
    c, top = p.c, int(p.c.words[0])
    was = int(c.free[top - 1 - second])
    c.free[top - 1 - second] = int(c.free[top - 1 - first])
    for _ in range(5):
        refused(p, lambda: c.extend(ints([1]), ints([16 * (second + 1)])), pi.PI_CACHE_EPAGE)
        refused(p, lambda: c.extend(ints([1, 2, 3]), ints([16 * 400, 16, 16 * 700])), pi.PI_CACHE_EPAGE)
        refused(p, lambda: c.extend(ints([1, 9]), ints([16 * 1100, 1])), pi.PI_CACHE_EPAGE | pi.PI_CACHE_ESLOT)
        if second < 5:
            refused(p, lambda: c.fork(ints([0] * 5), ints([1, 2, 3, 4, 5])), pi.PI_CACHE_EPAGE)
    c.free[top - 1 - second] = was
    p.m.extend([1, 2], [16 * 1100, 3])
    c.extend(ints([1, 2]), ints([16 * 1100, 3]))
    p.m.fork([0] * 3, [3, 4, 5])
    c.fork(ints([0] * 3), ints([3, 4, 5]))
    p.check()


def test_a_free_page_in_a_parents_table():
    """The page that a copy would go to is the parent's own last page by its table, and counted as free."""
    p = Pair(1, 12, 1, 16, 8, 6, 8)
    p.extend_append([0], [30])
    page = int(p.c.table[0, 1])
    top = int(p.c.words[0])
    p.c.ref[page], p.c.free[top], p.c.words[0] = 0, page, top + 1
    for _ in range(5):
        refused(p, lambda: p.c.fork(ints([0]), ints([1])), pi.PI_CACHE_EPAGE)
