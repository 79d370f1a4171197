"""The paged cache's upkeep against a model of it in plain Python: every word has to be equal."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402

DEV = "cuda:0"


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Model:
    """What include/pi.h says the calls do, on lists; the pools hold a number per (layer, page, token)."""

    def __init__(self, layers, pages, page, slots, max_pages):
        self.layers, self.pages, self.page, self.slots, self.max_pages = layers, pages, page, slots, max_pages
        self.table = [[0] * max_pages for _ in range(slots)]
        self.lens, self.ref = [0] * slots, [0] * pages
        self.free, self.error, self.used = list(range(pages - 1, -1, -1)), 0, 0
        self.pool = [[[0.0] * page for _ in range(pages)] for _ in range(layers)]

    def held(self, n):
        return -(-n // self.page)

    def extend(self, seqs, counts):
        need = [self.held(self.lens[s] + c) - self.held(self.lens[s]) for s, c in zip(seqs, counts)]
        if any(self.lens[s] + c > self.max_pages * self.page for s, c in zip(seqs, counts)):
            self.error |= pi.PI_CACHE_ELENGTH
            return
        if sum(need) > len(self.free):
            self.error |= pi.PI_CACHE_EFULL
            return
        for s, c, n in zip(seqs, counts, need):
            at = self.held(self.lens[s])
            for j in range(n):
                p = self.free.pop()
                self.table[s][at + j], self.ref[p] = p, 1
            self.lens[s] += c

    def append(self, layer, values, cu, seqs):
        for i, s in enumerate(seqs):
            n = cu[i + 1] - cu[i]
            for j in range(n):
                pos = self.lens[s] - n + j
                self.pool[layer][self.table[s][pos // self.page]][pos % self.page] = values[cu[i] + j]

    def fork(self, parents, children):
        lens = [self.lens[p] for p in parents]
        part = [n % self.page != 0 for n in lens]
        if sum(part) > len(self.free):
            self.error |= pi.PI_CACHE_EFULL
            return
        for p, c, n, own in zip(parents, children, lens, part):
            whole = n // self.page
            for j in range(whole):
                self.table[c][j] = self.table[p][j]
                self.ref[self.table[p][j]] += 1
            if own:
                new, old = self.free.pop(), self.table[p][whole]
                self.table[c][whole], self.ref[new] = new, 1
                for layer in self.pool:
                    layer[new] = list(layer[old])
            self.lens[c] = n

    def release(self, seqs):
        empty = []
        for s in seqs:
            for j in range(self.held(self.lens[s])):
                p = self.table[s][j]
                self.ref[p] -= 1
                if self.ref[p] == 0:
                    empty.append(p)
            self.lens[s] = 0
        self.free += sorted(empty, reverse=True)

    def compact(self):
        used = sum(r > 0 for r in self.ref)
        holes = [p for p in range(used) if self.ref[p] == 0]
        movers = [p for p in range(used, self.pages) if self.ref[p] > 0]
        to = [p if r > 0 else -1 for p, r in enumerate(self.ref)]
        for h, m in zip(holes, movers):
            to[m] = h
            self.ref[h], self.ref[m] = self.ref[m], 0
            for layer in self.pool:
                layer[h] = list(layer[m])
        for s in range(self.slots):
            for j in range(self.held(self.lens[s])):
                self.table[s][j] = to[self.table[s][j]]
        self.free, self.used = list(range(self.pages - 1, used - 1, -1)), used
        return to


class Pair:
    """A cache and its model; values are numbers that the 16-bit types hold, spread over heads and dims."""

    def __init__(self, layers, pages, kv_heads, page, dim, slots, max_pages, dtype=torch.float16):
        self.c = pi.Cache.create(layers, pages, kv_heads, page, dim, slots, max_pages, dtype, DEV)
        self.m = Model(layers, pages, page, slots, max_pages)
        self.spread = (torch.arange(kv_heads * dim) % 7 + 1).view(kv_heads, dim).to(dtype)
        self.count = 0

    def rows(self, values):
        return (torch.tensor(values).to(self.spread.dtype).view(-1, 1, 1) * self.spread).to(DEV)

    def extend_append(self, seqs, counts):
        self.m.extend(seqs, counts)
        self.c.extend(ints(seqs), ints(counts))
        if self.m.error:
            return
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        for layer in range(self.m.layers):
            values = [float((self.count + i) % 31 + layer + 1) for i in range(cu[-1])]
            self.count += cu[-1]
            self.m.append(layer, values, cu, seqs)
            k = self.rows(values)
            self.c.append(layer, k, -k, ints(cu), ints(seqs))

    def check(self, pool=True):
        c, m = self.c, self.m
        assert c.errors() == m.error
        assert c.lens.tolist() == m.lens
        assert c.ref.tolist() == m.ref
        assert c.words.tolist() == [len(m.free), m.error, m.used, 0]
        assert c.free[:len(m.free)].tolist() == m.free
        table = c.table.tolist()
        for s in range(m.slots):
            n = m.held(m.lens[s])
            assert table[s][:n] == m.table[s][:n], s
        if pool:
            for layer in range(m.layers):
                want = (torch.tensor(m.pool[layer]).to(self.spread.dtype).view(m.pages, 1, m.page, 1)
                        * self.spread.view(1, -1, 1, self.spread.shape[1]))
                assert torch.equal(c.k_pool[layer].cpu(), want), layer
                assert torch.equal(c.v_pool[layer].cpu(), -want), layer


@pytest.mark.parametrize("layers,pages,kv_heads,page,dim,slots,dtype", [
    (2, 90, 2, 16, 64, 6, torch.float16),
    (1, 40, 1, 48, 8, 3, torch.bfloat16),
    (3, 300, 3, 32, 40, 12, torch.bfloat16),
])
def test_a_life_of_a_cache(layers, pages, kv_heads, page, dim, slots, dtype):
    """Prompts, single tokens, forks, releases and compactions in an order that the seed gives."""
    rnd = random.Random(pages)
    p = Pair(layers, pages, kv_heads, page, dim, slots, pages, dtype)
    for step in range(60):
        live = [s for s in range(slots) if p.m.lens[s]]
        idle = [s for s in range(slots) if not p.m.lens[s]]
        what = rnd.choice(["prompt", "token", "fork", "release", "compact"])
        if what == "prompt" and idle:
            seqs = rnd.sample(idle, rnd.randint(1, len(idle)))
            counts = [rnd.choice([0, 1, page - 1, page, page + 1, rnd.randint(1, 3 * page)]) for _ in seqs]
            if sum(p.m.held(n) for n in counts) <= len(p.m.free):
                p.extend_append(seqs, counts)
        elif what == "token" and live:
            if len(live) <= len(p.m.free):
                p.extend_append(live, [1] * len(live))
        elif what == "fork" and live and idle:
            kids = rnd.sample(idle, rnd.randint(1, len(idle)))
            parents = [rnd.choice(live + idle[:1]) for _ in kids]
            parents = [live[0] if q in kids else q for q in parents]
            if len(kids) <= len(p.m.free):
                p.m.fork(parents, kids)
                p.c.fork(ints(parents), ints(kids))
        elif what == "release" and live:
            gone = rnd.sample(live, rnd.randint(1, len(live))) + idle[:1]
            p.m.release(gone)
            p.c.release(ints(gone))
        else:
            moved = torch.full((pages,), -9, dtype=torch.int32, device=DEV) if step % 2 else None
            to = p.m.compact()
            p.c.compact(moved)
            assert moved is None or moved.tolist() == to
        p.check(pool=step % 5 == 0)
    p.check()


def test_pools_beyond_a_block_of_threads():
    """More pages, and more listed slots, than an accounting block has threads."""
    p = Pair(1, 5000, 1, 16, 8, 2600, 4)
    seqs = random.Random(1).sample(range(2600), 2500)
    p.extend_append(seqs, [(i * 7) % 29 + 1 for i in range(2500)])
    p.check()
    gone = seqs[::2]
    p.m.release(gone)
    p.c.release(ints(gone))
    p.check(pool=False)
    kids, parents = gone[:900], [seqs[2 * i + 1] for i in range(900)]
    p.m.fork(parents, kids)
    p.c.fork(ints(parents), ints(kids))
    p.check()
    p.m.compact()
    p.c.compact()
    p.check()


@pytest.mark.parametrize("live", [0, 1, 7, 8])
def test_compaction_of_empty_full_and_nearly_full_pools(live):
    p = Pair(2, 8, 1, 16, 64, 8, 2)
    p.extend_append(list(range(8)), [16] * 8)
    gone = list(range(8 - live))
    if gone:
        p.m.release(gone)
        p.c.release(ints(gone))
    p.m.compact()
    p.c.compact()
    p.check()
    if live < 8:                                       # the pool is whole: new tokens go in
        p.extend_append([0], [1])
        p.check()


def test_append_strides_and_rows_of_no_sequence():
    p = Pair(2, 20, 2, 16, 24, 3, 5)
    seqs, counts = [2, 0], [20, 5]
    p.m.extend(seqs, counts)
    p.c.extend(ints(seqs), ints(counts))
    values = [float(i + 1) for i in range(30)]
    p.m.append(1, values, [3, 23, 28], seqs)
    wide = torch.full((30, 4, 32), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, :2, 8:] = p.rows(values)
    wide[:, 2:, 8:] = -p.rows(values)
    p.c.append(1, wide[:, :2, 8:], wide[:, 2:, 8:].clone().transpose(0, 1).contiguous().transpose(0, 1),
               ints([3, 23, 28]), ints(seqs))
    p.check()
    p.c.append(0, wide[:0, :2, 8:], wide[:0, 2:, 8:], ints([0, 0, 0]), ints(seqs))
    p.check()


def refused(p, call, bits):
    """The call changes nothing but the error word."""
    meta, k = p.c.meta.clone(), p.c.k_pool.clone()
    call()
    assert p.c.errors() == bits
    meta[p.c.meta.numel() - 3] = bits
    assert torch.equal(p.c.meta, meta) and torch.equal(p.c.k_pool, k)
    p.c.words[1] = 0


def test_calls_that_cannot_be_carried_out_change_nothing():
    p = Pair(1, 12, 1, 16, 8, 6, 8)
    p.extend_append([0, 1], [40, 17])
    c = p.c
    refused(p, lambda: c.extend(ints([2]), ints([16 * 7 + 1])), pi.PI_CACHE_EFULL)     # 7 pages are free
    refused(p, lambda: c.extend(ints([0, 2]), ints([1, 8 * 16 + 1])), pi.PI_CACHE_ELENGTH)
    refused(p, lambda: c.extend(ints([0]), ints([(1 << 31) - 1])), pi.PI_CACHE_ELENGTH)
    refused(p, lambda: c.extend(ints([0, 1]), ints([1, -1])), pi.PI_CACHE_ELENGTH)
    refused(p, lambda: c.extend(ints([0, 6]), ints([1, 1])), pi.PI_CACHE_ESLOT)
    refused(p, lambda: c.extend(ints([-1]), ints([1])), pi.PI_CACHE_ESLOT)
    refused(p, lambda: c.extend(ints([3, 4, 3]), ints([1, 1, 1])), pi.PI_CACHE_ESLOT)
    refused(p, lambda: c.fork(ints([0]), ints([1])), pi.PI_CACHE_ESLOT)                # a child that holds tokens
    refused(p, lambda: c.fork(ints([0, 0]), ints([2, 2])), pi.PI_CACHE_ESLOT)
    refused(p, lambda: c.fork(ints([6]), ints([2])), pi.PI_CACHE_ESLOT)
    refused(p, lambda: c.fork(ints([0]), ints([-2])), pi.PI_CACHE_ESLOT)
    refused(p, lambda: c.release(ints([0, 0])), pi.PI_CACHE_ESLOT)
    refused(p, lambda: c.release(ints([1, 9])), pi.PI_CACHE_ESLOT)
    p.check()
    # a fork whose copies find no page
    p.extend_append([2], [16 * 7])
    refused(p, lambda: c.fork(ints([0]), ints([3])), pi.PI_CACHE_EFULL)
    p.m.fork([2], [3])                                 # whole pages need none
    c.fork(ints([2]), ints([3]))
    p.check()


def test_broken_tables_are_not_followed():
    p = Pair(1, 12, 1, 16, 8, 6, 8)
    p.extend_append([0, 1], [40, 17])
    c = p.c
    for bad in (-1, 12, 1 << 30):
        was = int(c.table[0, 1])
        c.table[0, 1] = bad
        refused(p, lambda: c.fork(ints([0]), ints([2])), pi.PI_CACHE_EPAGE)
        refused(p, lambda: c.release(ints([0])), pi.PI_CACHE_EPAGE)
        k = p.rows([1.0] * 40)
        pool = c.k_pool.clone()
        c.append(0, k, k, ints([0, 40]), ints([0]))
        assert c.errors() == pi.PI_CACHE_EPAGE
        c.words[1] = 0
        diff = (c.k_pool != pool).flatten(2).any(-1)[0].nonzero().flatten().tolist()
        assert set(diff) <= {int(c.table[0, 0]), int(c.table[0, 2])}
        c.k_pool.copy_(pool)
        c.v_pool.copy_(-pool)
        c.table[0, 1] = was
    for bad in (-1, 12, 1 << 30):                      # the stack's top entry, and a page on it that is in use
        was = int(c.free[int(c.words[0]) - 1])
        c.free[int(c.words[0]) - 1] = bad
        refused(p, lambda: c.extend(ints([3]), ints([1])), pi.PI_CACHE_EPAGE)
        c.free[int(c.words[0]) - 1] = was
    was = int(c.free[int(c.words[0]) - 1])
    c.free[int(c.words[0]) - 1] = int(c.table[1, 0])
    refused(p, lambda: c.extend(ints([3]), ints([1])), pi.PI_CACHE_EPAGE)
    c.free[int(c.words[0]) - 1] = was
    for bad in (-1, 13, 1 << 30):
        was = int(c.words[0])
        c.words[0] = bad
        refused(p, lambda: c.extend(ints([3]), ints([1])), pi.PI_CACHE_EPAGE)
        refused(p, lambda: c.release(ints([0])), pi.PI_CACHE_EPAGE)
        c.words[0] = was
    for bad in (-1, 8 * 16 + 1, (1 << 31) - 1):
        was = int(c.lens[1])
        c.lens[1] = bad
        refused(p, lambda: c.extend(ints([1]), ints([1])), pi.PI_CACHE_ELENGTH)
        refused(p, lambda: c.fork(ints([1]), ints([2])), pi.PI_CACHE_ELENGTH)
        refused(p, lambda: c.release(ints([1])), pi.PI_CACHE_ELENGTH)
        c.lens[1] = was
    p.check()
    # rows for a slot that is out of range, or with more rows than the slot has tokens
    k = p.rows([1.0] * 20)
    c.append(0, k, k, ints([0, 20]), ints([6]))
    assert c.errors() == pi.PI_CACHE_ESLOT
    c.words[1] = 0
    c.append(0, k[:18], k[:18], ints([0, 18]), ints([1]))
    assert c.errors() == pi.PI_CACHE_ELENGTH
    # a table entry of a page that is not in use, found by the compaction, stays as it was
    c.words[1] = 0
    c.table[0, 0] = int(c.free[0])
    was = int(c.table[0, 0])
    c.compact()
    assert c.errors() == pi.PI_CACHE_EPAGE and int(c.table[0, 0]) == was


def test_forks_and_compactions_in_a_graph():
    """A captured fork, release and compaction: every replay equals the model."""
    p = Pair(2, 30, 1, 16, 8, 4, 8)
    p.extend_append([0], [40])
    parents, kids = ints([0, 0]), ints([1, 2])

    def step():
        p.c.fork(parents, kids)
        p.c.release(kids[:1])
        p.c.compact()
        p.c.release(kids[1:])

    def model():
        p.m.fork([0, 0], [1, 2])
        p.m.release([1])
        p.m.compact()
        p.m.release([2])
    step(), model()
    p.check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        graph.replay()
        model()
        p.check()
        p.extend_append([0], [3])
        p.check()
