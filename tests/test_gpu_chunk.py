"""Attention of chunks of new tokens over a paged cache, against 64 bits (chunk_ref.py)."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import chunk_ref  # noqa: E402

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def normal(seed, *shape, dtype, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


def offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


class Held:
    """A cache whose slots hold lens tokens of random keys and values in pages that lie anywhere.  What is in no page, or in
    a page behind a slot's last token, is `rest`."""

    def __init__(self, seed, layers, kv_heads, page, dim, lens, dtype, rest=float("nan"), spare=3):
        held = [-(-n // page) for n in lens]
        pages = sum(held) + spare
        self.lens, self.page = lens, page
        self.cache = c = pi.Cache.create(layers, pages, kv_heads, page, dim, len(lens), max(max(held), 1) + 1, dtype=dtype,
                                         device=DEV)
        c.k_pool.fill_(rest), c.v_pool.fill_(rest)
        ids, at = random.Random(seed).sample(range(pages), sum(held)), 0
        self.k, self.v = [], []
        for i, (n, m) in enumerate(zip(lens, held)):
            mine = ids[at:at + m]
            at += m
            c.table[i, :m] = ints(mine)
            k, v = normal(seed + 2 * i, n, kv_heads, dim, dtype=dtype), normal(seed + 2 * i + 1, n, kv_heads, dim, dtype=dtype)
            self.k.append(k.cpu()), self.v.append(v.cpu())
            self.write(i, k, v)
        c.lens.copy_(ints(lens))

    def places(self, i, n):
        token = torch.arange(n, device=DEV)
        return self.cache.table[i, token // self.page].long(), token % self.page

    def write(self, i, k, v, layer=-1):
        """All tokens of a slot."""
        page, off = self.places(i, k.shape[0])
        self.cache.k_pool[layer][page, :, off] = k.to(DEV)
        self.cache.v_pool[layer][page, :, off] = v.to(DEV)


def run(held, q, counts, seqs=None, **kw):
    out = torch.full_like(q, float("nan"))
    pi.attn_chunk(held.cache, held.cache.layers - 1, q, out, ints(offsets(counts)), None if seqs is None else ints(seqs), **kw)
    return out


CHUNKS = [
    # heads, kv_heads, dim, page, lens, counts
    (4, 4, 128, 16, [1], [1]),
    (4, 2, 128, 16, [2, 1, 3], [1, 1, 3]),
    (32, 32, 128, 16, [1501], [1]),
    (8, 1, 128, 16, [64, 65, 63, 128], [1, 2, 63, 128]),
    (8, 2, 64, 32, [40, 200, 129, 64], [40, 7, 128, 33]),
    (6, 2, 96, 16, [100, 333], [37, 200]),
    (7, 1, 64, 48, [77, 1000], [60, 19]),
    (71, 1, 64, 16, [33, 500], [5, 1]),
    (16, 8, 256, 16, [20, 130], [20, 66]),
    (2, 2, 8, 16, [90, 40], [90, 1]),
    (3, 1, 24, 16, [129, 77], [100, 77]),
    (5, 5, 80, 64, [300], [150]),
    (1, 1, 136, 16, [333], [333]),
    (2, 1, 192, 16, [190, 20], [130, 0]),
    (128, 8, 64, 64, [513, 2, 70], [13, 2, 1]),
    (8, 8, 128, 16, [2500], [3]),
    (4, 1, 128, 4096, [4100, 9000], [2, 40]),
    (2, 1, 64, 16, [1037], [1037]),
    (28, 4, 128, 32, [700, 15], [129, 15]),
    (1, 1, 64, 16, [0, 70], [0, 70]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens,counts", CHUNKS)
def test_chunk(heads, kv_heads, dim, page, lens, counts, dtype):
    """Pages hold NaN behind the last tokens."""
    h = Held(dim + lens[0], 2, kv_heads, page, dim, lens, TYPES[dtype])
    q = normal(7, sum(counts), heads, dim, dtype=TYPES[dtype])
    out = run(h, q, counts)
    chunk_ref.check(out, *chunk_ref.chunk(q, h.k, h.v, counts))
    assert h.cache.errors() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("cap,sloped,window", [(20.0, False, 0), (0.0, True, 0), (0.0, False, 1), (0.0, False, 2),
                                               (0.0, False, 63), (0.0, False, 64), (0.0, False, 65), (0.0, False, 200),
                                               (0.0, False, (1 << 31) - 1), (30.0, True, 100), (1024.0, True, 1000),
                                               (0.5, False, 0), (3.0, False, 33), (0.0, True, 1)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (6, 2, 128), (2, 1, 256)])
def test_scores(heads, kv_heads, dim, cap, sloped, window, dtype):
    lens, counts = [300, 70, 1000, 64], [150, 70, 3, 1]
    h = Held(dim, 1, kv_heads, 16, dim, lens, TYPES[dtype])
    q = normal(7, sum(counts), heads, dim, dtype=TYPES[dtype], scale=4.0 if cap else 1.0)
    slopes = None
    if sloped:
        slopes = torch.tensor([2.0 ** (-8 * (i + 1) / heads) * (-0.01 if i == 1 else 1) for i in range(heads)],
                              dtype=torch.float32, device=DEV)
    out = run(h, q, counts, cap=cap, slopes=slopes, window=window)
    chunk_ref.check(out, *chunk_ref.chunk(q, h.k, h.v, counts, cap=cap, slopes=None if slopes is None else slopes.tolist(),
                                          window=window))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 80])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window", [0, 70])
def test_unseen_keys_leave_no_trace(window, poison, dim, dtype):
    """A key and a value that are not finite reach their own row and later ones that see them, no other row."""
    n, c, heads, at = 300, 220, 4, 170
    h = Held(dim, 1, 2, 16, dim, [n], TYPES[dtype])
    q = normal(7, c, heads, dim, dtype=TYPES[dtype])
    ref, tol = chunk_ref.chunk(q, h.k, h.v, [c], window=window)
    first = at - (n - c)                               # the row of that token
    behind = first + window if window else c           # the first row that does not see it any more
    for which in ("k", "v", "kv"):
        k, v = h.k[0].clone(), h.v[0].clone()
        if "k" in which:
            k[at] = poison
        if "v" in which:
            v[at] = poison
        h.write(0, k, v)
        out = run(h, q, [c], window=window)
        chunk_ref.check(out[:first], ref[:first], tol[:first], which)
        chunk_ref.check(out[behind:], ref[behind:], tol[behind:], which)
        if which == "v":
            assert not torch.isfinite(out[first:behind]).any()
        if poison != poison:
            assert torch.isnan(out[first:behind]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_value_of_a_key_is_not_finite(dtype):
    """Only that dimension of the rows that see it is lost, in tiles that some rows see in part."""
    n, c, heads, dim = 130, 100, 3, 64
    h = Held(3, 1, 1, 16, dim, [n], TYPES[dtype])
    q = normal(7, c, heads, dim, dtype=TYPES[dtype])
    ref, tol = chunk_ref.chunk(q, h.k, h.v, [c])
    v = h.v[0].clone()
    v[100, 0, 5], v[101, 0, 6], v[120, 0, 63] = float("inf"), -float("inf"), float("nan")
    h.write(0, h.k[0], v)
    out = run(h, q, [c])
    lost = torch.zeros(c, heads, dim, dtype=torch.bool)
    lost[70:, :, 5] = lost[71:, :, 6] = lost[90:, :, 63] = True
    got = out.cpu().double()
    chunk_ref.check(torch.where(lost, ref, got), ref, tol)
    assert (got[70:, :, 5] == float("inf")).all() and (got[71:, :, 6] == -float("inf")).all() and torch.isnan(got[90:, :, 63]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_keys_that_score_minus_infinity(dtype):
    """Keys with a score of -inf weigh nothing; a row that sees only such keys is zero."""
    n, dim = 150, 64
    h = Held(3, 1, 1, 16, dim, [n], TYPES[dtype])
    q = normal(7, n, 1, dim, dtype=TYPES[dtype]).abs() + 0.125
    k = h.k[0].clone()
    k[:40] = -float("inf")
    k[90:120, :, 3] = -float("inf")
    h.write(0, k, h.v[0])
    out = run(h, q, [n])
    assert (out[:40] == 0).all()
    live = [i for i in range(40, n) if not 90 <= i < 120]
    hi = torch.tensor([sum(j <= i for j in live) for i in range(40, n)])
    ref, tol = chunk_ref.rows(q[40:, 0].cpu().double(), k[live, 0].double(), h.v[0][live, 0].double(), torch.zeros_like(hi), hi,
                              hi, dim ** -0.5, 0.0, 0.0, TYPES[dtype])
    chunk_ref.check(out[40:, 0], ref, tol)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mode", ["rising", "falling", "spiky", "tiny", "equal", "dominant"])
def test_ranges_of_scores(mode, dtype):
    n, c, heads, dim = 1400, 40, 4, 64
    h = Held(5, 1, 2, 16, dim, [n], TYPES[dtype])
    q = normal(7, c, heads, dim, dtype=TYPES[dtype])
    k, v = h.k[0].clone(), h.v[0].clone()
    ramp = torch.linspace(0, 4, n).view(n, 1, 1)
    if mode == "rising":
        q, k = q.abs(), (k.abs() * ramp).to(TYPES[dtype])
    elif mode == "falling":
        q, k = q.abs(), (k.abs() * (4 - ramp)).to(TYPES[dtype])
    elif mode == "spiky":
        k[::97] *= 12
    elif mode == "tiny":
        q, k = (q * 1e-3).to(TYPES[dtype]), (k * 1e-3).to(TYPES[dtype])
    elif mode == "equal":
        k[:] = k[0]
    else:                                              # a first token that outscores all others and has a small value
        q = q.abs() + 0.5
        k[0], v[0] = 2.0, 1e-4
        k[1:] *= 0.2
    h.write(0, k, v)
    chunk_ref.check(run(h, q, [c]), *chunk_ref.chunk(q, [k], [v], [c]))


def test_scale():
    h = Held(3, 1, 1, 16, 64, [100], torch.float16)
    q = normal(7, 30, 2, 64, dtype=torch.float16)
    chunk_ref.check(run(h, q, [30], scale=0.5), *chunk_ref.chunk(q, h.k, h.v, [30], scale=0.5))


@pytest.mark.parametrize("heads,kv_heads,n", [(4, 2, 65), (2, 1, 130), (64, 8, 100)])
def test_many_sequences(heads, kv_heads, n):
    """More sequences than a wave has lanes: some without rows, some long ones among short ones, in any order of slots."""
    r = random.Random(n)
    lens = [r.choice([1, 5, 40, 130]) for _ in range(n)]
    lens[n - 2], lens[3] = 3100, 2000
    counts = [r.choice([0, 1, min(m, 3), m if m < 50 else 1]) for m in lens]
    counts[n - 2], counts[3] = 2, 37
    h = Held(n, 1, kv_heads, 16, 64, lens, torch.bfloat16)
    order = list(range(n))
    r.shuffle(order)
    counts = [counts[i] for i in order]
    q = normal(7, sum(counts), heads, 64, dtype=torch.bfloat16)
    out = run(h, q, counts, order)
    chunk_ref.check(out, *chunk_ref.chunk(q, [h.k[i] for i in order], [h.v[i] for i in order], counts))
    assert h.cache.errors() == 0


def test_long_among_short():
    """One long chunk behind many tokens and single tokens: its keys are shared out, theirs are not."""
    lens, counts = [7000, 30, 1, 900], [200, 1, 1, 2]
    h = Held(3, 1, 2, 16, 128, lens, torch.float16)
    q = normal(7, sum(counts), 8, 128, dtype=torch.float16)
    chunk_ref.check(run(h, q, counts), *chunk_ref.chunk(q, h.k, h.v, counts))


def test_a_slot_twice_and_rows_of_no_sequence():
    h = Held(3, 1, 1, 16, 64, [100, 50], torch.float16)
    q = normal(7, 60, 2, 64, dtype=torch.float16)
    out = torch.full_like(q, 7.0)
    pi.attn_chunk(h.cache, 0, q, out, ints([5, 15, 15, 35]), ints([0, 1, 0]))
    ref, tol = chunk_ref.chunk(q[5:35], [h.k[0], h.k[1], h.k[0]], [h.v[0], h.v[1], h.v[0]], [10, 0, 20])
    chunk_ref.check(out[5:35], ref, tol)
    assert (out[:5] == 7).all() and (out[35:] == 7).all()


def test_offsets_that_cannot_be_stay_inside():
    h = Held(3, 1, 1, 16, 64, [100, 50], torch.float16)
    q = normal(7, 60, 2, 64, dtype=torch.float16)
    out = torch.full_like(q, 7.0)
    pi.attn_chunk(h.cache, 0, q, out, ints([-5, 30, 1 << 30]))
    chunk_ref.check(out, *chunk_ref.chunk(q, h.k, h.v, [30, 30]))
    out.fill_(7.0)
    pi.attn_chunk(h.cache, 0, q, out, ints([0, 50, 20]))    # the second holds nothing
    chunk_ref.check(out[:50], *chunk_ref.chunk(q[:50], h.k[:1], h.v[:1], [50]))
    assert (out[50:] == 7).all()


def test_offsets_that_do_not_ascend_stay_inside():
    """Sequences that overlap, more rows in all than the tensor has, behind many tokens: what comes out is not said, but nothing
    outside the rows is written, and the next call is not led astray."""
    n, t, heads, dim = 40, 60, 4, 64
    h = Held(3, 1, 1, 16, dim, [3000] * 2, torch.float16)
    q = normal(7, t, heads, dim, dtype=torch.float16)
    big = torch.full((t + 400, heads, dim), 7.0, dtype=torch.float16, device=DEV)
    pi.attn_chunk(h.cache, 0, normal(8, 400, heads, dim, dtype=torch.float16), big[:400], ints([0, 200, 400]))   # leaves its marks
    big.fill_(7.0)
    for cu in ([0, t] * (n // 2) + [0], [t, 0, t, 0, t], [0, t, 5, t, 7, t, 9, t]):
        pi.attn_chunk(h.cache, 0, q, big[200:200 + t], ints(cu), ints([i % 2 for i in range(len(cu) - 1)]))
    torch.cuda.synchronize()
    assert (big[:200] == 7).all() and (big[200 + t:] == 7).all()
    chunk_ref.check(run(h, q, [20, 40]), *chunk_ref.chunk(q, h.k, h.v, [20, 40]))


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 40, 90, 41])
def test_chunks_longer_than_their_slots(window):
    """Rows before a slot's first token are zero, the others see what there is, whatever the window."""
    h = Held(3, 1, 1, 16, 64, [90, 40], torch.bfloat16)
    for counts in ([120, 50], [91, 41]):
        q = normal(7, sum(counts), 2, 64, dtype=torch.bfloat16)
        out = run(h, q, counts, window=window)
        at = 0
        for i, c in enumerate(counts):
            miss = c - h.lens[i]
            assert (out[at:at + miss] == 0).all()
            sl = slice(at + miss, at + c)
            chunk_ref.check(out[sl], *chunk_ref.chunk(q[sl], h.k[i:i + 1], h.v[i:i + 1], [h.lens[i]], window=window))
            at += c
    assert h.cache.errors() == pi.PI_CACHE_ELENGTH


def test_tensors_that_want_a_gradient_are_refused():
    h = Held(3, 1, 1, 16, 64, [90], torch.bfloat16)
    q = normal(7, 3, 2, 64, dtype=torch.bfloat16)
    want, cu, rope = q.clone().requires_grad_(), ints([0, 3]), pi.Rope(64, device=DEV)
    k = q[:, :1].contiguous()
    for call in (lambda x: pi.attn_chunk(h.cache, 0, x, torch.empty_like(q), cu),
                 lambda x: pi.rope_heads(rope, ints([0, 1, 2]), x, torch.empty_like(q)),
                 lambda x: h.cache.append_rope(0, rope, x, torch.empty_like(q), k, k, cu, ints([0]))):
        with pytest.raises(pi.PiError, match="gradient"):
            call(want)
        with torch.no_grad():
            call(want)
    torch.cuda.synchronize()


def test_what_cannot_be():
    """Slots and lengths that cannot be, pages that cannot be: zeros, or those keys are not seen, and the error word."""
    lens, dim = [100, 50, 300], 64
    q = normal(7, 12, 2, dim, dtype=torch.bfloat16)

    def broken(change, seqs, counts=(4, 8)):
        h = Held(3, 1, 1, 16, dim, lens, torch.bfloat16)
        change(h.cache)
        return run(h, q, list(counts), seqs), h.cache.errors(), h
    out, err, h = broken(lambda c: None, [3, 1])
    assert err == pi.PI_CACHE_ESLOT and (out[:4] == 0).all()
    chunk_ref.check(out[4:], *chunk_ref.chunk(q[4:], h.k[1:2], h.v[1:2], [8]))
    assert broken(lambda c: None, [-1, 1])[1] == pi.PI_CACHE_ESLOT
    for n in (-1, -(1 << 31), 1 << 30, (1 << 31) - 1):
        out, err, _ = broken(lambda c: c.lens.fill_(n), [0, 1])
        assert err == pi.PI_CACHE_ELENGTH and (out == 0).all()
    # fewer tokens than the chunk: the first rows see nothing
    out, err, h = broken(lambda c: c.lens.copy_(ints([100, 5, 300])), [0, 1])
    assert err == pi.PI_CACHE_ELENGTH and (out[4:7] == 0).all()
    chunk_ref.check(out[7:], *chunk_ref.chunk(q[7:], [h.k[1][:5]], [h.v[1][:5]], [5]))
    for bad in (-1, 1 << 20, 1 << 30, -(1 << 31)):
        def change(c):
            c.table[2, 4] = bad
        out, err, h = broken(change, [0, 2])
        keep = torch.tensor([j for j in range(300) if not 64 <= j < 80])
        assert err == pi.PI_CACHE_EPAGE
        chunk_ref.check(out[4:], *chunk_ref.chunk(q[4:], [h.k[2][keep]], [h.v[2][keep]], [8]))
    out, err, _ = broken(lambda c: c.table.fill_(-1), [0, 2])
    assert err == pi.PI_CACHE_EPAGE and (out == 0).all()


@pytest.mark.parametrize("order", ["heads_first", "padded", "in_place"])
def test_strides(order):
    t, heads, dim, lens, counts = 31, 4, 64, [200, 40], [30, 1]
    h = Held(3, 1, 2, 16, dim, lens, torch.float16)

    def make(seed):
        if order == "heads_first":
            return normal(seed, heads, t, dim, dtype=torch.float16).transpose(0, 1)
        return normal(seed, t, heads, dim + 24, dtype=torch.float16)[:, :, 8:8 + dim]
    q = make(1)
    out = q if order == "in_place" else make(2)
    ref, tol = chunk_ref.chunk(q, h.k, h.v, counts)
    pi.attn_chunk(h.cache, 0, q, out, ints(offsets(counts)))
    chunk_ref.check(out, ref, tol)
    if order == "padded":
        base, was = out.as_strided((t, heads, dim + 24), out.stride(), 0), normal(2, t, heads, dim + 24, dtype=torch.float16)
        assert torch.equal(base[:, :, :8], was[:, :, :8]) and torch.equal(base[:, :, 8 + dim:], was[:, :, 8 + dim:])


def test_pages_past_32_bits():
    """A pool of more than 2^32 elements whose last pages are used."""
    heads, g, dim, page, pages = 8, 8, 128, 64, 66000
    cache = pi.Cache(torch.empty(1, pages, g, page, dim, dtype=torch.float16, device=DEV),
                     torch.empty(1, pages, g, page, dim, dtype=torch.float16, device=DEV),
                     torch.zeros(pi.Cache.meta_words(1, 4, pages), dtype=torch.int32, device=DEV), 1, 4)
    k, v = (normal(i, 200, g, dim, dtype=torch.float16) for i in (1, 2))
    q, raw = normal(3, 50, heads, dim, dtype=torch.float16), normal(4, 200, heads, dim, dtype=torch.float16)
    cache.table[0] = ints([pages - 1, 0, pages - 2, pages - 3])
    cache.lens[0] = 200
    out, turned, rope = torch.empty_like(q), torch.empty_like(raw), pi.Rope(dim, device=DEV)
    cache.append_rope(0, rope, raw, turned, k, v, ints([0, 200]), ints([0]))
    pi.attn_chunk(cache, 0, q, out, ints([0, 50]))
    kk = torch.empty_like(k)
    pi.rope_heads(rope, ints(range(200)), k, kk)
    chunk_ref.check(out, *chunk_ref.chunk(q, [kk.cpu()], [v.cpu()], [50]))


def test_a_million_tokens():
    """A long sequence whose table names the same pages again and again: each key counts as often as it comes."""
    heads, dim, page, period, times = 2, 64, 16, 8, 8192
    cache = pi.Cache.create(1, period, 1, page, dim, 1, period * times, dtype=torch.bfloat16, device=DEV)
    cache.k_pool.copy_(normal(1, *cache.k_pool.shape, dtype=torch.bfloat16))
    cache.v_pool.copy_(normal(2, *cache.v_pool.shape, dtype=torch.bfloat16))
    cache.table[0] = ints(list(range(period)) * times)
    n = period * page * times                          # 2^20
    cache.lens[0] = n
    q, out = normal(3, 1, heads, dim, dtype=torch.bfloat16), torch.empty(1, heads, dim, dtype=torch.bfloat16, device=DEV)
    pi.attn_chunk(cache, 0, q, out, ints([0, 1]))
    k, v = cache.k_pool[0, :, 0].reshape(1, -1, 1, dim).cpu()[0], cache.v_pool[0, :, 0].reshape(1, -1, 1, dim).cpu()[0]
    ref, tol = chunk_ref.chunk(q, [k], [v], [1])
    # a share of n / 64 keys or fewer is summed 64 keys a tile: at most 32 float32 additions each to a weight's and a value's
    # sum, so 2 (32 n / 64 / 64) 2^-24 of A, which is at most the largest value, beside the bound for one period
    chunk_ref.check(out, ref, tol + 2 * (32 * n / 64 / 64) * 2.0 ** -24 * v.double().abs().max())
    pi.attn_chunk(cache, 0, q, out, ints([0, 1]), window=period * page + 1)    # the last period and its own key once more
    kk, vv = torch.cat([k[-1:], k]), torch.cat([v[-1:], v])
    chunk_ref.check(out, *chunk_ref.chunk(q, [kk], [vv], [1]))


def test_repeats_streams_and_graphs():
    """The same bits every time, on any stream, and in two replayed graphs that share the workspace."""
    lens, counts = [2000, 300, 77], [5, 64, 1]
    h = Held(3, 1, 2, 16, 128, lens, torch.bfloat16)
    q = normal(7, sum(counts), 8, 128, dtype=torch.bfloat16)
    cu, few = ints(offsets(counts)), ints([0, 1])
    want, one = run(h, q, counts), torch.zeros_like(q[:1])
    pi.attn_chunk(h.cache, 0, q[:1], one, few, cap=30.0, window=500)
    torch.cuda.synchronize()
    out, side = torch.zeros_like(q), torch.cuda.Stream()
    for stream in (None, side):
        out.zero_()
        torch.cuda.synchronize()
        pi.attn_chunk(h.cache, 0, q, out, cu, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    a, b, got = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.zeros_like(one)
    with torch.cuda.graph(a):
        pi.attn_chunk(h.cache, 0, q, out, cu)
    with torch.cuda.graph(b):
        pi.attn_chunk(h.cache, 0, q[:1], got, few, cap=30.0, window=500)
    for i in range(4):
        out.zero_(), got.zero_()
        for g in ((a, b), (b, a))[i % 2]:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(got, one)
        pi.attn_chunk(h.cache, 0, q, out, cu)
        _ = torch.randn(1000, device=DEV).sum().item()


def test_workspace_grows_outside_captures_only():
    h = Held(3, 1, 2, 16, 64, [40], torch.float16)
    q = normal(7, 40, 4, 64, dtype=torch.float16)
    out, cu = torch.zeros_like(q), ints([0, 40])
    with pytest.raises(pi.PiError, match="capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            pi.attn_chunk(h.cache, 0, q, out, cu)
    torch.cuda.synchronize()
    h.cache.reserve_chunk(40, 4, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.attn_chunk(h.cache, 0, q, out, cu)
    graph.replay()
    torch.cuda.synchronize()
    ref, tol = chunk_ref.chunk(q, h.k, h.v, [40])
    chunk_ref.check(out, ref, tol)
    mine = torch.empty(h.cache.chunk_workspace(40, 4, 1).numel(), dtype=torch.uint8, device=DEV)
    out.zero_()
    pi.attn_chunk(h.cache, 0, q, out, cu, ws=mine)
    chunk_ref.check(out, ref, tol)


def test_no_tokens():
    h = Held(3, 1, 1, 16, 64, [10], torch.float16)
    e = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    pi.attn_chunk(h.cache, 0, e, e.clone(), ints([0, 0]))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pieces", [[200], [1] * 20 + [180], [64, 64, 72], [7, 150, 43]])
def test_a_prompt_in_pieces(pieces, dtype):
    """Room, norm, rotation, append and attention piece by piece, two sequences side by side, the second one step behind:
    the same as over the whole text."""
    heads, g, dim, layers = 8, 2, 64, 2
    total = sum(pieces)
    cache = pi.Cache.create(layers, 40, g, 16, dim, 2, 16, dtype=TYPES[dtype], device=DEV)
    rope, wq, wk = pi.Rope(dim, layout="pairs", device=DEV), 1 + normal(1, dim, dtype=torch.float32, scale=0.2), \
        1 + normal(2, dim, dtype=torch.float32, scale=0.2)
    texts = [normal(3 + i, total, heads + 2 * g, dim, dtype=TYPES[dtype]) for i in range(2)]
    outs = [torch.zeros(total, heads, dim, dtype=TYPES[dtype], device=DEV) for _ in range(2)]
    done = [0, 0]
    for step in range(len(pieces) + 1):
        counts = [pieces[step] if step < len(pieces) else 0, pieces[step - 1] if step else 0]
        qkv = torch.cat([texts[i][done[i]:done[i] + counts[i]] for i in range(2)])
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + g], qkv[:, heads + g:]
        cu, seqs = ints(offsets(counts)), ints([0, 1])
        cache.extend(seqs, ints(counts))
        turned, out = torch.empty_like(q), torch.empty_like(q)
        for layer in range(layers):
            cache.append_rope(layer, rope, q, turned, k, v, cu, seqs, q_norm=wq, k_norm=wk)
            pi.attn_chunk(cache, layer, turned, out, cu, seqs)
        for i, rows in enumerate(out.split(counts)):
            outs[i][done[i]:done[i] + counts[i]] = rows
            done[i] += counts[i]
    assert cache.errors() == 0 and cache.lens.tolist() == [total, total]
    for text, out in zip(texts, outs):
        q, k = torch.empty_like(text[:, :heads]), torch.empty_like(text[:, heads:heads + g])
        pi.rope_heads(rope, ints(range(total)), text[:, :heads], q, text[:, heads:heads + g], k, q_norm=wq, k_norm=wk)
        chunk_ref.check(out, *chunk_ref.chunk(q, [k.cpu()], [text[:, heads + g:].cpu()], [total]))


def test_single_tokens_beside_decode():
    """A chunk of one token a slot does what attn_decode does, forked slots with shared pages among them."""
    heads, g, dim = 16, 4, 128
    cache = pi.Cache.create(1, 200, g, 16, dim, 4, 60, dtype=torch.float16, device=DEV)
    k, v = (normal(i, 701, g, dim, dtype=torch.float16) for i in (1, 2))
    cache.extend(ints([0]), ints([701]))
    cache.append(0, k, v, ints([0, 701]), ints([0]))
    cache.fork(ints([0, 0]), ints([1, 2]))
    q, out, ref = normal(3, 4, heads, dim, dtype=torch.float16), torch.zeros(4, heads, dim, dtype=torch.float16, device=DEV), None
    ref = torch.zeros_like(out)
    pi.attn_chunk(cache, 0, q[:3], out[:3], ints([0, 1, 2, 3]))
    pi.attn_decode(cache, 0, q, ref)
    want, tol = chunk_ref.chunk(q[:3], [k.cpu()] * 3, [v.cpu()] * 3, [1, 1, 1])
    chunk_ref.check(out[:3], want, tol)
    chunk_ref.check(ref[:3], want, tol)
    assert cache.errors() == 0
