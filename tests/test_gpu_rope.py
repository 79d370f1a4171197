"""Norms and rotary positions of heads, on their own and on the way into the paged cache, against 64 bits (chunk_ref.py)."""
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


def weights(seed, dim):
    return 1 + normal(seed, dim, dtype=torch.float32, scale=0.3)


def offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


SHAPES = [
    # heads, kv_heads, dim, rotary, tokens
    (4, 2, 128, 128, 1),
    (4, 4, 128, 128, 9),
    (32, 8, 128, 64, 70),
    (71, 1, 64, 64, 13),
    (8, 2, 64, 30, 33),
    (3, 1, 80, 80, 17),
    (5, 5, 80, 38, 5),
    (2, 1, 96, 32, 40),
    (16, 8, 256, 256, 11),
    (2, 2, 256, 254, 3),
    (4, 1, 256, 64, 6),
    (3, 3, 8, 8, 21),
    (2, 1, 8, 2, 4),
    (2, 2, 24, 16, 19),
    (1, 1, 136, 120, 7),
    (6, 2, 40, 20, 130),
    (64, 8, 128, 128, 1300),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,rotary,tokens", SHAPES)
def test_heads(heads, kv_heads, dim, rotary, tokens, normed, layout, dtype):
    qkv = normal(dim + tokens, tokens, heads + 2 * kv_heads, dim, dtype=TYPES[dtype])
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv_heads]
    keep = qkv.clone()
    r = random.Random(tokens)
    pos = [r.choice([0, 1, i, r.randrange(1 << 20), -5]) for i in range(tokens)]
    rope = pi.Rope(rotary, layout=layout, device=DEV)
    wq, wk = (weights(1, dim), weights(2, dim)) if normed else (None, None)
    q_out, k_out = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    pi.rope_heads(rope, ints(pos), q, q_out, k, k_out, q_norm=wq, k_norm=wk)
    freqs, _ = chunk_ref.frequencies(rotary, 10000.0, None)
    chunk_ref.check(q_out, *chunk_ref.turn(q, pos, freqs, layout, norm=wq), "q")
    chunk_ref.check(k_out, *chunk_ref.turn(k, pos, freqs, layout, norm=wk), "k")
    assert torch.equal(qkv, keep)
    # in place, with the strides of a projection's output: the same bits, and the values beside them stay
    pi.rope_heads(rope, ints(pos), q, q, k, k, q_norm=wq, k_norm=wk)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(qkv[:, heads + kv_heads:], keep[:, heads + kv_heads:])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_parts_of_a_call(dtype):
    """Queries alone, a norm of one of both, norms without a rotation, no tokens."""
    t, h, g, d = 20, 6, 2, 128
    q, k = normal(1, t, h, d, dtype=TYPES[dtype]), normal(2, t, g, d, dtype=TYPES[dtype])
    pos, rope, w = list(range(t)), pi.Rope(d, device=DEV), weights(3, d)
    freqs, _ = chunk_ref.frequencies(d, 10000.0, None)
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    pi.rope_heads(rope, ints(pos), q, q_out)
    chunk_ref.check(q_out, *chunk_ref.turn(q, pos, freqs, "half"))
    pi.rope_heads(rope, ints(pos), q, q_out, k, k_out, k_norm=w, eps=0.5)
    chunk_ref.check(q_out, *chunk_ref.turn(q, pos, freqs, "half"))
    chunk_ref.check(k_out, *chunk_ref.turn(k, pos, freqs, "half", norm=w, eps=0.5))
    pi.rope_heads(None, None, q, q_out, k, k_out, q_norm=w)
    chunk_ref.check(q_out, *chunk_ref.turn(q, pos, [], "half", norm=w))
    assert torch.equal(k_out, k)                       # neither normed nor turned: as it was
    e = torch.empty(0, h, d, dtype=TYPES[dtype], device=DEV)
    pi.rope_heads(rope, ints([]), e, e.clone())
    torch.cuda.synchronize()


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("rotary", [64, 30])
def test_what_does_not_turn_keeps_its_bits(rotary, layout):
    """Dimensions behind the rotary ones, infinities and NaN among them, without a norm."""
    t, h, d = 7, 3, 128
    q = normal(5, t, h, d, dtype=torch.bfloat16)
    q[:, :, rotary:rotary + 3] = torch.tensor([float("inf"), -float("inf"), float("nan")], device=DEV)
    out = torch.zeros_like(q)
    pi.rope_heads(pi.Rope(rotary, layout=layout, magnitude=3.0, device=DEV), ints(range(t)), q, out)
    assert torch.equal(out[..., rotary:].view(torch.int16), q[..., rotary:].view(torch.int16))
    freqs, _ = chunk_ref.frequencies(rotary, 10000.0, None)
    ref, tol = chunk_ref.turn(q[..., :rotary].contiguous(), range(t), freqs, layout, magnitude=3.0)
    chunk_ref.check(out[..., :rotary], ref, tol)


def test_values_that_are_not_finite_stay_in_their_row():
    t, h, d = 5, 4, 64
    q = normal(5, t, h, d, dtype=torch.float16)
    ref, rope, w = torch.zeros_like(q), pi.Rope(d, device=DEV), weights(1, d)
    pi.rope_heads(rope, ints(range(t)), q, ref, q_norm=w)
    q[2, 1, 7], q[3, 0, 60] = float("nan"), float("inf")
    out = torch.zeros_like(q)
    pi.rope_heads(rope, ints(range(t)), q, out, q_norm=w)
    hit = torch.zeros(t, h, dtype=torch.bool)
    hit[2, 1] = hit[3, 0] = True
    assert torch.isnan(out[2, 1]).all() and not torch.isfinite(out[3, 0, 28])
    assert torch.equal(out[~hit.to(DEV)], ref[~hit.to(DEV)])
    zero = torch.zeros(2, 1, d, dtype=torch.float16, device=DEV)
    pi.rope_heads(rope, ints([0, 9]), zero, zero, q_norm=w)
    assert (zero == 0).all()


@pytest.mark.parametrize("pos", [0, 1, -1, 12345, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)])
def test_far_positions(pos):
    """Angles keep their precision at any position, for frequencies that are given."""
    d, freqs = 64, [1.0, 0.5, 3.25, -0.75, 1e-4, 2.0 ** -40, 0.0, 6.5] * 4
    q = normal(3, 1, 2, d, dtype=torch.float16)
    out = torch.zeros_like(q)
    pi.rope_heads(pi.Rope(d, freqs=freqs, device=DEV), ints([pos]), q, out)
    chunk_ref.check(out, *chunk_ref.turn(q, [pos], freqs, "half"))


@pytest.mark.parametrize("order", ["heads_first", "padded"])
@pytest.mark.parametrize("rotary", [64, 30])
def test_strides(order, rotary):
    t, h, d = 31, 4, 64

    def make(seed):
        if order == "heads_first":
            return normal(seed, h, t, d, dtype=torch.bfloat16).transpose(0, 1)
        return normal(seed, t, h, d + 24, dtype=torch.bfloat16)[:, :, 8:8 + d]
    q, out, pos = make(1), make(2), list(range(100, 100 + t))
    pi.rope_heads(pi.Rope(rotary, device=DEV), ints(pos), q, out)
    freqs, _ = chunk_ref.frequencies(rotary, 10000.0, None)
    chunk_ref.check(out, *chunk_ref.turn(q, pos, freqs, "half"))
    if order == "padded":                              # what lies between the rows stays as it was
        base, was = out.as_strided((t, h, d + 24), out.stride(), 0), normal(2, t, h, d + 24, dtype=torch.bfloat16)
        assert torch.equal(base[:, :, :8], was[:, :, :8]) and torch.equal(base[:, :, 8 + d:], was[:, :, 8 + d:])


def test_streams_and_graphs():
    t, h, g, d = 40, 8, 2, 128
    q, k, pos, rope = normal(1, t, h, d, dtype=torch.float16), normal(2, t, g, d, dtype=torch.float16), ints(range(t)), \
        pi.Rope(d, device=DEV)
    want_q, want_k = torch.zeros_like(q), torch.zeros_like(k)
    pi.rope_heads(rope, pos, q, want_q, k, want_k)
    torch.cuda.synchronize()
    out_q, out_k, side = torch.zeros_like(q), torch.zeros_like(k), torch.cuda.Stream()
    pi.rope_heads(rope, pos, q, out_q, k, out_k, stream=side)
    side.synchronize()
    assert torch.equal(out_q, want_q) and torch.equal(out_k, want_k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.rope_heads(rope, pos, q, out_q, k, out_k)
    for _ in range(3):
        out_q.zero_(), out_k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_q, want_q) and torch.equal(out_k, want_k)
        pi.rope_heads(rope, pos, q, out_q)
    pos += 1                                           # a replay takes the positions there are then
    pi.rope_heads(rope, pos, q, want_q, k, want_k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_q, want_q) and torch.equal(out_k, want_k)


# ------------------------------------------------------------ into the cache
def a_cache(seed, layers, kv_heads, page, dim, lens, dtype, spare=3):
    """A cache whose slots hold lens tokens in pages that lie anywhere; the pool holds 7 everywhere."""
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    cache = pi.Cache.create(layers, pages, kv_heads, page, dim, len(lens), max(max(held), 1) + 1, dtype=dtype, device=DEV)
    cache.k_pool.fill_(7), cache.v_pool.fill_(7)
    ids, at = random.Random(seed).sample(range(pages), sum(held)), 0
    for i, n in enumerate(held):
        cache.table[i, :n] = ints(ids[at:at + n])
        at += n
    cache.lens.copy_(ints(lens))
    return cache


def held(cache, layer, slot):
    """Keys and values of a slot [tokens, kv_heads, dim] in a layer."""
    n, page = int(cache.lens[slot]), cache.page
    ids = cache.table[slot, :-(-n // page)].long()
    return tuple(pool[layer][ids].transpose(1, 2).reshape(-1, cache.kv_heads, cache.dim)[:n].cpu()
                 for pool in (cache.k_pool, cache.v_pool))


APPENDS = [
    # heads, kv_heads, dim, page, lens, counts, rotary, layout
    (32, 32, 128, 16, [1501], [1], 128, "half"),
    (64, 8, 128, 16, [5, 100, 16, 33], [1, 1, 1, 1], 128, "half"),
    (8, 2, 64, 32, [70, 40, 31], [70, 0, 20], 32, "pairs"),
    (4, 4, 80, 48, [200, 1], [150, 1], 38, "half"),
    (71, 1, 64, 16, [20, 30], [20, 7], 64, "pairs"),
    (2, 1, 256, 16, [300], [299], 256, "half"),
    (3, 1, 24, 16, [40, 40], [3, 40], 22, "half"),
    (2, 1, 64, 16, [3] * 70 + [9, 17], [1, 0] * 35 + [9, 2], 64, "half"),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens,counts,rotary,layout", APPENDS)
def test_append(heads, kv_heads, dim, page, lens, counts, rotary, layout, normed, dtype):
    t = sum(counts)
    cache = a_cache(t, 2, kv_heads, page, dim, lens, TYPES[dtype])
    qkv = normal(t + 1, t, heads + 2 * kv_heads, dim, dtype=TYPES[dtype])
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    wq, wk = (weights(1, dim), weights(2, dim)) if normed else (None, None)
    rope = pi.Rope(rotary, 5000.0, layout, device=DEV)
    q_out, order = torch.full_like(q, float("nan")), list(range(len(lens)))
    random.Random(t).shuffle(order)                    # the slots in any order
    lens_of, cu = [lens[i] for i in range(len(lens))], ints(offsets([counts[i] for i in order]))
    cache.append_rope(1, rope, q, q_out, k, v, cu, ints(order), q_norm=wq, k_norm=wk)
    pos = [p for i in order for p in range(lens_of[i] - counts[i], lens_of[i])]
    freqs, _ = chunk_ref.frequencies(rotary, 5000.0, None)
    chunk_ref.check(q_out, *chunk_ref.turn(q, pos, freqs, layout, norm=wq), "q")
    # the same bits as without the cache
    alone_q, alone_k = torch.zeros_like(q), torch.zeros_like(k)
    pi.rope_heads(rope, ints(pos), q, alone_q, k, alone_k, q_norm=wq, k_norm=wk)
    assert torch.equal(q_out, alone_q)
    at = 0
    for i in order:
        kk, vv = held(cache, 1, i)
        first = lens[i] - counts[i]
        assert torch.equal(kk[first:], alone_k[at:at + counts[i]].cpu()) and torch.equal(vv[first:], v[at:at + counts[i]].cpu())
        assert (kk[:first] == 7).all() and (vv[:first] == 7).all()
        at += counts[i]
    assert (cache.k_pool[0] == 7).all() and (cache.v_pool[0] == 7).all()
    for pool in (cache.k_pool, cache.v_pool):          # nothing else was written
        assert int((pool[1] != 7).any(-1).sum()) <= t * kv_heads
    assert cache.errors() == 0


def test_append_of_keys_alone_and_of_norms_alone():
    lens, counts, g, d = [20, 5], [4, 5], 2, 64
    cache = a_cache(1, 1, g, 16, d, lens, torch.float16)
    k, v, w = normal(1, 9, g, d, dtype=torch.float16), normal(2, 9, g, d, dtype=torch.float16), weights(1, d)
    cu, seqs = ints(offsets(counts)), ints([0, 1])
    cache.append_rope(0, None, None, None, k, v, cu, seqs, k_norm=w)
    got = torch.cat([held(cache, 0, i)[0][lens[i] - counts[i]:] for i in range(2)])
    chunk_ref.check(got, *chunk_ref.turn(k, range(9), [], "half", norm=w))
    cache.append_rope(0, None, None, None, k, v, cu, seqs)       # neither: append
    other = a_cache(1, 1, g, 16, d, lens, torch.float16)
    other.append(0, k, v, cu, seqs)
    assert torch.equal(cache.k_pool, other.k_pool) and torch.equal(cache.v_pool, other.v_pool)


def test_append_what_cannot_be():
    """Slots, lengths and pages that cannot be set the error word; rows outside the offsets are not touched."""
    lens, g, h, d = [20, 5, 40], 1, 2, 64
    q, k, v = normal(1, 12, h, d, dtype=torch.float16), normal(2, 12, g, d, dtype=torch.float16), \
        normal(3, 12, g, d, dtype=torch.float16)
    rope = pi.Rope(d, device=DEV)

    def run(change, cu, seqs):
        cache = a_cache(1, 1, g, 16, d, lens, torch.float16)
        change(cache)
        out = torch.full_like(q, 7.0)
        cache.append_rope(0, rope, q, out, k, v, ints(cu), ints(seqs))
        return cache.errors(), (out != 7).flatten(1).any(1).tolist(), int((cache.k_pool != 7).any(-1).sum())

    none = [False] * 12
    assert run(lambda c: None, [2, 4, 9], [0, 2]) == (0, none[:2] + [True] * 7 + none[:3], 7)
    assert run(lambda c: None, [0, 3], [3]) == (pi.PI_CACHE_ESLOT, none, 0)
    assert run(lambda c: None, [0, 3], [-1]) == (pi.PI_CACHE_ESLOT, none, 0)
    assert run(lambda c: None, [0, 6], [1]) == (pi.PI_CACHE_ELENGTH, none[:1] + [True] * 5 + none[:6], 5)
    assert run(lambda c: c.lens.fill_(-1), [0, 6], [1]) == (pi.PI_CACHE_ELENGTH, none, 0)
    assert run(lambda c: c.lens.fill_(1 << 30), [0, 6], [1]) == (pi.PI_CACHE_ELENGTH, none, 0)
    # a broken page: its keys go nowhere, the queries are turned all the same
    assert run(lambda c: c.table[2].fill_(-7), [0, 6], [2]) == (pi.PI_CACHE_EPAGE, [True] * 6 + none[:6], 0)
    assert run(lambda c: c.table[2].fill_(1 << 20), [0, 6], [2]) == (pi.PI_CACHE_EPAGE, [True] * 6 + none[:6], 0)


def test_append_in_a_graph():
    lens, g, h, d = [1, 1], 2, 4, 128
    cache = pi.Cache.create(1, 8, g, 16, d, 2, 3, device=DEV)
    q, k, v, out = (normal(i, 2, n, d, dtype=torch.float16) for i, n in ((1, h), (2, g), (3, g), (4, h)))
    rope, cu, seqs, one = pi.Rope(d, device=DEV), ints([0, 1, 2]), ints([0, 1]), ints([1, 1])
    cache.extend(seqs, one)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.append_rope(0, rope, q, out, k, v, cu, seqs)
        cache.extend(seqs, one)
    freqs, _ = chunk_ref.frequencies(d, 10000.0, None)
    for step in range(20):
        graph.replay()
        torch.cuda.synchronize()
        chunk_ref.check(out, *chunk_ref.turn(q, [step, step], freqs, "half"))
        assert torch.equal(held(cache, 0, 1)[1][step], v[1].cpu())
        _ = torch.randn(1000, device=DEV).sum().item()
    assert cache.errors() == 0 and lens == [1, 1]
