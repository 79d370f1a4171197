"""Attention over packed prompts and of single new tokens over a paged cache, against 64 bits (tests/attn_ref.py)."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import attn_ref  # noqa: E402

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def normal(seed, *shape, dtype, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


def offsets(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


# ------------------------------------------------------------------ prompts
PROMPTS = [
    # heads, kv_heads, dim, lengths
    (4, 4, 128, [1]),
    (4, 2, 128, [2, 1, 3]),
    (2, 1, 128, [61]),
    (3, 3, 128, [63, 64, 65]),
    (8, 2, 64, [31, 32, 33, 127, 128, 129]),
    (4, 1, 128, [255, 256, 257]),
    (2, 2, 64, [511, 1, 513]),
    (2, 1, 96, [70, 130, 5]),
    (2, 1, 80, [300]),
    (2, 2, 8, [40, 200]),
    (3, 1, 24, [129, 77]),
    (2, 1, 256, [1, 65, 200]),
    (1, 1, 192, [190]),
    (2, 1, 136, [333]),
    (6, 2, 64, [1] * 70 + [3, 0, 2, 0, 0, 129]),
    (1, 1, 128, [1037]),
    (1, 1, 64, [0, 0, 1500]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,lengths", PROMPTS)
def test_prompt(heads, kv_heads, dim, lengths, dtype):
    t = sum(lengths)
    qkv = normal(7 * t + dim, t, heads + 2 * kv_heads, dim, dtype=TYPES[dtype])
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    out = torch.full((t, heads, dim), float("nan"), dtype=TYPES[dtype], device=DEV)
    pi.attn_prompt(q, k, v, out, ints(offsets(lengths)))
    attn_ref.check(out, *attn_ref.prompt(q, k, v, lengths))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("order", ["heads_first", "padded", "one_head"])
def test_prompt_strides(order, dtype):
    t, h, g, d, lengths = 201, 4, 2, 64, [150, 51]
    def make(seed, n):
        if order == "heads_first":
            return normal(seed, n, t, d, dtype=TYPES[dtype]).transpose(0, 1)
        if order == "padded":
            return normal(seed, t, n, d + 24, dtype=TYPES[dtype])[:, :, 8:8 + d]
        return normal(seed, t, n, d, dtype=TYPES[dtype])
    if order == "one_head":
        h = g = 1
    q, k, v, out = make(1, h), make(2, g), make(3, g), make(4, h)
    keep = out.clone()
    pi.attn_prompt(q, k, v, out, ints(offsets(lengths)))
    attn_ref.check(out, *attn_ref.prompt(q, k, v, lengths))
    if order == "padded":                              # what lies between the rows stays as it was
        base, was = out.as_strided((t, h, d + 24), out.stride(), 0), normal(4, t, h, d + 24, dtype=TYPES[dtype])
        assert torch.equal(base[:, :, :8], was[:, :, :8]) and torch.equal(base[:, :, 8 + d:], was[:, :, 8 + d:])
    assert keep.shape == out.shape


def test_prompt_rows_of_no_sequence_are_not_written():
    t, h, d = 90, 2, 64
    q, k, v = (normal(i, t, h, d, dtype=torch.float16) for i in range(3))
    out = torch.full((t, h, d), 7.0, dtype=torch.float16, device=DEV)
    pi.attn_prompt(q, k, v, out, ints([10, 40, 40, 75]))
    ref, tol = attn_ref.prompt(q[10:75], k[10:75], v[10:75], [30, 0, 35])
    attn_ref.check(out[10:75], ref, tol)
    assert (out[:10] == 7).all() and (out[75:] == 7).all()


def test_prompt_offsets_that_cannot_be_stay_inside():
    """Offsets beyond the tensors, negative ones and ones that go down are cut to the rows there are."""
    t, h, d = 70, 2, 64
    q, k, v = (normal(i, t, h, d, dtype=torch.bfloat16) for i in range(3))
    out = torch.zeros(t, h, d, dtype=torch.bfloat16, device=DEV)
    pi.attn_prompt(q, k, v, out, ints([-5, 30, 1 << 30]))
    attn_ref.check(out, *attn_ref.prompt(q, k, v, [30, 40]))
    out.zero_()
    pi.attn_prompt(q, k, v, out, ints([0, 50, 20]))    # the second holds nothing
    attn_ref.check(out[:50], *attn_ref.prompt(q[:50], k[:50], v[:50], [50]))
    assert (out[50:] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 80])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
def test_prompt_later_keys_leave_no_trace(dtype, dim, poison):
    """A key and a value that are not finite reach their own row and later ones, no earlier row."""
    t, h, at = 200, 2, 100
    q, k, v = (normal(i, t, h, dim, dtype=TYPES[dtype]) for i in range(3))
    ref, tol = attn_ref.prompt(q[:at], k[:at], v[:at], [at])
    for tensors in ((k,), (v,), (k, v)):
        kk, vv = k.clone(), v.clone()
        for x in tensors:
            (kk if x is k else vv)[at] = poison
        out = torch.zeros_like(q)
        pi.attn_prompt(q, kk, vv, out, ints([0, t]))
        attn_ref.check(out[:at], ref, tol)
        if tensors[0] is v:
            assert not torch.isfinite(out[at:]).any()
        if poison != poison:
            assert torch.isnan(out[at:]).all()
    # neighbours in the packing: another sequence's values leave no trace either
    vv = v.clone()
    vv[at:] = poison
    out = torch.zeros_like(q)
    pi.attn_prompt(q, k, vv, out, ints([0, at, t]))
    attn_ref.check(out[:at], ref, tol)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompt_keys_that_score_minus_infinity(dtype):
    """Keys with a score of -inf weigh nothing; a row that sees only such keys is zero."""
    t, h, d = 150, 1, 64
    q, k, v = (normal(i, t, h, d, dtype=TYPES[dtype]) for i in range(3))
    q = q.abs() + 0.125
    k[:40] = -float("inf")
    k[90:120, :, 3] = -float("inf")
    out = torch.full_like(q, float("nan"))
    pi.attn_prompt(q, k, v, out, ints([0, t]))
    assert (out[:40] == 0).all()
    live = torch.tensor([i for i in range(40, t) if not 90 <= i < 120])
    q64, k64, v64 = (x[:, 0].cpu().double() for x in (q, k, v))
    last = torch.tensor([int((live <= i).sum()) for i in range(40, t)])
    ref, tol = attn_ref.rows(q64[40:], k64[live], v64[live], last, d ** -0.5, TYPES[dtype])
    attn_ref.check(out[40:, 0], ref, tol)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mode", ["rising", "falling", "spiky", "tiny", "equal"])
def test_prompt_ranges_of_scores(dtype, mode):
    """The running maximum: growing in every tile, never, by leaps; scores far apart; all weights equal."""
    t, h, d = 700, 2, 64
    q, k, v = (normal(i + 5, t, h, d, dtype=TYPES[dtype]) for i in range(3))
    ramp = torch.linspace(0, 4, t, device=DEV).view(t, 1, 1)
    if mode == "rising":
        q, k = q.abs(), (k.abs() * ramp).to(TYPES[dtype])
    elif mode == "falling":
        q, k = q.abs(), (k.abs() * (4 - ramp)).to(TYPES[dtype])
    elif mode == "spiky":
        k[::97] *= 12
    elif mode == "tiny":
        q, k = q * 1e-3, k * 1e-3
    else:
        k[:] = k[0]
    out = torch.zeros_like(q)
    pi.attn_prompt(q, k, v, out, ints([0, t]))
    attn_ref.check(out, *attn_ref.prompt(q, k, v, [t]))


def test_prompt_scale():
    t, h, d = 100, 2, 64
    q, k, v = (normal(i, t, h, d, dtype=torch.float16) for i in range(3))
    out = torch.zeros_like(q)
    pi.attn_prompt(q, k, v, out, ints([0, t]), scale=0.5)
    attn_ref.check(out, *attn_ref.prompt(q, k, v, [t], scale=0.5))


def test_prompt_no_tokens():
    e = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    pi.attn_prompt(e, e, e, e.clone(), ints([0, 0]))
    torch.cuda.synchronize()


def test_prompt_repeats_and_other_streams():
    """The same bits every time, on any stream, and in a replayed graph between eager calls."""
    lengths = [77, 300, 1, 129]
    t, h, g, d = sum(lengths), 4, 2, 128
    q, k, v = (normal(i, t, n, d, dtype=torch.bfloat16) for i, n in ((0, h), (1, g), (2, g)))
    cu, want = ints(offsets(lengths)), torch.empty(t, h, d, dtype=torch.bfloat16, device=DEV)
    pi.attn_prompt(q, k, v, want, cu)
    torch.cuda.synchronize()
    out, side = torch.zeros_like(want), torch.cuda.Stream()
    with torch.cuda.stream(side):
        pi.attn_prompt(q, k, v, out, cu)
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    pi.attn_prompt(q, k, v, out, cu, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.attn_prompt(q, k, v, out, cu)
    for i in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        eager = torch.zeros_like(want)
        pi.attn_prompt(q, k, v, eager, cu)
        assert torch.equal(eager, want)


# ------------------------------------------------------------------ decoding
def make_cache(seed, dtype, kv_heads, dim, page, lens, shared=0, layers=2, spare=3, wide=2):
    """A cache whose slots hold lens tokens in scattered pages; the first `shared` pages of slots that hold them are the
    same.  Pages and the ends of last pages that nobody uses hold NaN."""
    rnd = random.Random(seed)
    held = [-(-n // page) for n in lens]
    own = [max(0, n - shared) if n >= shared else n for n in held]
    pages = shared + sum(own) + spare
    ids = rnd.sample(range(pages), pages)
    cache = pi.Cache.create(layers, pages, kv_heads, page, dim, len(lens), max(max(held) + wide, 1), TYPES[dtype], DEV)
    k = normal(seed, layers, pages, kv_heads, page, dim, dtype=TYPES[dtype]).cpu()
    v = normal(seed + 1, layers, pages, kv_heads, page, dim, dtype=TYPES[dtype]).cpu()
    table = torch.full((len(lens), cache.max_pages), -1, dtype=torch.int32)
    at, ref = shared, [0] * pages
    for i, n in enumerate(held):
        row = (ids[:shared] if n >= shared else []) + ids[at:at + own[i]]
        at += own[i]
        table[i, :n] = torch.tensor(row, dtype=torch.int32)
        for p in row:
            ref[p] += 1
    for i, n in enumerate(lens):
        if n % page:
            last = int(table[i, held[i] - 1])
            if ref[last] == 1:
                k[:, last, :, n % page:] = float("nan")
                v[:, last, :, n % page:] = float("nan")
    for p in range(pages):
        if ref[p] == 0:
            k[:, p], v[:, p] = float("nan"), float("inf")
    cache.k_pool.copy_(k)
    cache.v_pool.copy_(v)
    cache.table.copy_(table)
    cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    cache.ref.copy_(torch.tensor(ref, dtype=torch.int32))
    return cache


def held_by(cache, layer):
    """Per slot its keys and values [tokens, kv_heads, dim] on the CPU."""
    k, v, table, lens = cache.k_pool[layer].cpu(), cache.v_pool[layer].cpu(), cache.table.cpu(), cache.lens.cpu()
    ks, vs = [], []
    for i in range(cache.slots):
        n = int(lens[i])
        ids = table[i, :-(-n // cache.page)].long()
        ks.append(k[ids].transpose(1, 2).reshape(-1, cache.kv_heads, cache.dim)[:n])
        vs.append(v[ids].transpose(1, 2).reshape(-1, cache.kv_heads, cache.dim)[:n])
    return ks, vs


def check_decode(cache, q, layer=1, prefix=None, seqs=None, scale=None, errors=0):
    out = torch.full_like(q, float("nan"))
    pi.attn_decode(cache, layer, q, out, prefix=None if prefix is None else ints([prefix]),
                   seqs=None if seqs is None else ints(seqs), scale=scale or 0.0)
    assert cache.errors() == errors
    ks, vs = held_by(cache, layer)
    if seqs is not None:
        ks, vs = [ks[i] for i in seqs], [vs[i] for i in seqs]
    attn_ref.check(out, *attn_ref.decode(q, ks[:q.shape[0]], vs[:q.shape[0]], scale))
    return out


DECODES = [
    # heads, kv_heads, dim, page, lens
    (4, 4, 128, 16, [1]),
    (4, 2, 128, 16, [0, 1, 2]),
    (8, 8, 128, 16, [15, 16, 17, 31, 32, 33]),
    (8, 1, 64, 64, [63, 64, 65, 200]),
    (32, 2, 64, 16, [511, 1, 257]),
    (34, 2, 64, 32, [129, 600]),
    (40, 1, 64, 16, [77, 300]),
    (6, 3, 96, 16, [100, 47]),
    (8, 2, 80, 32, [1, 333]),
    (2, 2, 8, 16, [40, 0, 0, 300]),
    (3, 1, 24, 48, [129, 97]),
    (4, 2, 256, 16, [65, 200]),
    (5, 1, 192, 16, [190]),
    (2, 1, 136, 80, [333, 1]),
    (2, 2, 128, 16, [3001]),
    (2, 1, 128, 128, [5000, 3]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens", DECODES)
def test_decode(heads, kv_heads, dim, page, lens, dtype):
    cache = make_cache(heads + dim, dtype, kv_heads, dim, page, lens)
    check_decode(cache, normal(3, len(lens), heads, dim, dtype=TYPES[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page,shared,lens", [
    (8, 2, 128, 16, 4, [64, 65, 100, 300]),            # one slot holds the prefix alone
    (8, 1, 64, 16, 33, [33 * 16 + i for i in range(17)]),
    (16, 1, 64, 64, 9, [600, 577, 1000]),
    (32, 2, 64, 32, 40, [40 * 32 + 7 * i for i in range(12)]),
    (4, 4, 128, 16, 70, [70 * 16 + 1] * 5),
    (2, 1, 80, 16, 20, [330, 321, 320]),
    (6, 2, 256, 16, 12, [200, 193]),
    (4, 2, 24, 48, 3, [144, 200, 145]),
    (8, 2, 128, 16, 10, [161, 0, 200, 0]),             # empty slots take no part
    (64, 2, 64, 16, 5, [81] * 9),
])
def test_decode_shared_prefix(heads, kv_heads, dim, page, shared, lens, dtype):
    cache = make_cache(heads + dim + shared, dtype, kv_heads, dim, page, lens, shared)
    q = normal(4, len(lens), heads, dim, dtype=TYPES[dtype])
    for prefix in (shared, shared // 2, 1, 0, None):
        check_decode(cache, q, prefix=prefix)


def test_decode_prefix_longer_than_some_slot():
    """A slot that is too short to hold the prefix has none of it in common; the others still do."""
    lens = [40, 161, 0, 200, 15]
    cache = make_cache(11, "f16", 2, 64, 16, lens, shared=10)
    q = normal(4, len(lens), 8, 64, dtype=torch.float16)
    check_decode(cache, q, prefix=10)


@pytest.mark.parametrize("prefix", [-1, -(1 << 31), 1 << 20, (1 << 31) - 1])
def test_decode_prefix_that_cannot_be(prefix):
    lens = [170, 200]
    cache = make_cache(12, "bf16", 2, 64, 16, lens, shared=10)
    q = normal(4, 2, 8, 64, dtype=torch.bfloat16)
    check_decode(cache, q, prefix=prefix)


def test_decode_slots_by_list_strides_and_scale():
    lens = [100, 0, 31, 260, 7]
    cache = make_cache(5, "f16", 2, 64, 16, lens)
    q = normal(4, 3, 8, 2 * 64, dtype=torch.float16)[:, :, 64:]
    check_decode(cache, q, seqs=[3, 1, 0], layer=0)
    check_decode(cache, normal(5, 8, 6, 64, dtype=torch.float16).transpose(0, 1)[:, :8], seqs=[4, 4, 2, 2, 3, 0],
                 scale=0.25)


def test_decode_many_rows():
    """More rows than one pass over the lengths takes at a time."""
    lens = [i % 23 for i in range(700)]
    cache = make_cache(6, "bf16", 1, 64, 16, lens)
    check_decode(cache, normal(4, 700, 2, 64, dtype=torch.bfloat16))


def test_decode_mixed_lengths():
    """One long row among short ones: its keys are split, theirs are not."""
    lens = [4000] + [5, 0, 130, 64] * 6
    cache = make_cache(16, "bf16", 2, 128, 16, lens)
    check_decode(cache, normal(4, len(lens), 8, 128, dtype=torch.bfloat16))


def test_decode_bad_slots_pages_and_lengths():
    """Numbers that cannot be are not followed: the row is zero or goes without the page, and the error word says so."""
    lens = [40, 50, 60, 70]
    q = normal(4, 4, 4, 64, dtype=torch.float16)
    cache = make_cache(8, "f16", 2, 64, 16, lens)
    out = torch.full_like(q, float("nan"))
    pi.attn_decode(cache, 0, q, out, seqs=ints([0, -1, 4, 1 << 30]))
    assert cache.errors() == pi.PI_CACHE_ESLOT
    assert (out[1:] == 0).all() and torch.isfinite(out[0]).all()

    for value in (-1, cache.pages, 1 << 30, -(1 << 31)):
        cache = make_cache(8, "f16", 2, 64, 16, lens)
        ks, vs = held_by(cache, 0)
        cache.table[1, 1] = value
        pi.attn_decode(cache, 0, q, out)
        assert cache.errors() == pi.PI_CACHE_EPAGE
        keep = list(range(16)) + list(range(32, 50))
        ks[1], vs[1] = ks[1][keep], vs[1][keep]
        attn_ref.check(out, *attn_ref.decode(q, ks, vs))

    for value in (-1, cache.max_pages * 16 + 1, (1 << 31) - 1):
        cache = make_cache(8, "f16", 2, 64, 16, lens)
        ks, vs = held_by(cache, 0)
        cache.lens[2] = value
        pi.attn_decode(cache, 0, q, out)
        assert cache.errors() == pi.PI_CACHE_ELENGTH
        assert (out[2] == 0).all()
        ks[2], vs[2] = ks[2][:0], vs[2][:0]
        attn_ref.check(out, *attn_ref.decode(q, ks, vs))


def test_decode_bad_page_in_the_prefix():
    lens = [100, 120]
    cache = make_cache(9, "bf16", 1, 64, 16, lens, shared=5)
    ks, vs = held_by(cache, 0)
    cache.table[:, 2] = cache.pages + 7
    q = normal(4, 2, 4, 64, dtype=torch.bfloat16)
    out = torch.full_like(q, float("nan"))
    pi.attn_decode(cache, 0, q, out, prefix=ints([5]))
    assert cache.errors() == pi.PI_CACHE_EPAGE
    for i, n in enumerate(lens):
        keep = [j for j in range(n) if not 32 <= j < 48]
        ks[i], vs[i] = ks[i][keep], vs[i][keep]
    attn_ref.check(out, *attn_ref.decode(q, ks, vs))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("prefix", [None, 6])
def test_decode_keys_that_score_minus_infinity(dtype, prefix):
    """A row whose keys all score -inf is zero; single such keys weigh nothing."""
    lens = [96, 130, 130]
    cache = make_cache(10, dtype, 1, 64, 16, lens, shared=6 if prefix else 0)
    q = normal(4, 3, 4, 64, dtype=TYPES[dtype]).abs() + 0.125
    table = cache.table.cpu()
    for j in range(6):
        cache.k_pool[1, int(table[0, j])] = -float("inf")
    out = torch.full_like(q, float("nan"))
    pi.attn_decode(cache, 1, q, out, prefix=None if prefix is None else ints([prefix]))
    assert (out[0] == 0).all()
    ks, vs = held_by(cache, 1)
    for i in (1, 2):
        live = torch.isfinite(ks[i]).all(-1).all(-1)
        ks[i], vs[i] = ks[i][live], vs[i][live]
    ref, tol = attn_ref.decode(q, ks, vs)
    attn_ref.check(out[1:], ref[1:], tol[1:])


def test_decode_far_pages():
    """A pool whose later layers and pages lie past 2^32 bytes, and element offsets past 2^31."""
    layers, pages, kv, page, dim = 3, 70000, 8, 16, 128      # 1.15e9 elements a layer
    k = torch.zeros(layers, pages, kv, page, dim, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    assert k.numel() > 1 << 31
    lens, slots, wide = [40, 33], 2, 4
    meta = torch.zeros(pi.Cache.meta_words(slots, wide, pages), dtype=torch.int32, device=DEV)
    cache = pi.Cache(k, v, meta, slots, wide)
    ids = [[pages - 1, 3, pages - 2], [pages - 3, 65536, 7]]
    for i in range(2):
        cache.table[i, :3] = ints(ids[i])
        for p in ids[i]:
            k[2, p] = normal(p, kv, page, dim, dtype=torch.float16)
            v[2, p] = normal(p + 1, kv, page, dim, dtype=torch.float16)
    cache.lens.copy_(ints(lens))
    q = normal(4, 2, 16, dim, dtype=torch.float16)
    out = torch.zeros_like(q)
    pi.attn_decode(cache, 2, q, out)
    ks = [k[2][torch.tensor(ids[i], device=DEV)].transpose(1, 2).reshape(-1, kv, dim)[:lens[i]].cpu() for i in range(2)]
    vs = [v[2][torch.tensor(ids[i], device=DEV)].transpose(1, 2).reshape(-1, kv, dim)[:lens[i]].cpu() for i in range(2)]
    attn_ref.check(out, *attn_ref.decode(q, ks, vs))


def test_decode_repeats_in_a_graph():
    """A captured step follows the cache as it grows; every replay equals the eager call."""
    lens = [100, 0, 170, 33]
    cache = make_cache(14, "bf16", 2, 128, 16, lens, wide=3, spare=20)
    cache.free[:20].copy_(torch.tensor([p for p, r in enumerate(cache.ref.tolist()) if r == 0], dtype=torch.int32))
    cache.words[0] = 20
    cache.k_pool.nan_to_num_(0.0)
    cache.v_pool.nan_to_num_(0.0, 0.0, 0.0)
    q = normal(4, 4, 8, 128, dtype=torch.bfloat16)
    kv = normal(5, 4, 4, 128, dtype=torch.bfloat16)
    k, v = kv[:, :2], kv[:, 2:]
    out, seqs, ones, cu = torch.empty_like(q), ints([0, 1, 2, 3]), ints([1] * 4), ints([0, 1, 2, 3, 4])

    def step():
        cache.extend(seqs, ones)
        cache.append(1, k, v, cu, seqs)
        pi.attn_decode(cache, 1, q, out)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        kv.copy_(normal(50 + i, 4, 4, 128, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert cache.errors() == 0
        assert cache.lens.tolist() == [n + 2 + i for n in lens]
        ks, vs = held_by(cache, 1)
        attn_ref.check(out, *attn_ref.decode(q, ks, vs), what=i)
        for b, (kk, vv) in enumerate(zip(ks, vs)):
            assert torch.equal(kk[-1], k[b].cpu()) and torch.equal(vv[-1], v[b].cpu())
        eager = torch.zeros_like(out)
        pi.attn_decode(cache, 1, q, eager)
        assert torch.equal(eager, out), i
