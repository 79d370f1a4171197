"""Attention where one key outscores all others: what the others weigh is not lost.

The bounds are those of tests/attn_ref.py but for float16's rounding of the weights p_j.  The kernels keep the largest p_j
at 2^11 or more (own keys of a decoding step: 2^15), and binary16 rounds what lies below 2^-14 by at most 2^-25: 2^-36 a
key, relative to the largest.  A row's sums are cut among at least 64 waves where the keys are many (`depth` below),
so at most m / 64 additions and 256 of the joins follow one another.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import attn_ref  # noqa: E402
from test_gpu_attention import DEV, TYPES, held_by, ints, make_cache, normal  # noqa: E402


def rows(q, k, v, last, scale, dtype, depth):
    """attn_ref.rows with the bound above; depth: additions one after the other."""
    d, m = q.shape[1], k.shape[0]
    seen = torch.arange(m)[None, :] < last[:, None]
    s = torch.where(seen, (q @ k.T) * scale, torch.tensor(-math.inf, dtype=torch.float64))
    p = torch.exp(s - s.max(1, keepdim=True).values)
    total = p.sum(1, keepdim=True)
    o, a = p @ v / total, p @ v.abs() / total
    u = attn_ref.half_step(dtype)
    mag = torch.where(seen, (q.abs() @ k.abs().T) * scale, torch.zeros_like(s)).max(1, keepdim=True).values
    ds = d * 2.0 ** -24 * mag + 2.0 ** -22 * (1 + 2 * mag)
    tol = u * o.abs() + (u + 2 * ds + 2 * (depth + 64) * 2.0 ** -24) * a
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 + m * 2.0 ** -36 * v.abs().max() / total
    return o, tol * (1 + 2 * u)


def sink(t, heads, dim, nats, dtype, seed):
    """q, k, v [t, heads, dim]: key 0 scores `nats` for every query and has the value 0, the others score about 0."""
    q, k, v = (normal(seed + i, t, heads, dim, dtype=torch.float32) for i in range(3))
    q[..., 0], k[..., 0] = 4, 0
    k[:, :, 1:] *= 0.25
    k[0] = 0
    k[0, :, 0] = nats * dim ** 0.5 / 4
    v = v * 64
    v[0] = 0
    return q.to(dtype), k.to(dtype), v.to(dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nats", [6, 10, 13, 16])
def test_prompt_behind_a_dominant_key(nats, dim, dtype):
    t, h = 1500, 2
    q, k, v = sink(t, h, dim, nats, TYPES[dtype], 3)
    out = torch.zeros_like(q)
    pi.attn_prompt(q, k, v, out, ints([0, t]))
    for i in range(h):
        ref = rows(q[:, i].cpu().double(), k[:, i].cpu().double(), v[:, i].cpu().double(), torch.arange(1, t + 1),
                   dim ** -0.5, TYPES[dtype], t)
        attn_ref.check(out[:, i], *ref, what=i)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompt_whose_dominant_keys_come_by_steps(dtype):
    """Tiles are taken from the last one down, so these rise by 3 powers of two a tile: less than what makes the kernel move
    its reference point."""
    t, dim = 900, 64
    q, k, v = sink(t, 1, dim, 0, TYPES[dtype], 5)
    for j in range(0, t, 64):
        k[j, 0, 0] = (t - j) / 64 * 3 * math.log(2) * dim ** 0.5 / 4
        v[j] = 0
    out = torch.zeros_like(q)
    pi.attn_prompt(q, k, v, out, ints([0, t]))
    attn_ref.check(out[:, 0], *rows(q[:, 0].cpu().double(), k[:, 0].cpu().double(), v[:, 0].cpu().double(),
                                    torch.arange(1, t + 1), dim ** -0.5, TYPES[dtype], t))


def check_decode(cache, q, prefix, depth):
    out = torch.full_like(q, float("nan"))
    pi.attn_decode(cache, 1, q, out, prefix=None if prefix is None else ints([prefix]))
    assert cache.errors() == 0
    ks, vs = held_by(cache, 1)
    per = q.shape[1] // cache.kv_heads
    for b in range(q.shape[0]):
        for g in range(cache.kv_heads):
            sl = slice(g * per, (g + 1) * per)
            ref = rows(q[b, sl].cpu().double(), ks[b][:, g].double(), vs[b][:, g].double(),
                       torch.full((per,), ks[b].shape[0]), cache.dim ** -0.5, q.dtype, depth)
            attn_ref.check(out[b, sl], *ref, what=(b, g))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("prefix", [None, 0, 100])
@pytest.mark.parametrize("nats", [6, 10, 13, 16])
def test_decode_behind_a_dominant_key(nats, prefix, dtype):
    lens = [1603, 1700, 2000]
    cache = make_cache(21, dtype, 2, 64, 16, lens, shared=100)
    q = normal(4, 3, 8, 64, dtype=TYPES[dtype])
    q[..., 0] = 4
    cache.k_pool[..., 0] = 0
    cache.k_pool[..., 1:] *= 0.25
    cache.v_pool.mul_(64)
    first = int(cache.table[0, 0])
    cache.k_pool[:, first, :, 0] = 0
    cache.k_pool[:, first, :, 0, 0] = nats * 2
    cache.v_pool[:, first, :, 0] = 0
    check_decode(cache, q, prefix, 2000)


@pytest.mark.parametrize("first_value", [0.0, 1.0])
@pytest.mark.parametrize("prefix", [None, 1000])
def test_decode_of_many_keys_of_small_weight(prefix, first_value):
    """70000 keys whose weights are 2^-25.05 of the first one's, all values 1 but the first one's."""
    lens = [70000, 70001, 69999]
    cache = make_cache(22, "f16", 1, 64, 64, lens, shared=1000)
    cache.k_pool.zero_()
    cache.v_pool.fill_(1.0)
    first = int(cache.table[0, 0])
    q = torch.zeros(3, 2, 64, dtype=torch.float16, device=DEV)
    q[..., 0] = 4
    cache.k_pool[:, first, :, 0, 0] = 25.05 * math.log(2) * 2
    cache.v_pool[:, first, :, 0] = first_value
    check_decode(cache, q, prefix, 70000 / 64 + 256)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shared", [1, 3, 5, 22, 23])
def test_decode_infinite_value_in_the_last_common_keys(shared, dim, dtype):
    """An infinite value of a key that is seen makes the result infinite, whatever stands behind the common keys."""
    lens = [16 * shared + 1, 16 * shared + 40]
    cache = make_cache(23, dtype, 1, dim, 16, lens, shared=shared)
    cache.v_pool[:, int(cache.table[0, shared - 1]), :, 7, 3] = float("inf")
    q = normal(4, 2, 4, dim, dtype=TYPES[dtype])
    out = torch.full_like(q, float("nan"))
    pi.attn_decode(cache, 1, q, out, prefix=ints([shared]))
    assert (out[..., 3] == float("inf")).all()
    ks, vs = held_by(cache, 1)
    ref, tol = attn_ref.decode(q, ks, vs)
    keep = [i for i in range(dim) if i != 3]
    attn_ref.check(out[..., keep], ref[..., keep], tol[..., keep])
