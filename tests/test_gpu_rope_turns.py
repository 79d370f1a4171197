"""Norms and rotary positions of so many heads that a wave takes two or four turns of them: parts that queries, keys and values
share, last parts that are not full.  The bits are those of calls of few tokens, where a wave takes one turn; some tokens are
checked against 64 bits (chunk_ref.py)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import chunk_ref  # noqa: E402
from test_gpu_rope import TYPES, DEV, a_cache, held, ints, normal, offsets, weights  # noqa: E402

EPS, BASE = 1e-6, 10000.0
# heads, kv_heads, dim, rotary, layout, heads a turn
FORMS = [
    (24, 16, 128, 128, "half", 8),
    (24, 16, 128, 128, "pairs", 8),
    (12, 8, 128, 62, "half", 4),
    (12, 8, 128, 62, "pairs", 8),
    (40, 8, 80, 38, "half", 8),
    (64, 1, 64, 64, "half", 16),
    (10, 2, 256, 254, "half", 2),
    (7, 3, 128, 64, "half", 8),
    (24, 16, 128, 0, "half", 8),
]
form = pytest.mark.parametrize("heads,kv_heads,dim,rotary,layout,per", FORMS)
normed = pytest.mark.parametrize("norm", [False, True])
most = pytest.mark.parametrize("turns_a_wave,dtype", [(2, "f16"), (2, "bf16"), (4, "f16"), (4, "bf16")])


def tokens_for(turns, turns_a_wave):
    """So many that waves take that many turns: from 8192 turns of all tokens on two, from 16384 on four (of tokens with more
    than two)."""
    return -(-(16384 if turns_a_wave == 4 and turns > 2 else 8192) // turns)


def picked(t):
    return sorted({0, 1, 2, 63, 64, t // 3, t // 2, t - 2, t - 1} & set(range(t)))


@most
@normed
@form
def test_heads(heads, kv_heads, dim, rotary, layout, per, norm, turns_a_wave, dtype):
    turns = -(-heads // per) + -(-kv_heads // per)
    t = tokens_for(turns, turns_a_wave)
    qkv = normal(dim + t, t, heads + 2 * kv_heads, dim, dtype=TYPES[dtype])
    keep = qkv.clone()
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv_heads]
    pos = [(i * 7919) % 100003 for i in range(t)]
    at = ints(pos)
    rope = pi.Rope(rotary, BASE, layout, device=DEV) if rotary else None
    wq, wk = (weights(1, dim), weights(2, dim)) if norm else (None, None)
    q_out, k_out = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    pi.rope_heads(rope, at, q, q_out, k, k_out, q_norm=wq, k_norm=wk, eps=EPS)
    freqs = chunk_ref.frequencies(rotary, BASE, None)[0] if rotary else []
    some = picked(t)
    for x, y, w in ((q, q_out, wq), (k, k_out, wk)):
        chunk_ref.check(y[some], *chunk_ref.turn(x[some], [pos[i] for i in some], freqs, layout, norm=w, eps=EPS))
    step = 8191 // turns                               # a turn a wave
    q_one, k_one = torch.zeros_like(q_out), torch.zeros_like(k_out)
    for a in range(0, t, step):
        s = slice(a, min(a + step, t))
        pi.rope_heads(rope, at[s].clone(), q[s], q_one[s], k[s], k_one[s], q_norm=wq, k_norm=wk, eps=EPS)
    assert torch.equal(q_out, q_one) and torch.equal(k_out, k_one)
    assert torch.equal(qkv, keep)
    pi.rope_heads(rope, at, q, q, k, k, q_norm=wq, k_norm=wk, eps=EPS)   # in place
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(qkv[:, heads + kv_heads:], keep[:, heads + kv_heads:])


@most
@normed
@form
def test_append(heads, kv_heads, dim, rotary, layout, per, norm, turns_a_wave, dtype):
    turns = -(-heads // per) + 2 * -(-kv_heads // per)
    t = tokens_for(turns, turns_a_wave)
    counts = [t // 3, 1, t - t // 3 - 1 - 40, 40]
    lens = [t // 3 + 5, 1, t - t // 3 - 41 + 33, 40]
    cache = a_cache(t, 2, kv_heads, 16, dim, lens, TYPES[dtype])
    qkv = normal(t + 1, t, heads + 2 * kv_heads, dim, dtype=TYPES[dtype])
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    rope = pi.Rope(rotary, BASE, layout, device=DEV) if rotary else None
    wq, wk = (weights(1, dim), weights(2, dim)) if norm else (None, None)
    q_out = torch.full_like(q, float("nan"))
    cache.append_rope(1, rope, q, q_out, k, v, ints(offsets(counts)), ints([0, 1, 2, 3]), q_norm=wq, k_norm=wk, eps=EPS)
    pos = [p for n, c in zip(lens, counts) for p in range(n - c, n)]
    at, step = ints(pos), 8191 // (-(-heads // per) + -(-kv_heads // per))
    q_one, k_one = torch.zeros_like(q_out), torch.zeros(t, kv_heads, dim, dtype=TYPES[dtype], device=DEV)
    for a in range(0, t, step):
        s = slice(a, min(a + step, t))
        pi.rope_heads(rope, at[s].clone(), q[s], q_one[s], k[s], k_one[s], q_norm=wq, k_norm=wk, eps=EPS)
    assert torch.equal(q_out, q_one)
    row = 0
    for i, (n, c) in enumerate(zip(lens, counts)):
        kk, vv = held(cache, 1, i)
        assert torch.equal(kk[n - c:], k_one[row:row + c].cpu()) and torch.equal(vv[n - c:], v[row:row + c].cpu())
        assert (kk[:n - c] == 7).all() and (vv[:n - c] == 7).all()
        row += c
    assert (cache.k_pool[0] == 7).all() and (cache.v_pool[0] == 7).all()
    for pool in (cache.k_pool, cache.v_pool):          # nothing else was written
        assert int((pool[1] != 7).any(-1).sum()) <= t * kv_heads
    some = picked(t)
    freqs = chunk_ref.frequencies(rotary, BASE, None)[0] if rotary else []
    for x, y, w in ((q, q_out, wq), (k, k_one, wk)):
        chunk_ref.check(y[some], *chunk_ref.turn(x[some], [pos[i] for i in some], freqs, layout, norm=w, eps=EPS))
    assert cache.errors() == 0
