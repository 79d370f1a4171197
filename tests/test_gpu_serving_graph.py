"""A serving step (room, append with norms and rotation, attention of the new tokens) captured once and replayed while its
sequences grow: positions, pages and shares come from what the cache holds then."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import chunk_ref  # noqa: E402
from test_gpu_rope import DEV, TYPES, held, ints, normal, offsets, weights  # noqa: E402


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,per,kw", [
    (8, 2, 128, 1, {}),
    (8, 2, 64, 1, dict(cap=20.0, window=70)),
    (16, 1, 64, 5, {}),                                # 80 rows a sequence
    (4, 2, 256, 20, dict(window=33)),
])
def test_steps(heads, kv_heads, dim, per, kw, dtype):
    start, steps, layers = [0, 14, 700], 24, 2
    n, t = len(start), per * len(start)
    qkv = torch.zeros(t, heads + 2 * kv_heads, dim, dtype=TYPES[dtype], device=DEV)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    rope, wq, wk = pi.Rope(dim, 50000.0, device=DEV), weights(1, dim), weights(2, dim)
    cu, seqs, more = ints(offsets([per] * n)), ints(list(range(n))), ints([per] * n)

    def a_cache():
        c = pi.Cache.create(layers, 150, kv_heads, 16, dim, n, 80, dtype=TYPES[dtype], device=DEV)
        old = [m for m in start if m]
        slots = ints([i for i, m in enumerate(start) if m])
        c.extend(slots, ints(old))
        for layer in range(layers):
            c.append(layer, normal(3, sum(old), kv_heads, dim, dtype=TYPES[dtype]),
                     normal(4, sum(old), kv_heads, dim, dtype=TYPES[dtype]), ints(offsets(old)), slots)
        c.reserve_chunk(t, heads, n)
        return c

    def step(c, turned, outs):
        c.extend(seqs, more)
        for layer in range(layers):
            c.append_rope(layer, rope, q, turned, k, v, cu, seqs, q_norm=wq, k_norm=wk)
            pi.attn_chunk(c, layer, turned, outs[layer], cu, seqs, **kw)

    one, two = a_cache(), a_cache()
    turned, mine = torch.zeros_like(q), torch.zeros_like(q)
    outs, want = ([torch.zeros(t, heads, dim, dtype=TYPES[dtype], device=DEV) for _ in range(layers)] for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(one, turned, outs)
    for i in range(steps):
        qkv.copy_(normal(100 + i, *qkv.shape, dtype=TYPES[dtype]))
        graph.replay()
        step(two, mine, want)
        torch.cuda.synchronize()
        assert torch.equal(turned, mine) and all(torch.equal(a, b) for a, b in zip(outs, want))
        _ = torch.randn(1000, device=DEV).sum().item()
    assert one.errors() == 0 and one.lens.tolist() == [m + steps * per for m in start]
    keys, values = zip(*(held(one, 1, i) for i in range(n)))
    chunk_ref.check(outs[1], *chunk_ref.chunk(turned, keys, values, [per] * n, **kw))
