"""The workspaces that a cache and a matrix hold: how much memory they take, graphs that use them, and streams."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
from test_gpu_attention import DEV, ints, make_cache, normal  # noqa: E402

HEADS, ROWS = 16, 32


def setup():
    cache = make_cache(41, "bf16", 2, 64, 16, [100 + 3 * i for i in range(ROWS)], shared=4)
    q = normal(4, ROWS, HEADS, 64, dtype=torch.bfloat16)
    return cache, q, torch.zeros_like(q)


def needs(cache, n):
    return int(pi.lib().pi_attn_workspace_bytes(cache._ref, n, HEADS))


def held(before):
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before


@pytest.mark.parametrize("order", ["up", "down"])
def test_memory_of_many_batch_sizes(order):
    """All sizes together hold less than four times the largest one's workspace (a buffer of up to twice what is needed,
    and the smaller ones before it), not the sum over the sizes."""
    cache, q, out = setup()
    largest, before = max(needs(cache, n) for n in range(1, ROWS + 1)), held(0)
    sizes = range(1, ROWS + 1) if order == "up" else range(ROWS, 0, -1)
    for n in sizes:
        pi.attn_decode(cache, 1, q[:n], out[:n])
    assert 0 < held(before) <= 4 * largest + 4096


def test_no_call_takes_memory_after_reserve():
    cache, q, out = setup()
    cache.reserve(ROWS, HEADS)
    before = held(0)
    for n in [1, 32, 7, 16, 31] + list(range(1, ROWS + 1)):
        pi.attn_decode(cache, 1, q[:n], out[:n])
    assert held(before) == 0


def test_reserve_makes_a_first_call_fit_a_capture():
    cache, q, out = setup()
    want = torch.zeros_like(q)
    cache.reserve(ROWS, HEADS)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.attn_decode(cache, 1, q, out)
    pi.attn_decode(cache, 1, q, want)
    for i in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_a_graph_outlives_the_growth_of_the_workspace():
    cache, q, out = setup()
    want, other = torch.zeros_like(q), torch.zeros_like(q)
    pi.attn_decode(cache, 1, q[:2], want[:2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.attn_decode(cache, 1, q[:2], out[:2])
    for n in (5, 12, 32):
        pi.attn_decode(cache, 1, q[:n], other[:n])
        junk = [torch.full((needs(cache, 2) // 4,), float("nan"), device=DEV) for _ in range(4)]
        out.zero_()
        graph.replay()
        pi.attn_decode(cache, 1, q[:n], other[:n])
        torch.cuda.synchronize()
        assert torch.equal(out[:2], want[:2]) and torch.equal(other[:2], want[:2]) and all(torch.isnan(j).all() for j in junk)


def test_growth_inside_a_capture_is_refused():
    cache, q, out = setup()
    pi.attn_decode(cache, 1, q[:2], out[:2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(pi.PiError) as e:
            pi.attn_decode(cache, 1, q, out)
        pi.attn_decode(cache, 1, q[:2], out[:2])
    assert e.value.status == pi.PI_EINVAL
    graph.replay()
    torch.cuda.synchronize()
