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


def busy_reader(n):
    """Memory of n bytes that the current stream reads a while from now, given back already; the copy, and what it has to be."""
    block = torch.arange(n // 4, dtype=torch.int32, device=DEV)
    want, copy = block.clone(), torch.empty_like(block)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    copy.copy_(block)
    del block
    return copy, want


def test_first_call_on_another_stream_leaves_the_current_ones_memory_alone():
    cache, q, out = setup()
    want, side = torch.zeros_like(q), torch.cuda.Stream()
    cache2, _, _ = setup()
    pi.attn_decode(cache2, 1, q, want)
    for _ in range(2):
        copy, same = busy_reader(needs(cache, ROWS))
        pi.attn_decode(cache, 1, q, out, stream=side)  # the first time takes the memory that was given back
        torch.cuda.synchronize()
        assert torch.equal(copy, same) and torch.equal(out, want)


def test_products_on_another_stream_leave_the_current_ones_memory_alone():
    rows, cols, batch = 2048, 1024, 32
    q = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device=DEV)
    sc = torch.rand(rows, cols // 32, device=DEV).half()
    x, side = torch.randn(batch, cols, device=DEV), torch.cuda.Stream()
    want, y = torch.empty(batch, rows, device=DEV), torch.zeros(batch, rows, device=DEV)
    pi.matvec(pi.Q4Matrix(q, sc, batch=batch), x, want)
    copy, same = busy_reader(int(pi.lib().pi_matvec_workspace_bytes(rows, cols, batch)) // 4 * 4)
    mat = pi.Q4Matrix(q, sc, batch=batch)
    pi.matvec(mat, x, y, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, same) and torch.equal(y, want)


def test_calls_captured_on_a_stream_of_their_own():
    """A graph's stream is another one than the memory was taken on; what is captured runs all the same."""
    cache, q, out = setup()
    want = torch.zeros_like(q)
    pi.attn_decode(cache, 1, q, want)
    torch.cuda.synchronize()
    side = pi.HipStream()
    graph = pi.HipGraph(side, lambda s: pi.attn_decode(cache, 1, q, out, stream=s))
    for i in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        side.synchronize()
        assert torch.equal(out, want), i


@pytest.mark.parametrize("batch", [1, 8])
def test_ffn_calls_without_a_workspace_on_another_stream(batch):
    """The memory that such a call took and gave back is not handed to the current stream while the call's work runs."""
    import workload
    layer = pi.DeviceLayer.upload(workload.make_layer(workload.CONFIGS[1].with_(d=512, ffn=1100, rank=128, n_layers=1), 0))
    x, side = torch.randn(batch, 512, device=DEV), torch.cuda.Stream()
    want, y = torch.empty_like(x), torch.zeros_like(x)
    pi.ffn_stack([layer], x, want, batch=batch)
    n = pi.workspace_bytes([layer], batch)
    torch.cuda.synchronize()
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        pi.ffn_stack([layer], x, y, batch=batch, stream=side)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(y, want) and all((j == 255).all() for j in junk)


def test_workspace_of_layers_given_one_by_one():
    import workload
    cfg = workload.CONFIGS[1].with_(d=512, ffn=1100, rank=128, n_layers=2)
    layers = [pi.DeviceLayer.upload(workload.make_layer(cfg, i)) for i in range(2)]
    ws = pi.alloc_workspace((layer for layer in layers), 4)
    assert ws.numel() == pi.workspace_bytes(layers, 4) and ws.device == layers[0].A.device
