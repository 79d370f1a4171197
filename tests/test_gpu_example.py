"""examples/decode.py: every operator of every layer against 64 bits, from the inputs it was given there."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attn_ref  # noqa: E402
import oracle  # noqa: E402
import workload  # noqa: E402
from test_gpu_attention import held_by  # noqa: E402
from test_gpu_matvec import check as check_matvec  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DIMS = dict(layers=2, width=512, ffn=1100, rank=128, heads=8, kv_heads=2, dim=64, page=16, pages=64, slots=6, max_pages=12)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def check_layer(d, i, t, attention, host):
    """One layer's record; attention: (o, tol) of its queries."""
    n = t["x"].shape[0]
    for a in range(0, n, 32):
        sl = slice(a, min(a + 32, n))
        check_matvec(d.qkv[i].nibbles.cpu(), d.qkv[i].scales.cpu(), None, t["x"][sl], t["qkv"][sl].reshape(-1, d.qkv[i].rows))
        check_matvec(d.proj[i].nibbles.cpu(), d.proj[i].scales.cpu(), None, t["attn"][sl].reshape(-1, d.heads * d.dim),
                     t["y"][sl])
    attn_ref.check(t["attn"], *attention)
    # the sparse FFN as tests/test_gpu_parity.py holds it: a row whose scores keep clear of the threshold
    h = t["h"].cpu().numpy()
    ref = oracle.layer_forward(host[i], h)
    want = oracle.rms_glue(h.astype(np.float64), ref["y"])
    clear = (np.abs(ref["scores"]) >= 1e-4).all(-1)
    assert clear.any()
    got = t["out"].cpu().numpy().astype(np.float64)
    assert np.abs(got[clear] - want[clear]).max() <= 1e-3 * np.abs(want).max()


def test_every_operator_where_it_is_used(example):
    d = example.Decoder(**DIMS)
    cfg = workload.CONFIGS[1].with_(d=512, ffn=1100, rank=128, n_layers=2)
    host = [workload.make_layer(cfg, i) for i in range(2)]
    gen = torch.Generator().manual_seed(3)
    text = torch.randn(75, 512, generator=gen).cuda()
    trace = []
    d.prompt(text, 0, trace)
    h, g = d.heads, d.kv_heads
    for i, t in enumerate(trace):
        q, k, v = t["qkv"][:, :h], t["qkv"][:, h:h + g], t["qkv"][:, h + g:]
        check_layer(d, i, t, attn_ref.prompt(q, k, v, [75]), host)
        ks, vs = held_by(d.cache, i)
        assert torch.equal(ks[0], k.cpu()) and torch.equal(vs[0], v.cpu())
    d.share(0, [1, 2, 4], 75)
    assert d.prefix.item() == 4 and d.cache.lens.tolist() == [75, 75, 75, 0, 75, 0]
    seqs = d.ints([4, 1, 2])
    x = torch.randn(3, 512, generator=gen).cuda()
    for step in range(3):
        trace = []
        x = d.step(x, seqs, trace)
        for i, t in enumerate(trace):
            ks, vs = held_by(d.cache, i)
            check_layer(d, i, t, attn_ref.decode(t["qkv"][:, :h], [ks[s] for s in (4, 1, 2)], [vs[s] for s in (4, 1, 2)]),
                        host)
    d.cache.release(d.ints([0, 2]))
    d.cache.compact()
    assert d.cache.errors() == 0 and d.cache.lens.tolist() == [0, 78, 0, 0, 78, 0]
    trace = []
    d.step(x[:2].contiguous(), d.ints([4, 1]), trace)
    for i, t in enumerate(trace):
        ks, vs = held_by(d.cache, i)
        check_layer(d, i, t, attn_ref.decode(t["qkv"][:, :h], [ks[4], ks[1]], [vs[4], vs[1]]), host)


def test_a_replayed_step_equals_an_eager_one(example):
    a, b = example.Decoder(**DIMS), example.Decoder(**DIMS)
    text = torch.randn(40, 512, generator=torch.Generator().manual_seed(4)).cuda()
    x = torch.randn(2, 512, generator=torch.Generator().manual_seed(5)).cuda()
    for d in (a, b):
        d.prompt(text, 0)
        d.share(0, [1, 2], 40)
    seqs = a.ints([1, 2])
    y = x.clone()
    x.copy_(a.step(x, seqs))
    y.copy_(b.step(y, seqs))
    torch.cuda.synchronize()
    assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(a.step(x, seqs))
    for i in range(20):
        graph.replay()
        y.copy_(b.step(y, seqs))
        torch.cuda.synchronize()
        assert torch.equal(x, y), i
        assert a.cache.errors() == b.cache.errors() == 0
    assert torch.equal(a.cache.lens, b.cache.lens)


def test_the_command_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decode.py"), "--width", "512", "--ffn", "1100", "--rank",
                        "128", "--heads", "8", "--kv-heads", "2", "--dim", "64", "--text", "100", "--questions", "3",
                        "--tokens", "20"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "error word 0" in r.stdout
