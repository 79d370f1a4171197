"""examples/decode.py with its text in pieces: every piece's attention against 64 bits over what the pieces before it left."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import chunk_ref  # noqa: E402
import decode  # noqa: E402


@pytest.mark.parametrize("piece", [1, 40, 64, 300])
def test_text_in_pieces(piece):
    heads, kv_heads, dim, layers, text = 8, 2, 64, 2, 9 if piece == 1 else 150
    d = decode.Decoder(layers=layers, width=512, ffn=1100, rank=128, heads=heads, kv_heads=kv_heads, dim=dim, pages=40, slots=3,
                       max_pages=20, piece=piece, device="cuda:0")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(3)
    x, trace = torch.randn(text, 512, generator=gen, device="cuda:0"), []
    y = d.prompt(x, 0, trace)
    assert y.shape == x.shape and torch.isfinite(y).all() and d.cache.errors() == 0 and int(d.cache.lens[0]) == text
    assert len(trace) == layers * -(-text // piece)
    for layer in range(layers):
        k = v = torch.empty(0, kv_heads, dim, dtype=torch.float16)
        for t in trace[layer::layers]:
            qkv = t["qkv"]
            k = torch.cat([k, qkv[:, heads:heads + kv_heads].cpu()])
            v = torch.cat([v, qkv[:, heads + kv_heads:].cpu()])
            chunk_ref.check(t["attn"], *chunk_ref.chunk(qkv[:, :heads], [k], [v], [qkv.shape[0]]))
    d.share(0, [1, 2], text)                           # and on with answers
    y = d.step(torch.randn(2, 512, generator=gen, device="cuda:0"), d.ints([1, 2]))
    assert torch.isfinite(y).all() and d.cache.errors() == 0 and d.cache.lens.tolist() == [text, text + 1, text + 1]
