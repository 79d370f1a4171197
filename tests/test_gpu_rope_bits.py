"""What neither turns nor has a norm is moved bit by bit, NaN with a payload and signalling NaN among it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import chunk_ref  # noqa: E402
from test_gpu_rope import TYPES, DEV, a_cache, held, ints, normal  # noqa: E402

# signalling and quiet NaN with payloads, of both signs, an infinity, a subnormal value, -0
BITS = {"f16": [0x7c01, 0xfc55, 0x7d23, 0x7e77, 0xff01, 0xfc00, 0x0001, 0x8000],
        "bf16": [0x7f81, 0xff95, 0x7fa3, 0x7fd7, 0xffc1, 0xff80, 0x0001, 0x8000]}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("rotary,dim", [(64, 128), (62, 128), (30, 64), (2, 16), (10, 24), (40, 80), (0, 64)])
def test_bits(rotary, dim, layout, dtype):
    t, h, g = 9, 3, 2
    bits = torch.tensor([x - (1 << 16) if x >> 15 else x for x in BITS[dtype]], dtype=torch.int16)
    behind = dim - rotary
    still = bits[torch.arange(t * (h + 2 * g) * behind) * 5 % 8].view(t, h + 2 * g, behind).to(DEV)
    x = normal(5, t, h + 2 * g, dim, dtype=TYPES[dtype])
    x.view(torch.int16)[:, :, rotary:] = still
    q, k, v = x[:, :h], x[:, h:h + g], x[:, h + g:]
    rope = pi.Rope(rotary, layout=layout, device=DEV) if rotary else None
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    pi.rope_heads(rope, ints(range(t)), q, q_out, k, k_out)
    freqs = chunk_ref.frequencies(rotary, 10000.0, None)[0] if rotary else []

    def same(got, src):
        assert torch.equal(got[..., rotary:].contiguous().view(torch.int16), src[..., rotary:].contiguous().view(torch.int16))
        if rotary:
            ref, tol = chunk_ref.turn(src[..., :rotary].contiguous(), range(t), freqs, layout)
            chunk_ref.check(got[..., :rotary], ref, tol)
    same(q_out, q), same(k_out, k)
    cache, q_in = a_cache(1, 1, g, 16, dim, [t], TYPES[dtype]), torch.zeros_like(q)
    cache.append_rope(0, rope, q, q_in, k, v, ints([0, t]), ints([0]))
    keys, values = held(cache, 0, 0)
    same(q_in, q), same(keys, k.cpu())
    assert torch.equal(values.contiguous().view(torch.int16), v.contiguous().cpu().view(torch.int16))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_bits_of_a_call_whose_other_heads_have_a_norm(dtype):
    t, h, g, dim, rotary = 9, 3, 2, 64, 30
    bits = torch.tensor([x - (1 << 16) if x >> 15 else x for x in BITS[dtype]], dtype=torch.int16)
    q, k = normal(5, t, h, dim, dtype=TYPES[dtype]), normal(6, t, g, dim, dtype=TYPES[dtype])
    k.view(torch.int16)[:, :, rotary:] = bits[torch.arange(t * g * (dim - rotary)) % 8].view(t, g, -1).to(DEV)
    rope, w = pi.Rope(rotary, layout="pairs", device=DEV), 1 + normal(7, dim, dtype=torch.float32, scale=0.3)
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    pi.rope_heads(rope, ints(range(t)), q, q_out, k, k_out, q_norm=w)
    assert torch.equal(k_out[..., rotary:].contiguous().view(torch.int16), k[..., rotary:].contiguous().view(torch.int16))
    freqs = chunk_ref.frequencies(rotary, 10000.0, None)[0]
    chunk_ref.check(q_out, *chunk_ref.turn(q, range(t), freqs, "pairs", norm=w))
