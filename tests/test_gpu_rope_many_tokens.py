"""Norms and rotary positions of more tokens than one dimension of a launch has threads for."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import chunk_ref  # noqa: E402
from test_gpu_rope import DEV, weights  # noqa: E402


def test_many_tokens():
    t, d = (1 << 26) + 9, 8                            # a wave of 64 threads each
    gen = torch.Generator(device=DEV).manual_seed(3)
    q = torch.empty(t, 1, d, dtype=torch.float16, device=DEV).normal_(generator=gen)
    pos = torch.arange(t, dtype=torch.int32, device=DEV)
    rope, w, out = pi.Rope(d, layout="pairs", device=DEV), weights(1, d), torch.zeros_like(q)
    pi.rope_heads(rope, pos, q, out, q_norm=w)
    some = [0, 1, 1000, t // 2, (1 << 26) - 1, 1 << 26, t - 2, t - 1]
    chunk_ref.check(out[some], *chunk_ref.turn(q[some], some, chunk_ref.frequencies(d, 10000.0, None)[0], "pairs", norm=w))
    step, part = 1 << 24, torch.empty_like(q[:1 << 24])
    for a in range(0, t, step):
        b = min(a + step, t)
        pi.rope_heads(rope, pos[a:b].clone(), q[a:b], part[:b - a], q_norm=w)
        assert torch.equal(out[a:b], part[:b - a])
