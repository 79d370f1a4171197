"""examples/decode.py with slots that do not hold the same text: nobody reads another text's pages."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attn_ref  # noqa: E402
from test_gpu_attention import held_by  # noqa: E402
from test_gpu_example import DIMS, example  # noqa: E402, F401


def check_step(d, x, slots):
    trace = []
    d.step(x[:len(slots)].contiguous(), d.ints(slots), trace)
    assert d.cache.errors() == 0
    for i, t in enumerate(trace):
        ks, vs = held_by(d.cache, i)
        attn_ref.check(t["attn"], *attn_ref.decode(t["qkv"][:, :d.heads], [ks[s] for s in slots], [vs[s] for s in slots]))


def test_a_second_text_beside_a_shared_one(example):  # noqa: F811
    d = example.Decoder(**DIMS)
    gen = torch.Generator().manual_seed(7)
    texts = [torch.randn(n, 512, generator=gen).cuda() for n in (75, 90)]
    x = torch.randn(4, 512, generator=gen).cuda()
    d.prompt(texts[0], 0)
    d.share(0, [1, 2], 75)
    assert d.prefix.item() == 4
    check_step(d, x, [1, 2])
    d.prompt(texts[1], 3)
    check_step(d, x, [1, 3, 2])
    d.share(3, [4], 90)
    check_step(d, x, [4, 1, 3, 2])


def test_a_fork_of_a_fork(example):  # noqa: F811
    d = example.Decoder(**DIMS)
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(3, 512, generator=gen).cuda()
    d.prompt(torch.randn(63, 512, generator=gen).cuda(), 0)
    d.share(0, [1, 2], 63)
    for _ in range(2):
        check_step(d, x, [1, 2])
    d.share(1, [3], 65)                                # a page more than slot 2 has in common with it
    check_step(d, x, [2, 3, 1])
