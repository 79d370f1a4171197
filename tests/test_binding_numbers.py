"""Numbers that the C types do not hold, on the host: ctypes would hand over what is left of them, without a word."""
import pytest

torch = pytest.importorskip("torch")

from test_binding_arguments import ints, pi, refused, spy  # noqa: E402, F401


@pytest.fixture
def held(pi, spy):  # noqa: F811
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    c.reserve(3, 4), c.reserve_chunk(3, 4, 1)
    return c, torch.zeros(3, 4, 64, dtype=torch.float16)


def windows_seen(spy, monkeypatch):  # noqa: F811
    seen, real = [], type(spy).__getattr__

    def look(self, name):
        call = real(self, name)
        if name != "pi_attn_chunk":
            return call

        def with_window(*args):
            seen.append(args[12])
            return call(*args)
        return with_window
    monkeypatch.setattr(type(spy), "__getattr__", look)
    return seen


def test_windows(pi, spy, held, monkeypatch):  # noqa: F811
    c, q = held
    seen = windows_seen(spy, monkeypatch)
    for window in (0, 5, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 63) - 1, -1, -(1 << 32) + 5):
        pi.attn_chunk(c, 0, q, q.clone(), ints(0, 3), window=window)
    most = (1 << 31) - 1
    assert seen == [0, 5, most, most, most, most, -1, -1]


@pytest.mark.parametrize("small", [1e-46, 1e-300])
def test_scales_and_caps_that_round_to_zero(pi, spy, held, small):  # noqa: F811
    c, q = held
    kv = torch.zeros(3, 2, 64, dtype=torch.float16)
    refused(pi, spy, lambda: pi.attn_chunk(c, 0, q, q.clone(), ints(0, 3), cap=small), "cap")
    refused(pi, spy, lambda: pi.attn_chunk(c, 0, q, q.clone(), ints(0, 3), scale=small), "scale")
    refused(pi, spy, lambda: pi.attn_decode(c, 0, q, q.clone(), scale=small), "scale")
    refused(pi, spy, lambda: pi.attn_prompt(q, kv, kv, q.clone(), ints(0, 3), scale=small), "scale")


def test_more_tokens_than_an_int32_counts(pi, spy, held):  # noqa: F811
    c, _ = held
    many = torch.zeros(1, 4, 64, dtype=torch.float16).expand((1 << 32) + 3, 4, 64)
    keys = torch.zeros(1, 2, 64, dtype=torch.float16).expand((1 << 32) + 3, 2, 64)
    w = torch.ones(64)
    refused(pi, spy, lambda: pi.rope_heads(None, None, many, many, q_norm=w))
    refused(pi, spy, lambda: c.append_rope(0, None, None, None, keys, keys, ints(0, 3), ints(0), k_norm=w))
    refused(pi, spy, lambda: c.append(0, keys, keys, ints(0, 3), ints(0)))
    refused(pi, spy, lambda: pi.attn_prompt(many, keys, keys, many, ints(0, 3)))
    with pytest.raises(pi.PiError):
        pi.attn_chunk(c, 0, many, many, ints(0, 3))
