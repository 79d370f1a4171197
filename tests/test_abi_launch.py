"""Calls that would take more threads than a launch counts (2^32 - 1) are refused, on the host: through the C ABI with addresses
that are never followed.  (The runtime cuts such a launch off without an error.)"""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_abi_chunk import EUNSUPPORTED, FAKE, cache, heads, pi  # noqa: E402, F401


@pytest.mark.parametrize("tokens,h,kv_heads,n", [((1 << 24) + 1, 1, 1, (1 << 24) + 1), (1 << 20, 64, 64, 1 << 20),
                                                 ((1 << 31) - 1, 4, 4, 1)])
def test_prompt(pi, tokens, h, kv_heads, n):  # noqa: F811
    x = heads(pi, token=8 * h, head=8)
    assert pi.lib().pi_attn_prompt(x, x, x, x, tokens, h, kv_heads, 8, pi.PI_F16, FAKE, n, 0.0, None) == EUNSUPPORTED


@pytest.mark.parametrize("tokens", [1 << 28, (1 << 31) - 1])
def test_append(pi, tokens):  # noqa: F811
    x = heads(pi, token=128, head=64)
    assert pi.lib().pi_cache_append(ctypes.byref(cache(pi)), 0, x, x, tokens, FAKE, FAKE, 1, None) == EUNSUPPORTED


@pytest.mark.parametrize("dim,tokens,n", [(256, (1 << 18) - 1, 4096), (136, (1 << 18) - 1, 4096)])
def test_chunk(pi, dim, tokens, n):  # noqa: F811
    L, c = pi.lib(), ctypes.byref(cache(pi, kv_heads=1024, dim=dim))
    x = heads(pi, token=4096 * dim, head=dim)
    size = L.pi_attn_chunk_workspace_bytes(c, tokens, 4096, n)
    assert size > 0
    assert L.pi_attn_chunk(c, 0, x, x, tokens, 4096, FAKE, FAKE, n, 0.0, 0.0, None, 0, FAKE, size, None) == EUNSUPPORTED
