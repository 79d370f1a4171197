"""Outputs that lie over inputs or over themselves, on the host: refused before anything is enqueued, so the addresses are
never followed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_abi_operators import EINVAL, FAKE, cache, pi  # noqa: E402, F401


@pytest.mark.parametrize("x,y", [
    (dict(), dict()),                                  # the same rows
    (dict(), dict(p=FAKE + 4 * 127)),                  # the last element of the first row
    (dict(p=FAKE + 4 * 127), dict()),
    (dict(ld=512), dict(p=FAKE + 4 * (512 * 2 + 100), ld=512)),          # the third row
    (dict(ld=512), dict(p=FAKE + 4 * (128 + 300), ld=512)),              # y's first over x's second
    (dict(t=1), dict(p=FAKE + 2 * 127, t=1)),
    (dict(t=3), dict(p=FAKE + 2 * (128 * 3 - 2), t=0)),
])
def test_matvec_y_over_x(pi, x, y):  # noqa: F811
    L, m = pi.lib(), pi.PiMat(FAKE << 4, FAKE << 5)
    rows, cols, batch = 128, 128, 3
    n = L.pi_matvec_workspace_bytes(rows, cols, batch)
    x, y = dict(dict(p=FAKE, t=0, ld=128), **x), dict(dict(p=FAKE, t=0, ld=128), **y)
    assert L.pi_matvec(ctypes.byref(m), rows, cols, None, x["p"], x["t"], x["ld"], y["p"], y["t"], y["ld"], batch, FAKE << 6, n,
                       None) == EINVAL


@pytest.mark.parametrize("token,head", [(0, 64), (64, 64), (256, 0), (0, 0), (256, 56), (56, 256), (128, 64), (64, 256),
                                        (200, 64), (160, 96)])
def test_attention_outputs_whose_rows_lie_over_each_other(pi, token, head):  # noqa: F811
    """5 rows of 4 heads of 64."""
    L, q, out = pi.lib(), ctypes.byref(pi.PiHeads(FAKE, 512, 64)), ctypes.byref(pi.PiHeads(FAKE << 4, token, head))
    assert L.pi_attn_prompt(q, q, q, out, 5, 4, 2, 64, pi.PI_F16, FAKE, 1, 0.0, None) == EINVAL
    c = ctypes.byref(cache(pi, slots=5))
    n = L.pi_attn_workspace_bytes(c, 5, 4)
    assert L.pi_attn_decode(c, 0, q, out, 5, 4, None, None, 0.0, FAKE << 5, n, None) == EINVAL
