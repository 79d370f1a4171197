"""Products with a value that is far larger than the rest of its row, where its weight is 0.

x goes into the matrix instruction behind a power of two that brings its row's largest value into [2^14, 2^15), a float32
value as two binary16 numbers of which the second stands for 2^-11 times itself.  binary16 rounds what is below 2^-14 by at
most 2^-25, so the row's largest value L adds to the error of every x
  float32: 2^-25 2^-11 / 2^14 L = 2^-50 L,    bfloat16: 2^-25 / 2^14 L = 2^-39 L (where its 8 bits go below 2^-24).
float16 rows go in as they are.  The other terms are test_gpu_matvec's."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
from test_gpu_matvec import DEV, TYPES, matrix, weights  # noqa: E402


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch", [1, 4, 20])
@pytest.mark.parametrize("power", [10, 20, 25, 30, 38, 60])
def test_a_large_value_with_a_weight_of_zero(power, batch, x_type):
    rows, cols = 64, 512
    q, sc = matrix(13, rows, cols)
    q[::2, 5] = (q[::2, 5] & 0xf0) | 8                 # weight 5 of the first block is 0 in every other row
    x = torch.randn(batch, cols, generator=torch.Generator().manual_seed(power))
    x[:, 5] = 2.0 ** (min(power, 14) if x_type == "f16" else power)
    x = x.to(TYPES[x_type]).to(DEV)
    y = torch.empty(batch, rows, device=DEV)
    pi.matvec(pi.Q4Matrix(q.to(DEV), sc.to(DEV), batch=batch), x, y)
    w, xd = weights(q, sc), x.cpu().double()
    assert (w[::2, 5] == 0).all()
    ref, mass = xd @ w.T, xd.abs() @ w.abs().T
    lost = {"f32": 2.0 ** -50, "bf16": 2.0 ** -39, "f16": 0.0}[x_type] * xd.abs().max(1, keepdim=True).values * w.abs().sum(1)
    tol = 2.0 ** -24 * ref.abs() + ((cols / 16 + 64) * 2.0 ** -24 + 2.0 ** -22) * mass + lost
    off = (y.cpu().double() - ref).abs()
    assert (off <= tol).all(), float((off / tol).max())
