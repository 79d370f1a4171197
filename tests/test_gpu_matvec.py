"""Products with Q4_0 matrices against 64 bits.

A product is off by at most
  - the output's own rounding, half a step of its type,
  - x as it goes into the matrix instruction: exact for 16-bit rows, 2^-23 relative for float32 rows (values below
    2^-39 of the row's largest may lose more, 2^-39 of the largest each),
  - float32 sums: one rounding per addition, at most (cols / 16 + 64) one after the other, and a few more for
    the scales, each 2^-24 of the sum of |w x|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def matrix(seed, rows, cols, spread=0.0):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (rows, cols // 2), generator=gen, dtype=torch.uint8)
    sc = torch.randn(rows, cols // 32, generator=gen) / cols ** 0.5
    if spread:
        sc = sc * torch.exp2(torch.randn(rows, cols // 32, generator=gen) * spread)
    return q, sc.to(torch.float16)


def weights(q, scale):
    """[rows][cols] float64: byte j of a block of 32 holds weights j (low half) and j + 16."""
    b = q.view(q.shape[0], -1, 16)
    w = torch.cat([(b & 15), (b >> 4)], 2).double() - 8
    return (w * scale.double().unsqueeze(-1)).flatten(1)


def check(q, scale, bias, x, y):
    w, xd = weights(q, scale), x.cpu().double()
    ref = xd @ w.T
    mass = xd.abs() @ w.abs().T
    if bias is not None:
        ref = ref + bias.cpu().double()
        mass = mass + bias.cpu().double().abs()
    u = torch.finfo(y.dtype).eps / 2
    cols = q.shape[1] * 2
    depth = cols / 16 + 64
    tol = u * ref.abs() + (depth * 2.0 ** -24 + 2.0 ** -22) * mass
    if x.dtype == torch.float32:
        tol = tol + 2.0 ** -39 * xd.abs().max(1, keepdim=True).values * w.abs().sum(1)
    tol = tol * (1 + 2 * u) + torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps
    off = (y.cpu().double() - ref).abs()
    assert (off <= tol).all(), (float((off / tol).max()), [int(i) for i in (off > tol).nonzero()[0]])


SIZES = [(1, 32, 1), (16, 64, 1), (17, 32, 2), (100, 96, 3), (33, 128, 5), (64, 160, 7), (48, 1056, 8), (257, 512, 9),
         (1000, 352, 15), (96, 2048, 16), (31, 4096, 17), (320, 736, 24), (128, 1024, 31), (515, 544, 32), (4099, 128, 1),
         (5, 12288, 1), (7, 12320, 32), (2050, 96, 32)]


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("rows,cols,batch", SIZES)
def test_sizes(rows, cols, batch, x_type):
    q, sc = matrix(rows + cols, rows, cols)
    gen = torch.Generator().manual_seed(batch)
    x = torch.randn(batch, cols, generator=gen).to(TYPES[x_type]).to(DEV)
    y_types = list(TYPES) if rows <= 100 else ["f32", "bf16" if rows % 2 else "f16"]
    for i, y_type in enumerate(y_types):
        bias = torch.randn(rows, generator=gen).to(DEV) if i % 2 == 0 else None
        mat = pi.Q4Matrix(q.to(DEV), sc.to(DEV), bias, batch=batch)
        y = torch.full((batch, rows), float("nan"), dtype=TYPES[y_type], device=DEV)
        pi.matvec(mat, x, y)
        check(q, sc, bias, x, y)


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("batch", [1, 4, 20])
def test_strided_rows_and_what_lies_between(x_type, batch):
    rows, cols = 130, 256
    q, sc = matrix(1, rows, cols)
    gen = torch.Generator().manual_seed(2)
    wide_x = torch.randn(batch, cols + 11, generator=gen).to(TYPES[x_type]).to(DEV)
    wide_y = torch.full((batch, rows + 9), 3.0, dtype=torch.bfloat16, device=DEV)
    x, y = wide_x[:, 3:3 + cols], wide_y[:, 5:5 + rows]
    pi.matvec(pi.Q4Matrix(q.to(DEV), sc.to(DEV), batch=32), x, y)
    check(q, sc, None, x, y)
    assert (wide_y[:, :5] == 3).all() and (wide_y[:, 5 + rows:] == 3).all()


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("batch", [1, 3])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-8, 1e8, 1e30])
def test_ranges_of_x(scale, batch, x_type):
    """Rows far outside binary16's range, and rows whose values are far apart."""
    rows, cols = 48, 256
    q, sc = matrix(3, rows, cols)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(batch, cols, generator=gen) * scale
    if batch > 1:
        x[1, ::2] *= 1e-6
        x[2] = 0
    x = x.to(TYPES[x_type]).to(DEV)
    y = torch.empty(batch, rows, device=DEV)
    pi.matvec(pi.Q4Matrix(q.to(DEV), sc.to(DEV), batch=batch), x, y)
    check(q, sc, None, x, y)
    if batch > 1:
        assert (y[2] == 0).all()


def test_scales_of_every_size():
    """Block scales over binary16's whole range, subnormal and negative ones among them."""
    rows, cols = 40, 512
    q, sc = matrix(5, rows, cols, spread=6)
    x = torch.randn(4, cols, generator=torch.Generator().manual_seed(6)).to(DEV)
    y = torch.empty(4, rows, device=DEV)
    pi.matvec(pi.Q4Matrix(q.to(DEV), sc.to(DEV), batch=4), x, y)
    check(q, sc, None, x, y)


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("batch", [1, 3, 20])
def test_values_that_are_not_finite_stay_in_their_row(poison, x_type, batch):
    rows, cols = 40, 320
    q, sc = matrix(7, rows, cols)
    sc = sc.abs() + 1e-3
    x = torch.randn(batch, cols, generator=torch.Generator().manual_seed(8)).to(TYPES[x_type])
    x[batch // 2, 77] = poison
    if x_type != "f16":
        x[batch // 2, 78] = 3e38                       # a large value beside it does not count as infinite
    x = x.to(DEV)
    y = torch.empty(batch, rows, device=DEV)
    pi.matvec(pi.Q4Matrix(q.to(DEV), sc.to(DEV), batch=batch), x, y)
    rest = [b for b in range(batch) if b != batch // 2]
    if rest:
        check(q, sc, None, x[rest], y[rest])
    w = weights(q, sc)[:, 77]
    got = y[batch // 2].cpu()
    want = torch.full((rows,), poison).double() * w    # 0 times an infinity is NaN
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep].double(), want[keep])


def test_a_bias_or_scale_that_is_not_finite():
    rows, cols = 20, 64
    q, sc = matrix(9, rows, cols)
    bias = torch.zeros(rows)
    bias[3], bias[4] = float("inf"), float("nan")
    x = torch.randn(2, cols, generator=torch.Generator().manual_seed(1)).to(DEV)
    y = torch.empty(2, rows, device=DEV)
    pi.matvec(pi.Q4Matrix(q.to(DEV), sc.to(DEV), bias.to(DEV), batch=2), x, y)
    assert (y[:, 3] == float("inf")).all() and torch.isnan(y[:, 4]).all()
    keep = [i for i in range(rows) if i not in (3, 4)]
    check(q[keep], sc[keep], None, x, y[:, keep])
    bad = sc.clone()
    bad[5, 1] = float("nan")
    pi.matvec(pi.Q4Matrix(q.to(DEV), bad.to(DEV), batch=2), x, y)
    assert torch.isnan(y[:, 5]).all()
    keep = [i for i in range(rows) if i != 5]
    check(q[keep], sc[keep], None, x, y[:, keep])


def test_matrices_of_the_host():
    """Q4Matrix.upload takes the host generator's layout."""
    import workload
    lw = workload.make_layer(workload.CONFIGS[4].with_(d=256, ffn=100, rank=64, n_layers=1), 0)
    mat = pi.Q4Matrix.upload(lw.up, batch=2)
    x = torch.randn(2, mat.cols, generator=torch.Generator().manual_seed(1)).to(DEV)
    y = torch.empty(2, mat.rows, device=DEV)
    pi.matvec(mat, x, y)
    sc = torch.from_numpy(np.ascontiguousarray(lw.up.scales).view(np.float16).copy()).view(mat.rows, -1)
    check(torch.from_numpy(np.ascontiguousarray(lw.up.nibbles).copy()).view(mat.rows, -1), sc, None, x, y)


def test_repeats_streams_and_graphs():
    rows, cols, batch = 600, 1024, 5
    q, sc = matrix(11, rows, cols)
    mat = pi.Q4Matrix(q.to(DEV), sc.to(DEV), batch=batch)
    x = torch.randn(batch, cols, generator=torch.Generator().manual_seed(12)).to(DEV)
    want, y = torch.empty(batch, rows, device=DEV), torch.zeros(batch, rows, device=DEV)
    pi.matvec(mat, x, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pi.matvec(mat, x, y)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.matvec(mat, x, y)
    for i in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        eager = torch.zeros_like(y)
        pi.matvec(mat, x, eager)
        assert torch.equal(eager, want)
