"""Products whose blocks take several row tiles, or several groups of columns: the pipelines in their steady state.

Sampled rows of the matrix are checked, so that the 64-bit form stays small."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
from test_gpu_matvec import DEV, TYPES, check  # noqa: E402


def product(rows, cols, batch, x_type, y_type="f32", bias=True):
    gen = torch.Generator(device=DEV).manual_seed(rows + cols + batch)
    q = torch.randint(0, 256, (rows, cols // 2), generator=gen, dtype=torch.uint8, device=DEV)
    sc = (torch.randn(rows, cols // 32, generator=gen, device=DEV) / cols ** 0.5).half()
    x = torch.randn(batch, cols, generator=gen, device=DEV).to(TYPES[x_type])
    b = torch.randn(rows, generator=gen, device=DEV) if bias else None
    y = torch.full((batch, rows), float("nan"), dtype=TYPES[y_type], device=DEV)
    pi.matvec(pi.Q4Matrix(q, sc, b, batch=batch), x, y)
    # rows of every tile, at changing places of it, and the last ones
    pick = torch.unique(torch.cat([torch.arange(0, rows, 16 * 7 + 3), torch.arange(max(0, rows - 40), rows)]))
    at = pick.to(DEV)
    check(q[at].cpu(), sc[at].cpu(), None if b is None else b[at], x, y[:, at])
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("x_type,batch", [("f32", 1), ("f32", 2), ("f32", 3), ("f32", 4), ("f32", 8), ("f16", 1), ("f16", 5),
                                          ("f16", 16), ("bf16", 4), ("bf16", 8), ("bf16", 16)])
@pytest.mark.parametrize("rows,cols", [(20003, 256), (20003, 512), (33000, 96), (66003, 64), (40000, 1056), (18001, 1248), (17000, 2304)])
def test_few_columns_several_row_tiles_a_block(rows, cols, batch, x_type):
    """At most 1024 blocks of 16 rows are there at once; groups of 8 blocks of 32 columns go to 8 waves: fewer than that, as
    many and a little more, and rows that end inside a group."""
    product(rows, cols, batch, x_type)


@pytest.mark.parametrize("rows,cols,batch,x_type", [(9219, 8224, n, t) for n in (17, 24, 32) for t in ("f32", "bf16")]
                         + [(9219, 8224, 9, "f32"), (4100, 16384, 32, "f16"), (30011, 2080, 20, "bf16"),
                            (70000, 1024, 32, "f32"), (140001, 416, 17, "f32")])
def test_many_columns_several_groups_a_share(rows, cols, batch, x_type):
    """Five groups a block and more, so that every place of the operand's and weights' buffers is filled again; one to four
    column tiles."""
    product(rows, cols, batch, x_type, "bf16" if batch == 24 else "f32")


def test_one_row_too_wide_for_lds():
    """A row whose operand no block makes for itself."""
    for x_type in TYPES:
        product(100, 49152, 1, x_type)
