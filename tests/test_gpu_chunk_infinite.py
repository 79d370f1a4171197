"""Keys and values that are not finite under attention of chunks: every kernel (chunks of few rows; four waves a block; eight,
for wide heads), tiles that all rows of a block see and tiles that some see, keys shared out and not."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import chunk_ref  # noqa: E402
from test_gpu_chunk import TYPES, Held, normal, run  # noqa: E402

INF, NAN = float("inf"), float("nan")
# heads, kv_heads, dim, tokens of the slot, of the chunk.  Up to 32 rows (tokens times heads of a key head): k_chunk_few.
FORMS = [
    (4, 2, 64, 300, 5),
    (8, 2, 128, 3000, 8),        # two tiles of 16 rows a block, keys shared out
    (4, 1, 256, 1000, 6),
    (2, 2, 80, 90, 1),           # one row
    (2, 1, 128, 2500, 1),        # one row, keys shared out
    (4, 2, 64, 300, 220),
    (4, 2, 128, 2600, 70),       # 128 rows a block, keys shared out
    (2, 1, 192, 300, 220),       # eight waves
    (4, 2, 256, 1900, 90),       # eight waves, keys shared out
    (2, 1, 256, 290, 290),
]
form = pytest.mark.parametrize("heads,kv_heads,dim,n,c", FORMS)
both = pytest.mark.parametrize("dtype", ["f16", "bf16"])


def seen_by(n, c, window):
    """[c, n]: which keys the rows see."""
    back = torch.arange(n - c, n)[:, None] - torch.arange(n)[None, :]
    return (back >= 0) & (back < window) if window else back >= 0


def lost(v, n, c, heads, window):
    """What becomes of elements [c, heads, dim] that see values which are not finite: the infinity, or NaN where there is a NaN
    or infinities of both signs; 0 for the others."""
    seen = seen_by(n, c, window).float()
    up, down, nan = (torch.einsum("ck,kgd->cgd", seen, x.float()) > 0 for x in (v == INF, v == -INF, torch.isnan(v)))
    out = torch.zeros(up.shape, dtype=torch.float64)
    out[up], out[down], out[nan | up & down] = INF, -INF, NAN
    return out.repeat_interleave(heads // v.shape[1], 1)


def check(out, ref, tol, gone):
    got = out.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(gone))
    assert torch.equal(torch.where(torch.isinf(got), got, 0.0), torch.where(torch.isinf(gone), gone, 0.0))
    chunk_ref.check(torch.where(gone == 0, got, ref), ref, tol)


@both
@form
@pytest.mark.parametrize("poison", [NAN, INF, -INF])
@pytest.mark.parametrize("window", [0, 70])
def test_unseen_keys_leave_no_trace(window, poison, heads, kv_heads, dim, n, c, dtype):
    """A token inside the chunk, and one that a window hides from some rows or all."""
    h = Held(dim, 1, kv_heads, 16, dim, [n], TYPES[dtype])
    q = normal(7, c, heads, dim, dtype=TYPES[dtype])
    ref, tol = chunk_ref.chunk(q, h.k, h.v, [c], window=window)
    for at in (n - (c + 1) // 2, n - c // 2 - 70):
        if at < 0:
            continue
        hit = seen_by(n, c, window)[:, at]
        for which in ("k", "v", "kv"):
            k, v = h.k[0].clone(), h.v[0].clone()
            if "k" in which:
                k[at] = poison
            if "v" in which:
                v[at] = poison
            h.write(0, k, v)
            out = run(h, q, [c], window=window)
            chunk_ref.check(out[~hit], ref[~hit], tol[~hit], which)
            if which == "v":
                assert not torch.isfinite(out[hit]).any()
            if poison != poison:
                assert torch.isnan(out[hit]).all()


@both
@form
@pytest.mark.parametrize("window", [0, 130])
def test_values_here_and_there(window, heads, kv_heads, dim, n, c, dtype):
    """Single values in a chunk, before it and far before it: only their dimensions of the rows that see them are lost."""
    h = Held(dim, 1, kv_heads, 16, dim, [n], TYPES[dtype])
    q = normal(7, c, heads, dim, dtype=TYPES[dtype])
    ref, tol = chunk_ref.chunk(q, h.k, h.v, [c], window=window)
    v = h.v[0].clone()
    for i, (at, d, x) in enumerate(((n - 1, 0, INF), (n - (c + 1) // 2, 5, -INF), (n - c, 7, NAN), (max(0, n - c - 100), 9, INF),
                                    (0, dim - 1, -INF), (3, dim - 2, NAN), (1, 11, INF), (n - 1, 11, -INF), (n // 2, 13, INF),
                                    (n // 2 + 1, 13, INF))):
        v[at, i % kv_heads, d] = x
    h.write(0, h.k[0], v)
    check(run(h, q, [c], window=window), ref, tol, lost(v, n, c, heads, window))


@both
@form
@pytest.mark.parametrize("how", ["far below", "minus infinity"])
def test_infinite_values_of_keys_without_weight(how, heads, kv_heads, dim, n, c, dtype):
    """An infinite value reaches the rows that see its key, wherever its tile lies and however small the key's weight is: it is
    not 0 times infinity."""
    h = Held(dim, 1, kv_heads, 16, dim, [n], TYPES[dtype])
    q = normal(7, c, heads, dim, dtype=TYPES[dtype]).abs() + 0.5
    k, v = h.k[0].clone() * 0.25, h.v[0].clone()
    tokens = sorted({0, 5, n // 2, max(0, n - c - 70), max(0, n - c - 3), n - (c + 1) // 2} - {n - 1})
    for i, at in enumerate(tokens):
        k[at] = -60.0 if how == "far below" else -INF      # scores of -240 and less
        v[at, :, 8 * (i % 2):8 * (i % 2) + 4] = -INF if i % 3 == 2 else INF
    h.write(0, k, v)
    live = torch.ones(n, dtype=torch.bool)
    live[tokens] = False
    seen = seen_by(n, c, 0)
    gone = lost(v, n, c, heads, 0)
    ref, tol = torch.zeros(c, heads, dim, dtype=torch.float64), torch.zeros(c, heads, dim, dtype=torch.float64)
    hi = seen[:, live].sum(1)                              # of the keys that have a weight, how many each row sees
    for i in range(heads):
        g = i // (heads // kv_heads)
        ref[:, i], tol[:, i] = chunk_ref.rows(q[:, i].cpu().double(), k[live, g].double(), v[live, g].double(),
                                              torch.zeros_like(hi), hi, hi, dim ** -0.5, 0.0, 0.0, TYPES[dtype])
    rows = hi > 0                                          # a row of nothing but such keys has their values, or zeros
    check(run(h, q, [c])[rows], ref[rows], tol[rows], gone[rows])


@both
@pytest.mark.parametrize("c", [1, 60])
def test_nan_scores_outweigh_infinite_values(c, dtype):
    """NaN scores make a row NaN in all its dimensions, whatever its values are."""
    n, heads, dim = 700, 4, 64
    h = Held(dim, 1, 2, 16, dim, [n], TYPES[dtype])
    q = normal(7, c, heads, dim, dtype=TYPES[dtype])
    k, v = h.k[0].clone(), h.v[0].clone()
    k[100, :, 3], v[200, :, 9] = NAN, INF
    h.write(0, k, v)
    assert torch.isnan(run(h, q, [c])).all()
