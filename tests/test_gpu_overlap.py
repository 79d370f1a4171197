"""Inputs and outputs that share a buffer without lying over each other."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import activation_sparse_predict_amd as pi  # noqa: E402
import attn_ref  # noqa: E402
from test_gpu_attention import held_by, ints, make_cache, normal  # noqa: E402
from test_gpu_matvec import DEV, check, matrix  # noqa: E402


@pytest.mark.parametrize("batch", [1, 3, 20])
def test_matvec_columns_of_one_buffer(batch):
    rows, cols = 96, 256
    q, sc = matrix(1, rows, cols)
    mat = pi.Q4Matrix(q.to(DEV), sc.to(DEV), batch=batch)
    buf = torch.randn(batch, cols + rows, device=DEV)
    x = buf[:, :cols].clone()
    pi.matvec(mat, buf[:, :cols], buf[:, cols:])
    check(q, sc, None, x, buf[:, cols:])
    buf = torch.randn(2 * batch, cols, device=DEV)     # rows one after the other
    x = buf[:batch].clone()
    pi.matvec(mat, buf[:batch], buf[batch:, :rows])
    check(q, sc, None, x, buf[batch:, :rows])


def test_attention_in_place_of_the_queries():
    t, h, g, d = 300, 8, 2, 64
    qkv = normal(3, t, h + 2 * g, d, dtype=torch.float16)
    q, k, v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
    ref = attn_ref.prompt(q, k, v, [211, 89])
    pi.attn_prompt(q, k, v, q, ints([0, 211, 300]))
    attn_ref.check(q, *ref)


@pytest.mark.parametrize("prefix", [None, 5])
def test_decode_in_place_of_the_queries(prefix):
    lens = [90, 3001, 81, 0, 700]
    cache = make_cache(51, "bf16", 2, 64, 16, lens, shared=5)
    q = normal(4, 5, 40, 64, dtype=torch.bfloat16)
    ks, vs = held_by(cache, 1)
    ref = attn_ref.decode(q, ks, vs)
    pi.attn_decode(cache, 1, q, q, prefix=None if prefix is None else ints([prefix]))
    attn_ref.check(q, *ref)


@pytest.mark.parametrize("tokens,heads,token,head", [(2, 3, 40, 24), (3, 2, 24, 40), (1, 4, 0, 8), (5, 1, 8, 0), (4, 3, 24, 8),
                                                     (4, 3, 8, 32)])
def test_outputs_between_each_others_rows(tokens, heads, token, head):
    """Rows of 8, in any order of strides, that do not meet."""
    q, k, v = (normal(i, tokens, n, 8, dtype=torch.float16) for i, n in ((0, heads), (1, heads), (2, heads)))
    size = (tokens - 1) * token + (heads - 1) * head + 8
    out = torch.zeros(size, dtype=torch.float16, device=DEV).as_strided((tokens, heads, 8), (token, head, 1))
    pi.attn_prompt(q, k, v, out, ints([0, tokens]))
    attn_ref.check(out, *attn_ref.prompt(q, k, v, [tokens]))
