"""What the attention half's entry points refuse, on the host: through the C ABI with addresses that are never
followed, and through the binding.  Every call returns before anything is enqueued, so no GPU is needed."""
import ctypes
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20                                         # 256-byte aligned, never dereferenced
EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def pi():
    import activation_sparse_predict_amd as pi
    if not os.path.exists(pi.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build_library()
    pi.lib()
    return pi


def cache(pi, **kw):
    base = dict(k=FAKE, v=FAKE, meta=FAKE, layers=2, pages=100, kv_heads=2, page=16, dim=64, dtype=pi.PI_F16, slots=4,
                max_pages=10)
    base.update(kw)
    return pi.PiCache(*(base[f] for f, _ in pi.PiCache._fields_))


def heads(pi, p=FAKE, token=512, head=64):
    return pi.PiHeads(p, token, head)


BAD_CACHES = [(dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(meta=None), EINVAL), (dict(k=FAKE + 8), EINVAL),
              (dict(v=FAKE + 2), EINVAL), (dict(meta=FAKE + 2), EINVAL), (dict(layers=0), EINVAL), (dict(pages=0), EINVAL),
              (dict(kv_heads=0), EINVAL), (dict(page=0), EINVAL), (dict(page=24), EINVAL), (dict(dim=0), EINVAL),
              (dict(dim=20), EINVAL), (dict(slots=0), EINVAL), (dict(max_pages=0), EINVAL), (dict(slots=-1), EINVAL),
              (dict(dtype=0), EUNSUPPORTED), (dict(dtype=2), EINVAL), (dict(dtype=9), EINVAL),
              (dict(dim=264), EUNSUPPORTED), (dict(page=4112), EUNSUPPORTED), (dict(kv_heads=1025), EUNSUPPORTED),
              (dict(pages=(1 << 20) + 1), EUNSUPPORTED), (dict(layers=16385), EUNSUPPORTED),
              (dict(max_pages=1 << 27), EUNSUPPORTED), (dict(max_pages=1 << 20, slots=1025), EUNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(pi, kw, status):
    L, c, h = pi.lib(), ctypes.byref(cache(pi, **kw)), ctypes.byref(heads(pi))
    big = 1 << 40
    assert L.pi_cache_workspace_bytes(c) == 0
    assert L.pi_cache_extend(c, FAKE, FAKE, 1, None) == status
    assert L.pi_cache_append(c, 0, h, h, 1, FAKE, FAKE, 1, None) == status
    assert L.pi_cache_fork(c, FAKE, FAKE, 1, FAKE, big, None) == status
    assert L.pi_cache_release(c, FAKE, 1, None) == status
    assert L.pi_cache_compact(c, None, FAKE, big, None) == status
    assert L.pi_attn_workspace_bytes(c, 1, 4) == 0
    assert L.pi_attn_decode(c, 0, h, h, 1, 4, None, None, 0.0, FAKE, big, None) == status


def test_no_cache_at_all(pi):
    L = pi.lib()
    assert L.pi_cache_extend(None, FAKE, FAKE, 1, None) == EINVAL
    assert L.pi_cache_workspace_bytes(None) == 0 and L.pi_attn_workspace_bytes(None, 1, 4) == 0


def test_meta_words(pi):
    L = pi.lib()
    assert L.pi_cache_meta_words(3, 5, 7) == 15 + 3 + 14 + 4
    assert L.pi_cache_meta_words(4096, 1 << 18, 1 << 20) == (1 << 30) + 4096 + (1 << 21) + 4
    for bad in ((0, 5, 7), (3, 0, 7), (3, 5, 0), (-1, 5, 7)):
        assert L.pi_cache_meta_words(*bad) == 0


def test_lists_of_slots(pi):
    L, c, big = pi.lib(), ctypes.byref(cache(pi)), 1 << 40
    for a, n, status in ((None, 1, EINVAL), (FAKE + 2, 1, EINVAL), (FAKE, 0, EINVAL), (FAKE, -1, EINVAL),
                         (FAKE, 4097, EUNSUPPORTED)):
        assert L.pi_cache_extend(c, a, FAKE, n, None) == status
        assert L.pi_cache_extend(c, FAKE, a, n, None) == status
        assert L.pi_cache_release(c, a, n, None) == status
        assert L.pi_cache_fork(c, a, FAKE, n, FAKE, big, None) == status
        assert L.pi_cache_fork(c, FAKE, a, n, FAKE, big, None) == status
    h = ctypes.byref(heads(pi))
    for layer, tokens, cu, seqs, n in ((-1, 1, FAKE, FAKE, 1), (2, 1, FAKE, FAKE, 1), (0, -1, FAKE, FAKE, 1),
                                       (0, 1, None, FAKE, 1), (0, 1, FAKE + 1, FAKE, 1), (0, 1, FAKE, None, 1),
                                       (0, 1, FAKE, FAKE + 2, 1), (0, 1, FAKE, FAKE, 0)):
        assert L.pi_cache_append(c, layer, h, h, tokens, cu, seqs, n, None) == EINVAL
    assert L.pi_cache_append(c, 0, h, h, 0, FAKE, FAKE, 1, None) == 0      # nothing to write: nothing is enqueued


BAD_HEADS = [dict(p=None), dict(p=FAKE + 8), dict(token=4), dict(head=12)]


@pytest.mark.parametrize("kw", BAD_HEADS)
def test_tensors_of_heads(pi, kw):
    L, good, bad = pi.lib(), heads(pi), heads(pi, **kw)
    c, G, B, big = ctypes.byref(cache(pi)), ctypes.byref(good), ctypes.byref(bad), 1 << 40
    assert L.pi_cache_append(c, 0, B, G, 5, FAKE, FAKE, 1, None) == EINVAL
    assert L.pi_cache_append(c, 0, G, B, 5, FAKE, FAKE, 1, None) == EINVAL
    assert L.pi_cache_append(c, 0, None, G, 5, FAKE, FAKE, 1, None) == EINVAL
    assert L.pi_attn_decode(c, 0, B, G, 1, 4, None, None, 0.0, FAKE, big, None) == EINVAL
    assert L.pi_attn_decode(c, 0, G, B, 1, 4, None, None, 0.0, FAKE, big, None) == EINVAL
    for i in range(4):
        four = [G] * 4
        four[i] = B
        assert L.pi_attn_prompt(*four, 5, 4, 2, 64, pi.PI_F16, FAKE, 1, 0.0, None) == EINVAL
        four[i] = None
        assert L.pi_attn_prompt(*four, 5, 4, 2, 64, pi.PI_F16, FAKE, 1, 0.0, None) == EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), EINVAL), (dict(kv_heads=0), EINVAL), (dict(heads=5), EINVAL), (dict(dim=0), EINVAL),
    (dict(dim=12), EINVAL), (dict(dim=264), EUNSUPPORTED), (dict(heads=4098), EUNSUPPORTED), (dict(dtype=0), EUNSUPPORTED),
    (dict(dtype=2), EINVAL), (dict(dtype=7), EINVAL), (dict(tokens=-1), EINVAL), (dict(n=0), EINVAL), (dict(cu=None), EINVAL),
    (dict(cu=FAKE + 1), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(scale=3e38), EINVAL),
    (dict(tokens=(1 << 31) - 1, heads=4096, kv_heads=4096), EUNSUPPORTED),
])
def test_prompt_arguments(pi, kw, status):
    a = dict(tokens=5, heads=4, kv_heads=2, dim=64, dtype=pi.PI_F16, cu=FAKE, n=1, scale=0.0)
    a.update(kw)
    h = ctypes.byref(heads(pi))
    assert pi.lib().pi_attn_prompt(h, h, h, h, a["tokens"], a["heads"], a["kv_heads"], a["dim"], a["dtype"], a["cu"], a["n"],
                                   a["scale"], None) == status


@pytest.mark.parametrize("token", [(1 << 24) + 8, -8])
def test_prompt_strides_of_keys_and_values(pi, token):
    good, bad = ctypes.byref(heads(pi)), ctypes.byref(heads(pi, token=token))
    for k, v in ((bad, good), (good, bad)):
        assert pi.lib().pi_attn_prompt(good, k, v, good, 5, 4, 2, 64, pi.PI_F16, FAKE, 1, 0.0, None) == EUNSUPPORTED


def test_prompt_of_no_tokens_enqueues_nothing(pi):
    h = ctypes.byref(heads(pi, p=None))
    assert pi.lib().pi_attn_prompt(h, h, h, h, 0, 4, 2, 64, pi.PI_BF16, FAKE, 3, 0.0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), EINVAL), (dict(layer=2), EINVAL), (dict(batch=0), EINVAL), (dict(batch=5), EINVAL),
    (dict(batch=4097, seqs=FAKE), EUNSUPPORTED), (dict(heads=0), EINVAL), (dict(heads=5), EINVAL),
    (dict(heads=4098), EUNSUPPORTED), (dict(seqs=FAKE + 2), EINVAL), (dict(prefix=FAKE + 1), EINVAL),
    (dict(scale=-0.5), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(ws=None), EWORKSPACE),
    (dict(ws=FAKE + 128), EWORKSPACE), (dict(short=1), EWORKSPACE),
])
def test_decode_arguments(pi, kw, status):
    L, c, h = pi.lib(), ctypes.byref(cache(pi)), ctypes.byref(heads(pi))
    a = dict(layer=0, batch=3, heads=4, seqs=None, prefix=None, scale=0.0, ws=FAKE, short=0)
    a.update(kw)
    n = L.pi_attn_workspace_bytes(c, a["batch"], a["heads"])
    assert (n > 0 and n % 256 == 0) or status in (EINVAL, EUNSUPPORTED)
    assert L.pi_attn_decode(c, a["layer"], h, h, a["batch"], a["heads"], a["seqs"], a["prefix"], a["scale"], a["ws"],
                            n - a["short"] if n else 1 << 40, None) == status


def test_cache_workspaces(pi):
    L, c = pi.lib(), ctypes.byref(cache(pi))
    n = L.pi_cache_workspace_bytes(c)
    assert n > 0 and n % 256 == 0
    for ws, size in ((None, n), (FAKE + 64, n), (FAKE, n - 1)):
        assert L.pi_cache_fork(c, FAKE, FAKE, 1, ws, size, None) == EWORKSPACE
        assert L.pi_cache_compact(c, None, ws, size, None) == EWORKSPACE
    assert L.pi_cache_compact(c, FAKE + 2, FAKE, n, None) == EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), EINVAL), (dict(cols=0), EINVAL), (dict(cols=48), EINVAL), (dict(batch=0), EINVAL), (dict(batch=33), EINVAL),
    (dict(rows=(1 << 28) + 1, ldy=1 << 40), EUNSUPPORTED), (dict(cols=(1 << 22) + 32, ldx=1 << 40), EUNSUPPORTED),
    (dict(w=None), EINVAL), (dict(w=FAKE + 8), EINVAL), (dict(scale=None), EINVAL), (dict(scale=FAKE + 1), EINVAL),
    (dict(bias=FAKE + 2), EINVAL), (dict(x=None), EINVAL), (dict(x=FAKE + 2), EINVAL), (dict(x=FAKE + 1, xt=1), EINVAL),
    (dict(y=None), EINVAL), (dict(y=FAKE + 2), EINVAL), (dict(y=FAKE + 1, yt=3), EINVAL), (dict(xt=2), EINVAL),
    (dict(xt=4), EINVAL), (dict(yt=2), EINVAL), (dict(yt=-1), EINVAL), (dict(ldx=127), EINVAL), (dict(ldy=99), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(ws=FAKE + 16), EWORKSPACE), (dict(short=1), EWORKSPACE),
])
def test_matvec_arguments(pi, kw, status):
    L = pi.lib()
    a = dict(rows=100, cols=128, batch=2, w=FAKE, scale=FAKE, bias=None, x=FAKE, xt=0, ldx=128, y=FAKE, yt=0, ldy=100, ws=FAKE,
             short=0)
    a.update(kw)
    m = pi.PiMat(a["w"], a["scale"])
    n = L.pi_matvec_workspace_bytes(a["rows"], a["cols"], a["batch"])
    assert (n > 0) == (not any(k in kw for k in ("rows", "cols", "batch")))
    assert L.pi_matvec(ctypes.byref(m), a["rows"], a["cols"], a["bias"], a["x"], a["xt"], a["ldx"], a["y"], a["yt"], a["ldy"],
                       a["batch"], a["ws"], n - a["short"] if n else 1 << 40, None) == status


def test_matvec_without_a_matrix(pi):
    assert pi.lib().pi_matvec(None, 16, 32, None, FAKE, 0, 32, FAKE, 0, 16, 1, FAKE, 1 << 30, None) == EINVAL


def test_structures_match_the_header(pi, tmp_path):
    fields = {"pi_heads": pi.PiHeads, "pi_cache": pi.PiCache}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "pi.h"', "int main(void) {"]
    for st, cls in fields.items():
        lines.append(f'  printf("{st} %zu\\n", sizeof({st}));')
        lines += [f'  printf("{st}.{f} %zu\\n", offsetof({st}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o",
                    str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout
    got = dict(line.rsplit(" ", 1) for line in out.splitlines())
    for st, cls in fields.items():
        assert int(got[st]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{st}.{f}"]) == getattr(cls, f).offset
    with open(os.path.join(ROOT, "include", "pi.h")) as fh:
        header = fh.read()
    for name in ("PI_CACHE_ESLOT", "PI_CACHE_EPAGE", "PI_CACHE_EFULL", "PI_CACHE_ELENGTH"):
        assert int(re.search(rf"#define {name} (\d+)", header).group(1)) == getattr(pi, name)


# ------------------------------------------------------------------ the binding
def refuses(pi, call, status=EINVAL):
    with pytest.raises(pi.PiError) as e:
        call()
    assert e.value.status == status


def test_binding_refuses_tensors_of_the_host(pi):
    """A tensor that does not lie on a GPU never reaches a kernel."""
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    refuses(pi, lambda: pi.attn_prompt(q, q, q, q.clone(), cu))
    refuses(pi, lambda: pi.Cache.create(1, 4, 2, 16, 64, 2, 2, device="cpu"))
    refuses(pi, lambda: pi.Q4Matrix(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.float16)))


def test_binding_refuses_shapes_and_types(pi):
    cu = torch.tensor([0, 3], dtype=torch.int32)

    def t(*shape, dtype=torch.float16):
        return torch.zeros(*shape, dtype=dtype)
    q = t(3, 4, 64)
    for bad in ((t(3, 4, 64), t(3, 2, 64), t(3, 1, 64), t(3, 4, 64)), (q, t(2, 2, 64), t(2, 2, 64), q),
                (q, t(3, 2, 32), t(3, 2, 32), q), (q, q, q, t(3, 4, 32)), (q, q, q, t(3, 4, 64, dtype=torch.bfloat16)),
                (q[0], q[0], q[0], q[0]), (q.transpose(1, 2), q, q, q)):
        refuses(pi, lambda: pi.attn_prompt(*bad, cu))
    for bad in (cu.long(), cu.view(1, 2), cu[:1], torch.zeros(6, dtype=torch.int32)[::2]):
        refuses(pi, lambda: pi.attn_prompt(q, q, q, q.clone(), bad))
    pool = t(1, 4, 2, 16, 64)
    meta = torch.zeros(pi.Cache.meta_words(2, 3, 4), dtype=torch.int32)
    for bad in ((pool, pool[:, :3], meta, 2, 3), (pool, pool.bfloat16(), meta, 2, 3), (pool[0], pool[0], meta, 2, 3),
                (pool, pool, meta[:-1], 2, 3), (pool, pool, meta.float(), 2, 3), (pool, pool, meta, 0, 3),
                (pool.transpose(1, 2), pool.transpose(1, 2), meta, 2, 3), (pool.double(), pool.double(), meta, 2, 3)):
        refuses(pi, lambda: pi.Cache(*bad))
    nib, sc = torch.zeros(4, 32, dtype=torch.uint8), t(4, 2)
    for bad in ((nib.int(), sc), (nib[:, ::2], sc), (nib, sc.float()), (nib, t(4, 3)), (nib, sc, t(4)),
                (nib, sc, t(5, dtype=torch.float32)), (nib, sc, None, 0), (nib, sc, None, 33)):
        refuses(pi, lambda: pi.Q4Matrix(*bad))
