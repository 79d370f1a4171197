"""What rotary positions, the append that turns keys, and attention of chunks refuse, on the host: through the C ABI with
addresses that are never followed, and through the binding.  Every call returns before anything is enqueued, so no GPU is
needed.  The frequencies' rules and steps are computed on the host and checked here too."""
import ctypes
import math
import os
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

import chunk_ref  # noqa: E402

FAKE = 1 << 20                                         # 256-byte aligned, never dereferenced
EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
NAN, INF = float("nan"), float("inf")


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
    return ctypes.byref(pi.PiHeads(p, token, head))


def rope(pi, steps=FAKE, rotary=64, layout=0, magnitude=1.0):
    return ctypes.byref(pi.PiRope(steps, rotary, layout, magnitude))


BAD_ROPES = [dict(steps=None), dict(steps=FAKE + 8), dict(rotary=0), dict(rotary=-2), dict(rotary=7), dict(rotary=66),
             dict(layout=2), dict(layout=-1), dict(magnitude=-1.0), dict(magnitude=NAN), dict(magnitude=INF)]
BAD_HEADS = [dict(p=None), dict(p=FAKE + 8), dict(token=4), dict(head=12)]


def rope_heads(pi, **kw):
    h = heads(pi)
    a = dict(rope=rope(pi), pos=FAKE, q=h, q_out=h, heads=4, q_norm=None, k=h, k_out=h, kv_heads=2, k_norm=None, eps=1e-6,
             tokens=5, dim=64, dtype=pi.PI_F16)
    a.update(kw)
    return pi.lib().pi_rope_heads(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(pos=None), EINVAL), (dict(pos=FAKE + 2), EINVAL), (dict(q=None), EINVAL), (dict(q_out=None), EINVAL),
    (dict(heads=0), EINVAL), (dict(heads=-1), EINVAL), (dict(heads=4097), EUNSUPPORTED), (dict(k=None), EINVAL),
    (dict(k_out=None), EINVAL), (dict(kv_heads=0), EINVAL), (dict(kv_heads=-3), EINVAL), (dict(k=None, k_out=None), EINVAL),
    (dict(kv_heads=4097), EUNSUPPORTED), (dict(q_norm=FAKE + 4), EINVAL), (dict(k_norm=FAKE + 8), EINVAL),
    (dict(q_norm=FAKE, eps=0.0), EINVAL), (dict(k_norm=FAKE, eps=-1.0), EINVAL), (dict(q_norm=FAKE, eps=NAN), EINVAL),
    (dict(q_norm=FAKE, eps=INF), EINVAL), (dict(tokens=-1), EINVAL), (dict(dim=0), EINVAL), (dict(dim=60), EINVAL),
    (dict(dim=264), EUNSUPPORTED), (dict(dtype=0), EUNSUPPORTED), (dict(dtype=2), EINVAL), (dict(dtype=9), EINVAL),
    (dict(dim=32), EINVAL),                            # more turn than there are
])
def test_rope_arguments(pi, kw, status):
    assert rope_heads(pi, **kw) == status


@pytest.mark.parametrize("kw", BAD_ROPES)
def test_ropes(pi, kw):
    c, h = ctypes.byref(cache(pi)), heads(pi)
    assert rope_heads(pi, rope=rope(pi, **kw)) == EINVAL
    assert pi.lib().pi_cache_append_rope(c, 0, rope(pi, **kw), h, h, 4, None, h, h, None, 1e-6, 5, FAKE, FAKE, 1, None) == EINVAL


@pytest.mark.parametrize("kw", BAD_HEADS)
def test_tensors_of_heads(pi, kw):
    L, c, g, b = pi.lib(), ctypes.byref(cache(pi)), heads(pi), heads(pi, **kw)
    for name in ("q", "q_out", "k", "k_out"):
        assert rope_heads(pi, **{name: b}) == EINVAL
    for at in range(4):
        four = [g] * 4
        four[at] = b
        assert L.pi_cache_append_rope(c, 0, rope(pi), four[0], four[1], 4, None, four[2], four[3], None, 1e-6, 5, FAKE, FAKE, 1,
                                      None) == EINVAL
    big = 1 << 40
    assert L.pi_attn_chunk(c, 0, b, g, 5, 4, FAKE, None, 1, 0.0, 0.0, None, 0, FAKE, big, None) == EINVAL
    assert L.pi_attn_chunk(c, 0, g, b, 5, 4, FAKE, None, 1, 0.0, 0.0, None, 0, FAKE, big, None) == EINVAL


@pytest.mark.parametrize("kw", [dict(token=0), dict(token=32), dict(head=0), dict(token=64, head=64), dict(token=-32, head=1024)])
def test_outputs_whose_rows_lie_over_each_other(pi, kw):
    L, c, g, b, big = pi.lib(), ctypes.byref(cache(pi)), heads(pi), heads(pi, **kw), 1 << 40
    assert rope_heads(pi, q_out=b) == EINVAL and rope_heads(pi, k_out=b) == EINVAL
    assert L.pi_cache_append_rope(c, 0, rope(pi), g, b, 4, None, g, g, None, 1e-6, 5, FAKE, FAKE, 1, None) == EINVAL
    assert L.pi_attn_chunk(c, 0, g, b, 5, 4, FAKE, None, 1, 0.0, 0.0, None, 0, FAKE, big, None) == EINVAL


def test_rope_of_no_tokens_enqueues_nothing(pi):
    h = heads(pi, p=None)
    assert rope_heads(pi, tokens=0, q=h, q_out=h, k=h, k_out=h, pos=None) == 0
    assert rope_heads(pi, tokens=0, rope=None, pos=None, k=None, k_out=None, kv_heads=0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), EINVAL), (dict(layer=2), EINVAL), (dict(q=None), EINVAL), (dict(q_out=None), EINVAL), (dict(heads=0), EINVAL),
    (dict(heads=-1), EINVAL), (dict(heads=4097), EUNSUPPORTED), (dict(q=None, q_out=None), EINVAL), (dict(k=None), EINVAL),
    (dict(v=None), EINVAL), (dict(q_norm=FAKE + 4), EINVAL), (dict(k_norm=FAKE + 4), EINVAL), (dict(k_norm=FAKE, eps=0.0), EINVAL),
    (dict(tokens=-1), EINVAL), (dict(cu=None), EINVAL), (dict(cu=FAKE + 2), EINVAL), (dict(seqs=None), EINVAL),
    (dict(seqs=FAKE + 2), EINVAL), (dict(n=0), EINVAL), (dict(tokens=0), 0), (dict(tokens=0, q=None, q_out=None, heads=0), 0),
])
def test_append_arguments(pi, kw, status):
    h = heads(pi)
    a = dict(layer=0, rope=rope(pi), q=h, q_out=h, heads=4, q_norm=None, k=h, v=h, k_norm=None, eps=1e-6, tokens=5, cu=FAKE,
             seqs=FAKE, n=1)
    a.update(kw)
    assert pi.lib().pi_cache_append_rope(ctypes.byref(cache(pi)), *a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), EINVAL), (dict(layer=2), EINVAL), (dict(tokens=-1), EINVAL), (dict(heads=0), EINVAL), (dict(heads=5), EINVAL),
    (dict(heads=4098), EUNSUPPORTED), (dict(cu=None), EINVAL), (dict(cu=FAKE + 1), EINVAL), (dict(seqs=FAKE + 2), EINVAL),
    (dict(n=0), EINVAL), (dict(n=5), EINVAL), (dict(n=4097, seqs=FAKE), EUNSUPPORTED), (dict(scale=-0.5), EINVAL),
    (dict(scale=NAN), EINVAL), (dict(scale=INF), EINVAL), (dict(cap=-1.0), EINVAL), (dict(cap=NAN), EINVAL),
    (dict(cap=INF), EUNSUPPORTED), (dict(cap=1025.0), EUNSUPPORTED), (dict(cap=1e-38), EINVAL), (dict(slopes=FAKE + 2), EINVAL),
    (dict(window=-1), EINVAL), (dict(tokens=(1 << 31) - 1), EUNSUPPORTED), (dict(ws=None), EWORKSPACE),
    (dict(ws=FAKE + 128), EWORKSPACE), (dict(short=1), EWORKSPACE), (dict(tokens=0), 0),
])
def test_chunk_arguments(pi, kw, status):
    L, c, h = pi.lib(), ctypes.byref(cache(pi)), heads(pi)
    a = dict(layer=0, tokens=5, heads=4, cu=FAKE, seqs=None, n=3, scale=0.0, cap=0.0, slopes=None, window=0, ws=FAKE, short=0)
    a.update(kw)
    size = L.pi_attn_chunk_workspace_bytes(c, a["tokens"], a["heads"], a["n"]) - a["short"]
    assert L.pi_attn_chunk(c, a["layer"], h, h, a["tokens"], a["heads"], a["cu"], a["seqs"], a["n"], a["scale"], a["cap"],
                           a["slopes"], a["window"], a["ws"], max(size, 0), None) == status


BAD_CACHES = [(dict(k=None), EINVAL), (dict(meta=FAKE + 2), EINVAL), (dict(page=24), EINVAL), (dict(dim=20), EINVAL),
              (dict(slots=0), EINVAL), (dict(dtype=0), EUNSUPPORTED), (dict(dtype=9), EINVAL), (dict(dim=264), EUNSUPPORTED),
              (dict(max_pages=1 << 27), EUNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(pi, kw, status):
    L, c, h, big = pi.lib(), ctypes.byref(cache(pi, **kw)), heads(pi), 1 << 40
    assert L.pi_cache_append_rope(c, 0, None, None, None, 0, None, h, h, None, 1e-6, 1, FAKE, FAKE, 1, None) == status
    assert L.pi_attn_chunk_workspace_bytes(c, 1, 4, 1) == 0
    assert L.pi_attn_chunk(c, 0, h, h, 1, 4, FAKE, None, 1, 0.0, 0.0, None, 0, FAKE, big, None) == status
    assert L.pi_attn_chunk_workspace_bytes(None, 1, 4, 1) == 0


def test_workspace_never_shrinks(pi):
    """Room for more rows or chunks is room for fewer."""
    L, c = pi.lib(), ctypes.byref(cache(pi))
    sizes = [[L.pi_attn_chunk_workspace_bytes(c, t, 8, n) for n in (1, 2, 64, 4096)] for t in (0, 1, 7, 8, 9, 31, 32, 33, 5000)]
    assert all(s > 0 for row in sizes for s in row)
    for a, b in zip(sizes, sizes[1:]):
        assert all(x <= y for x, y in zip(a, b))
    assert all(x <= y for row in sizes for x, y in zip(row, row[1:]))


# ------------------------------------------------------------- frequencies
RULES = [(None, {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
         ("bands", dict(factor=8.0, trained=8192, low=1.0, high=4.0)), ("bands", dict(factor=2.5, trained=100, low=0.5, high=32.0)),
         ("ramp", dict(factor=16.0, trained=4096)), ("ramp", dict(factor=40.0, trained=4096, low=1.0, high=32.0)),
         ("ramp", dict(factor=2.0, trained=8, low=1.0, high=32.0)), ("ramp", dict(factor=2.0, trained=1e9))]


@pytest.mark.parametrize("rotary", [4, 30, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
@pytest.mark.parametrize("rule,kw", RULES)
def test_rules(pi, rule, kw, base, rotary):
    r = pi.Rope(rotary, base, scaling=rule, device="cpu", **kw)
    want, mag = chunk_ref.frequencies(rotary, base, rule, **{"high": 32.0, **kw})
    # a few operations and a power in double precision, whose exponent of up to 2^5 nats carries 2^-53 along
    assert all(abs(a - b) <= 2.0 ** -45 * b for a, b in zip(r.freqs, want)), (r.freqs, want)
    assert r.magnitude == pytest.approx(mag, rel=2.0 ** -24)


def test_steps(pi):
    """freq / (2 pi) turns in units of 2^-64, modulo 2^64."""
    pi_ = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    freqs = [1.0, 0.5, 1e-9, 2.0 ** -60, 0.0, 6.5, 1234.5, -0.25, -7.0, 3.0e5] + [10000.0 ** (-i / 37) for i in range(37)]
    freqs.append(0.125)
    r = pi.Rope(2 * len(freqs), freqs=freqs, device="cpu")
    for f, got in zip(freqs, r.steps.tolist()):
        exact = Fraction(f) / (2 * pi_) * 2 ** 64
        off = (Fraction(got) - exact) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # the quotient is rounded to 64 bits, which for more than a turn takes bits from the part of one
        assert off <= 1 + abs(exact) * Fraction(1, 2 ** 62), (f, got, float(off))


@pytest.mark.parametrize("kw", [dict(base=1.0), dict(base=0.5), dict(base=NAN), dict(base=INF), dict(rule=-1), dict(rule=5),
                                dict(rule=1, factor=0.5), dict(rule=1, factor=NAN), dict(rule=3, trained=0.0),
                                dict(rule=3, low=4.0), dict(rule=3, low=0.0), dict(rule=4, high=INF), dict(rule=4, trained=NAN),
                                dict(rotary=0), dict(rotary=3), dict(rotary=258), dict(rule=2, rotary=2)])
def test_rules_that_cannot_be(pi, kw):
    a = dict(base=10000.0, factor=2.0, trained=4096.0, low=1.0, high=4.0, rule=0, rotary=64)
    a.update(kw)
    out = (ctypes.c_double * 200)()
    s = pi.PiRopeScaling(a["base"], a["factor"], a["trained"], a["low"], a["high"], a["rule"])
    assert pi.lib().pi_rope_freqs(ctypes.byref(s), a["rotary"], out, None) == EINVAL
    assert pi.lib().pi_rope_freqs(None, 64, out, None) == EINVAL


def test_steps_that_cannot_be(pi):
    L, one, out = pi.lib(), (ctypes.c_double * 1)(1.0), (ctypes.c_uint64 * 1)()
    assert L.pi_rope_steps(one, 1, out) == 0
    assert L.pi_rope_steps(None, 1, out) == EINVAL and L.pi_rope_steps(one, 1, None) == EINVAL
    assert L.pi_rope_steps(one, 0, out) == EINVAL
    for bad in (NAN, INF, -INF):
        assert L.pi_rope_steps((ctypes.c_double * 1)(bad), 1, out) == EINVAL


# ------------------------------------------------------------------ the binding
def refused(pi, call):
    with pytest.raises(pi.PiError) as e:
        call()
    assert e.value.status == EINVAL


def test_binding_refuses(pi):
    r = pi.Rope(64, device="cpu")
    q, k = torch.zeros(5, 4, 64, dtype=torch.float16), torch.zeros(5, 2, 64, dtype=torch.float16)
    pos, w = torch.zeros(5, dtype=torch.int32), torch.ones(64)
    good = dict(rope=r, pos=pos, q=q, q_out=q, k=k, k_out=k)
    for bad in (dict(), dict(q=q[0]), dict(q_out=q[:4]), dict(q=q.float(), q_out=q.float()), dict(k=None), dict(k_out=None),
                dict(k=k[:, :, :32], k_out=k[:, :, :32]), dict(k=k.to(torch.bfloat16), k_out=k.to(torch.bfloat16)), dict(pos=None),
                dict(pos=pos[:4]), dict(pos=pos.long()), dict(q_norm=w[:32]), dict(q_norm=w.half()), dict(k_norm=w.view(1, 64))):
        refused(pi, lambda: pi.rope_heads(**{**good, **bad}))   # the first: tensors of the host
    for bad in (dict(layout="other"), dict(scaling="other"), dict(rotary=0), dict(rotary=31), dict(rotary=300),
                dict(magnitude=0.0), dict(magnitude=NAN), dict(freqs=[1.0]), dict(freqs=[NAN] * 32),
                dict(freqs=[1.0] * 32, scaling="linear", factor=2.0), dict(base=0.0), dict(scaling="bands")):
        refused(pi, lambda: pi.Rope(**{"rotary": 64, "device": "cpu", **bad}))
    assert math.isclose(pi.Rope(64, magnitude=2.0, device="cpu").magnitude, 2.0)
