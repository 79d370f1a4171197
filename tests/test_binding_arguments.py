"""Arguments that the binding refuses, on the host: tensors that say they lie on GPU 0, and a library that only writes down
what it is called with."""
import pytest

torch = pytest.importorskip("torch")

from test_binding_gpus import Spy, ints, pi  # noqa: E402, F401


@pytest.fixture
def spy(pi, monkeypatch):  # noqa: F811
    s = Spy(pi.lib(), [0])
    monkeypatch.setattr(pi, "_lib", s)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(pi, "_mark", lambda dev: None)
    monkeypatch.setattr(pi, "_capturing", lambda *a: False)
    return s


def refused(pi, spy, call, what=""):  # noqa: F811
    with pytest.raises(pi.PiError) as e:
        call()
    assert e.value.status == pi.PI_EINVAL and what in str(e.value)
    assert spy.calls == []


def test_workspace_of_a_decoding_step(pi, spy):  # noqa: F811
    """Its bytes have to be there: elements that repeat, or lie apart, are no memory of their number's size."""
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    n = int(pi.lib().pi_attn_workspace_bytes(c._ref, 3, 4))
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(n), torch.zeros(2 * n, dtype=torch.uint8)[::2],
               torch.zeros(64, n // 64, dtype=torch.uint8).t()):
        refused(pi, spy, lambda: pi.attn_decode(c, 0, q, q.clone(), ws=ws))
    pi.attn_decode(c, 0, q, q.clone(), ws=torch.zeros(n, dtype=torch.uint8))
    pi.attn_decode(c, 0, q, q.clone(), ws=torch.zeros(n // 4, dtype=torch.float32))
    assert [name for name, _, _ in spy.calls] == ["pi_attn_decode"] * 2


def test_tensors_that_want_a_gradient(pi, spy):  # noqa: F811
    """The outputs would carry none, without a word."""
    def t(*shape, dtype=torch.float16):
        return torch.zeros(*shape, dtype=dtype)
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    c.reserve(3, 4)
    mat = pi.Q4Matrix(torch.zeros(64, 32, dtype=torch.uint8), t(64, 2), batch=2)
    calls = {
        "attn_prompt": (lambda q, k, v, o: pi.attn_prompt(q, k, v, o, ints(0, 3)), [t(3, 4, 64), t(3, 2, 64), t(3, 2, 64), t(3, 4, 64)]),
        "attn_decode": (lambda q, o: pi.attn_decode(c, 0, q, o), [t(3, 4, 64), t(3, 4, 64)]),
        "append": (lambda k, v: c.append(0, k, v, ints(0, 3), ints(0)), [t(3, 2, 64), t(3, 2, 64)]),
        "matvec": (lambda x, y: pi.matvec(mat, x, y), [t(2, 64), t(2, 64)]),
    }
    for name, (call, args) in calls.items():
        for a in args:
            a.requires_grad_()
            refused(pi, spy, lambda: call(*args), "gradient")
            with torch.no_grad():
                call(*args)
            spy.calls.clear()
            a.requires_grad_(False)
        call(*args)
        spy.calls.clear()


def test_tensors_of_heads_are_handed_over_as_their_structure(pi):  # noqa: F811
    import ctypes
    t = torch.zeros(5, 3, 64, dtype=torch.float16)
    for x in (t, t[:, 1:], t.transpose(0, 1), t[:1], t[:, :1], t[:0]):
        raw = pi._heads(x, x.shape, "")
        assert len(raw) == ctypes.sizeof(pi.PiHeads)
        got = pi.PiHeads.from_buffer_copy(raw)
        want = (x.data_ptr() or None, x.stride(0) if x.shape[0] > 1 else 0, x.stride(1) if x.shape[1] > 1 else 0)
        assert (got.p, got.token_stride, got.head_stride) == want


def test_sizes_of_a_workspace_that_cannot_be(pi, spy):  # noqa: F811
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    for _ in range(2):                                 # without a buffer, and with one
        for batch, heads in ((0, 4), (-1, 4), (2, 0), (2, 5), (5000, 4)):
            with pytest.raises(pi.PiError):
                c.reserve(batch, heads)
            with pytest.raises(pi.PiError):
                c.attn_workspace(batch, heads)
        c.reserve(3, 4)
        assert c.attn_workspace(2, 4) is c.attn_workspace(3, 4)
