"""Which GPU and stream the binding's calls go to, on the host: tensors that say they lie on GPU 1 while GPU 0 is current,
and a library that only writes down what it is called with."""
import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pi():
    import activation_sparse_predict_amd as pi
    if not os.path.exists(pi.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build_library()
    pi.lib()
    return pi


class Spy:
    """The library, whose calls with a stream are not made: (name, current GPU, stream) goes to `calls` instead."""

    def __init__(self, real, gpus):
        self.real, self.gpus, self.calls = real, gpus, []

    def __getattr__(self, name):
        if "words" in name or "bytes" in name or name in ("pi_status_str", "pi_last_hip_error"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, self.gpus[-1], args[-1]))
            return 0
        return call


STREAMS = {0: 70, 1: 0}                                # the current stream of each GPU; 0 is a default stream


@pytest.fixture
def spy(pi, monkeypatch):
    gpus = [0]                                         # what was made current, in order
    s = Spy(pi.lib(), gpus)
    monkeypatch.setattr(pi, "_lib", s)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: gpus[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_setDevice", gpus.append, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", STREAMS.__getitem__, raising=False)
    monkeypatch.setattr(pi, "_capturing", lambda *a: False, raising=False)
    # events of the workspaces: where they are recorded, and which streams wait for them before which call
    monkeypatch.setattr(pi, "_mark", lambda dev: ("mark", dev), raising=False)
    s.waits = []
    monkeypatch.setattr(pi, "_wait_for", lambda *a: s.waits.append((len(s.calls), *a)) or True, raising=False)
    return s


def ints(*values):
    return torch.tensor(values, dtype=torch.int32)


def calls_of(pi, stream):
    """One call of each operator, name -> function."""
    half = dict(dtype=torch.float16)
    q, kv = torch.zeros(3, 4, 64, **half), torch.zeros(3, 2, 64, **half)
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    mat = pi.Q4Matrix(torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(64, 2, **half), batch=2)
    x = torch.zeros(2, 64)
    ws = torch.zeros(int(pi.lib().pi_attn_workspace_bytes(c._ref, 3, 4)), dtype=torch.uint8)
    layer = pi.DeviceLayer(d=64, ffn=64, rank=64, act="relu", w_dtype="f32", p_dtype="f32", A=x, B=x, bias=x, up=x, downT=x)
    some = torch.zeros(1 << 20, dtype=torch.uint8)
    return {
        "pi_cache_extend": lambda: c.extend(ints(0), ints(3), stream),
        "pi_cache_append": lambda: c.append(0, kv, kv, ints(0, 3), ints(0), stream),
        "pi_cache_fork": lambda: c.fork(ints(0), ints(1), stream),
        "pi_cache_release": lambda: c.release(ints(0), stream),
        "pi_cache_compact": lambda: c.compact(None, stream),
        "pi_attn_prompt": lambda: pi.attn_prompt(q, kv, kv, q.clone(), ints(0, 3), stream=stream),
        "pi_attn_decode": lambda: pi.attn_decode(c, 0, q, q.clone(), ws=ws, stream=stream),
        "pi_matvec": lambda: pi.matvec(mat, x, x.clone(), stream=stream),
        "pi_predict": lambda: pi.predict(layer, x, x, x, ws=some, stream=stream),
        "pi_sparse_ffn": lambda: pi.sparse_ffn(layer, x, x, x, x, ws=some, stream=stream),
        "pi_ffn_stack": lambda: pi.ffn_stack([layer], x, x, ws=some, stream=stream),
        "pi_ffn_stack_static": lambda: pi.ffn_stack_static([layer], x, x, stream=stream),
    }


def test_calls_go_to_the_gpu_of_their_tensors(pi, spy):
    for name, call in calls_of(pi, None).items():
        spy.calls.clear()
        call()
        assert spy.calls == [(name, 1, 0)]             # GPU 1 is current, and its own current stream is taken
        assert spy.gpus[-1] == 0, name                 # as it was before the call


def test_a_stream_that_is_given(pi, spy):
    class Stream:
        cuda_stream, device_index = 99, 1
    for name, call in calls_of(pi, Stream()).items():
        spy.calls.clear()
        call()
        assert spy.calls == [(name, 1, 99)]
    Stream.device_index = 0
    for name, call in calls_of(pi, Stream()).items():
        spy.calls.clear()
        with pytest.raises(pi.PiError) as e:
            call()
        assert e.value.status == pi.PI_EINVAL and not spy.calls, name


@pytest.mark.parametrize("name", ["pi_cache_fork", "pi_cache_compact", "pi_attn_decode", "pi_matvec"])
def test_another_stream_waits_for_memory_that_was_taken_on_the_current_one(pi, spy, name):
    """The memory may have been given back with work of the current stream still reading it."""
    class Stream:
        cuda_stream, device_index = 99, 1
    half, some = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(2, 64)
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    mat = pi.Q4Matrix(torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.float16), batch=2)
    if name == "pi_attn_decode":
        c.reserve(3, 4)

    def call(stream):
        if name == "pi_cache_fork":
            c.fork(ints(0), ints(1), stream)
        elif name == "pi_cache_compact":
            c.compact(None, stream)
        elif name == "pi_attn_decode":
            pi.attn_decode(c, 0, half, half.clone(), stream=stream)
        else:
            pi.matvec(mat, some, some.clone(), stream=stream)
    call(None)                                         # the stream it was taken on
    assert spy.waits == [] and len(spy.calls) == 1
    call(Stream())
    assert spy.waits == [(1, 1, 99, ("mark", 1))]      # before the second call
    call(Stream())
    call(None)
    assert len(spy.waits) == 1 and [c[2] for c in spy.calls] == [0, 99, 99, 0]


def test_the_current_gpu_comes_back_after_an_error(pi, spy, monkeypatch):
    def fails(*args):
        raise ValueError
    calls = calls_of(pi, None)
    monkeypatch.setattr(spy, "pi_matvec", fails, raising=False)
    mat = calls["pi_matvec"]
    with pytest.raises(ValueError):
        mat()
    assert spy.gpus[-1] == 0
