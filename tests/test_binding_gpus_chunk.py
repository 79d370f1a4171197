"""Which GPU and stream the calls of a serving step go to, on the host: tensors that say they lie on GPU 1 while GPU 0 is
current, and a library that only writes down what it is called with."""
import pytest

torch = pytest.importorskip("torch")

from test_binding_gpus import ints, pi, spy  # noqa: E402, F401


def calls_of(pi, rope, stream):  # noqa: F811
    """One call of each operator, name -> function."""
    half = dict(dtype=torch.float16)
    q, kv = torch.zeros(3, 4, 64, **half), torch.zeros(3, 2, 64, **half)
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    c.reserve_chunk(3, 4, 1)
    ws = torch.zeros(c.chunk_workspace(3, 4, 1).numel(), dtype=torch.uint8)
    return {
        "pi_rope_heads": lambda: pi.rope_heads(rope, ints(0, 1, 2), q, q.clone(), kv, kv.clone(), stream=stream),
        "pi_cache_append_rope": lambda: c.append_rope(0, rope, q, q.clone(), kv, kv, ints(0, 3), ints(0), stream=stream),
        "pi_attn_chunk": lambda: pi.attn_chunk(c, 0, q, q.clone(), ints(0, 3), ws=ws, stream=stream),
    }


@pytest.fixture
def rope(pi):  # noqa: F811
    return pi.Rope(64, device="cpu")


def test_calls_go_to_the_gpu_of_their_tensors(pi, rope, spy):  # noqa: F811
    for name, call in calls_of(pi, rope, None).items():
        spy.calls.clear()
        call()
        assert spy.calls == [(name, 1, 0)]
        assert spy.gpus[-1] == 0, name


def test_a_stream_that_is_given(pi, rope, spy):  # noqa: F811
    class Stream:
        cuda_stream, device_index = 99, 1
    for name, call in calls_of(pi, rope, Stream()).items():
        spy.calls.clear()
        call()
        assert spy.calls == [(name, 1, 99)]
    Stream.device_index = 0
    for name, call in calls_of(pi, rope, Stream()).items():
        spy.calls.clear()
        with pytest.raises(pi.PiError) as e:
            call()
        assert e.value.status == pi.PI_EINVAL and not spy.calls, name


def test_another_stream_waits_for_the_workspace(pi, spy):  # noqa: F811
    class Stream:
        cuda_stream, device_index = 99, 1
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    c = pi.Cache.create(1, 8, 2, 16, 64, 4, 4, device="cpu")
    c.reserve_chunk(3, 4, 1)

    def call(stream):
        pi.attn_chunk(c, 0, q, q.clone(), ints(0, 3), stream=stream)
    call(None)
    assert spy.waits == [] and len(spy.calls) == 1
    call(Stream())
    assert spy.waits == [(1, 1, 99, ("mark", 1))]
    call(Stream())
    call(None)
    assert len(spy.waits) == 1 and [x[2] for x in spy.calls] == [0, 99, 99, 0]


def test_tensors_of_two_gpus_are_refused(pi, rope, spy, monkeypatch):  # noqa: F811
    for name, call in calls_of(pi, rope, None).items():
        seen = iter([1, 0] + [1] * 20)                 # the second tensor lies elsewhere
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: next(seen))
        spy.calls.clear()
        with pytest.raises(pi.PiError):
            call()
        assert not spy.calls, name
