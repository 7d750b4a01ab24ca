"""Where the tensor forms of the products take their memory when they are
given a stream of their own: shown on the host, with stand-ins for the streams
and the library, because a block of memory that two streams use at once gives
wrong results only now and then."""
import contextlib

import pytest
import torch

import lossless_compression_float_amd as uz
import lossless_compression_float_amd.weights as weights

BF, F32 = torch.bfloat16, torch.float32
CPU = torch.device("cpu")


class Stream:
    def __init__(self, name, device=CPU):
        self.name, self.device, self.cuda_stream = name, device, 0

    def __repr__(self):
        return self.name


class Library:
    """Answers every call with success and every workspace question with 1,000 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append(name)
            return 1000 if name.endswith("_workspace_size") else uz.UZIP_OK
        return fn


@pytest.fixture
def streams(monkeypatch):
    main, side = Stream("main"), Stream("side")
    state = dict(current=main, made=[], recorded=[], main=main, side=side, lib=Library())

    @contextlib.contextmanager
    def current(s):
        before, state["current"] = state["current"], s
        yield
        state["current"] = before

    empty = torch.empty

    def logged(*a, **kw):
        t = empty(*a, **kw)
        state["made"].append((t, state["current"]))
        return t

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["current"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(torch, "empty", logged)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state["recorded"].append((t.data_ptr(), s)))
    monkeypatch.setattr(weights, "_lib", lambda: state["lib"])
    return state


M, N, K, E = 5, 32, 64, 3
X, DY, Z = torch.zeros(M, K, dtype=BF), torch.zeros(M, N, dtype=BF), torch.zeros(M, N)
OFF, T, F = torch.zeros(E + 1, dtype=torch.int32), torch.zeros(M, dtype=torch.int64), torch.zeros(M)


def packed(*shape):
    return uz.PackedWeight(torch.zeros(16, dtype=torch.uint8), shape, False)


CALLS = {
    "linear": lambda **kw: uz.linear(X, packed(N, K), act="silu", return_preact=True, **kw),
    "linear_backward": lambda **kw: uz.linear_backward(DY, X, packed(N, K), preact=Z, act="silu", need_bias=True, **kw),
    "grouped_linear": lambda **kw: uz.grouped_linear(X, OFF, packed(E, N, K), return_preact=True, **kw),
    "grouped_linear_backward": lambda **kw: uz.grouped_linear_backward(DY, X, OFF, packed(E, N, K), need_bias=True, **kw),
    "linear_cross_entropy": lambda **kw: uz.linear_cross_entropy(X, packed(N, K), T, **kw),
    "linear_cross_entropy_backward": lambda **kw: uz.linear_cross_entropy_backward(F, X, packed(N, K), T, F, **kw),
    "unpack_weight": lambda **kw: (uz.unpack_weight(packed(N, K), **kw),),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_another_stream_takes_its_memory_there(streams, name):
    """Results and workspace come from the memory of the stream that writes them, and the allocator knows that the
    caller's stream uses the results."""
    results = CALLS[name](stream=streams["side"])
    assert "uzip_" + ("weight_unpack" if name == "unpack_weight" else name) in streams["lib"].calls
    assert streams["made"] and all(s is streams["side"] for _, s in streams["made"]), streams["made"]
    for t in results:
        assert [s for p, s in streams["recorded"] if p == t.data_ptr()] == [streams["main"]]
    assert streams["current"] is streams["main"]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_the_current_stream_records_nothing(streams, name):
    CALLS[name]()
    CALLS[name](stream=streams["main"])
    assert all(s is streams["main"] for _, s in streams["made"]) and not streams["recorded"]


def test_the_callers_own_output_and_workspace_are_recorded_for_the_stream(streams):
    out, ws = torch.zeros(M, N, dtype=BF), torch.zeros(2000, dtype=torch.uint8)
    y = uz.linear(X, packed(N, K), out=out, ws=ws, stream=streams["side"])
    assert y is out and not streams["made"]
    assert set(streams["recorded"]) == {(out.data_ptr(), streams["side"]), (ws.data_ptr(), streams["side"])}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_stream_of_another_device_is_refused(streams, name):
    with pytest.raises(ValueError, match="stream is on"):
        CALLS[name](stream=Stream("far", torch.device("cuda", 1)))
    assert not [c for c in streams["lib"].calls if not c.endswith("_workspace_size")]
