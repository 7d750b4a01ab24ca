"""The router, the expert layer and the sampler without a GPU: sizes, argument
errors of the C entry points (returned before anything is launched) and the
refusals of the tensor forms (raised before the library is called)."""
import ctypes
import math

import pytest
import torch

import lossless_compression_float_amd as uz
import lossless_compression_float_amd.experts as experts
import lossless_compression_float_amd.sampling as sampling
from test_linear_args import FAKE, INVALID, weight
from test_linear_streams import Stream, streams  # noqa: F401

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
BIG = 1 << 50


def test_structs_have_the_headers_sizes():
    assert [ctypes.sizeof(t) for t in (uz.uzip_moe_route_args, uz.uzip_moe_args, uz.uzip_sample_args)] == [112, 112, 112]


# ---- C entry points ---------------------------------------------------------------

def route_args(**kw):
    base = dict(logits=FAKE, logits_stride=8, tokens=5, bias=None, experts=FAKE, weights=FAKE, order=FAKE, offsets=FAKE,
                dweights=FAKE, dlogits=FAKE, dlogits_stride=8, num_experts=8, k=2, logits_dtype=uz.UZIP_FP32, scores=0,
                renormalize=1, scale=1.0)
    return uz.uzip_moe_route_args(**{**base, **kw})


def test_route_argument_errors():
    assert uz.uzip_moe_route_workspace_size(route_args()) == 0  # few tokens need none
    many = route_args(tokens=1000)
    need = uz.uzip_moe_route_workspace_size(many)
    assert need > 4 * 9 * 60
    for ws, size in ((FAKE, need - 1), (None, need), (FAKE + 4, need)):
        assert uz.uzip_moe_route(many, ws, size, None) == INVALID
    for kw in [dict(num_experts=0), dict(num_experts=1025), dict(k=0), dict(k=9), dict(k=65, num_experts=100, logits_stride=100),
               dict(logits=FAKE + 2), dict(logits_stride=7), dict(logits_dtype=0), dict(logits_dtype=3), dict(scores=2),
               dict(renormalize=2), dict(experts=None), dict(weights=None), dict(order=None), dict(offsets=None),
               dict(offsets=FAKE + 2), dict(order=FAKE + 1), dict(bias=FAKE), dict(bias=FAKE + 2, scores=1),
               dict(tokens=(1 << 24) + 1), dict(tokens=1 << 62), dict(logits=None, bias=FAKE, scores=1)]:
        assert uz.uzip_moe_route(route_args(**kw), FAKE, BIG, None) == INVALID, kw
        assert uz.uzip_moe_route_workspace_size(route_args(**kw)) == 0, kw
    assert uz.uzip_moe_route(None, FAKE, BIG, None) == INVALID
    for kw in [dict(num_experts=0), dict(k=0), dict(k=9), dict(logits=None), dict(logits_stride=7), dict(dlogits=None),
               dict(dlogits_stride=7), dict(dlogits=FAKE + 2), dict(dweights=None), dict(dweights=FAKE + 2), dict(experts=None),
               dict(logits_dtype=9), dict(scores=7), dict(tokens=1 << 62)]:
        assert uz.uzip_moe_route_backward(route_args(**kw), None) == INVALID, kw
    assert uz.uzip_moe_route_backward(route_args(tokens=0, logits=None, dlogits=None), None) == uz.UZIP_OK
    assert uz.uzip_moe_route_backward(None, None) == INVALID


def moe_args(**kw):
    base = dict(x=FAKE, x_stride=64, tokens=5, weights=FAKE, order=FAKE, offsets=FAKE, up_bias=None, down_bias=None,
                residual=None, residual_stride=0, y=FAKE, y_stride=48, k=2, act=0, bias_dtype=0, y_dtype=uz.UZIP_BF16)
    return uz.uzip_moe_args(**{**base, **kw})


def test_moe_argument_errors():
    up, down = weight(rows=32, cols=64, matrices=3), weight(rows=48, cols=32, matrices=3)
    for tokens in (5, 2000):  # both ways
        need = uz.uzip_moe_workspace_size(up, down, moe_args(tokens=tokens))
        assert need > 0
        for ws, size in ((FAKE, need - 1), (None, need), (FAKE + 4, need)):
            assert uz.uzip_moe(up, down, moe_args(tokens=tokens), ws, size, None) == INVALID
        for kw in [dict(x=None), dict(x=FAKE + 1), dict(x_stride=63), dict(weights=None), dict(weights=FAKE + 2), dict(order=None),
                   dict(order=FAKE + 2), dict(offsets=None), dict(offsets=FAKE + 1), dict(y=None), dict(y_stride=47), dict(y_dtype=0),
                   dict(y=FAKE + 2, y_dtype=2), dict(k=0), dict(k=65), dict(act=6), dict(act=5), dict(up_bias=FAKE),
                   dict(down_bias=FAKE + 1, bias_dtype=1), dict(up_bias=FAKE + 2, bias_dtype=2), dict(residual=FAKE, residual_stride=47),
                   dict(residual=FAKE + 1, residual_stride=48), dict(tokens=1 << 25), dict(tokens=1 << 62)]:
            a = moe_args(**{**dict(tokens=tokens), **kw})
            assert uz.uzip_moe(up, down, a, FAKE, BIG, None) == INVALID, kw
            assert uz.uzip_moe_workspace_size(up, down, a) == 0, kw
    gated = weight(rows=64, cols=64, matrices=3, gated=1)
    assert uz.uzip_moe_workspace_size(gated, down, moe_args(act=5)) > 0
    for u, d, kw in [(gated, down, {}), (up, gated, {}), (weight(rows=32, matrices=2), down, {}), (up, weight(rows=48, cols=33, matrices=3), {}),
                     (None, down, {}), (up, None, {}), (weight(rows=0, matrices=3), down, {}), (up, weight(rows=48, cols=32, matrices=3, data=FAKE + 8), {}),
                     (weight(rows=32, matrices=1025), weight(rows=48, cols=32, matrices=1025), {})]:
        assert uz.uzip_moe(u, d, moe_args(**kw), FAKE, BIG, None) == INVALID
        assert uz.uzip_moe_workspace_size(u, d, moe_args(**kw)) == 0
    assert uz.uzip_moe(up, down, None, FAKE, BIG, None) == INVALID
    assert uz.uzip_moe(up, down, moe_args(tokens=0, x=None, y=None, order=None), None, 0, None) == uz.UZIP_OK


def test_moe_of_few_tokens_takes_no_workspace_for_rows_that_cannot_be_read_whole():
    up, down = weight(rows=32, cols=64, matrices=3), weight(rows=48, cols=32, matrices=3)
    plain = uz.uzip_moe_workspace_size(up, down, moe_args())
    for kw in (dict(x=FAKE + 2), dict(x_stride=65), dict(x_stride=1 << 30)):
        assert uz.uzip_moe_workspace_size(up, down, moe_args(**kw)) == plain


def sample_args(**kw):
    base = dict(logits=FAKE, logits_stride=100, rows=3, vocab=100, u=FAKE, temperature=None, top_k=None, top_p=None, min_p=None,
                token=FAKE, logprob=FAKE, temperature_all=1.0, top_k_all=0, top_p_all=1.0, min_p_all=0.0,
                logits_dtype=uz.UZIP_FP32, u_double=0)
    return uz.uzip_sample_args(**{**base, **kw})


def test_sample_argument_errors():
    need = uz.uzip_sample_workspace_size(sample_args())
    assert need > 0
    for ws, size in ((FAKE, need - 1), (None, need), (FAKE + 4, need)):
        assert uz.uzip_sample(sample_args(), ws, size, None) == INVALID
    for kw in [dict(logits=None), dict(logits=FAKE + 2), dict(logits_stride=99), dict(vocab=0), dict(vocab=(1 << 22) + 1, logits_stride=1 << 23),
               dict(rows=(1 << 21) + 1), dict(rows=1 << 62), dict(rows=1 << 20, vocab=1 << 20, logits_stride=1 << 20), dict(u=None),
               dict(u=FAKE + 2), dict(u=FAKE + 4, u_double=1), dict(u_double=2), dict(token=None), dict(token=FAKE + 4),
               dict(logprob=FAKE + 2), dict(logits_dtype=0), dict(logits_dtype=3), dict(temperature_all=-1.0),
               dict(temperature_all=math.nan), dict(temperature_all=math.inf), dict(top_p_all=math.nan), dict(min_p_all=math.nan),
               dict(temperature=FAKE + 2), dict(top_k=FAKE + 1), dict(top_p=FAKE + 2), dict(min_p=FAKE + 2)]:
        assert uz.uzip_sample(sample_args(**kw), FAKE, BIG, None) == INVALID, kw
        assert uz.uzip_sample_workspace_size(sample_args(**kw)) == 0, kw
    assert uz.uzip_sample(None, FAKE, BIG, None) == INVALID
    assert uz.uzip_sample(sample_args(rows=0, logits=None, u=None, token=None), None, 0, None) == uz.UZIP_OK


# ---- tensor forms -----------------------------------------------------------------

@pytest.fixture
def device(monkeypatch, streams):  # noqa: F811
    """Tensors on the CPU pass for device tensors; the library is a stand-in that answers every call."""
    monkeypatch.setattr(experts, "_lib", lambda: streams["lib"])
    monkeypatch.setattr(sampling, "_lib", lambda: streams["lib"])
    monkeypatch.setattr(experts, "_device", lambda t, what: t.device)
    monkeypatch.setattr(sampling, "_device", lambda t: t.device)
    return streams


T, E, K, D, F = 5, 8, 2, 64, 32


def packed(*shape, gated=False):
    return uz.PackedWeight(torch.zeros(16, dtype=torch.uint8), shape, gated)


def routing(tokens=T, k=K, num=E):
    return uz.Routing(torch.zeros(tokens, k, dtype=I32), torch.zeros(tokens, k), torch.zeros(tokens * k, dtype=I32),
                      torch.zeros(num + 1, dtype=I32))


X = torch.zeros(T, D, dtype=BF)
UP, DOWN = packed(E, 2 * F, D, gated=True), packed(E, D, F)
LOGITS = torch.zeros(T, E)
CALLS = {
    "moe_route": lambda **kw: uz.moe_route(LOGITS, K, **kw),
    "moe_group": lambda **kw: uz.moe_group(torch.zeros(T, K, dtype=I32), torch.zeros(T, K), E, **kw),
    "moe_route_backward": lambda **kw: uz.moe_route_backward(torch.zeros(T, K), LOGITS, routing(), **kw),
    "moe": lambda **kw: uz.moe(X, routing(), UP, DOWN, **kw),
    "sample": lambda **kw: uz.sample(LOGITS, torch.zeros(T), **kw),
}


def results(r):
    return (r.experts, r.weights, r.order, r.offsets) if isinstance(r, uz.Routing) else r if isinstance(r, tuple) else (r,)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_another_stream_takes_its_memory_there(device, name):
    out = results(CALLS[name](stream=device["side"]))
    assert device["made"] and all(s is device["side"] for _, s in device["made"])
    for t in out:
        assert [s for p, s in device["recorded"] if p == t.data_ptr()] == [device["main"]]
    assert device["current"] is device["main"]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_the_current_stream_records_nothing(device, name):
    CALLS[name]()
    CALLS[name](stream=device["main"])
    assert all(s is device["main"] for _, s in device["made"]) and not device["recorded"]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_stream_of_another_device_is_refused(device, name):
    with pytest.raises(ValueError, match="stream is on"):
        CALLS[name](stream=Stream("far", torch.device("cuda", 1)))
    assert not [c for c in device["lib"].calls if not c.endswith("_workspace_size")]


def test_calls_without_rows_launch_nothing(device):
    assert uz.moe(X[:0], routing(0), UP, DOWN).shape == (0, D)
    token, logprob = uz.sample(LOGITS[:0], torch.zeros(0))
    assert token.shape == logprob.shape == (0,)
    assert not [c for c in device["lib"].calls if c in ("uzip_moe", "uzip_sample")]


ROUTE_BAD = [
    (TypeError, "logits", dict(logits=[1])), (TypeError, "logits", dict(logits=LOGITS.half())), (ValueError, "logits", dict(logits=LOGITS[0])),
    (ValueError, "1024", dict(logits=torch.zeros(2, 1025))), (ValueError, "rows", dict(logits=torch.zeros(E, T).t())),
    (ValueError, "k must", dict(k=0)), (ValueError, "k must", dict(k=9)), (ValueError, "k must", dict(k=True)), (ValueError, "k must", dict(k=2.0)),
    (ValueError, "scores", dict(scores="relu")), (ValueError, "bias goes", dict(bias=torch.zeros(E))),
    (TypeError, "bias", dict(bias=torch.zeros(E, dtype=BF), scores="sigmoid")), (ValueError, "bias", dict(bias=torch.zeros(E + 1), scores="sigmoid")),
    (ValueError, "autograd", dict(logits=torch.zeros(T, E, requires_grad=True))), (ValueError, "ws", dict(ws=torch.zeros(4))),
]


@pytest.mark.parametrize("error,match,kw", ROUTE_BAD)
def test_route_refusals(device, error, match, kw):
    with pytest.raises(error, match=match):
        uz.moe_route(**{**dict(logits=LOGITS, k=K), **kw})
    assert "uzip_moe_route" not in device["lib"].calls


@pytest.mark.parametrize("error,match,args", [
    (TypeError, "experts", (torch.zeros(T, K), torch.zeros(T, K), E)), (TypeError, "weights", (torch.zeros(T, K, dtype=I32), torch.zeros(T, K, dtype=BF), E)),
    (ValueError, "shape", (torch.zeros(T, K, dtype=I32), torch.zeros(T, K + 1), E)), (ValueError, "shape", (torch.zeros(T, 65, dtype=I32), torch.zeros(T, 65), E)),
    (ValueError, "num_experts", (torch.zeros(T, K, dtype=I32), torch.zeros(T, K), 0)), (ValueError, "num_experts", (torch.zeros(T, K, dtype=I32), torch.zeros(T, K), 1025)),
    (ValueError, "autograd", (torch.zeros(T, K, dtype=I32), torch.zeros(T, K, requires_grad=True), E)),
])
def test_group_refusals(device, error, match, args):
    with pytest.raises(error, match=match):
        uz.moe_group(*args)


@pytest.mark.parametrize("error,match,kw", [
    (TypeError, "experts", dict(experts=torch.zeros(T, K))), (ValueError, "up to", dict(experts=torch.zeros(T, dtype=I32))),
    (ValueError, "up to", dict(experts=torch.zeros(T, 65, dtype=I32))), (ValueError, "up to", dict(offsets=torch.zeros(1026, dtype=I32))),
    (ValueError, "experts", dict(experts=torch.zeros(K, T, dtype=I32).t())), (TypeError, "weights", dict(weights=torch.zeros(T, K, dtype=BF))),
    (ValueError, "weights", dict(weights=torch.zeros(T, K + 1))), (TypeError, "order", dict(order=torch.zeros(T * K, dtype=torch.int64))),
    (ValueError, "order", dict(order=torch.zeros(T * K - 1, dtype=I32))), (TypeError, "offsets", dict(offsets=torch.zeros(E + 1))),
    (ValueError, "offsets", dict(offsets=torch.zeros(2, E + 1, dtype=I32)[:, ::2])),
    (ValueError, "scores", dict(scores="linear")),
])
def test_a_routing_of_other_tensors_is_checked(error, match, kw):
    base = dict(experts=torch.zeros(T, K, dtype=I32), weights=torch.zeros(T, K), order=torch.zeros(T * K, dtype=I32),
                offsets=torch.zeros(E + 1, dtype=I32))
    with pytest.raises(error, match=match):
        uz.Routing(**{**base, **kw})
    assert uz.Routing(**base).num_experts == E


@pytest.mark.parametrize("error,match,args", [
    (TypeError, "Routing", (torch.zeros(T, K), LOGITS, None)), (ValueError, "shape", (torch.zeros(T, K), LOGITS[:, :-1].contiguous(), routing())),
    (TypeError, "dweights", (torch.zeros(T, K, dtype=BF), LOGITS, routing())), (ValueError, "dweights", (torch.zeros(K, T).t(), LOGITS, routing())),
])
def test_route_backward_refusals(device, error, match, args):
    with pytest.raises(error, match=match):
        uz.moe_route_backward(*args)


MOE_BAD = [
    (TypeError, "Routing", dict(routing=None)), (TypeError, "PackedWeight", dict(up=X)), (TypeError, "PackedWeight", dict(down=X)),
    (ValueError, "stack", dict(up=packed(2 * F, D, gated=True))), (ValueError, "gated", dict(down=packed(E, D, F, gated=True))),
    (ValueError, "swiglu", dict(act="silu")), (ValueError, "act must", dict(act="tanh")), (ValueError, "down must", dict(down=packed(E, D, F + 1))),
    (ValueError, "down must", dict(down=packed(E - 1, D, F))), (ValueError, "routing is of", dict(routing=routing(T + 1))),
    (ValueError, "routing is of", dict(routing=routing(num=E + 1))), (TypeError, "x must", dict(x=X.float())), (ValueError, "x must", dict(x=X[:, 1:])),
    (ValueError, "x must", dict(x=X[0])), (TypeError, "out_dtype", dict(out_dtype=torch.float16)), (ValueError, "up_bias", dict(up_bias=torch.zeros(E, F))),
    (ValueError, "down_bias", dict(down_bias=torch.zeros(D, E).t())), (TypeError, "one type", dict(up_bias=torch.zeros(E, 2 * F), down_bias=torch.zeros(E, D, dtype=BF))),
    (TypeError, "residual", dict(residual=torch.zeros(T, D))), (ValueError, "residual", dict(residual=X[:, :-1])), (ValueError, "overlap x", dict(out=X)),
    (ValueError, "autograd", dict(x=torch.zeros(T, D, dtype=BF, requires_grad=True))), (ValueError, "ws", dict(ws=torch.zeros(8))),
]


@pytest.mark.parametrize("error,match,kw", MOE_BAD)
def test_moe_refusals(device, error, match, kw):
    with pytest.raises(error, match=match):
        uz.moe(**{**dict(x=X, routing=routing(), up=UP, down=DOWN), **kw})
    assert "uzip_moe" not in device["lib"].calls


def test_a_result_may_take_its_residuals_place_but_not_part_of_it(device):
    room = torch.zeros(T + 1, D, dtype=BF)
    assert uz.moe(X, routing(), UP, DOWN, residual=room[1:], out=room[1:]).data_ptr() == room[1:].data_ptr()
    with pytest.raises(ValueError, match="residual itself"):
        uz.moe(X, routing(), UP, DOWN, residual=room[1:], out=room[:-1])


U = torch.zeros(T)
SAMPLE_BAD = [
    (TypeError, "tensors", dict(logits=[1.0])), (TypeError, "tensors", dict(u=0.5)), (TypeError, "logits", dict(logits=LOGITS.half())),
    (ValueError, "logits", dict(logits=LOGITS[0])), (ValueError, "logits", dict(logits=LOGITS[:, :0])), (TypeError, "u must", dict(u=U.half())),
    (ValueError, "u must", dict(u=U[1:])), (ValueError, "u must", dict(u=torch.zeros(T, 2)[:, 0])), (ValueError, "temperature", dict(temperature=-0.1)),
    (ValueError, "temperature", dict(temperature=math.inf)), (TypeError, "temperature", dict(temperature=math.nan)), (TypeError, "temperature", dict(temperature="1")),
    (TypeError, "temperature", dict(temperature=U.double())), (ValueError, "temperature", dict(temperature=U[1:])), (ValueError, "top_k", dict(top_k=-1)),
    (ValueError, "top_k", dict(top_k=1.5)), (TypeError, "top_k", dict(top_k=U.long())), (ValueError, "top_p", dict(top_p=1.1)), (ValueError, "top_p", dict(top_p=-0.1)),
    (ValueError, "min_p", dict(min_p=1.1)), (TypeError, "min_p", dict(min_p=None)), (ValueError, "autograd", dict(logits=torch.zeros(T, E, requires_grad=True))),
    (ValueError, "ws", dict(ws=torch.zeros(8))),
]


@pytest.mark.parametrize("error,match,kw", SAMPLE_BAD)
def test_sample_refusals(device, error, match, kw):
    with pytest.raises(error, match=match):
        uz.sample(**{**dict(logits=LOGITS, u=U), **kw})
    assert "uzip_sample" not in device["lib"].calls


def test_host_tensors_are_refused():
    for call in ("moe_route", "moe_group", "sample"):
        with pytest.raises(ValueError, match="device tensors"):
            CALLS[call]()


C_SRC = r"""
#include <stdio.h>
#include "uzip.h"

int main(int argc, char **argv) {
    (void)argv;
    uzip_weight w = {0};
    uzip_moe_route_args r = {0};
    uzip_moe_args m = {0};
    uzip_sample_args s = {0};
    r.scores = UZIP_SCORES_SIGMOID;
    if (argc > 100) {  /* never taken: type-checks every call */
        int st = uzip_moe_route(&r, 0, uzip_moe_route_workspace_size(&r), 0) | uzip_moe_route_backward(&r, 0);
        st |= uzip_moe(&w, &w, &m, 0, uzip_moe_workspace_size(&w, &w, &m), 0);
        return st | uzip_sample(&s, 0, uzip_sample_workspace_size(&s), 0);
    }
    printf("%zu %zu %zu\n", sizeof r, sizeof m, sizeof s);
    return 0;
}
"""


def test_the_structs_and_calls_from_c(tmp_path):
    import os
    import subprocess
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text(C_SRC)
    root, lib = os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(uz.LIB_PATH)
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Wextra", "-pedantic", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I" + root + "/include",
                           "-isystem", "/opt/rocm/include", "-o", str(exe), str(src), "-L" + lib, "-luzip", "-Wl,-rpath," + lib])
    sizes = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    assert sizes == [ctypes.sizeof(t) for t in (uz.uzip_moe_route_args, uz.uzip_moe_args, uz.uzip_sample_args)]
