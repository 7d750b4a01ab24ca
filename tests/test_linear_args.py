"""The products with packed weights without a GPU: sizes, argument errors of
the C entry points (returned before anything is launched) and the refusals of
the tensor forms (raised before the library is called)."""
import ctypes

import pytest
import torch

import lossless_compression_float_amd as uz

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its checks first
BF, F32 = torch.bfloat16, torch.float32
INVALID = uz.UZIP_ERR_INVALID_ARGUMENT


def weight(rows=32, cols=64, matrices=1, gated=0, **kw):
    base = dict(data=FAKE, bytes=1 << 40, matrices=matrices, rows=rows, cols=cols, gated=gated, reserved=0)
    return uz.uzip_weight(**{**base, **kw})


def linear_args(**kw):
    base = dict(x=FAKE, x_stride=64, tokens=5, offsets=None, bias=None, residual=None, residual_stride=0, y=FAKE,
                y_stride=32, preact=None, preact_stride=0, bias_dtype=0, y_dtype=uz.UZIP_BF16, act=0, preact_dtype=uz.UZIP_BF16, clear_rest=0, reserved=0)
    return uz.uzip_linear_args(**{**base, **kw})


def backward_args(**kw):
    base = dict(dy=FAKE, dy_stride=32, x=FAKE, x_stride=64, preact=FAKE, preact_stride=32, tokens=5, offsets=None, dx=FAKE,
                dx_stride=64, dw=FAKE, dbias=FAKE, dy_dtype=uz.UZIP_BF16, dbias_dtype=uz.UZIP_BF16, act=0, preact_dtype=uz.UZIP_BF16, clear_rest=0, reserved=0)
    return uz.uzip_linear_backward_args(**{**base, **kw})


def loss_args(**kw):
    base = dict(x=FAKE, x_stride=64, tokens=5, target=FAKE, ignore_index=-100, loss=FAKE, lse=FAKE, dloss=FAKE, dx=FAKE,
                dx_stride=64, dw=FAKE)
    return uz.uzip_loss_args(**{**base, **kw})


def test_structs_have_the_headers_sizes():
    assert [ctypes.sizeof(t) for t in (uz.uzip_weight, uz.uzip_linear_args, uz.uzip_linear_backward_args,
                                       uz.uzip_loss_args)] == [48, 112, 120, 88]


def test_packed_sizes():
    tiles = (4096 // 16) * (14336 // 64)
    assert uz.uzip_weight_max_size(1, 4096, 14336) == 256 + 16 * tiles + 1536 * tiles + 1024 * tiles
    assert uz.uzip_weight_max_size(1, 1, 1) == 512 + 2560
    # halves of 17 rows take two row blocks each, one matrix of 34 rows three
    assert uz.uzip_weight_max_size(3, 34, 65, 1) - 256 >= 3 * 4 * 2 * 2560 > uz.uzip_weight_max_size(3, 34, 65, 0)
    for bad in [(0, 1, 1, 0), (1, 0, 1, 0), (1, 1, 0, 0), (1, 3, 4, 1), (1, 2, 4, 2), (65536, 1, 1, 0), (1, 1 << 31, 1, 0),
                (1, 1, 1 << 31, 0), (1, 1 << 20, 1 << 20, 0), (1 << 63, 1 << 63, 4, 0)]:
        assert uz.uzip_weight_max_size(*bad) == 0 and uz.uzip_weight_workspace_size(*bad) == 0, bad


def test_pack_argument_errors():
    cap, ws = uz.uzip_weight_max_size(1, 32, 64), uz.uzip_weight_workspace_size(1, 32, 64)

    def call(**kw):
        return uz.uzip_weight_pack(**{**dict(d_in=FAKE, matrices=1, rows=32, cols=64, row_stride=64, matrix_stride=0, gated=0,
                                             d_out=FAKE, out_capacity=cap, d_out_size=FAKE, d_workspace=FAKE,
                                             workspace_bytes=ws - 1, stream=None), **kw})

    assert call() == INVALID  # workspace one byte short
    for kw in [dict(d_in=None), dict(d_in=FAKE + 1), dict(matrices=0), dict(rows=0), dict(cols=0), dict(row_stride=63),
               dict(rows=33, gated=1), dict(gated=2), dict(d_out=None), dict(d_out=FAKE + 8), dict(d_out_size=None),
               dict(d_out_size=FAKE + 4), dict(d_workspace=None), dict(d_workspace=FAKE + 8)]:
        assert call(**{**dict(workspace_bytes=ws), **kw}) == INVALID, kw
    assert call(workspace_bytes=ws, out_capacity=cap - 1) == uz.UZIP_ERR_CAPACITY


def bad_weights(rows=32):
    return [weight(data=None), weight(data=FAKE + 8), weight(bytes=256), weight(rows=0), weight(cols=0), weight(matrices=0),
            weight(reserved=1), weight(gated=2), weight(rows=33, gated=1), None]


@pytest.mark.parametrize("grouped", [False, True])
def test_linear_argument_errors(grouped):
    fn = uz.uzip_grouped_linear if grouped else uz.uzip_linear
    w = weight(matrices=3) if grouped else weight()
    off = dict(offsets=FAKE) if grouped else {}
    assert uz.uzip_linear_workspace_size(w, linear_args(**off)) == 0  # few rows: no workspace
    many = linear_args(tokens=5000, x_stride=65, **off)
    need = uz.uzip_linear_workspace_size(w, many)
    assert need > 0
    assert fn(w, many, FAKE, need - 1, None) == INVALID
    assert fn(w, many, None, need, None) == INVALID
    assert fn(w, many, FAKE + 4, need, None) == INVALID
    for b in bad_weights():
        assert fn(b, linear_args(**off), FAKE, 1 << 30, None) == INVALID
        assert uz.uzip_linear_workspace_size(b, linear_args(**off)) == 0
    assert fn(w, None, FAKE, 1 << 30, None) == INVALID
    for kw in [dict(x=None), dict(x=FAKE + 1), dict(x_stride=63), dict(y=None), dict(y_stride=31), dict(y_dtype=3),
               dict(y_dtype=0), dict(act=6), dict(act=5), dict(reserved=1), dict(clear_rest=2), dict(preact=FAKE, preact_stride=32, preact_dtype=0),
               dict(preact=FAKE + 2, preact_stride=32, preact_dtype=2), dict(tokens=1 << 31), dict(bias=FAKE),
               dict(bias=FAKE + 1, bias_dtype=1), dict(bias=FAKE + 2, bias_dtype=2), dict(preact=FAKE, preact_stride=31),
               dict(residual=FAKE, residual_stride=31), dict(y=FAKE + 2, y_dtype=2),
               dict(offsets=None if grouped else FAKE), dict(residual=FAKE, residual_stride=32) if grouped else dict(act=9)]:
        a = linear_args(**{**off, **kw})
        assert fn(w, a, FAKE, 1 << 30, None) == INVALID, kw
    if grouped:
        assert fn(w, linear_args(offsets=FAKE + 2), FAKE, 1 << 30, None) == INVALID
    else:
        assert fn(weight(matrices=2), linear_args(), FAKE, 1 << 30, None) == INVALID
    gated = weight(gated=1, matrices=w.matrices)
    assert fn(gated, linear_args(act=4, **off), FAKE, 1 << 30, None) == INVALID  # a gated weight takes swiglu only
    # nothing to do: no launch, whatever the pointers
    assert fn(w, linear_args(tokens=0, x=None, y=None, **off), FAKE, need, None) == uz.UZIP_OK


def test_calls_beyond_the_launch_grids_are_refused():
    big = 1 << 40
    w = weight(rows=1 << 20, cols=64)
    for tokens in [1 << 20, (1 << 25) + 1, 1 << 63]:
        a = linear_args(tokens=tokens, y_stride=1 << 20)
        assert uz.uzip_linear(w, a, FAKE, big, None) == INVALID
        assert uz.uzip_linear_backward(w, backward_args(tokens=tokens, dy_stride=1 << 20), FAKE, big, None) == INVALID
        assert uz.uzip_linear_cross_entropy(w, loss_args(tokens=tokens), FAKE, big, None) == INVALID
    assert uz.uzip_linear(weight(), linear_args(tokens=(1 << 25) + 1), FAKE, big, None) == INVALID


def test_matrices_too_wide_for_a_product_are_refused():
    """A tile's rows are addressed with 32 bits; such weights can be packed all the same."""
    big, most = 1 << 45, (1 << 22) - 512
    for kw in (dict(rows=64, cols=most + 1), dict(rows=most + 1, cols=64)):
        w = weight(**kw)
        assert uz.uzip_weight_max_size(1, kw["rows"], kw["cols"]) > 0
        rows, cols = kw["rows"], kw["cols"]
        a = linear_args(x_stride=cols, y_stride=rows)
        assert uz.uzip_linear(w, a, FAKE, big, None) == INVALID
        b = backward_args(dy_stride=rows, x_stride=cols, dx_stride=cols)
        assert uz.uzip_linear_backward(w, b, FAKE, big, None) == INVALID
        l = loss_args(x_stride=cols, dx_stride=cols)
        assert uz.uzip_linear_cross_entropy(w, l, FAKE, big, None) == INVALID
        assert uz.uzip_linear_cross_entropy_backward(w, l, FAKE, big, None) == INVALID
    w = weight(rows=64, cols=most)
    assert uz.uzip_linear_workspace_size(w, linear_args(x_stride=most + 1, y_stride=64)) > 2 * most


def test_linear_workspace_holds_a_copy_of_rows_that_cannot_be_read_whole():
    small = uz.uzip_linear_workspace_size(weight(), linear_args(tokens=1000))
    for kw in [dict(x=FAKE + 2), dict(x_stride=65)]:
        assert uz.uzip_linear_workspace_size(weight(), linear_args(tokens=1000, **kw)) >= small + 1000 * 64 * 2
    odd = uz.uzip_linear_workspace_size(weight(cols=63), linear_args(tokens=1000))
    assert odd >= small + 1000 * 64 * 2


@pytest.mark.parametrize("grouped", [False, True])
def test_backward_argument_errors(grouped):
    fn = uz.uzip_grouped_linear_backward if grouped else uz.uzip_linear_backward
    w = weight(matrices=3) if grouped else weight()
    off = dict(offsets=FAKE) if grouped else {}
    need = uz.uzip_linear_backward_workspace_size(w, backward_args(**off))
    assert fn(w, backward_args(**off), FAKE, need - 1, None) == INVALID
    for b in bad_weights():
        assert fn(b, backward_args(**off), FAKE, 1 << 30, None) == INVALID
    for kw in [dict(dy=None), dict(dy_stride=31), dict(dy_dtype=5), dict(dx_stride=63), dict(x=None), dict(x_stride=1),
               dict(act=1, preact=None), dict(act=1, preact_stride=31), dict(act=5), dict(act=77), dict(dbias_dtype=0),
               dict(dbias=FAKE + 1), dict(dw=FAKE + 1), dict(act=1, preact_dtype=3), dict(reserved=1), dict(clear_rest=2), dict(tokens=1 << 32),
               dict(offsets=None if grouped else FAKE)]:
        assert fn(w, backward_args(**{**off, **kw}), FAKE, 1 << 30, None) == INVALID, kw


def test_loss_argument_errors():
    w = weight()
    for fn, size in ((uz.uzip_linear_cross_entropy, uz.uzip_linear_cross_entropy_workspace_size),
                     (uz.uzip_linear_cross_entropy_backward, uz.uzip_linear_cross_entropy_backward_workspace_size)):
        need = size(w, loss_args())
        assert need > 0 and fn(w, loss_args(), FAKE, need - 1, None) == INVALID
        for b in bad_weights() + [weight(gated=1), weight(matrices=2)]:
            assert fn(b, loss_args(), FAKE, 1 << 30, None) == INVALID and size(b, loss_args()) == 0
        for kw in [dict(x=None), dict(x_stride=3), dict(target=None), dict(target=FAKE + 4), dict(lse=None),
                   dict(tokens=1 << 31)]:
            assert fn(w, loss_args(**kw), FAKE, 1 << 30, None) == INVALID, kw
        assert fn(w, None, FAKE, 1 << 30, None) == INVALID
    assert uz.uzip_linear_cross_entropy(w, loss_args(loss=None), FAKE, 1 << 30, None) == INVALID
    for kw in [dict(dloss=None), dict(dx_stride=63), dict(dw=FAKE + 1)]:
        assert uz.uzip_linear_cross_entropy_backward(w, loss_args(**kw), FAKE, 1 << 30, None) == INVALID, kw


def test_loss_backward_holds_one_piece_of_the_logits():
    """The workspace does not grow with the vocabulary once it is cut."""
    a = loss_args(tokens=8192)
    small = uz.uzip_linear_cross_entropy_backward_workspace_size(weight(rows=32768), a)
    large = uz.uzip_linear_cross_entropy_backward_workspace_size(weight(rows=262144), a)
    assert small == large < 8192 * 262144 * 2 // 8


# ---- the tensor forms ---------------------------------------------------------------

def packed(shape=(32, 64), gated=False):
    return uz.PackedWeight(torch.zeros(16, dtype=torch.uint8), shape, gated)


def test_pack_weight_refusals():
    with pytest.raises(TypeError):
        uz.pack_weight(torch.zeros(4, 4))
    with pytest.raises(TypeError):
        uz.pack_weight([1.0])
    with pytest.raises(ValueError):
        uz.pack_weight(torch.zeros(4, 4, dtype=BF))  # not on a device
    with pytest.raises(TypeError):
        uz.unpack_weight(torch.zeros(4, 4, dtype=BF))


X = torch.zeros(5, 64, dtype=BF)
OFF = torch.zeros(4, dtype=torch.int32)


@pytest.mark.parametrize("kw,error", [
    (dict(weight=X), TypeError), (dict(weight=packed((3, 32, 64))), ValueError), (dict(x=X.float()), TypeError),
    (dict(x=X[:, :63]), ValueError), (dict(x=X[0]), ValueError), (dict(x=[1]), TypeError),
    (dict(x=torch.zeros(64, 5, dtype=BF).t()), ValueError), (dict(x=X[:1].expand(5, 64)), ValueError),
    (dict(act="tanh"), ValueError), (dict(act="swiglu"), ValueError), (dict(weight=packed(gated=True)), ValueError),
    (dict(bias=torch.zeros(31, dtype=BF)), ValueError), (dict(bias=torch.zeros(32, dtype=torch.float16)), TypeError),
    (dict(bias=3.0), TypeError), (dict(residual=torch.zeros(5, 32)), TypeError),
    (dict(residual=torch.zeros(4, 32, dtype=BF)), ValueError), (dict(out_dtype=torch.float16), TypeError)])
def test_linear_refusals(kw, error):
    with pytest.raises(error):
        uz.linear(**{**dict(x=X, weight=packed()), **kw})


def test_linear_refuses_an_output_over_its_inputs():
    square = packed((64, 64))
    both = torch.zeros(5, 128, dtype=BF)
    for out, x, residual in [(X, X, None), (both[:, :64], both[:, 63:127], None), (both[:, :64], X, both[:, 1:65]),
                             (both[1:5, :64], X[:4], both[:4, :64])]:
        with pytest.raises(ValueError, match="overlap"):
            uz.linear(x, square, out=out, residual=residual)
    from lossless_compression_float_amd.weights import _overlap
    assert not _overlap(both[:, :64], both[:, 64:]) and not _overlap(both[:2], both[2:]) and not _overlap(X[:0], X)
    assert _overlap(both[:, 60:70], both[:, :61]) and _overlap(both[1:2, :3], both[:, 2:])


@pytest.mark.parametrize("kw,error", [
    (dict(weight=packed()), ValueError), (dict(offsets=OFF.long()), TypeError), (dict(offsets=OFF[:3]), ValueError),
    (dict(offsets=[0, 1, 2, 3]), TypeError), (dict(bias=torch.zeros(32, dtype=BF)), ValueError)])
def test_grouped_linear_refusals(kw, error):
    with pytest.raises(error):
        uz.grouped_linear(**{**dict(x=X, offsets=OFF, weight=packed((3, 32, 64))), **kw})


@pytest.mark.parametrize("kw,error", [
    (dict(dy=torch.zeros(5, 31, dtype=BF)), ValueError), (dict(dy=torch.zeros(5, 32, dtype=torch.float16)), TypeError),
    (dict(act="silu"), ValueError), (dict(act="silu", preact=torch.zeros(5, 31, dtype=BF)), ValueError),
    (dict(x=None), TypeError), (dict(bias_dtype=torch.float16), TypeError), (dict(x=X[:4]), ValueError)])
def test_linear_backward_refusals(kw, error):
    with pytest.raises(error):
        uz.linear_backward(**{**dict(dy=torch.zeros(5, 32, dtype=BF), x=X, weight=packed()), **kw})


@pytest.mark.parametrize("kw,error", [
    (dict(target=torch.zeros(5, dtype=torch.int32)), TypeError), (dict(target=torch.zeros(4, dtype=torch.int64)), ValueError),
    (dict(weight=packed(gated=True)), ValueError), (dict(weight=packed((2, 32, 64))), ValueError),
    (dict(x=X.float()), TypeError)])
def test_loss_refusals(kw, error):
    args = dict(x=X, weight=packed(), target=torch.zeros(5, dtype=torch.int64))
    with pytest.raises(error):
        uz.linear_cross_entropy(**{**args, **kw})
    with pytest.raises(error):
        uz.linear_cross_entropy_backward(**{**args, **dict(dloss=torch.zeros(5), lse=torch.zeros(5)), **kw})


def test_loss_backward_refusals():
    args = dict(dloss=torch.zeros(5), x=X, weight=packed(), target=torch.zeros(5, dtype=torch.int64), lse=torch.zeros(5))
    for kw in (dict(dloss=torch.zeros(4)), dict(lse=torch.zeros(5, 1))):
        with pytest.raises(ValueError):
            uz.linear_cross_entropy_backward(**{**args, **kw})
    with pytest.raises(TypeError):
        uz.linear_cross_entropy_backward(**{**args, **dict(lse=torch.zeros(5, dtype=BF))})
