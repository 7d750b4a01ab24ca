"""The products with packed weights against their plain 64-bit forms on an
MI355X: packing bit for bit, linear, grouped_linear and linear_cross_entropy
with their gradients, at the sizes, layouts and values where they can go
wrong.  The bounds are derived in linear_testlib."""
import pytest
import torch

import lossless_compression_float_amd as uz
from linear_testlib import backward64, close, linear64, loss64, loss_backward64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def bits(t):
    return t.contiguous().view(torch.int16)


# ---- packing ----------------------------------------------------------------------

def weight_of(kind, g, shape):
    n = 1
    for s in shape:
        n *= s
    if kind == "normal":
        return normal(g, *shape, scale=0.02)
    if kind == "bits":      # every pattern, NaN payloads included
        return torch.randint(-32768, 32768, (n,), generator=g, dtype=torch.int32).to(torch.int16).view(BF).reshape(shape).to(DEV)
    if kind == "zeros":
        return torch.zeros(shape, dtype=BF, device=DEV)
    if kind == "pruned":    # half of the values exactly zero, of either sign
        w = normal(g, *shape, scale=0.02)
        m = torch.rand(shape, generator=g).to(DEV)
        return torch.where(m < 0.3, torch.zeros_like(w), torch.where(m < 0.5, torch.full_like(w, -0.0), w))
    if kind == "tiny":      # denormals and the smallest exponents
        return torch.randint(0, 0x600, (n,), generator=g, dtype=torch.int32).to(torch.int16).view(BF).reshape(shape).to(DEV)
    if kind == "spread":    # ever more values outside a tile's window: lists of every length, then exponent bytes
        e = torch.arange(n) % 977
        w = torch.randn(n, generator=g) * torch.where(torch.rand(n, generator=g) < e / 6000.0, 1e-9, 1.0)
        return w.to(BF).reshape(shape).to(DEV)
    w = normal(g, *shape, scale=0.02)
    flat = w.view(torch.int16).reshape(-1)
    pos = torch.randint(0, n, (max(1, n // 200),), generator=g).to(DEV)
    flat[pos] = torch.randint(-32768, 32768, (pos.numel(),), generator=g, dtype=torch.int32).to(torch.int16).to(DEV)
    return w


KINDS = ["normal", "bits", "zeros", "pruned", "tiny", "spread", "specials"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,gated", [((1, 1), False), ((16, 64), False), ((17, 65), False), ((250, 1000), False),
                                         ((1024, 512), False), ((3, 34, 130), False), ((2, 66, 200), True), ((62, 129), True)])
def test_pack_is_lossless(kind, shape, gated):
    w = weight_of(kind, gen(1), shape)
    p = uz.pack_weight(w, gated=gated)
    assert torch.equal(bits(uz.unpack_weight(p)), bits(w))
    q = uz.pack_weight(w, gated=gated, trim=False)
    assert q.nbytes == uz.uzip_weight_max_size(shape[0] if len(shape) == 3 else 1, shape[-2], shape[-1], int(gated))
    assert torch.equal(q.data[:p.nbytes], p.data)
    assert torch.equal(bits(uz.unpack_weight(q)), bits(w))


def test_pack_of_normal_weights_takes_three_quarters():
    w = normal(gen(2), 2048, 4096, scale=0.02)
    p = uz.pack_weight(w)
    assert p.nbytes / (2 * w.numel()) < 0.76
    raw = uz.pack_weight(weight_of("bits", gen(3), (1024, 1024)))
    assert raw.nbytes == 256 + 1024 * (16 + 1536 + 1024)  # 1024 tiles that keep their exponents


def test_pack_reads_strided_weights():
    g = gen(4)
    big = normal(g, 2, 70, 300)
    w = big[:, 3:67, 7:207]
    p = uz.pack_weight(w)
    assert torch.equal(bits(uz.unpack_weight(p)), bits(w))
    row = big[0, :1, 5:6]
    assert torch.equal(bits(uz.unpack_weight(uz.pack_weight(row))), bits(row))


# ---- linear --------------------------------------------------------------------------

def check_linear(m, n, k, act="none", bias=None, residual=False, out=BF, kind="normal", seed=10, x=None, keep=F32):
    g = gen(seed)
    gated = act == "swiglu"
    w = weight_of(kind, g, (n, k))
    x = normal(g, m, k) if x is None else x
    b = normal(g, n, dtype=bias) if bias is not None else None
    r = normal(g, m, n // 2 if gated else n, dtype=out) if residual else None
    p = uz.pack_weight(w, gated=gated)
    y, z = uz.linear(x, p, bias=b, act=act, residual=r, out_dtype=out, return_preact=True, preact_dtype=keep)
    assert z.dtype is keep
    z64, ez, y64, ey = linear64(x, w, b, act, r, out, keep)
    close(z, z64, ez, "preact")
    close(y, y64, ey, "y")
    assert torch.equal(uz.linear(x, p, bias=b, act=act, residual=r, out_dtype=out), y)
    return w, x, p, z


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("n,k", [(16, 64), (130, 200), (48, 1000), (257, 65)])
def test_linear_sizes(m, n, k):
    check_linear(m, n, k)


@pytest.mark.parametrize("m", [1, 16, 40, 64, 200])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("bias,residual,out", [(BF, True, BF), (F32, False, F32), (None, True, F32)])
def test_linear_epilogues(m, act, bias, residual, out):
    check_linear(m, 156, 136, act, bias, residual, out)


@pytest.mark.parametrize("m", [1, 3, 33, 64, 130])
@pytest.mark.parametrize("n,k", [(2, 1), (30, 7), (66, 63), (514, 129), (64, 72)])
def test_linear_gated_odd(m, n, k):
    check_linear(m, n, k, "swiglu", BF, True)


@pytest.mark.parametrize("m", [1, 50, 150])
@pytest.mark.parametrize("kind", ["pruned", "tiny", "spread", "zeros"])
def test_linear_tile_kinds(m, kind):
    check_linear(m, 300, 500, kind=kind)


@pytest.mark.parametrize("m,n,k", [(600, 700, 300), (513, 2048, 136), (2048, 2100, 64), (4100, 4096, 72)])
def test_linear_large_tiles(m, n, k):
    check_linear(m, n, k, "silu", BF, True)


@pytest.mark.parametrize("m", [5, 90])
def test_linear_infinities_and_nans_stay_in_their_rows(m):
    g = gen(11)
    k, n = 96, 80
    x = normal(g, m, k).abs()
    x[1, 3], x[2, 5], x[3, 7] = float("inf"), float("-inf"), float("nan")
    w = normal(g, n, k, scale=0.02).abs()
    w[7, 11] = float("inf")
    w[9, 13] = float("nan")
    y = uz.linear(x, uz.pack_weight(w))
    want = x.double().cpu() @ w.double().cpu().T
    _, _, y64, ey = linear64(torch.where(x.isfinite(), x, 0), torch.where(w.isfinite(), w, 0), None, "none", None, BF)
    close(y, torch.where(want.isfinite(), y64, want), ey, "y")


@pytest.mark.parametrize("m", [3, 77])
def test_linear_garbage_behind_the_rows_is_not_read_into_results(m):
    """NaNs in the columns behind x's rows, and in rows behind the last."""
    g = gen(12)
    n, k = 40, 104
    for pad in (8, 3):
        store = torch.full((m + 70, k + pad), float("nan"), dtype=BF, device=DEV)
        x = store[:m, :k]
        x.copy_(normal(g, m, k))
        ystore = torch.full((m + 3, n + 5), 7.0, dtype=BF, device=DEV)
        w = normal(g, n, k, scale=0.02)
        out = ystore[:m, :n]
        y = uz.linear(x, uz.pack_weight(w), out=out)
        assert y.data_ptr() == ystore.data_ptr()
        _, _, y64, ey = linear64(x, w, None, "none", None, BF)
        close(ystore[:m, :n], y64, ey, "y")
        assert (ystore[m:] == 7).all() and (ystore[:, n:] == 7).all()


@pytest.mark.parametrize("m", [4, 100])
def test_linear_unaligned_arguments(m):
    g = gen(13)
    n, k = 72, 80
    x = normal(g, m * k + 1)[1:].view(m, k)
    w = normal(g, n * k + 1, scale=0.1)[1:].view(n, k)
    b = normal(g, n + 1)[1:]
    r = normal(g, m * n + 1)[1:].view(m, n)
    y, z = uz.linear(x, uz.pack_weight(w), bias=b, residual=r, act="silu", return_preact=True)
    z64, ez, y64, ey = linear64(x, w, b, "silu", r, BF)
    close(y, y64, ey, "y")
    dy = normal(g, m * n + 1)[1:].view(m, n)
    dx, dw, db = uz.linear_backward(dy, x, uz.pack_weight(w), preact=z, act="silu", need_bias=True)
    want = backward64(dy, x, w, z, "silu", BF)
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
        close(got, *want[name], name)


def test_linear_without_tokens():
    p = uz.pack_weight(normal(gen(14), 32, 40))
    assert uz.linear(torch.empty(0, 40, dtype=BF, device=DEV), p).shape == (0, 32)
    x = torch.empty(0, 40, dtype=BF, device=DEV)
    dx, dw, db = uz.linear_backward(torch.empty(0, 32, dtype=BF, device=DEV), x, p, need_bias=True)
    assert dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("keep", [F32, BF])
@pytest.mark.parametrize("m", [1, 20, 64, 130, 515])
@pytest.mark.parametrize("n,k,act", [(96, 64, "none"), (100, 72, "silu"), (33, 65, "gelu"), (70, 50, "swiglu"),
                                     (514, 264, "swiglu"), (300, 129, "relu"), (128, 256, "gelu_tanh")])
def test_linear_backward(m, n, k, act, keep):
    w, x, p, z = check_linear(m, n, k, act, BF, seed=20, keep=keep)
    g = gen(21)
    for dtype, bd in ((BF, F32), (F32, BF)):
        dy = normal(g, m, n // 2 if act == "swiglu" else n, dtype=dtype)
        dx, dw, db = uz.linear_backward(dy, x, p, preact=z, act=act, need_bias=True, bias_dtype=bd)
        want = backward64(dy, x, w, z, act, bd)
        for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
            close(got, *want[name], name)
    only = uz.linear_backward(dy, None, p, preact=z, act=act, need_weight=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    assert torch.equal(uz.linear_backward(dy, x, p, preact=z, act=act, need_x=False)[1], dw)


@pytest.mark.parametrize("m,n,k", [(2100, 2048, 264), (300, 2304, 2050)])
def test_linear_backward_large_tiles(m, n, k):
    w, x, p, z = check_linear(m, n, k, "silu", BF, seed=22)
    dy = normal(gen(23), m, n)
    dx, dw, db = uz.linear_backward(dy, x, p, preact=z, act="silu", need_bias=True)
    want = backward64(dy, x, w, z, "silu", BF)
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
        close(got, *want[name], name)


def test_linear_gradient_against_differences():
    """The directional derivative of sum(dy y) by central differences of the
    64-bit form agrees with the kernels' gradients."""
    g = gen(24)
    m, n, k = 24, 60, 70
    w, x, b = normal(g, n, k, scale=0.1), normal(g, m, k), normal(g, n)
    p = uz.pack_weight(w, gated=True)
    y, z = uz.linear(x, p, bias=b, act="swiglu", return_preact=True)
    dy = normal(g, m, n // 2)
    grads = uz.linear_backward(dy, x, p, preact=z, act="swiglu", need_bias=True, bias_dtype=F32)
    at = [x.double().cpu(), w.double().cpu(), b.double().cpu()]

    def f(x, w, b):
        return float((linear64(x, w, b, "swiglu", None, BF)[2] * dy.double().cpu()).sum())

    for i, gr in enumerate(grads):
        d = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        plus = [t + h * d if j == i else t for j, t in enumerate(at)]
        minus = [t - h * d if j == i else t for j, t in enumerate(at)]
        num = (f(*plus) - f(*minus)) / (2 * h)
        # each gradient is within 2^-7 of its terms (dz and the result are rounded to bf16), in directions that do not add up: sqrt of the squares' sum, and four times that
        slack = 4 * 2.0 ** -7 * float((gr.double().cpu() * d).norm())
        assert abs(float((gr.double().cpu() * d).sum()) - num) < slack + 1e-3


# ---- grouped ----------------------------------------------------------------------------

def offsets_of(counts, first=0):
    return torch.tensor([first] + counts).cumsum(0).to(torch.int32).to(DEV)


def check_grouped(counts, n, k, act, bias, first=0, tail=0, seed=30, backward=True, kind="normal"):
    g = gen(seed)
    e, t = len(counts), first + sum(counts) + tail
    gated = act == "swiglu"
    w = weight_of(kind, g, (e, n, k))
    x = normal(g, t, k)
    b = normal(g, e, n, dtype=bias) if bias is not None else None
    off = offsets_of(counts, first)
    p = uz.pack_weight(w, gated=gated)
    width = n // 2 if gated else n
    out = torch.full((t, width), 5.0, dtype=BF, device=DEV)
    y, z = uz.grouped_linear(x, off, p, bias=b, act=act, return_preact=True, out=out)
    fresh = uz.grouped_linear(x, off, p, bias=b, act=act)
    dy = normal(g, t, width)
    grads = uz.grouped_linear_backward(dy, x, off, p, preact=z, act=act, need_bias=True, bias_dtype=F32) if backward else None
    at = first
    for i, c in enumerate(counts):
        s = slice(at, at + c)
        at += c
        if c:
            z64, ez, y64, ey = linear64(x[s], w[i], None if b is None else b[i], act, None, BF)
            close(z[s], z64, ez, "preact of group %d" % i)
            close(y[s], y64, ey, "y of group %d" % i)
        if not backward:
            continue
        dx, dw, db = grads
        if c:
            want = backward64(dy[s], x[s], w[i], z[s], act, F32)
            close(dx[s], *want["dx"], "dx of group %d" % i)
            close(dw[i], *want["dw"], "dw of group %d" % i)
            close(db[i], *want["dbias"], "dbias of group %d" % i)
        else:
            assert (dw[i] == 0).all() and (db[i] == 0).all()
    for rows in (slice(0, first), slice(at, t)):
        assert (out[rows] == 5).all() and (fresh[rows] == 0).all()
        if backward:
            assert (grads[0][rows] == 0).all()
    assert torch.equal(fresh[first:at], y[first:at])


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1], [5, 0, 17, 2], [16, 16, 16, 16], [0, 64, 0, 0, 0, 0, 0, 0],
                                    [130, 0, 1, 255], [0, 0, 0, 700], [128, 256, 129, 127]])
@pytest.mark.parametrize("act,bias,n,k", [("none", None, 48, 72), ("silu", BF, 100, 130), ("swiglu", F32, 134, 64)])
def test_grouped(counts, act, bias, n, k):
    check_grouped(counts, n, k, act, bias)


def test_grouped_rows_of_no_group_are_left():
    check_grouped([3, 0, 40], 40, 64, "silu", BF, first=2, tail=5)
    check_grouped([300, 7], 70, 136, "silu", BF, first=9, tail=31)
    check_grouped([0, 0], 40, 64, "none", None, first=1, tail=3)


def test_grouped_many_experts():
    g = gen(31)
    counts = torch.randint(0, 9, (200,), generator=g).tolist()
    check_grouped(counts, 32, 64, "silu", BF)
    counts[77] = 900
    check_grouped(counts, 32, 64, "silu", BF)
    counts = torch.randint(0, 60, (130,), generator=g).tolist()
    check_grouped(counts, 32, 72, "swiglu", None)


def test_grouped_large_tiles():
    check_grouped([700, 1500, 0, 1900], 1100, 96, "swiglu", BF)


@pytest.mark.parametrize("offsets", [[-5, 3, 9], [0, 100, 200], [4, 2, 12], [12, 0, 3]])
def test_grouped_offsets_out_of_order_or_range_are_clamped(offsets):
    g = gen(32)
    t, n, k = 12, 40, 64
    x, w, dy = normal(g, t, k), normal(g, 2, n, k), normal(g, t, n)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    p = uz.pack_weight(w)
    y = uz.grouped_linear(x, off, p)
    uz.grouped_linear_backward(dy, x, off, p, need_bias=True)
    c = [min(max(o, 0), t) for o in offsets]
    for i in range(2):
        if c[i + 1] > c[i]:
            s = slice(c[i], c[i + 1])
            _, _, y64, ey = linear64(x[s], w[i], None, "none", None, BF)
            close(y[s], y64, ey, "y")


# ---- loss -----------------------------------------------------------------------------------

def check_loss(m, v, k, seed=40, scale=0.3, backward=True, targets=None, ignore=-100):
    g = gen(seed)
    x, w = normal(g, m, k), normal(g, v, k, scale=scale)
    t = torch.randint(0, v, (m,), generator=g).to(DEV) if targets is None else targets
    if targets is None and m > 2:
        t[1] = ignore
        t[0], t[-1] = v - 1, 0
    p = uz.pack_weight(w)
    loss, lse = uz.linear_cross_entropy(x, p, t, ignore_index=ignore)
    loss64_, lse64_, eloss, el, _, _ = loss64(x, w, t, ignore)
    close(lse, lse64_, el, "lse")
    close(loss, loss64_, eloss, "loss")
    if m > 2 and targets is None:
        assert loss[1] == 0
    if backward:
        dl = torch.randn(m, generator=g).to(DEV)
        dx, dw = uz.linear_cross_entropy_backward(dl, x, p, t, lse, ignore_index=ignore)
        wx, ww = loss_backward64(dl, x, w, t, ignore)
        close(dx, *wx, "dx")
        close(dw, *ww, "dw")
        assert torch.equal(uz.linear_cross_entropy_backward(dl, x, p, t, lse, ignore_index=ignore, need_weight=False)[0], dx)
        assert torch.equal(uz.linear_cross_entropy_backward(dl, x, p, t, lse, ignore_index=ignore, need_x=False)[1], dw)


@pytest.mark.parametrize("m", [1, 3, 64, 129, 300])
@pytest.mark.parametrize("v,k", [(1, 8), (2, 64), (17, 65), (1000, 72), (4097, 40), (9001, 136)])
def test_loss(m, v, k):
    check_loss(m, v, k)


def test_loss_large_tiles_and_pieces():
    check_loss(2050, 8300, 72)  # 256-wide tiles
    check_loss(20, 270001, 16)  # two pieces would need more tokens: one here


def test_loss_pieces():
    check_loss(17000, 5000, 16, backward=True)  # two pieces of 4,096 rows


def test_loss_gradient_of_a_mean():
    """One dloss for all tokens, halfway between two bf16 values, 2^-8 of itself away from both: rounded with the logit
    gradients it would be missing from, or added to, every target's alike.  The gradients' errors are those of two
    roundings that know nothing of each other, each uniform over up to +-2^-8 of a value: 2^-8 sqrt(2 / 3) = 0.0032 of the
    whole, 0.0039 and more with the other.  The unit's reduction also meets NaN and infinity where no token counts."""
    g = gen(48)
    m, v, k = 500, 3001, 136
    x, w = normal(g, m, k), normal(g, v, k, scale=0.02)
    t = torch.randint(0, v, (m,), generator=g).to(DEV)
    t[3:9] = -100
    t[11] = v
    dl = torch.full((m,), (1 + 2.0 ** -8) / 512, device=DEV)
    p = uz.pack_weight(w)
    _, lse = uz.linear_cross_entropy(x, p, t)
    dl[3], dl[4], dl[11] = float("nan"), float("inf"), 3e38
    dx, dw = uz.linear_cross_entropy_backward(dl, x, p, t, lse)
    dl[3], dl[4], dl[11] = 0, 0, 0
    t[11] = -100
    (wx, _), (ww, _) = loss_backward64(dl, x, w, t, -100)
    for got, want in ((dx, wx), (dw, ww)):
        off = (got.double().cpu() - want).norm() / want.norm()
        assert off < 2.0 ** -8 * (2 / 3) ** 0.5, off


def test_loss_gradients_of_any_size():
    """dloss over twenty decades; tiny; none at all."""
    g = gen(49)
    m, v, k = 40, 300, 64
    x, w = normal(g, m, k), normal(g, v, k, scale=0.1)
    t = torch.randint(0, v, (m,), generator=g).to(DEV)
    p = uz.pack_weight(w)
    _, lse = uz.linear_cross_entropy(x, p, t)
    for dl in (torch.logspace(-10, 10, m, device=DEV), torch.full((m,), 1e-30, device=DEV), torch.zeros(m, device=DEV)):
        dx, dw = uz.linear_cross_entropy_backward(dl, x, p, t, lse)
        (wx, ex), (ww, ew) = loss_backward64(dl, x, w, t, -100)
        close(dx, wx, ex, "dx")
        close(dw, ww, ew, "dw")


def test_loss_large_logits():
    check_loss(40, 600, 64, scale=20.0)


def test_loss_targets():
    g = gen(41)
    m, v, k = 6, 50, 64
    x, w = normal(g, m, k), normal(g, v, k, scale=0.2)
    t = torch.tensor([3, -100, 50, -1, 49, 2 ** 40], device=DEV)
    p = uz.pack_weight(w)
    loss, lse = uz.linear_cross_entropy(x, p, t)
    ok = torch.tensor([0, 4])
    good = t[ok.to(DEV)]
    l64, s64, el, es, _, _ = loss64(x[ok.to(DEV)], w, good, -100)
    close(loss[ok.to(DEV)], l64, el, "loss")
    assert loss[1] == 0 and torch.isnan(loss[[2, 3, 5]]).all() and torch.isfinite(lse).all()
    dl = torch.ones(m, device=DEV)
    dx, dw = uz.linear_cross_entropy_backward(dl, x, p, t, lse)
    assert (dx[[1, 2, 3, 5]] == 0).all()
    wx, ww = loss_backward64(dl[ok.to(DEV)], x[ok.to(DEV)], w, good, -100)
    close(dx[ok.to(DEV)], *wx, "dx")
    close(dw, *ww, "dw")
    # an ignored target inside the vocabulary
    t2 = torch.tensor([7, 7, 3, 7, 1, 0], device=DEV)
    assert torch.equal(uz.linear_cross_entropy(x, p, t2, ignore_index=7)[0] == 0, (t2 == 7))


def test_loss_infinite_logits():
    g = gen(42)
    m, v, k = 5, 300, 64
    x, w = normal(g, m, k).abs(), normal(g, v, k).abs()
    w[40, 3] = float("inf")            # logit 40 is +inf in every row
    x[1, 5] = float("nan")
    t = torch.tensor([40, 1, 2, 40, 299], device=DEV)
    loss, lse = uz.linear_cross_entropy(x, uz.pack_weight(w), t)
    z = x.double().cpu() @ w.double().cpu().T
    want = torch.logsumexp(z, 1)
    assert torch.equal(torch.isnan(lse.cpu()), torch.isnan(want)) and torch.equal(lse.cpu()[[0, 2, 3, 4]].double(), want[[0, 2, 3, 4]])
    lw = want - z.gather(1, t.cpu()[:, None])[:, 0]
    assert torch.equal(torch.isnan(loss.cpu()), torch.isnan(lw)) and torch.equal(loss.cpu()[[2, 4]].double(), lw[[2, 4]])
    w = normal(g, v, k).abs()
    w[:, 0] = float("-inf")            # every logit -inf
    loss, lse = uz.linear_cross_entropy(normal(g, 2, k).abs() + 0.5, uz.pack_weight(w), t[:2])
    assert (lse == float("-inf")).all() and torch.isnan(loss).all()


def test_loss_without_tokens():
    p = uz.pack_weight(normal(gen(43), 100, 40))
    x = torch.empty(0, 40, dtype=BF, device=DEV)
    t, f = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    assert uz.linear_cross_entropy(x, p, t)[0].shape == (0,)
    dx, dw = uz.linear_cross_entropy_backward(f, x, p, t, f)
    assert dx.shape == (0, 40) and (dw == 0).all()
