"""The products with packed weights where their contract has an edge: groups
out of order, rows of no group, the activations' tails, masked tokens, runs of
the contraction joined behind every epilogue.  The bounds are derived in
linear_testlib or beside the test."""
import math

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


# ---- groups out of order --------------------------------------------------------

OUT_OF_ORDER = {
    # tokens, offsets: descending pairs are empty groups, the others may lie anywhere and leave gaps
    "behind the first": (12, [4, 2, 12]), "before the first": (12, [12, 0, 3]), "ends low": (12, [0, 10, 5]),
    "gap": (12, [5, 10, 0, 3]), "two gaps": (40, [30, 36, 12, 20, 2, 7]), "none": (9, [9, 5, 0]),
    "many rows": (900, [700, 900, 300, 520, 1, 290]), "runs": (150, [100, 150, 20, 75])}


@pytest.mark.parametrize("name", sorted(OUT_OF_ORDER))
@pytest.mark.parametrize("n,k,act,out", [(40, 64, "none", BF), (134, 72, "swiglu", F32), (272, 1024, "silu", BF)])
def test_groups_out_of_order_keep_their_rows(name, n, k, act, out):
    """Rows of a group are its results, whatever the order of the groups, and all other rows of a new output are zero."""
    t, offsets = OUT_OF_ORDER[name]
    g = gen(1)
    e, width = len(offsets) - 1, n // 2 if act == "swiglu" else n
    x, w, dy = normal(g, t, k), normal(g, e, n, k, scale=0.1), normal(g, t, width)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    p = uz.pack_weight(w, gated=act == "swiglu")
    for _ in range(3):
        junk = [torch.full((t, c), float("nan"), device=DEV) for c in (width, k)]  # what a new output's memory may hold
        torch.cuda.synchronize()
        del junk
        y = uz.grouped_linear(x, off, p, act=act, out_dtype=out)
        _, z = uz.grouped_linear(x, off, p, act=act, return_preact=True)
        dx, dw, _ = uz.grouped_linear_backward(dy, x, off, p, preact=z, act=act)
        rest = torch.ones(t, dtype=torch.bool, device=DEV)
        for i in range(e):
            s = slice(offsets[i], offsets[i + 1])
            if offsets[i + 1] <= offsets[i]:
                assert (dw[i] == 0).all()
                continue
            rest[s] = False
            _, _, y64, ey = linear64(x[s], w[i], None, act, None, out)
            close(y[s], y64, ey, "y of group %d" % i)
            want = backward64(dy[s], x[s], w[i], z[s], act, BF)
            close(dx[s], *want["dx"], "dx of group %d" % i)
            close(dw[i], *want["dw"], "dw of group %d" % i)
        assert (y[rest] == 0).all() and (dx[rest] == 0).all()


@pytest.mark.parametrize("n,k,rows", [(40, 64, 9), (300, 136, 40)])
def test_many_groups_in_descending_order(n, k, rows):
    """A hundred groups from the last rows to the first, every third right below the one before, the others with gaps."""
    g = gen(12)
    offsets, at = [], 110 * rows
    for i in range(100):
        begin = at - 1 - int(torch.randint(0, rows, (1,), generator=g))
        offsets += [begin, at]
        at = begin if i % 3 == 0 else begin - int(torch.randint(0, 4, (1,), generator=g))
    t, e = 110 * rows + 3, len(offsets) - 1
    assert offsets[-2] >= 0
    x, w = normal(g, t, k), normal(g, e, n, k, scale=0.1)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    p = uz.pack_weight(w)
    junk = [torch.full((t, c), float("nan"), device=DEV) for c in (n, n, k)]
    torch.cuda.synchronize()
    del junk
    y, z = uz.grouped_linear(x, off, p, act="relu", return_preact=True)
    dx, _, _ = uz.grouped_linear_backward(y, x, off, p, preact=z, act="relu", need_weight=False)
    rest = torch.ones(t, dtype=torch.bool, device=DEV)
    for i in range(0, e, 2):
        s = slice(offsets[i], offsets[i + 1])
        rest[s] = False
        z64, ez, y64, ey = linear64(x[s], w[i], None, "relu", None, BF)
        close(z[s], z64, ez, "preact of group %d" % i)
        close(y[s], y64, ey, "y of group %d" % i)
        close(dx[s], *backward64(y[s], x[s], w[i], z[s], "relu", BF)["dx"], "dx of group %d" % i)
    for v in (y, z, dx):
        assert (v[rest] == 0).all()


@pytest.mark.parametrize("keep", [F32, BF])
@pytest.mark.parametrize("own_out", [False, True])
@pytest.mark.parametrize("offsets,t", [([3, 5, 5, 9], 20), ([100, 180, 181, 400], 450), ([0, 0, 0, 0], 40), ([7, 9, 2, 6], 12)])
@pytest.mark.parametrize("n,k,act", [(40, 64, "silu"), (134, 72, "swiglu"), (256, 2048, "gelu")])
def test_the_pre_activation_of_rows_of_no_group_is_zero(offsets, t, n, k, act, own_out, keep):
    g = gen(3)
    w, x = normal(g, 3, n, k, scale=0.1), normal(g, t, k)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    p = uz.pack_weight(w, gated=act == "swiglu")
    width = n // 2 if act == "swiglu" else n
    out = torch.full((t, width), 5.0, dtype=BF, device=DEV) if own_out else None
    junk = [torch.full((t, n), float("nan"), dtype=keep, device=DEV) for _ in range(4)]  # what new memory may hold
    torch.cuda.synchronize()
    del junk
    y, z = uz.grouped_linear(x, off, p, act=act, return_preact=True, preact_dtype=keep, out=out)
    rest = torch.ones(t, dtype=torch.bool, device=DEV)
    for i in range(3):
        s = slice(offsets[i], offsets[i + 1])
        if offsets[i + 1] > offsets[i]:
            rest[s] = False
            z64, ez, y64, ey = linear64(x[s], w[i], None, act, None, BF, keep)
            close(z[s], z64, ez, "preact")
            close(y[s], y64, ey, "y")
    assert (z[rest] == 0).all() and (y[rest] == (5 if own_out else 0)).all()


# ---- a stream of the call's own ----------------------------------------------------

def test_memory_of_a_call_on_another_stream_is_that_streams_own():
    """Blocks that the current stream's pending work still uses are not handed to a call on another stream."""
    m, n, k, act = 300, 320, 4096, "silu"
    g = gen(2)
    x, dy, wt = normal(g, m, k), normal(g, m, n), normal(g, n, k, scale=0.05)
    w, t, dl = uz.pack_weight(wt), torch.randint(0, n, (m,), generator=g).to(DEV), torch.ones(m, device=DEV)

    def calls(**kw):
        p = uz.pack_weight(wt, **kw)
        y, z = uz.linear(x, w, act=act, return_preact=True, **kw)
        dx, dw, db = uz.linear_backward(dy, x, w, preact=z, act=act, need_bias=True, **kw)
        loss, lse = uz.linear_cross_entropy(x, w, t, **kw)
        lx, lw = uz.linear_cross_entropy_backward(dl, x, w, t, lse, **kw)
        return [p.data, uz.unpack_weight(w, **kw), y, z, dx, dw, db, loss, lse, lx, lw]

    want = calls()
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = [torch.empty(s, dtype=torch.uint8, device=DEV) for s in (512, m * n * 2, m * n * 4, 1 << 21, 1 << 25, 1 << 25)]
    for b in busy:
        b.zero_()
    del b, busy  # free for the current stream's next work, and only for that
    side.wait_stream(main)
    got = calls(stream=side)
    blocks = [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
              if s["stream"] == side.cuda_stream]
    for r in got:
        assert any(a <= r.data_ptr() < e for a, e in blocks), (r.shape, r.dtype)
    main.wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


# ---- tails of the activations --------------------------------------------------------

STEP = 2.0 ** -24
K0, K1 = math.sqrt(2 / math.pi), 0.044715


def scalar64(z, act):
    """(act(z), act'(z), how far fp32 may be off relative to each of its terms, act's two terms) in 64 bits.  The
    function's argument passes through up to 2 (gelu: a rounded constant and a product) or 8 roundings (tanh form: 2 u);
    erfc(t) then moves by at most t (2 t + 1.2) = z^2 + 0.9 |z| times the argument's relative error, exp(-2 u) by 2 |u| times it,
    exp(-z^2 / 2) by z^2 / 2 times two roundings.  2^-20 covers the functions themselves and the products around them."""
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        slope = z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        rel = 2 * STEP * (z * z + 0.9 * z.abs()) + 2.0 ** -20
        return z * cdf, cdf + slope, rel, (cdf, slope)
    u2 = 2 * K0 * (z + K1 * z ** 3)
    s, r = torch.sigmoid(u2), torch.sigmoid(-u2)
    slope = z * s * r * 2 * K0 * (1 + 3 * K1 * z * z)
    return z * s, s + slope, 2 * 8 * STEP * u2.abs() + 2.0 ** -20, (s, slope)


TINY = 2.0 ** -120  # results that have run out of exponents: exp(2 u) passes fp32's range at 2 u = 88


@pytest.mark.parametrize("m", [1, 200])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_gelu_keeps_its_bits_in_the_negative_tail(m, act):
    z = torch.cat((torch.linspace(-12, 12, 1531), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 100.0, -13.0]))).to(BF)
    n = z.numel()
    w = torch.zeros(n, 8, dtype=BF, device=DEV)
    w[:, 0] = z.to(DEV)
    x = torch.zeros(m, 8, dtype=BF, device=DEV)
    x[:, 0] = 1
    p = uz.pack_weight(w)
    y, pre = uz.linear(x, p, act=act, out_dtype=F32, return_preact=True)
    z = z.double()
    assert torch.equal(pre.cpu().double(), z.expand(m, n))
    y64, _, rel, _ = scalar64(z, act)
    close(y, y64.expand(m, n), ((rel + STEP) * y64.abs() + TINY).expand(m, n), "y")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_gelus_gradient_keeps_its_bits_in_the_negative_tail(act):
    """One row of dy, whose bias gradient is the unrounded gradient of the pre-activation."""
    z = torch.cat((torch.linspace(-12, 12, 4000), torch.tensor([0.0, 1e-30, 100.0, -13.0])))
    n = z.numel()
    p = uz.pack_weight(torch.zeros(n, 8, dtype=BF, device=DEV))
    _, _, db = uz.linear_backward(torch.ones(1, n, device=DEV), None, p, preact=z[None].to(DEV), act=act, need_x=False,
                                  need_weight=False, need_bias=True, bias_dtype=F32)
    _, d64, rel, (a, b) = scalar64(z.double(), act)
    close(db, d64, (rel + STEP) * (a.abs() + b.abs()) + TINY, "gradient")


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
def test_huge_values_have_the_gradient_of_the_limit(act):
    """0 to the left, 1 to the right (swiglu: times the other half, 1 here), past where z^2 and z^3 leave fp32."""
    big = torch.tensor([1e3, 1e10, 1e13, 2e19, 1e25, 3e38])
    z = torch.cat((big, -big))
    n = z.numel()
    gated = act == "swiglu"
    pre = torch.cat((z, torch.ones(n)))[None] if gated else z[None]
    p = uz.pack_weight(torch.zeros(pre.shape[1], 8, dtype=BF, device=DEV), gated=gated)
    _, _, db = uz.linear_backward(torch.ones(1, n, device=DEV), None, p, preact=pre.to(DEV), act=act, need_x=False,
                                  need_weight=False, need_bias=True, bias_dtype=F32)
    assert torch.equal(db.cpu()[:n], (z > 0).float()), db
    if gated:
        assert torch.equal(db.cpu()[n:], z.clamp(min=0))


# ---- masked tokens of the loss ----------------------------------------------------------

@pytest.mark.parametrize("m,v,k", [(5, 50, 64), (70, 1000, 65), (300, 515, 1024), (1030, 4200, 72)])
@pytest.mark.parametrize("pad", [0, 3])
def test_masked_tokens_may_hold_anything(m, v, k, pad):
    """Rows of padding hold infinities and NaNs: tokens that do not count leave no trace in the gradients."""
    g = gen(4)
    x = torch.zeros(m, k + pad, dtype=BF, device=DEV)[:, :k]
    x.copy_(normal(g, m, k))
    w = normal(g, v, k, scale=0.1)
    t = torch.randint(0, v, (m,), generator=g).to(DEV)
    off = torch.randperm(m, generator=g)[:max(3, m // 4)].to(DEV)
    t[off[0::3]], t[off[1::3]], t[off[2::3]] = -100, v, -1
    p = uz.pack_weight(w)
    clean = x.clone()
    clean[off] = 0
    x[off[0::2]], x[off[1::2]] = float("nan"), float("inf")
    before = x.clone()
    loss, lse = uz.linear_cross_entropy(x, p, t)
    dl = torch.randn(m, generator=g).to(DEV)
    dl[off[0]] = float("nan")
    dx, dw = uz.linear_cross_entropy_backward(dl, x, p, t, lse)
    kept = torch.where((t >= 0) & (t < v), t, -100)
    l64, s64, el, es, _, _ = loss64(clean, w, kept, -100)
    on = torch.ones(m, dtype=torch.bool, device=DEV)
    on[off] = False
    close(loss[on], l64[on.cpu()], el[on.cpu()], "loss")
    close(lse[on], s64[on.cpu()], es[on.cpu()], "lse")
    assert (loss[t == -100] == 0).all() and torch.isnan(loss[(t == -1) | (t == v)]).all()
    dl[off[0]] = 0
    wx, ww = loss_backward64(dl, clean, w, kept, -100)
    close(dx, *wx, "dx")
    close(dw, *ww, "dw")
    assert (dx[off] == 0).all()
    one = uz.linear_cross_entropy_backward(dl, x, p, t, lse, need_x=False)[1]
    assert torch.equal(one, dw)
    assert torch.equal(uz.linear_cross_entropy_backward(dl, x, p, t, lse, need_weight=False)[0], dx)
    assert torch.equal(x.view(torch.int16), before.view(torch.int16))


# ---- runs of the contraction, joined behind every epilogue --------------------------------

def cut(w, x, **kw):
    """Whether a forward call with these rows of x (aligned, so not staged) has its contraction cut: only then does it need
    a workspace."""
    a = uz.uzip_linear_args(x=x.data_ptr(), x_stride=x.stride(0), tokens=x.shape[0], y=x.data_ptr(), y_stride=1 << 20,
                            y_dtype=uz.UZIP_BF16, **kw)
    return uz.uzip_linear_workspace_size(w._c, a) > 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("bias", [BF, F32, None])
@pytest.mark.parametrize("m,n,k,act", [(100, 256, 2048, "swiglu"), (40, 516, 4096, "swiglu"), (100, 300, 2048, "gelu"),
                                       (130, 515, 1096, "silu")])
def test_joined_runs_of_linear(m, n, k, act, bias, out):
    g = gen(5)
    gated = act == "swiglu"
    x, w = normal(g, m, k), normal(g, n, k, scale=0.02)
    b = None if bias is None else normal(g, n, dtype=bias)
    r = normal(g, m, n // 2 if gated else n, dtype=out)
    p = uz.pack_weight(w, gated=gated)
    assert cut(p, x, act=uz.ACTIVATIONS[act])
    for keep in (F32, BF):
        y, z = uz.linear(x, p, bias=b, act=act, residual=r, out_dtype=out, return_preact=True, preact_dtype=keep)
        z64, ez, y64, ey = linear64(x, w, b, act, r, out, keep)
        close(z, z64, ez, "preact")
        close(y, y64, ey, "y")


@pytest.mark.parametrize("out,keep,grad", [(BF, F32, BF), (F32, BF, F32), (F32, F32, BF)])
@pytest.mark.parametrize("act,bias", [("silu", BF), ("swiglu", F32), ("none", None)])
@pytest.mark.parametrize("counts,n,k,runs", [([40, 0, 60], 256, 4096, True), ([100, 300, 7], 130, 1096, True),
                                             ([3, 0, 9], 256, 520, False), ([400, 500, 300], 1100, 136, False)])
def test_grouped_types_and_joined_runs(counts, n, k, runs, act, bias, out, keep, grad):
    """fp32 results, pre-activations in bf16 and dy in fp32, whole and in runs of the contraction."""
    g = gen(6)
    e, first, t = len(counts), 2, sum(counts) + 5
    gated = act == "swiglu"
    width = n // 2 if gated else n
    w, x = normal(g, e, n, k, scale=0.05), normal(g, t, k)
    b = None if bias is None else normal(g, e, n, dtype=bias)
    off = torch.tensor([first] + counts).cumsum(0).to(torch.int32).to(DEV)
    p = uz.pack_weight(w, gated=gated)
    assert cut(p, x, offsets=off.data_ptr(), act=uz.ACTIVATIONS[act]) == runs
    y, z = uz.grouped_linear(x, off, p, bias=b, act=act, out_dtype=out, return_preact=True, preact_dtype=keep)
    dy = normal(g, t, width, dtype=grad)
    dx, dw, db = uz.grouped_linear_backward(dy, x, off, p, preact=z, act=act, need_bias=True, bias_dtype=F32)
    assert y.dtype is out and z.dtype is keep
    at = first
    for i, c in enumerate(counts):
        s = slice(at, at + c)
        at += c
        if not c:
            assert (dw[i] == 0).all() and (db[i] == 0).all()
            continue
        z64, ez, y64, ey = linear64(x[s], w[i], None if b is None else b[i], act, None, out, keep)
        close(z[s], z64, ez, "preact")
        close(y[s], y64, ey, "y")
        want = backward64(dy[s], x[s], w[i], z[s], act, F32)
        close(dx[s], *want["dx"], "dx")
        close(dw[i], *want["dw"], "dw")
        close(db[i], *want["dbias"], "dbias")
    for v in (y, z, dx):
        assert (v[:first] == 0).all() and (v[at:] == 0).all()


@pytest.mark.parametrize("m,v,k,runs", [(100, 300, 1024, True), (33, 4097, 2048, True), (200, 129, 4096, True),
                                        (64, 5000, 1000, True), (129, 1, 512, False)])
def test_joined_runs_of_the_loss(m, v, k, runs):
    """The loss's own join and that of the logit gradients: odd vocabularies, targets at both ends, masked tokens."""
    g = gen(7)
    x, w = normal(g, m, k), normal(g, v, k, scale=0.05)
    t = torch.randint(0, v, (m,), generator=g).to(DEV)
    t[0], t[1], t[2] = v - 1, 0, -100
    p = uz.pack_weight(w)
    a = uz.uzip_loss_args(x=x.data_ptr(), x_stride=k, tokens=m, target=t.data_ptr(), ignore_index=-100, loss=x.data_ptr(),
                          lse=x.data_ptr())
    tiles = 8 * m * -(-v // 128) + 4 * m + 3 * 256
    # (more than the tokens' references, sums and picked logits, with their alignment)
    assert (uz.uzip_linear_cross_entropy_workspace_size(p._c, a) > tiles) == runs
    loss, lse = uz.linear_cross_entropy(x, p, t)
    l64, s64, el, es, _, _ = loss64(x, w, t, -100)
    close(loss, l64, el, "loss")
    close(lse, s64, es, "lse")
    dl = torch.randn(m, generator=g).to(DEV)
    dx, dw = uz.linear_cross_entropy_backward(dl, x, p, t, lse)
    wx, ww = loss_backward64(dl, x, w, t, -100)
    close(dx, *wx, "dx")
    close(dw, *ww, "dw")


def test_joined_runs_of_the_loss_with_infinite_logits():
    g = gen(8)
    m, v, k = 70, 300, 1024
    x, w = normal(g, m, k).abs(), normal(g, v, k).abs()
    w[40, 3], x[1, 5] = float("inf"), float("nan")
    t = torch.randint(0, v, (m,), generator=g).to(DEV)
    t[0] = 40
    loss, lse = uz.linear_cross_entropy(x, uz.pack_weight(w), t)
    z = x.double().cpu() @ w.double().cpu().T
    want = torch.logsumexp(z, 1)
    assert torch.equal(torch.isnan(lse.cpu()), torch.isnan(want)) and bool((lse.cpu()[~torch.isnan(want)] == float("inf")).all())
    lw = want - z.gather(1, t.cpu()[:, None])[:, 0]
    assert torch.equal(torch.isnan(loss.cpu()), torch.isnan(lw))
    w = normal(g, v, k).abs()
    w[:, 0] = float("-inf")
    loss, lse = uz.linear_cross_entropy(x[:2] + 0.5, uz.pack_weight(w), t[:2])
    assert lse[0] == float("-inf") and torch.isnan(lse[1]) and torch.isnan(loss).all()


# ---- every shape of workgroup of the product for few rows ---------------------------------

@pytest.mark.parametrize("m", [1, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("n,k,act", [(4096, 200, "none"), (4097, 72, "silu"), (8192, 136, "swiglu"), (8194, 65, "swiglu"),
                                     (24576, 64, "swiglu"), (24578, 72, "swiglu")])
def test_few_rows_on_both_sides_of_each_rule(m, n, k, act):
    """256 and 257 row blocks; gated 256, 257, 768 and 769 of each half."""
    g = gen(10)
    gated = act == "swiglu"
    x, w, b = normal(g, m, k), normal(g, n, k, scale=0.05), normal(g, n)
    r = normal(g, m, n // 2 if gated else n)
    y, z = uz.linear(x, uz.pack_weight(w, gated=gated), bias=b, act=act, residual=r, return_preact=True)
    z64, ez, y64, ey = linear64(x, w, b, act, r, BF)
    close(z, z64, ez, "preact")
    close(y, y64, ey, "y")


@pytest.mark.parametrize("counts", [[16, 0, 3, 13], [40, 0, 0, 24]])
@pytest.mark.parametrize("n,act", [(1024, "silu"), (1040, "silu"), (6144, "swiglu"), (6176, "swiglu")])
def test_few_grouped_rows_on_both_sides_of_each_rule(counts, n, act):
    g = gen(11)
    k, e, t = 136, len(counts), sum(counts)
    gated = act == "swiglu"
    x, w = normal(g, t, k), normal(g, e, n, k, scale=0.05)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    y = uz.grouped_linear(x, off, uz.pack_weight(w, gated=gated), act=act)
    at = 0
    for i, c in enumerate(counts):
        if c:
            _, _, y64, ey = linear64(x[at:at + c], w[i], None, act, None, BF)
            close(y[at:at + c], y64, ey, "y of group %d" % i)
        at += c


# ---- the largest calls, and captured ones on other streams ----------------------------------

def small(seed, *shape):
    """-1, 0 and 1: sums of their products are exact."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device=DEV, dtype=torch.int8).to(BF)


MOST = 1 << 25  # tokens of a call


def test_the_most_tokens_of_a_product():
    n, k = 16, 64
    w, x = small(1, n, k), small(2, MOST, k)
    p = uz.pack_weight(w)
    y = uz.linear(x, p)
    for c in range(0, MOST, 1 << 22):
        s = slice(c, c + (1 << 22))
        assert torch.equal(y[s].float(), x[s].float() @ w.float().t())
    at = torch.tensor([0, 1, 255, 256, MOST // 2 + 77, MOST - 257, MOST - 1], device=DEV)
    dy = torch.zeros(MOST, n, dtype=BF, device=DEV)
    dy[at] = small(3, at.numel(), n)
    dx, dw, db = uz.linear_backward(dy, x, p, need_bias=True, bias_dtype=F32)
    assert torch.equal(dx[at].float(), dy[at].float() @ w.float())
    dx[at] = 0
    assert not bool(dx.any())
    assert torch.equal(dw.float(), dy[at].float().t() @ x[at].float()) and torch.equal(db, dy[at].float().sum(0))


def test_the_most_tokens_of_a_loss():
    """Logits are exact.  A sum of 16 exponentials good to 2^-20, its logarithm and lse each rounded once, below 2^7."""
    v, k = 16, 64
    w, x = small(4, v, k), small(5, MOST, k)
    t = torch.arange(MOST, device=DEV) % (v + 1) - 1  # (every 17th target is no row of w)
    p = uz.pack_weight(w)
    loss, lse = uz.linear_cross_entropy(x, p, t, ignore_index=-1)
    bound = 16 * STEP + 2.0 ** -20 + 2 * 2.0 ** 7 * STEP
    for c in range(0, MOST, 1 << 22):
        s = slice(c, c + (1 << 22))
        z = (x[s].float() @ w.float().t()).double()
        want = torch.logsumexp(z, 1)
        assert float((lse[s].double() - want).abs().max()) < bound
        picked = z.gather(1, t[s].clamp(min=0)[:, None])[:, 0]
        off = (loss[s].double() - torch.where(t[s] < 0, 0.0, want - picked)).abs()
        assert float(off.max()) < bound + 2.0 ** 7 * STEP
    at = torch.tensor([1, 300, MOST // 2 + 78, MOST - 1], device=DEV)
    assert bool((t[at] >= 0).all())
    g = torch.zeros(MOST, device=DEV)
    g[at] = 1.0
    dx, dw = uz.linear_cross_entropy_backward(g, x, p, t, lse, ignore_index=-1)
    wx, ww = loss_backward64(g[at], x[at], w, t[at], -1)
    close(dx[at], *wx, "dx")
    close(dw, *ww, "dw")
    dx[at] = 0
    assert not bool(dx.any())


def test_the_most_matrices_of_a_stack():
    e, n, k = 65535, 16, 64
    w = small(6, e, n, k)
    p = uz.pack_weight(w)
    assert torch.equal(uz.unpack_weight(p), w)
    for rows in ({0: 3, 777: 1, 65534: 5}, {0: 30, 64: 700, 40000: 1, 65533: 2, 65534: 300}):
        counts = torch.zeros(e, dtype=torch.int64)
        for i, c in rows.items():
            counts[i] = c
        off = torch.cat((torch.tensor([2]), 2 + counts.cumsum(0))).to(torch.int32).to(DEV)
        t = int(off[-1]) + 3
        x, dy = small(7, t, k), small(8, t, n)
        of = torch.repeat_interleave(torch.arange(e), counts).to(DEV)
        y = uz.grouped_linear(x, off, p)
        dx, dw, db = uz.grouped_linear_backward(dy, x, off, p, need_bias=True, bias_dtype=F32)
        s = slice(2, t - 3)
        assert torch.equal(y[s].float(), (w[of].float() @ x[s].float()[:, :, None])[:, :, 0])
        assert torch.equal(dx[s].float(), (dy[s].float()[:, None] @ w[of].float())[:, 0])
        for i in rows:
            r = s.start + int(counts[:i].sum())
            r = slice(r, r + rows[i])
            assert torch.equal(dw[i].float(), (dy[r].float().t() @ x[r].float()).to(BF).float())
            assert torch.equal(db[i], dy[r].float().sum(0))
        hit = torch.tensor(sorted(rows), device=DEV)
        dw[hit], db[hit] = 0, 0
        assert not bool(dw.any()) and not bool(db.any())
        for v in (y, dx):
            assert not bool(v[:2].any()) and not bool(v[t - 3:].any())


def test_captured_on_another_stream_and_from_packing_on():
    """Packing without a wait, products on a second stream of the capture, their memory the graph's; replayed with new
    values between eager calls."""
    g = gen(9)
    m, n, k = 100, 256, 4096
    wt, x, dy = normal(g, n, k, scale=0.02), normal(g, m, k), normal(g, m, n)
    t, dl = torch.randint(0, n, (m,), generator=g).to(DEV), torch.ones(m, device=DEV)
    off = torch.tensor([60, 90, 10, 40], dtype=torch.int32, device=DEV)
    stack = normal(g, 3, n, k, scale=0.02)
    side = torch.cuda.Stream()

    def calls(stream):
        main = torch.cuda.current_stream()
        kw = {}
        if stream is not None:
            stream.wait_stream(main)
            kw["stream"] = stream
        w, ws = uz.pack_weight(wt, trim=False, **kw), uz.pack_weight(stack, trim=False, **kw)
        y, z = uz.linear(x, w, act="gelu", return_preact=True, **kw)
        dx, dw, db = uz.linear_backward(dy, x, w, preact=z, act="gelu", need_bias=True, **kw)
        gy, gz = uz.grouped_linear(x, off, ws, act="silu", return_preact=True, **kw)
        gdx, gdw, _ = uz.grouped_linear_backward(dy, x, off, ws, preact=gz, act="silu", **kw)
        loss, lse = uz.linear_cross_entropy(x, w, t, **kw)
        lx, lw = uz.linear_cross_entropy_backward(dl, x, w, t, lse, **kw)
        back = uz.unpack_weight(w, **kw)
        if stream is not None:
            main.wait_stream(stream)
        return [y, z, dx, dw, db, gy, gz, gdx, gdw, loss, lse, lx, lw, back]

    calls(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(side)
    for i in range(4):
        for v, s in ((wt, 0.02), (x, 1.0), (dy, 1.0), (stack, 0.02)):
            v.copy_(normal(g, *v.shape, scale=s))
        want = [o.clone() for o in calls(None)]
        graph.replay()
        if i & 1:
            torch.cuda.synchronize()
        eager = calls(side)
        torch.cuda.synchronize()
        for a, b, c in zip(want, outs, eager):
            for o in (b, c):
                assert torch.equal(a.reshape(-1).view(torch.uint8), o.reshape(-1).view(torch.uint8))
