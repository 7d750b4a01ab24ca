"""The router, its gradient and the expert layer against plain forms in 64
bits, with the bounds of linear_testlib."""
import math

import pytest
import torch

import lossless_compression_float_amd as uz
from linear_testlib import ACC, FUN, HALF, close, linear64

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


# ---- the router -----------------------------------------------------------------

def choice64(logits, k, scores, bias):
    """The choice one place at a time, and the scores, on the CPU in 64 bits."""
    z = logits.double().cpu()
    p = torch.sigmoid(z) if scores == "sigmoid" else torch.softmax(z, 1)
    by = z.clone() if bias is None else torch.where(z > -math.inf, torch.sigmoid(z) + bias.double().cpu(), -math.inf)
    by = torch.where(by.isnan(), -math.inf, by)
    experts = torch.full((z.shape[0], k), -1)
    for t in range(z.shape[0]):
        for j in range(k):
            top = by[t].max()
            if top == -math.inf:
                break
            e = int((by[t] == top).nonzero()[0])
            experts[t, j] = e
            by[t, e] = -math.inf
    return experts, p


def weights64(p, experts, renorm, scale):
    w = torch.where(experts >= 0, p.gather(1, experts.clamp(min=0)), 0.0)
    s = w.sum(1, keepdim=True)
    return scale * (torch.where(s > 0, w / s.clamp(min=1e-300), w) if renorm else w)


def check_groups(r):
    """order and offsets from the experts: stable, those without an expert behind the last."""
    flat = r.experts.cpu().reshape(-1).long()
    last = torch.where(flat < 0, r.num_experts, flat)
    assert torch.equal(r.order.cpu().long(), torch.sort(last, stable=True).indices)
    counts = torch.bincount(last, minlength=r.num_experts + 1)[:r.num_experts]
    assert r.offsets.cpu().tolist() == [0] + counts.cumsum(0).tolist()


ROUTES = [(1, 1, 1), (1, 128, 8), (3, 5, 5), (4, 64, 6), (17, 65, 3), (63, 60, 4), (64, 128, 8), (65, 256, 8), (100, 257, 2),
          (777, 60, 4), (1000, 1024, 64), (4097, 7, 1), (5000, 64, 8)]


@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("tokens,num,k", ROUTES)
def test_route(tokens, num, k, scores, renorm):
    g = gen(tokens * 31 + num)
    dtype = BF if tokens % 2 else F32
    wide = normal(g, tokens, num + 3, scale=2.0, dtype=dtype)
    logits = wide[:, 1:num + 1]  # rows that are no multiple of anything apart
    bias = normal(g, num, scale=0.2, dtype=F32) if scores == "sigmoid" and num % 2 == 0 else None
    r = uz.moe_route(logits, k, scores=scores, bias=bias, renormalize=renorm, scale=1.5)
    experts, p = choice64(logits, k, scores, bias)
    assert torch.equal(r.experts.cpu().long(), experts)
    check_groups(r)
    want = weights64(p, experts, renorm, 1.5)
    # e^x of an argument up to 20 off by 2^-24 of it, sums of up to 1,024 values, three more roundings
    close(r.weights, want, want * (40 + num + 16) * 2.0 ** -23, "weights")


def test_route_masks_nans_and_infinities():
    ninf, nan, inf = -math.inf, math.nan, math.inf
    rows = [[ninf] * 6, [ninf, 1, ninf, ninf, ninf, ninf], [0, 0, 0, 0, 0, 0], [nan, 1, 2, 3, 4, 5], [nan] * 6,
            [inf, 1, inf, 0, 0, 0], [-3e38, 3e38, 0, ninf, ninf, 1], [0.0, -0.0, ninf, ninf, 0.0, ninf]]
    logits = torch.tensor(rows, device=DEV)
    for tokens in (len(rows), 40 * len(rows)):
        z = logits.repeat(tokens // len(rows), 1)
        for scores in ("softmax", "sigmoid"):
            r = uz.moe_route(z, 3, scores=scores, renormalize=True)
            e, w = r.experts[:8].cpu().tolist(), r.weights[:8].cpu()
            assert torch.equal(r.experts[-8:].cpu(), r.experts[:8].cpu())
            assert e[0] == [-1] * 3 and w[0].tolist() == [0] * 3
            assert e[1] == [1, -1, -1] and w[1].tolist() == [1, 0, 0]
            assert e[2] == [0, 1, 2] and torch.allclose(w[2], torch.full((3,), 1 / 3), rtol=1e-6)
            assert e[3] == [5, 4, 3] and w[3].isnan().all()
            assert e[4] == [-1] * 3 and w[4].tolist() == [0] * 3
            assert e[5][:2] == [0, 2] and not w[5].isnan().any()
            if scores == "softmax":
                assert w[5].tolist() == [0.5, 0.5, 0]
            assert e[6] == [1, 5, 2] and not w[6].isnan().any()
            assert sorted(e[7]) == [0, 1, 4] and not w[7].isnan().any()  # (both zeros are equal in the scores)
            check_groups(r)


def test_sigmoid_scores_of_very_negative_logits_keep_their_ratio():
    r = uz.moe_route(torch.tensor([[-200.0, -201.0, -300.0]], device=DEV), 2, scores="sigmoid")
    assert r.experts.tolist() == [[0, 1]]
    assert torch.allclose(r.weights.cpu(), torch.softmax(torch.tensor([[-200.0, -201.0]]), 1), rtol=1e-6)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_sigmoid_scores_that_all_vanish_keep_their_ratio(dtype, bias):
    """Below e^-745, masked by the type's lowest value among them."""
    low = torch.finfo(dtype).min
    rows = [[low] * 4, [-720.0, -721, low, low], [-1e5, -1e5, -1.5e5, low], [-800, -801, -802, -math.inf], [-660, -670, -672, -1000],
            [low, 0.5, low, low]]
    logits = torch.tensor(rows, device=DEV).to(dtype)
    b = torch.zeros(4, device=DEV) if bias else None
    for n in (1, 20):
        z = logits.repeat(n, 1)
        r = uz.moe_route(z, 3, scores="sigmoid", bias=b)
        # scores of exactly 0 are equal to the biased choice, which then takes the lowest index
        s = torch.nn.functional.logsigmoid(z.double()).cpu().gather(1, r.experts.cpu().long())
        want = torch.softmax(s, 1)
        # one rounding to 24 bits, exponents of less than 1,000 in 64 bits
        close(r.weights, want, want * (2.0 ** -24 + 1e-12) + 2.0 ** -126, "weights")
        dw = normal(gen(n), z.shape[0], 3, dtype=F32)
        d = dw.double().cpu()
        rest = torch.sigmoid(-z.double()).cpu().gather(1, r.experts.cpu().long())
        dz = torch.zeros(z.shape, dtype=torch.float64).scatter(1, r.experts.cpu().long(), want * rest * (d - (d * want).sum(1, keepdim=True)))
        got = uz.moe_route_backward(dw, z, r)
        close(got, dz, dz.abs() * (HALF[dtype] + 2.0 ** -24) + d.abs().max() * 1e-12, "dlogits")


def test_a_bias_decides_and_does_not_weigh():
    z = torch.zeros((70, 8), device=DEV)
    bias = torch.tensor([0, 3, 0, 2.0, -1, 0, 1, 0], device=DEV)
    r = uz.moe_route(z, 3, scores="sigmoid", bias=bias)
    assert (r.experts == torch.tensor([1, 3, 6], device=DEV)).all()
    assert torch.allclose(r.weights, torch.full_like(r.weights, 1 / 3))


def test_group_drops_what_is_no_expert_and_joins_what_is_named_twice():
    e = torch.tensor([[2, 2, 0], [5, -1, 1], [1, 2, 1], [0, 0, 0], [7, -9, 6]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1, 2, 4], [1, 2, 4], [1, 2, 4], [1, 2, 4], [1, 2, 4.0]], device=DEV)
    for n in (1, 30):
        r = uz.moe_group(e.repeat(n, 1), w.repeat(n, 1), 5)
        assert r.experts[-5:].tolist() == [[2, -1, 0], [-1, -1, 1], [1, 2, -1], [0, -1, -1], [-1, -1, -1]]
        assert r.weights[-5:].tolist() == [[3, 0, 4], [0, 0, 4], [5, 2, 0], [7, 0, 0], [0, 0, 0]]
        check_groups(r)
    assert e[0].tolist() == [2, 2, 0] and w[0].tolist() == [1, 2, 4]


def test_no_tokens():
    r = uz.moe_route(torch.empty((0, 9), device=DEV), 2)
    assert r.offsets.tolist() == [0] * 10 and r.experts.shape == (0, 2)
    assert uz.moe_route_backward(torch.empty((0, 2), device=DEV), torch.empty((0, 9), device=DEV), r).shape == (0, 9)


@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("tokens,num,k", [(1, 1, 1), (5, 5, 5), (130, 64, 6), (77, 130, 8), (9, 1000, 40)])
def test_route_backward(tokens, num, k, scores, renorm):
    g = gen(num)
    for dtype in (F32, BF):
        logits = normal(g, tokens, num + 2, scale=1.5, dtype=dtype)[:, :num]
        dw = normal(g, tokens, k, dtype=F32)
        r = uz.moe_route(logits, k, scores=scores, renormalize=renorm, scale=0.7)
        got = uz.moe_route_backward(dw, logits, r)
        z = logits.double().cpu().requires_grad_(True)
        p = torch.sigmoid(z) if scores == "sigmoid" else torch.softmax(z, 1)
        w = p.gather(1, r.experts.cpu().long())
        w = 0.7 * (w / w.sum(1, keepdim=True) if renorm else w)
        want, = torch.autograd.grad(w, z, dw.double().cpu())
        # dz_i = p_i (g_i - sum g p): each factor off by what the scores are (see test_route), the difference by both
        size = 0.7 * dw.double().cpu().abs().max(1, keepdim=True).values
        share = (w / w.sum(1, keepdim=True)).detach() if renorm else w.detach() / 0.7
        each = p.detach() if not renorm else torch.zeros_like(p).detach().scatter(1, r.experts.cpu().long(), share)
        # (and the 64-bit form's own roundings: where renorm leaves exactly nothing of p (g - sum g p), it leaves 2^-53 of them)
        bound = 4 * each * size * (40 + num + 16) * 2.0 ** -23 + 64 * p.detach() * size * 2.0 ** -53
        close(got, want, bound + HALF[dtype] * (want.abs() + bound), "dlogits")


def test_route_backward_against_differences():
    g = gen(5)
    logits, dw = normal(g, 6, 20, dtype=F32), normal(g, 6, 4, dtype=F32)
    for scores in ("softmax", "sigmoid"):
        for renorm in (True, False):
            r = uz.moe_route(logits, 4, scores=scores, renormalize=renorm)
            got = uz.moe_route_backward(dw, logits, r).double().cpu()
            step = 2.0 ** -13
            for e in range(20):
                up, down = (logits.double().cpu() for _ in range(2))
                up[:, e] += step
                down[:, e] -= step
                ex = r.experts.cpu().long()

                def value(z):
                    p = torch.sigmoid(z) if scores == "sigmoid" else torch.softmax(z, 1)
                    return (weights64(p, ex, renorm, 1.0) * dw.double().cpu()).sum(1)
                # the third derivative of a score is below 1, dw below 5: step^2 * 4 * 5 / 6; fp32 results
                assert torch.allclose(got[:, e], (value(up) - value(down)) / (2 * step), atol=1e-6, rtol=0)


def test_route_backward_of_tokens_without_experts_and_of_nans():
    ninf = -math.inf
    logits = torch.tensor([[ninf] * 4, [1, ninf, ninf, 2], [math.nan, 0, 1, 2]], device=DEV)
    for scores in ("softmax", "sigmoid"):
        for renorm in (True, False):
            r = uz.moe_route(logits, 3, scores=scores, renormalize=renorm)
            d = uz.moe_route_backward(torch.ones((3, 3), device=DEV), logits, r).cpu()
            assert d[0].tolist() == [0] * 4 and torch.isfinite(d[1]).all() and d[1, 1] == d[1, 2] == 0
            assert d[2].isnan().all()


# ---- the layer --------------------------------------------------------------------

def layer64(x, r, up, down, act, up_bias, down_bias, residual, out_dtype):
    """(y, its bound) on the CPU in 64 bits from the routing's own experts and weights."""
    experts, weights = r.experts.cpu(), r.weights.double().cpu()
    y = torch.zeros((x.shape[0], down.shape[1]), dtype=torch.float64)
    err, size = torch.zeros_like(y), torch.zeros_like(y)
    for e in range(up.shape[0]):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        if t.numel() == 0:
            continue
        _, _, h, eh = linear64(x[t], up[e], None if up_bias is None else up_bias[e], act, None, BF)
        d = down[e].double().cpu()
        w = weights[t, j][:, None]
        eh = eh + 2.0 ** -23 * h.abs()  # (the weight times the activation, rounded to fp32 before)
        o = h @ d.T
        eo = eh @ d.abs().T + (d.shape[1] * r.k + 24) * ACC * ((h.abs() + eh) @ d.abs().T)
        if down_bias is not None:
            o = o + down_bias[e].double().cpu()
            eo = eo + ACC * o.abs()
        y.index_add_(0, t, w * o)
        err.index_add_(0, t, w.abs() * eo)
        size.index_add_(0, t, w.abs() * o.abs())
    err = err + (r.k + 2) * ACC * size
    if residual is not None:
        y = y + residual.double().cpu()
    err = err + ACC * y.abs()
    return y, err + HALF[out_dtype] * (y.abs() + err)


def layer(tokens, num, k, d, f, act="swiglu", bias=False, residual=False, out_dtype=BF, seed=0, logits=None, out_cols=None,
          x=None):
    g = gen(seed + tokens + 7 * num + d)
    rows = 2 * f if act == "swiglu" else f
    up, down = normal(g, num, rows, d, scale=0.05), normal(g, num, out_cols or d, f, scale=0.05)
    x = normal(g, tokens, d) if x is None else x
    logits = normal(g, tokens, num, dtype=F32) if logits is None else logits
    r = uz.moe_route(logits, k) if not isinstance(logits, uz.Routing) else logits
    bd = F32 if d % 2 else BF
    ub = normal(g, num, rows, scale=0.3, dtype=bd) if bias else None
    db = normal(g, num, out_cols or d, scale=0.3, dtype=bd) if bias else None
    res = normal(g, tokens, out_cols or d, dtype=out_dtype) if residual else None
    y = uz.moe(x, r, uz.pack_weight(up, gated=act == "swiglu"), uz.pack_weight(down), act=act, up_bias=ub, down_bias=db,
               residual=res, out_dtype=out_dtype)
    want, bound = layer64(x, r, up, down, act, ub, db, res, out_dtype)
    close(y, want, bound, "y")
    return y, x, r, up, down


LAYERS = [(1, 1, 1, 16, 16), (1, 128, 8, 64, 48), (1, 8, 2, 512, 1024), (2, 3, 3, 65, 17), (5, 4, 2, 1, 1), (13, 7, 3, 127, 133),
          (15, 16, 4, 256, 96), (16, 16, 4, 256, 96), (17, 16, 4, 256, 96), (31, 2, 1, 130, 200), (32, 5, 5, 64, 64),
          (33, 40, 8, 192, 80), (63, 8, 8, 128, 64), (64, 64, 8, 128, 96), (65, 64, 8, 128, 96), (129, 128, 4, 96, 64),
          (200, 9, 2, 257, 65), (500, 4, 2, 128, 256), (1500, 3, 2, 256, 128)]


@pytest.mark.parametrize("tokens,num,k,d,f", LAYERS)
def test_layer(tokens, num, k, d, f):
    layer(tokens, num, k, d, f, residual=tokens % 2 == 0, out_dtype=F32 if tokens % 3 == 0 else BF)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("tokens", [1, 7, 40, 90])
def test_layer_activations_and_biases(tokens, act):
    layer(tokens, 6, 3, 72 + tokens, 52, act=act, bias=True, residual=True, out_dtype=F32, out_cols=100)


@pytest.mark.parametrize("tokens", [1, 16, 30, 64, 80])
def test_all_tokens_to_one_expert_and_none_to_others(tokens):
    z = torch.full((tokens, 20), -math.inf, device=DEV)
    z[:, 13] = 1.0
    y, x, r, up, down = layer(tokens, 20, 2, 96, 80, logits=z)
    assert (r.experts == torch.tensor([13, -1], device=DEV, dtype=torch.int32)).all()


@pytest.mark.parametrize("tokens", [9, 48, 100])
def test_tokens_without_experts_get_the_residual(tokens):
    g = gen(4)
    z = normal(g, tokens, 6, dtype=F32)
    z[::3] = -math.inf
    x = normal(g, tokens, 64)
    x[::3] = math.nan  # never read into a result
    y, *_ = layer(tokens, 6, 2, 64, 40, logits=z, x=x)
    assert (y[::3] == 0).all() and torch.isfinite(y).all()
    z[:] = -math.inf
    y, *_ = layer(tokens, 6, 2, 64, 40, logits=z, x=x, residual=True)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("tokens", [5, 64, 100])
def test_experts_named_twice(tokens):
    g = gen(6)
    e = torch.randint(-1, 5, (tokens, 4), generator=g, device=DEV, dtype=torch.int32)
    r = uz.moe_group(e, normal(g, tokens, 4, dtype=F32), 4)
    layer(tokens, 4, 4, 96, 64, logits=r)


@pytest.mark.parametrize("tokens", [3, 64, 90])
def test_strides_and_places(tokens):
    """Rows of any stride at any value's address, a result in place of its residual, memory around it untouched."""
    g = gen(8)
    num, k, d, f = 5, 2, 70, 36
    up, down = normal(g, num, 2 * f, d, scale=0.05), normal(g, num, d, f, scale=0.05)
    pu, pd = uz.pack_weight(up, gated=True), uz.pack_weight(down)
    r = uz.moe_route(normal(g, tokens, num, dtype=F32), k)
    x = normal(g, tokens, d + 5)[:, 3:d + 3]
    for dtype in (BF, F32):
        room = normal(g, tokens + 2, d + 9, dtype=dtype)
        before = room.clone()
        res = room[1:-1, 4:d + 4]
        want, bound = layer64(x, r, up, down, "swiglu", None, None, res, dtype)
        got = uz.moe(x, r, pu, pd, residual=res, out=res)
        assert got is res
        close(res, want, bound, "y")
        room[1:-1, 4:d + 4] = before[1:-1, 4:d + 4]
        assert torch.equal(room, before)


@pytest.mark.parametrize("tokens", [3, 30, 80])
@pytest.mark.parametrize("d", [1, 7, 8, 9, 60, 63, 64, 65, 120, 129, 200])
def test_nothing_beside_the_rows_of_x_is_used(tokens, d):
    """Rows of every width among NaNs, 16 bytes apart and not."""
    g = gen(d)
    num, k, f = 4, 2, 40
    up, down = normal(g, num, f, d, scale=0.2), normal(g, num, 33, f, scale=0.2)
    pu, pd = uz.pack_weight(up), uz.pack_weight(down)
    r = uz.moe_route(normal(g, tokens, num, dtype=F32), k)
    for lead, wide in ((8, (d + 23) // 8 * 8), (3, d + 7)):
        room = torch.full((tokens, wide), math.nan, dtype=BF, device=DEV)
        x = room[:, lead:lead + d]
        x.copy_(normal(g, tokens, d))
        want, bound = layer64(x, r, up, down, "silu", None, None, None, F32)
        close(uz.moe(x, r, pu, pd, act="silu", out_dtype=F32), want, bound, "y")


def test_rows_of_x_far_apart():
    g = gen(9)
    num, k, d, f = 4, 2, 72, 40
    up, down = normal(g, num, f, d, scale=0.2), normal(g, num, 33, f, scale=0.2)
    pu, pd = uz.pack_weight(up), uz.pack_weight(down)
    r = uz.moe_route(normal(g, 3, num, dtype=F32), k)
    for stride in ((1 << 22) + 8, (1 << 31) + 8):
        x = torch.empty(2 * stride + d, dtype=BF, device=DEV).as_strided((3, d), (stride, 1))
        x.copy_(normal(g, 3, d))
        want, bound = layer64(x, r, up, down, "silu", None, None, None, F32)
        close(uz.moe(x, r, pu, pd, act="silu", out_dtype=F32), want, bound, "y")


def test_a_call_gives_the_same_bits_again_and_in_a_larger_batch_the_same_values():
    g = gen(9)
    num, k, d, f = 16, 4, 256, 128
    pu, pd = uz.pack_weight(normal(g, num, 2 * f, d, scale=0.05), gated=True), uz.pack_weight(normal(g, num, d, f, scale=0.05))
    x, z = normal(g, 64, d), normal(g, 64, num, dtype=F32)
    y = [uz.moe(x, uz.moe_route(z, k), pu, pd) for _ in range(3)]
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_routing_that_does_not_fit_its_tokens_reads_nothing_out_of_range():
    """order and offsets are data: whatever they hold, only results may be wrong."""
    g = gen(10)
    for tokens in (4, 40, 100):
        num, k, d, f = 6, 2, 64, 32
        pu, pd = uz.pack_weight(normal(g, num, 2 * f, d), gated=True), uz.pack_weight(normal(g, num, d, f))
        r = uz.moe_route(normal(g, tokens, num, dtype=F32), k)
        for bad in (-1, 1 << 30, tokens * k):
            o = r.order.clone()
            o[::2] = bad
            uz.moe(normal(g, tokens, d), uz.Routing(r.experts, r.weights, o, r.offsets), pu, pd)
            e = r.offsets.clone()
            e[1::2] = bad
            uz.moe(normal(g, tokens, d), uz.Routing(r.experts, r.weights, r.order, e), pu, pd)
    torch.cuda.synchronize()
