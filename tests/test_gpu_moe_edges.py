"""The expert layer with routings of a program's own, and what each of its two
ways promises."""
import pytest
import torch

import lossless_compression_float_amd as uz
from linear_testlib import ACC, HALF, close, linear64
from test_gpu_moe import gen, layer64, normal

pytestmark = pytest.mark.gpu
DEV, BF, F32, I32 = "cuda", torch.bfloat16, torch.float32, torch.int32


def grouped(experts, weights, num):
    """A Routing of these experts as they are: a token may name one twice."""
    flat = experts.reshape(-1).long()
    last = torch.where(flat < 0, num, flat)
    counts = torch.bincount(last, minlength=num + 1)[:num]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return uz.Routing(experts.contiguous(), weights, torch.sort(last, stable=True).indices.to(I32), offsets.to(I32))


@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("tokens,num,k", [(1, 4, 4), (2, 1, 8), (3, 2, 64), (8, 3, 3), (40, 20, 5), (120, 70, 8), (300, 3, 4)])
def test_a_token_that_names_an_expert_twice_gets_both(tokens, num, k, act):
    """In both ways of the layer, each of the row blocks and waves that the second product takes, and whatever order the
    pairs of an expert are in."""
    g = gen(tokens)
    for d, f in ((64, 48), (200, 136)):
        rows = 2 * f if act == "swiglu" else f
        up, down = normal(g, num, rows, d, scale=0.1), normal(g, num, d, f, scale=0.1)
        bias = normal(g, num, d, dtype=F32)
        pu, pd = uz.pack_weight(up, gated=act == "swiglu"), uz.pack_weight(down)
        x, w = normal(g, tokens, d), normal(g, tokens, k, dtype=F32)
        every = torch.randint(-1, num, (tokens, k), generator=g, device=DEV, dtype=I32)
        same = torch.randint(0, num, (tokens, 1), generator=g, device=DEV, dtype=I32).expand(tokens, k)
        for e in (every, same):
            r = grouped(e, w, num)
            order = r.order.clone()
            for i in range(num):  # the pairs of an expert in another order
                a, b = int(r.offsets[i]), int(r.offsets[i + 1])
                order[a:b] = order[a:b][torch.randperm(b - a, generator=g, device=DEV)]
            for s in (r, uz.Routing(r.experts, r.weights, order, r.offsets)):
                want, bound = layer64(x, s, up, down, act, None, bias, None, F32)
                close(uz.moe(x, s, pu, pd, act=act, down_bias=bias, out_dtype=F32), want, bound, "y")


def meant(r):
    """The experts of each token as order and offsets have them: a pair that order does not name within a group has none."""
    pairs = r.tokens * r.k
    experts = torch.full((pairs,), -1, dtype=I32)
    at = [min(max(v, 0), pairs) for v in r.offsets.tolist()]
    order = r.order.tolist()
    for e in range(r.num_experts):
        for s in range(at[e], at[e + 1]):
            if 0 <= order[s] < pairs:
                experts[order[s]] = e
    return uz.Routing(experts.view(r.tokens, r.k), r.weights.cpu(), r.order.cpu(), r.offsets.cpu())


@pytest.mark.parametrize("tokens", [4, 40, 100, 300])
def test_entries_out_of_range_and_rows_of_no_group_are_left_out(tokens):
    """Both ways of the layer (the last two gather rows), over workspaces that hold other numbers."""
    g = gen(tokens)
    num, k, d, f = 6, 2, 72, 48
    pairs = tokens * k
    up, down = normal(g, num, 2 * f, d, scale=0.2), normal(g, num, d, f, scale=0.2)
    pu, pd = uz.pack_weight(up, gated=True), uz.pack_weight(down)
    x, r = normal(g, tokens, d), uz.moe_route(normal(g, tokens, num, dtype=F32), k)
    bias = normal(g, num, d, dtype=F32)
    orders, offsets = [r.order], [r.offsets]
    for bad in (-1, -1 << 31, pairs, 1 << 30):
        o = r.order.clone()
        o[::3] = bad
        orders.append(o)
    h, q = pairs // 2, pairs // 3
    rows = r.offsets.tolist()
    for o in ([q] + [max(q, v) for v in rows[1:]], rows[:-1] + [rows[-2]], [-5] + rows[1:-1] + [1 << 30], [0] * (num + 1), [pairs] * (num + 1),
              [h, pairs, 0, q, h, h, h], [h, pairs, 0, q, q, q, q], [pairs, 0, 0, q, q, h, h], [1 << 30, -7, q, h, h, h, pairs - 1]):
        offsets.append(torch.tensor(o, dtype=I32, device=DEV))
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)
    for order in orders:
        for o in offsets:
            s = uz.Routing(r.experts, r.weights, order, o)
            want, bound = layer64(x, meant(s), up, down, "swiglu", None, bias, x.float(), F32)
            got = uz.moe(x, s, pu, pd, down_bias=bias, residual=x.float(), out_dtype=F32, ws=ws)
            close(got, want, bound, "y of offsets %s" % o.tolist())


def two_value64(x, r, up, down, act, up_bias, keep):
    """(y, its bound) of a call that takes two kernels: the weight times the activation as two bf16 values (off by 2^-17 of
    itself: half a step of the second, which is at most half a step of the first), fp32 else.  keep: what becomes of it here."""
    experts, weights = r.experts.cpu(), r.weights.double().cpu()
    y = torch.zeros((x.shape[0], down.shape[1]), dtype=torch.float64)
    err = torch.zeros_like(y)
    for e in range(up.shape[0]):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        if t.numel() == 0:
            continue
        _, _, h, eh = linear64(x[t], up[e], None if up_bias is None else up_bias[e], act, None, F32)
        w, d = weights[t, j][:, None], down[e].double().cpu()
        h, eh = w * h, w.abs() * (eh + (2.0 ** -17 + 2.0 ** -23) * (h.abs() + eh))
        y.index_add_(0, t, keep(h) @ d.T)
        err.index_add_(0, t, eh @ d.abs().T + (d.shape[1] * r.k + 24) * ACC * ((h.abs() + eh) @ d.abs().T))
    return y, err + HALF[F32] * (y.abs() + err)


# each shape of the two kernels' workgroups: 1, 2 and 4 row blocks, one and two columns of tiles, 4, 8 and 16 waves, splits
FEW = [(1, 8, 2, 64, 40, 72), (1, 300, 1, 32, 16, 17), (7, 7, 1, 64, 64, 100), (16, 4, 1, 64, 48, 2000), (33, 16, 2, 40, 32, 64), (64, 8, 2, 64, 64, 130),
       (100, 8, 1, 56, 24, 600), (128, 16, 2, 64, 32, 64), (200, 64, 2, 24, 48, 80), (256, 32, 2, 64, 40, 64), (60, 100, 2, 64, 64, 1000),
       (64, 128, 2, 24, 112, 64), (256, 128, 3, 24, 112, 40), (64, 128, 2, 24, 200, 64), (256, 128, 3, 24, 200, 40)]


@pytest.mark.parametrize("act", ["swiglu", "none", "gelu"])
@pytest.mark.parametrize("tokens,num,k,d,f,out", FEW)
def test_activations_between_the_two_kernels_keep_17_bits(tokens, num, k, d, f, out, act):
    assert tokens <= 256 and tokens * k <= 16 * num
    g = gen(tokens + f)
    rows = 2 * f if act == "swiglu" else f
    up, down = normal(g, num, rows, d, scale=0.2), normal(g, num, out, f, scale=0.2)
    x, bias = normal(g, tokens, d), normal(g, num, rows, dtype=F32)
    r = uz.moe_route(normal(g, tokens, num, dtype=F32), k)
    want, bound = two_value64(x, r, up, down, act, bias, lambda h: h)
    one, _ = two_value64(x, r, up, down, act, bias, lambda h: h.bfloat16().double())
    assert ((one - want).abs() > 2 * bound).any()  # with one bf16 value it would show
    got = uz.moe(x, r, uz.pack_weight(up, gated=act == "swiglu"), uz.pack_weight(down), act=act, up_bias=bias, out_dtype=F32)
    close(got, want, bound, "y")


def test_a_token_alone_and_in_batches_is_within_what_each_way_promises():
    g = gen(12)
    num, k, d, f = 16, 2, 64, 48
    up, down = normal(g, num, 2 * f, d, scale=0.2), normal(g, num, d, f, scale=0.2)
    pu, pd = uz.pack_weight(up, gated=True), uz.pack_weight(down)
    x, z = normal(g, 600, d), normal(g, 600, num, dtype=F32)
    whole = uz.moe_route(z, k)
    want, bound = two_value64(x, whole, up, down, "swiglu", None, lambda h: h)
    rough, wide = layer64(x, whole, up, down, "swiglu", None, None, None, F32)
    for tokens in (1, 2, 9, 40, 128, 600):
        r = uz.moe_route(z[:tokens], k)
        assert torch.equal(r.experts, whole.experts[:tokens]) and torch.equal(r.weights, whole.weights[:tokens])
        got = [uz.moe(x[:tokens], r, pu, pd, out_dtype=F32) for _ in range(2)]
        assert torch.equal(*got)
        close(got[0], want[:tokens] if tokens <= 128 else rough, bound[:tokens] if tokens <= 128 else wide, "y")


def test_the_weights_gradients_of_a_training_step():
    """From grouped_linear's rows to the router's logits, as a program that trains the layer takes them, against autograd in 64
    bits over the same rows."""
    g = gen(13)
    tokens, num, k, d, f = 50, 6, 2, 72, 40
    up, down = uz.pack_weight(normal(g, num, 2 * f, d, scale=0.2), gated=True), uz.pack_weight(normal(g, num, d, f, scale=0.2))
    x, scores, dy = normal(g, tokens, d), normal(g, tokens, num, dtype=F32), normal(g, tokens, d, dtype=F32)
    scores[3] = -float("inf")
    scores[4, 1:] = -float("inf")
    r = uz.moe_route(scores, k)
    h = uz.grouped_linear(x[r.order // k], r.offsets, up, act="swiglu")
    o = uz.grouped_linear(h, r.offsets, down, out_dtype=F32)
    dweights = torch.empty_like(r.weights)
    dweights.view(-1)[r.order] = (dy[r.order // k] * o).sum(-1)
    got = uz.moe_route_backward(dweights, scores, r)
    z = scores.double().cpu().requires_grad_(True)
    chosen = r.experts.cpu().long()
    p = torch.where(chosen >= 0, torch.exp(z.gather(1, chosen.clamp(min=0))), 0.0)
    s = p.sum(1, keepdim=True)
    w = torch.where(s > 0, p / torch.where(s > 0, s, 1.0), 0.0)
    rows = torch.empty((tokens * k, d), dtype=torch.float64)
    rows[r.order.cpu().long()] = o.double().cpu()
    rows = rows.view(tokens, k, d)
    y = (w[:, :, None] * rows).sum(1)
    want, = torch.autograd.grad(y, z, dy.double().cpu())
    # dweights: a sum of d products in fp32; its gradient then by at most the share times that, twice, and the share's own error
    size = (dy.double().cpu().abs()[:, None, :] * rows.abs()).sum(2).max(1, keepdim=True).values
    close(got, want, 4 * (d + 8 + 40 + num + 16) * ACC * size * torch.ones_like(want), "dlogits")
