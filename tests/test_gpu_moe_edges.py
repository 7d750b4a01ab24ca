"""The expert layer with routings of a program's own, and what each of its two
ways promises."""
import pytest
import torch

import lossless_compression_float_amd as uz
from linear_testlib import close
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
