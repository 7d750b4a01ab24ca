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
