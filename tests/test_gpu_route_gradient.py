"""The router's gradient where one expert has nearly all of a token."""
import pytest
import torch

import lossless_compression_float_amd as uz
from linear_testlib import HALF, close
from test_gpu_moe import normal

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


def gradient64(logits, experts, dw, scores, renorm, scale):
    """(dlogits, the sum of its terms' magnitudes) in 64 bits, without differences that cancel: with p_i the shares and g_i
    the gradients of the weights (0 for those not chosen), dz_j = p_j sum_i p_i (g_j - g_i), i not j; with sigmoid scores
    times 1 - s_j."""
    z = logits.double().cpu()
    e = experts.cpu().long()
    chosen = torch.zeros_like(z).scatter(1, e, 1.0)
    g = scale * torch.zeros_like(z).scatter(1, e, dw.double().cpu())
    s = torch.sigmoid(z) if scores == "sigmoid" else torch.exp(z - z.max(1, keepdim=True).values)
    own = torch.sigmoid(-z) if scores == "sigmoid" else torch.ones_like(z)  # the score's own derivative, over the score
    if scores == "sigmoid" and not renorm:
        return g * s * own, (g * s * own).abs()
    if renorm:
        s = s * chosen
    p = s / s.sum(1, keepdim=True)
    terms = p[:, None, :] * (g[:, :, None] - g[:, None, :])  # [token, j, i]
    sizes = p[:, None, :] * (g[:, :, None].abs() + g[:, None, :].abs()) * (1 - torch.eye(z.shape[1], dtype=torch.float64))
    return p * own * terms.sum(2), p * own * sizes.sum(2)


@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens,num,k", [(9, 4, 1), (40, 60, 6), (17, 130, 8), (5, 300, 2), (3, 1000, 64)])
def test_gradient_of_a_router_that_is_sure(tokens, num, k, dtype, scores, renorm):
    g = torch.Generator().manual_seed(num + k)
    for gap in (0.0, 12.0, 20.0, 40.0):
        z = torch.randn((tokens, num), generator=g)
        first = torch.randint(0, num, (tokens, 1), generator=g)
        z = (z - gap).scatter(1, first, torch.randn((tokens, 1), generator=g)).to(DEV, dtype)
        dw = torch.randn((tokens, k), generator=g).to(DEV)
        r = uz.moe_route(z, k, scores=scores, renormalize=renorm, scale=1.5)
        want, size = gradient64(z, r.experts, dw, scores, renorm, 1.5)
        got = uz.moe_route_backward(dw, z, r)
        # dz_j = p_j (g_j (1 - p_j) - the sum of p_i g_i over i not j): in fp32 each share is off by its exponent's rounding (up to
        # 50 of them) and a sum of up to num values, the sums alike, each relative to the terms' magnitudes; only where p_j is
        # below 1/2 may p_j g_j be among them, which is then below (1 - p_j) g_j: twice all of that
        rel = (2 * (50 + num) + k + 16) * 2.0 ** -23 if scores == "softmax" else 1e-12
        bound = rel * size + 2.0 ** -24 * want.abs() + 2.0 ** -126
        close(got, want, bound + HALF[dtype] * (want.abs() + bound), "dlogits, gap %g" % gap)


def test_the_gradients_of_a_token_sum_to_nothing():
    """With softmax scores; where one expert has all but 1e-9 of a token as well."""
    g = torch.Generator(device=DEV).manual_seed(1)
    z = normal(g, 64, 32, dtype=F32)
    z[:, 5] += 20.0
    for k in (1, 4):
        for renorm in (True, False):
            r = uz.moe_route(z, k, renormalize=renorm)
            d = uz.moe_route_backward(normal(g, 64, k, dtype=F32), z, r).double()
            # each of the 32 is off by what test_gradient_of_a_router_that_is_sure allows of its terms, which are those of the sum
            assert (d.sum(1).abs() <= (2 * (50 + 32) + 4 + 16) * 2.0 ** -23 * 4 * d.abs().sum(1)).all()
