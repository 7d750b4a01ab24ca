"""The sampler where its paths end: rows read whole, borders far out in a flat
tail, the ends of u."""
import math

import pytest
import torch

import lossless_compression_float_amd as uz
from test_gpu_sample import check, gen

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
INF = math.inf


def groups(kept, dtype):
    """How many groups of a lane's 16 tokens in half a segment have one that is kept."""
    i = torch.arange(kept.shape[1], device=DEV)
    of = i // 1024 * 64 + i // (4 if dtype is F32 else 8) % 64
    return torch.zeros((kept.shape[0], int(of[-1] // 64 + 1) * 64), device=DEV).index_add_(1, of, kept.float()).gt(0).sum(1)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [2, 40])
def test_min_p_alone_over_flat_rows(rows, dtype):
    """More groups with kept tokens than are read apart (2,048): the row is read whole, by min_p alone."""
    g = gen(rows)
    for vocab, spread, min_p in ((128256, 1.0, 0.02), (128256, 3.0, 0.001), (65551, 0.5, 0.01), (40000, 1.0, 1e-30)):
        z = (torch.randn((rows, vocab), generator=g, device=DEV) * spread).to(dtype)
        kept = torch.exp(z.double() - z.double().max(1, keepdim=True).values) >= min_p
        assert spread == 3.0 or (groups(kept, dtype) > 2048).all()
        check(z, torch.rand(rows, generator=g, device=DEV), min_p=min_p, rows=range(0, rows, 13))
