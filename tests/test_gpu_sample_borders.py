"""The sampler where its paths end: rows read whole, borders far out in a flat
tail, the ends of u."""
import math

import pytest
import torch

import lossless_compression_float_amd as uz
from test_gpu_sample import check, gen, row64

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


def compared(z, u, **f):
    """As check, where every row's draw has to be farther than 1e-12 from a border."""
    want = [row64(z[i], float(u[i]), *(float(torch.tensor(f.get(n, d), dtype=F32)) for n, d in
                                       (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)))) for i in range(z.shape[0])]
    assert all(room > 1e-12 for _, _, room in want)
    token, logprob = check(z, u, **f)
    assert token.tolist() == [t for t, _, _ in want]
    return token


TAILS = [(128256, 21.5, 0.0, 0.99998), (128256, 22.0, 1.0, 0.99999), (128256, 26.0, 2.0, 0.999999), (1000003, 24.0, 0.5, 0.9999),
         (40000, 21.0, 0.0, 1 - 2.0 ** -24), (9001, 20.0, 1.0, 1 - 2.0 ** -20), (70001, 14.0, 1.0, 0.9), (300, 30.0, 1.0, 1 - 2.0 ** -24)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab,above,spread,top_p", TAILS)
def test_top_p_ends_in_a_tail_of_faint_tokens(vocab, above, spread, top_p, dtype):
    """Tokens of less than 2^-32 of the sum, of which top-p keeps a part."""
    g = torch.Generator().manual_seed(vocab)
    z = (torch.randn((3, vocab), generator=g) * spread - above).to(DEV, dtype)
    z[0, 0] = z[1, vocab // 3] = z[2, vocab - 1] = 0
    for far in (1.0, 0.5, 1e-2, 1e-4):
        # draws among the last kept tokens, and anywhere
        u = (1 - torch.rand(3, generator=g, dtype=torch.float64) * min(1.0, far * 4 * vocab * math.exp(-above) + 1e-9)).to(DEV)
        compared(z, u, top_p=top_p)
        compared(z, u, top_p=top_p, min_p=math.exp(-above - 1))
        compared(z, u, top_p=top_p, min_p=math.exp(-above + 1))


@pytest.mark.parametrize("vocab", [7, 1000, 20000])
def test_top_p_over_the_whole_range_of_fp32(vocab):
    """Differences of logits past fp32's largest value, at temperatures that make them small."""
    z = torch.full((2, vocab), -3e38, device=DEV)
    z[0, 5] = 3e38
    z[1, 2:6] = 3e38
    z[1, ::3] = -2e38
    for heat in (1e38, 3e37):
        for top_p in (0.3, 0.9, 0.999):
            for u in (0.123456, 0.55555, 0.98765):
                compared(z, torch.full((2,), u, dtype=torch.float64, device=DEV), temperature=heat, top_p=top_p)
