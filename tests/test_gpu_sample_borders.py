"""The sampler where its paths end: rows read whole, borders far out in a flat
tail, the ends of u."""
import math

import pytest
import torch

import lossless_compression_float_amd as uz
from test_gpu_sample import FILTERS, check, gen, row64

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


def kept64(z, temperature, top_k, top_p, min_p):
    """(e where it is kept, else 0; the log-probabilities; how far top-p is from keeping one more or less, relative to the sum)
    of one row on the CPU in 64 bits.  A product by which min_p decides is exact in the rows used here, or far from it."""
    z = z.double().cpu()
    top, n = z.max(), z.numel()
    y = torch.where(z == top, torch.zeros_like(z), (z - top) / (temperature if temperature > 0 else 1.0))
    e = torch.exp(y)
    order = torch.sort(z, descending=True, stable=True).indices
    es = e[order]
    count = 1 if temperature == 0 else n if top_k <= 0 or top_k >= n else top_k
    run, room = es[:count].cumsum(0), 1.0
    if top_p < 1 and count > 1:
        before = run - es[:count]
        room = float((before / run[-1] - top_p).abs()[1:].min())
        count = max(1, int((before < top_p * run[-1]).sum()))
    count = max(1, int((es[:count] >= min(min_p, 1.0)).sum()))
    kept = torch.zeros(n, dtype=torch.float64)
    kept[order[:count]] = es[:count]
    return kept, y - e.sum().log(), room


def drawn(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Every token is one that is kept, and the running sum passes u there to 1e-12 of the whole; at u = 0 it is the first."""
    token, logprob = uz.sample(logits, u, temperature, top_k, top_p, min_p)
    f32 = lambda v: float(torch.tensor(v, dtype=F32))
    for i in range(logits.shape[0]):
        kept, logp, room = kept64(logits[i], f32(temperature), top_k, f32(top_p), f32(min_p))
        assert room > 1e-12
        run, t = kept.cumsum(0), int(token[i])
        total, at = float(run[-1]), float(u[i])
        what = (i, t, at, temperature, top_k, top_p, min_p)
        assert kept[t] > 0, what
        assert float(run[t]) >= (at - 1e-12) * total and float(run[t] - kept[t]) <= (at + 1e-12) * total, what
        if at == 0:
            assert t == int((kept > 0).nonzero()[0]), what
        assert abs(float(logprob[i]) - float(logp[t])) <= 2.0 ** -24 * abs(float(logp[t])) + 1e-12, what


ENDS = [0.0, 2.0 ** -70, 0.37, 1 - 2.0 ** -24, 1 - 2.0 ** -53]


def at(u, rows):
    return torch.full((rows,), u, dtype=torch.float64, device=DEV)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("u", ENDS)
def test_draws_at_the_ends_of_u(u, dtype):
    g = torch.Generator().manual_seed(2)
    for vocab in (7, 3001, 40000):
        z = torch.randn((4, vocab), generator=g) * 3
        z = z.scatter_add(1, torch.randint(0, vocab, (4, 4), generator=g), torch.rand((4, 4), generator=g) * 10).to(DEV, dtype)
        z[1:, ::7] = -INF
        z[2:, -1] = -INF
        z[3, 0:3] = -INF
        for f in FILTERS:
            drawn(z, at(u, 4), **f)


@pytest.mark.parametrize("u", ENDS)
def test_draws_at_the_ends_of_u_among_equal_logits_and_masks(u):
    for vocab in (5, 700, 70001):
        z = torch.zeros((5, vocab), device=DEV)
        z[1] = -7.5
        z[2] = (torch.arange(vocab, device=DEV) % 3).float()
        z[3, ::2] = -INF
        z[4, :-1] = -INF
        for f in (dict(), dict(top_k=3), dict(top_p=0.5003), dict(top_k=vocab // 2 + 1, top_p=0.7703), dict(temperature=0.0), dict(min_p=0.9),
                  dict(temperature=1e30, top_p=0.3301), dict(temperature=1e30), dict(min_p=1.0, top_k=2)):
            drawn(z, at(u, 5), **f)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_masked_tokens_are_not_a_segments_smallest(dtype):
    """What the draw takes from the survey of 2,048 tokens, in the workspace: were -inf the smallest value of a segment, a row's
    bins would reach down to 2^-80 of the largest, and ordinary masked rows would go the way of rows of equal logits."""
    vocab = 2 * 2048 + 700
    z = torch.randn((3, vocab), generator=torch.Generator().manual_seed(3)).to(DEV, dtype)
    z[1, 5] = z[1, 3000:3100] = z[1, -2:] = -INF
    z[2, :2048] = -INF
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    u = torch.full((3,), 0.4, device=DEV)
    token, _ = uz.sample(z, u, top_p=0.9, ws=ws)
    begin = -ws.data_ptr() % 256
    room = ws[begin:begin + 3 * 3 * 16].view(torch.float32).view(3, 3, 4).cpu()  # sum (64 bits), largest, smallest
    for r in range(3):
        for seg in range(3):
            part = z[r, seg * 2048:(seg + 1) * 2048].float().cpu()
            part = part[part > -INF]
            assert room[r, seg, 2] == (part.max() if len(part) else -INF) and room[r, seg, 3] == (part.min() if len(part) else INF)
    check(z, u, top_p=0.9)
