"""The sampler against its definition in 64 bits."""
import math

import pytest
import torch

import lossless_compression_float_amd as uz

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def row64(z, u, temperature, top_k, top_p, min_p):
    """(token, its log-probability, how far u is from moving the draw or the top-p border from moving, relative to the
    sums) of one row on the CPU in 64 bits."""
    z = z.double().cpu()
    if z.isnan().any() or z.max() == -INF or not temperature >= 0:
        return -1, NAN, 1.0
    top = z.max()
    heat = temperature if temperature > 0 else 1.0
    y = torch.where(z == top, torch.zeros_like(z), (z - top) / heat)
    e = torch.exp(y)
    order = torch.sort(z, descending=True, stable=True).indices
    es = e[order]
    n = z.numel()
    k = 1 if temperature == 0 else n if top_k <= 0 or top_k >= n else top_k
    keep = torch.arange(n) < k
    run = (es * keep).cumsum(0)
    before = run - es * keep
    room = 1.0
    if top_p < 1:
        room = float((before[keep] / run[-1] - top_p).abs()[1:].min()) if int(keep.sum()) > 1 else 1.0
        keep &= (before < top_p * run[-1]) | (torch.arange(n) == 0)
    keep &= (es >= min(min_p, 1.0)) | (torch.arange(n) == 0)
    kept = torch.zeros(n, dtype=torch.float64)
    kept[order] = es * keep
    run = kept.cumsum(0)
    token = int((run <= u * run[-1]).sum())
    room = min(room, float((run / run[-1] - u).abs().min()))
    return token, float(y[token] - e.sum().log()), room


def check(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=None):
    token, logprob = uz.sample(logits, u, temperature, top_k, top_p, min_p)
    f32 = lambda v, i: float(v[i]) if isinstance(v, torch.Tensor) else float(torch.tensor(v, dtype=F32))
    for i in range(logits.shape[0]) if rows is None else rows:
        want, lp, room = row64(logits[i], float(u[i]), f32(temperature, i), int(f32(top_k, i)), f32(top_p, i), f32(min_p, i))
        # e is off by 1.5e-14 of itself, sums of 2^17 of them by 2^17 2^-53 more at most: only a draw closer than that to a
        # border may fall on the other side of it
        if room > 1e-12:
            assert int(token[i]) == want, (i, int(token[i]), want, room)
        if int(token[i]) == want:
            got = float(logprob[i])
            # the exact difference and logarithm rounded once, and e's error
            assert (math.isnan(got) and math.isnan(lp)) or abs(got - lp) <= 2.0 ** -24 * abs(lp) + 1e-12, (i, got, lp)
    return token, logprob


def peaked(g, rows, vocab, spread=3.0, dtype=F32):
    z = torch.randn((rows, vocab), generator=g, device=DEV) * spread
    at = torch.randint(0, vocab, (rows, 4), generator=g, device=DEV)
    return z.scatter_add(1, at, torch.rand((rows, 4), generator=g, device=DEV) * 10).to(dtype)


FILTERS = [dict(), dict(temperature=0.0), dict(temperature=0.3), dict(top_k=1), dict(top_k=7), dict(top_k=50, top_p=0.9),
           dict(top_p=0.5), dict(top_p=0.999), dict(min_p=0.1), dict(min_p=0.01, top_p=0.95, top_k=300, temperature=1.7),
           dict(top_k=5000), dict(top_p=0.0), dict(min_p=1.0), dict(top_p=1.0, top_k=10 ** 6)]


@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 1000, 1024, 4097, 32003])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_filters(vocab, dtype):
    g = gen(vocab)
    for f in FILTERS:
        z = peaked(g, 6, vocab, dtype=dtype)
        check(z, torch.rand(6, generator=g, device=DEV), **f)


@pytest.mark.parametrize("vocab", [2000, 4097, 9001, 20000, 128256])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_large_top_k(vocab, dtype):
    """More than the row has groups of tokens, more than are sorted, among many equal ones (bf16)."""
    g = gen(vocab + 1)
    for k in (700, 1000, 3000, 5000, vocab - 1):
        for f in (dict(), dict(top_p=0.9), dict(min_p=0.01), dict(top_p=0.99, min_p=0.001, temperature=2.0)):
            z = peaked(g, 3, vocab, spread=1.0, dtype=dtype)
            z[1, ::5] = -INF
            check(z, torch.rand(3, generator=g, device=DEV), top_k=k, **f)


@pytest.mark.parametrize("rows", [1, 3, 300])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_large_vocabulary(rows, dtype):
    g = gen(rows)
    z = peaked(g, rows, 128256, spread=2.5, dtype=dtype)
    for f in (dict(), dict(top_k=50, top_p=0.9, temperature=0.7), dict(top_p=0.95), dict(top_p=0.95, temperature=1.5),
              dict(temperature=0.0), dict(min_p=0.02), dict(top_k=1000), dict(top_k=20000)):
        check(z, torch.rand(rows, generator=g, device=DEV), rows=range(0, rows, 61), **f)


def test_each_row_has_its_own_parameters():
    g = gen(1)
    rows = 200
    z = peaked(g, rows, 5003)
    pick = lambda vals, dt: torch.tensor(vals, dtype=dt, device=DEV)[torch.randint(0, len(vals), (rows,), generator=g, device=DEV)]
    check(z, torch.rand(rows, generator=g, device=DEV), pick([0.0, 0.5, 1.0, 2.0], F32), pick([-1, 0, 1, 3, 40, 6000], torch.int32),
          pick([0.0, 0.3, 0.9, 1.0, 2.0], F32), pick([0.0, 0.05, 1.0, 3.0], F32))


@pytest.mark.parametrize("u", [0.0, 0.5, 1 - 2.0 ** -24, 1 - 2.0 ** -53])
def test_the_ends_of_u(u):
    g = gen(2)
    z = peaked(g, 5, 3001)
    z[:, ::7] = -INF
    z[:, -1] = -INF
    z[:, 0] = -INF
    for f in FILTERS:
        check(z, torch.full((5,), u, dtype=torch.float64, device=DEV), **f)
        token, logprob = uz.sample(z, torch.full((5,), u, dtype=torch.float64, device=DEV), **f)
        assert torch.isfinite(z[torch.arange(5, device=DEV), token]).all() and torch.isfinite(logprob).all()


@pytest.mark.parametrize("vocab", [5, 1000, 70001])
def test_equal_logits_go_by_index(vocab):
    """A row of one value, and one of few: top-k and top-p end among equals."""
    z = torch.zeros((4, vocab), device=DEV)
    z[1] = -7.5
    z[2] = (torch.arange(vocab, device=DEV) % 3).float()
    z[3] = (torch.arange(vocab, device=DEV) % 2).float() * -100
    z[3, :2] = torch.tensor([-0.0, 0.0])
    for u in (0.0, 0.3, 0.99):
        uu = torch.full((4,), u, device=DEV)
        for f in (dict(), dict(top_k=3), dict(top_p=0.5), dict(top_k=vocab // 2 + 1, top_p=0.77), dict(temperature=0.0), dict(min_p=0.9)):
            check(z, uu, **f)
    token, _ = uz.sample(z, torch.full((4,), 0.99, device=DEV), top_k=2)
    assert token.tolist()[:2] == [1, 1]


def test_masks_nans_and_infinities():
    n = 700
    z = torch.zeros((9, n), device=DEV)
    z[0] = -INF
    z[1] = -INF
    z[1, 699] = -3e38
    z[2, 5] = NAN
    z[3, 10] = INF
    z[3, 600] = INF
    z[4] = torch.finfo(F32).min
    z[5] = torch.finfo(F32).min
    z[5, 3] = torch.finfo(F32).max
    z[6] = NAN
    z[7, 1:] = -INF
    z[8, ::2] = -INF
    for f in FILTERS:
        for u in (0.0, 0.7):
            token, logprob = check(z, torch.full((9,), u, device=DEV), **f)
            assert token[0] == token[2] == token[6] == -1
            assert token[1] == 699 and logprob[1] == 0 and token[5] == 3 and token[7] == 0 and token[3] in (10, 600)
    b = z.to(BF)
    token, _ = uz.sample(b, torch.full((9,), 0.5, device=DEV), top_p=0.9)
    assert token[0] == token[2] == -1 and token[1] == 699


def test_bad_parameters_of_a_row_make_only_that_row_invalid():
    g = gen(3)
    z = peaked(g, 4, 900)
    u = torch.rand(4, generator=g, device=DEV)
    t = torch.tensor([1.0, -1.0, NAN, 1.0], device=DEV)
    p = torch.tensor([0.9, 0.9, 0.9, NAN], device=DEV)
    token, logprob = uz.sample(z, u, temperature=t, top_p=p)
    assert token[0] >= 0 and (token[1:] == -1).all() and logprob[1:].isnan().all()
    token, logprob = uz.sample(z, u, min_p=p)
    assert (token[:3] >= 0).all() and token[3] == -1


def test_strides_and_odd_places():
    g = gen(4)
    for dtype in (F32, BF):
        wide = peaked(g, 5, 9000, dtype=dtype)
        for lo, hi in ((0, 8999), (1, 8000), (3, 4003), (8, 9000)):
            check(wide[:, lo:hi], torch.rand(5, generator=g, device=DEV), top_p=0.9)


def test_even_logits_are_drawn_evenly():
    """Flat rows, where every token is a border: the draw is floor(u n) exactly, as sums of ones are."""
    n = 65536
    z = torch.full((64, n), 2.5, device=DEV)
    u = torch.rand(64, generator=gen(5), device=DEV)
    token, logprob = uz.sample(z, u, temperature=0.8)
    assert torch.equal(token, (u.double() * n).floor().long())
    assert torch.allclose(logprob, torch.full_like(logprob, -math.log(n)), rtol=2.0 ** -23)


def test_wide_spread_at_low_temperature():
    g = gen(6)
    z = torch.randn((8, 20001), generator=g, device=DEV) * 1e4
    for t in (1e-30, 1e-3, 1.0, 1e4, 1e30):
        check(z, torch.rand(8, generator=g, device=DEV), temperature=t, top_p=0.99)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_masked_tokens_are_not_drawn_at_the_highest_temperatures(dtype):
    z = torch.randn((3, 3001), generator=gen(7), device=DEV).to(dtype)
    z[:, :40] = -INF
    z[1, 50::2] = -INF
    z[2, 41:] = torch.finfo(dtype).min
    for t in (1e20, 1e37, 3e38):
        for u in (0.0, 0.6):
            for f in (dict(), dict(top_p=1 - 2.0 ** -24), dict(top_p=0.3), dict(min_p=1e-30), dict(top_k=2999, top_p=0.9), dict(top_k=50)):
                token, _ = check(z, torch.full((3,), u, device=DEV), temperature=t, **f)
                assert (token >= 40).all()


def test_no_rows():
    token, logprob = uz.sample(torch.empty((0, 10), device=DEV), torch.empty(0, device=DEV))
    assert token.shape == logprob.shape == (0,)
