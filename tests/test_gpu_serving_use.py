"""The router, the expert layer and the sampler in use: a decode step from
packed weights, graphs, streams and threads at once, exact workspaces, stacks
and logits past 4 GiB."""
import threading

import pytest
import torch

import lossless_compression_float_amd as uz
from linear_testlib import ACC, close
from test_gpu_moe import gen, layer64, normal
from test_gpu_sample import check, peaked

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


class Model:
    """One layer of experts between a packed router and a packed head."""

    def __init__(self, seed, d=256, f=128, num=16, k=4, vocab=3001):
        g = gen(seed)
        self.k = k
        self.router_w = normal(g, num, d, scale=0.1)
        self.up_w, self.down_w = normal(g, num, 2 * f, d, scale=0.08), normal(g, num, d, f, scale=0.08)
        self.head_w = normal(g, vocab, d, scale=0.1)
        self.router, self.head = uz.pack_weight(self.router_w), uz.pack_weight(self.head_w)
        self.up, self.down = uz.pack_weight(self.up_w, gated=True), uz.pack_weight(self.down_w)

    def step(self, x, u, **kw):
        scores = uz.linear(x, self.router, out_dtype=F32)
        r = uz.moe_route(scores, self.k)
        y = uz.moe(x, r, self.up, self.down, residual=x)
        logits = uz.linear(y, self.head, out_dtype=F32)
        token, logprob = uz.sample(logits, u, **kw)
        return scores, r, y, logits, token, logprob


@pytest.mark.parametrize("tokens", [1, 7, 40, 150])
def test_a_decode_step(tokens):
    """Each part against the 64-bit form of what it was given; the log-probabilities against the loss of the same tokens."""
    m, g = Model(1), gen(tokens)
    x, u = normal(g, tokens, 256), torch.rand(tokens, generator=g, device=DEV)
    scores, r, y, logits, token, logprob = m.step(x, u)
    z = x.double().cpu() @ m.router_w.double().cpu().T
    close(scores, z, (256 + 8) * ACC * (x.double().cpu().abs() @ m.router_w.double().cpu().abs().T) + ACC * z.abs(), "scores")
    want, bound = layer64(x, r, m.up_w, m.down_w, "swiglu", None, None, x, BF)
    close(y, want, bound, "y")
    check(logits, u)
    loss, _ = uz.linear_cross_entropy(y, m.head, token)
    # both logits are off by (k + 8) 2^-23 of the sum of magnitudes, the loss by a few roundings of values up to 30
    size = (y.double().cpu().abs() @ m.head_w.double().cpu().abs().T).max()
    assert (loss + logprob).abs().max() <= 4 * (256 + 8) * ACC * float(size) + 64 * 2.0 ** -24 * 30
    # under a temperature and filters the token is one of the likeliest
    token, _ = uz.sample(logits, u, temperature=0.5, top_k=5)
    top = logits.topk(5).indices
    assert (top == token[:, None]).any(1).all()


def test_a_decode_step_in_a_graph():
    """Replayed with new inputs, with eager work of the same calls between the replays."""
    m, tokens = Model(2), 12
    x, u = torch.zeros(tokens, 256, dtype=BF, device=DEV), torch.zeros(tokens, device=DEV)
    heat = torch.full((tokens,), 0.8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        m.step(x, u, temperature=heat, top_p=0.9)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(x, u, temperature=heat, top_p=0.9)
    for i in range(4):
        g = gen(100 + i)
        x.copy_(normal(g, tokens, 256))
        u.copy_(torch.rand(tokens, generator=g, device=DEV))
        heat.fill_(0.5 + 0.3 * i)
        want = m.step(x, u, temperature=heat, top_p=0.9)
        graph.replay()
        torch.cuda.synchronize()
        again = m.step(x, u, temperature=heat, top_p=0.9)
        for a, b, c in zip(out, want, again):
            if isinstance(a, uz.Routing):
                for name in ("experts", "weights", "order", "offsets"):
                    assert torch.equal(getattr(a, name), getattr(b, name)) and torch.equal(getattr(b, name), getattr(c, name))
            else:
                assert torch.equal(a, b) and torch.equal(b, c)


def test_two_graphs_and_eager_calls_have_nothing_in_common():
    """Captures of the split second product, whose workgroups count each other, replayed in turn."""
    m = Model(3, d=1024, f=256, num=8, k=2)
    runs = []
    for tokens in (3, 20):
        x, z = normal(gen(tokens), tokens, 1024), normal(gen(tokens + 1), tokens, 8, dtype=F32)
        want = uz.moe(x, uz.moe_route(z, 2), m.up, m.down)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = uz.moe(x, uz.moe_route(z, 2), m.up, m.down)
        runs.append((graph, y, want, x, z))
    for _ in range(3):
        for graph, y, want, x, z in runs:
            y.zero_()
            graph.replay()
            eager = uz.moe(x, uz.moe_route(z, 2), m.up, m.down)
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(eager, want)


def test_threads_on_streams_of_their_own():
    m = Model(4)
    inputs = [(normal(gen(10 + i), 5 + 11 * i, 256), torch.rand(5 + 11 * i, generator=gen(20 + i), device=DEV)) for i in range(4)]
    want = [m.step(x, u, top_k=40) for x, u in inputs]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got[i] = m.step(*inputs[i], top_k=40)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(got, want):
        assert torch.equal(a[2], b[2]) and torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])


def test_a_stream_given_to_the_calls():
    m, tokens = Model(5), 9
    x, z, u = normal(gen(1), tokens, 256), normal(gen(2), tokens, 16, dtype=F32), torch.rand(tokens, device=DEV)
    logits = normal(gen(3), tokens, 5000, dtype=F32)
    want = uz.moe(x, uz.moe_route(z, 4), m.up, m.down), *uz.sample(logits, u, top_p=0.8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = uz.moe_route(z, 4, stream=s)
    got = uz.moe(x, r, m.up, m.down, stream=s), *uz.sample(logits, u, top_p=0.8, stream=s)
    grad = uz.moe_route_backward(r.weights, z, r, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(grad, uz.moe_route_backward(r.weights, z, r))


def exact_workspace(need):
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    return room, room[2048:2048 + need]


@pytest.mark.parametrize("tokens", [1, 16, 64, 200, 300])
def test_workspaces_of_the_size_that_is_asked_for(tokens, monkeypatch):
    """Nothing outside them is touched, and what they held before is no matter."""
    m, g = Model(6, num=40), gen(tokens)
    x, z, u = normal(g, tokens, 256), normal(g, tokens, 40, dtype=F32), torch.rand(tokens, generator=g, device=DEV)
    logits = peaked(g, tokens, 3001)
    rooms = []

    def given(nbytes, device):
        room, ws = exact_workspace(nbytes)
        rooms.append((room, nbytes))
        return ws

    want = uz.moe_route(z, 4), uz.moe(x, uz.moe_route(z, 4), m.up, m.down), uz.sample(logits, u, top_p=0.9)
    import lossless_compression_float_amd.experts as experts
    import lossless_compression_float_amd.sampling as sampling
    monkeypatch.setattr(experts, "workspace", given)
    monkeypatch.setattr(sampling, "workspace", given)
    got = uz.moe_route(z, 4), uz.moe(x, uz.moe_route(z, 4), m.up, m.down), uz.sample(logits, u, top_p=0.9)
    assert len(rooms) >= 2
    assert torch.equal(got[0].order, want[0].order) and torch.equal(got[1], want[1]) and torch.equal(got[2][0], want[2][0])
    for room, n in rooms:
        assert (room[:2048] == 0xA5).all() and (room[2048 + n:] == 0xA5).all()


def test_a_stack_past_4_gib():
    """700 experts of 2 x 1024 x 2048 and 2048 x 1024: 4.5 GB packed; the last ones and the first."""
    num, d, f = 700, 2048, 1024
    g = gen(7)

    def stack(rows, cols):
        w = torch.empty((num, rows, cols), dtype=BF, device=DEV)
        w.view(num, -1)[:] = normal(g, 1, rows * cols, scale=0.02)
        w[0] = normal(g, rows, cols, scale=0.02)
        w[num - 1] = normal(g, rows, cols, scale=0.02)
        return w

    up, down = stack(2 * f, d), stack(d, f)
    pu, pd = uz.pack_weight(up, gated=True), uz.pack_weight(down)
    assert pu.nbytes > 1 << 32
    for tokens in (2, 30):
        z = torch.full((tokens, num), -50.0, device=DEV)
        z[:, num - 1], z[:, 0], z[:, num - 2] = 1.0, 0.5, 0.1
        x = normal(g, tokens, d)
        r = uz.moe_route(z, 3)
        assert (r.experts == torch.tensor([num - 1, 0, num - 2], device=DEV, dtype=torch.int32)).all()
        pick = [0, num - 2, num - 1]
        few = uz.Routing(torch.tensor([2, 0, 1], dtype=torch.int32).repeat(tokens, 1), r.weights.cpu(), r.order.cpu(), torch.zeros(4, dtype=torch.int32))
        want, bound = layer64(x, few, up[pick], down[pick], "swiglu", None, None, None, BF)
        close(uz.moe(x, r, pu, pd), want, bound, "y")


def test_logits_past_4_gib():
    g = gen(8)
    rows, vocab = 8500, 128256
    z = torch.empty((rows, vocab), device=DEV)
    z[:] = peaked(g, 1, vocab)
    z[-3:] = peaked(g, 3, vocab)
    u = torch.rand(rows, generator=g, device=DEV)
    for f in (dict(), dict(top_k=20), dict(top_p=0.9)):
        token, logprob = uz.sample(z, u, **f)
        some = torch.tensor([0, rows // 2, rows - 3, rows - 1], device=DEV)
        alone = uz.sample(z[some], u[some], **f)
        assert torch.equal(token[some], alone[0]) and torch.equal(logprob[some], alone[1])


def test_the_largest_vocabulary():
    g = gen(9)
    for vocab in ((1 << 22), (1 << 22) - 1001, 600001):
        z = peaked(g, 2, vocab, spread=2.0)
        for f in (dict(), dict(top_k=50, top_p=0.9), dict(top_p=0.3), dict(min_p=0.2), dict(temperature=0.0), dict(top_k=3000)):
            check(z, torch.rand(2, generator=g, device=DEV), **f)
