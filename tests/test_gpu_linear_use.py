"""The products with packed weights as a program uses them: weights that
arrive compressed, are packed, multiplied and trained on; in graphs, on other
streams and threads, with buffers past 4 GiB; the same bits from the same
call."""
import threading

import pytest
import torch

import lossless_compression_float_amd as uz
import workloads
from linear_testlib import backward64, close, linear64, loss64, loss_backward64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def normal(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def same(a, b):
    return bool(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)))


def arrive(w):
    """A weight as a receiver gets it: compressed, sent, decompressed; then packed."""
    buf, size = uz.compress(w)
    torch.cuda.synchronize()
    frame = buf[:int(size.item())].clone()
    back, status = uz.decompress(frame, w.dtype, w.numel())
    assert int(status.item()) == 0
    return back.view(w.shape)


def test_a_block_from_compressed_weights():
    """Token rows through a projection with residual, experts, and the output
    head's loss, then back: every weight arrived compressed, every gradient
    agrees with the 64-bit form of its own operator."""
    m, h, f, e, v = 200, 256, 192, 4, 1000
    ws = {"o": normal(1, h, h, scale=0.05), "up": normal(2, e, 2 * f, h, scale=0.05), "down": normal(3, e, h, f, scale=0.05),
          "head": normal(4, v, h, scale=0.1)}
    got = {k: arrive(w) for k, w in ws.items()}
    for k in ws:
        assert torch.equal(got[k].view(torch.int16), ws[k].view(torch.int16))
    p = {k: uz.pack_weight(w, gated=k == "up") for k, w in got.items()}
    assert sum(w.nbytes for w in p.values()) < 0.8 * sum(2 * w.numel() for w in ws.values())
    x, attn = normal(5, m, h), normal(6, m, h)
    off = torch.tensor([0, 70, 70, 131, m], dtype=torch.int32, device=DEV)
    t = torch.randint(0, v, (m,), device=DEV)
    a = uz.linear(attn, p["o"], residual=x)
    u, z = uz.grouped_linear(a, off, p["up"], act="swiglu", return_preact=True)
    d = uz.grouped_linear(u, off, p["down"])
    loss, lse = uz.linear_cross_entropy(d, p["head"], t)
    dl = torch.full((m,), 1.0 / m, device=DEV)
    dd, dhead = uz.linear_cross_entropy_backward(dl, d, p["head"], t, lse)
    du, ddown, _ = uz.grouped_linear_backward(dd, u, off, p["down"])
    da, dup, _ = uz.grouped_linear_backward(du, a, off, p["up"], preact=z, act="swiglu")
    dattn, do, _ = uz.linear_backward(da, attn, p["o"])
    close(a, *linear64(attn, ws["o"], None, "none", x, BF)[2:], "a")
    l64, s64, el, es, _, _ = loss64(d, ws["head"], t, -100)
    close(loss, l64, el, "loss")
    wx, ww = loss_backward64(dl, d, ws["head"], t, -100)
    close(dd, *wx, "dd")
    close(dhead, *ww, "dhead")
    o = off.tolist()
    for i in range(e):
        s = slice(o[i], o[i + 1])
        if o[i] == o[i + 1]:
            assert (ddown[i] == 0).all() and (dup[i] == 0).all()
            continue
        close(u[s], *linear64(a[s], ws["up"][i], None, "swiglu", None, BF)[2:], "u")
        close(d[s], *linear64(u[s], ws["down"][i], None, "none", None, BF)[2:], "d")
        w = backward64(dd[s], u[s], ws["down"][i], None, "none", BF)
        close(du[s], *w["dx"], "du")
        close(ddown[i], *w["dw"], "ddown")
        w = backward64(du[s], a[s], ws["up"][i], z[s], "swiglu", BF)
        close(da[s], *w["dx"], "da")
        close(dup[i], *w["dw"], "dup")
    w = backward64(da, attn, ws["o"], None, "none", BF)
    close(dattn, *w["dx"], "dattn")
    close(do, *w["dw"], "do")
    # and the gradients go back over the wire
    assert torch.equal(arrive(dhead).view(torch.int16), dhead.view(torch.int16))


def test_weights_of_the_model_set_pack_losslessly():
    """One matrix of each shape of the 8B weight set, rows divided by 16."""
    total = packed = 0
    for w in workloads.llama3_8b_weights(DEV, seed=2, scale=16)[:10]:
        if w.dim() == 2:
            p = uz.pack_weight(w)
            assert torch.equal(uz.unpack_weight(p).view(torch.int16), w.view(torch.int16))
            total, packed = total + 2 * w.numel(), packed + p.nbytes
    assert packed < 0.765 * total


CALLS = {
    "token": (1, 320, 520, "none"), "rows": (50, 320, 520, "silu"), "tiles": (300, 320, 520, "gelu"),
    "runs": (100, 256, 4096, "relu"), "large": (2200, 2200, 136, "none")}


def step(w, x, res, dy, act, ws=None):
    """All of one layer's calls, their outputs in a list."""
    y, z = uz.linear(x, w, act=act, residual=res, return_preact=True)
    dx, dw, db = uz.linear_backward(dy, x, w, preact=z, act=act, need_bias=True)
    return [y, z, dx, dw, db]


def loss_step(w, x, t, dl):
    loss, lse = uz.linear_cross_entropy(x, w, t)
    dx, dw = uz.linear_cross_entropy_backward(dl, x, w, t, lse)
    return [loss, lse, dx, dw]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_same_call_same_bits(name):
    m, n, k, act = CALLS[name]
    w = uz.pack_weight(normal(10, n, k, scale=0.05))
    args = (w, normal(11, m, k), normal(12, m, n), normal(13, m, n), act)
    t, dl = torch.randint(0, n, (m,), device=DEV), normal(14, m, dtype=F32)
    first = step(*args) + loss_step(w, args[1], t, dl)
    for _ in range(5):
        torch.empty(1 << 26, dtype=torch.uint8, device=DEV).fill_(0xFF)  # (other contents in the workspaces' memory)
        for a, b in zip(first, step(*args) + loss_step(w, args[1], t, dl)):
            assert same(a, b)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_graph_replays_equal_eager(name):
    """Captured, replayed with new inputs, with eager calls and waits between."""
    m, n, k, act = CALLS[name]
    w = uz.pack_weight(normal(20, n, k, scale=0.05))
    x, res, dy = normal(21, m, k), normal(22, m, n), normal(23, m, n)
    t, dl = torch.randint(0, n, (m,), device=DEV), normal(24, m, dtype=F32)
    e = 3
    stack = uz.pack_weight(normal(25, e, n, k, scale=0.05))
    off = torch.tensor([0, m // 3, m // 3, m], dtype=torch.int32, device=DEV)

    def all_calls():
        g = uz.grouped_linear(x, off, stack, act=act)
        gb = uz.grouped_linear_backward(dy, x, off, stack)
        return step(w, x, res, dy, act) + loss_step(w, x, t, dl) + [g] + list(gb[:2])

    all_calls()
    torch.cuda.synchronize()
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_calls()
    with torch.cuda.graph(graph2):
        outs2 = all_calls()
    for i in range(4):
        x.copy_(normal(30 + i, m, k))
        dy.copy_(normal(40 + i, m, n))
        off.copy_(torch.tensor([0, min(i, m // 2), m // 2, m - (i > 1)], dtype=torch.int32))
        want = [o.clone() for o in all_calls()]
        graph.replay()
        if i & 1:
            torch.cuda.synchronize()
        graph2.replay()
        eager = all_calls()
        torch.cuda.synchronize()
        for a, b, c, d in zip(want, outs, outs2, eager):
            assert [same(a, b), same(a, c), same(a, d)] == [True] * 3


def test_two_threads_on_two_streams():
    jobs = []
    for i, name in enumerate(("tiles", "runs")):
        m, n, k, act = CALLS[name]
        w = uz.pack_weight(normal(50 + i, n, k, scale=0.05))
        args = (w, normal(60 + i, m, k), normal(70 + i, m, n), normal(80 + i, m, n), act)
        jobs.append((args, step(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    failures = []

    def work(args, want, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = step(*args)
                    stream.synchronize()
                    assert all(same(a, b) for a, b in zip(want, got))
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failures, failures


def test_stream_argument():
    m, n, k, act = CALLS["tiles"]
    wt = normal(90, n, k, scale=0.05)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w = uz.pack_weight(wt, stream=side)
    x, dy = normal(91, m, k), normal(92, m, n)
    side.wait_stream(torch.cuda.current_stream())
    y, z = uz.linear(x, w, act=act, return_preact=True, stream=side)
    dx, dw, _ = uz.linear_backward(dy, x, w, preact=z, act=act, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    w2 = uz.pack_weight(wt)
    assert torch.equal(w.data, w2.data)
    y2, z2 = uz.linear(x, w2, act=act, return_preact=True)
    dx2, dw2, _ = uz.linear_backward(dy, x, w2, preact=z2, act=act)
    for a, b in ((y, y2), (z, z2), (dx, dx2), (dw, dw2)):
        assert same(a, b)


def test_own_workspace_and_too_small_a_one():
    m, n, k, act = CALLS["runs"]
    w = uz.pack_weight(normal(95, n, k, scale=0.05))
    x = normal(96, m, k)
    want = uz.linear(x, w, act=act)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    assert torch.equal(uz.linear(x, w, act=act, ws=ws), want)
    with pytest.raises(uz.UzipError):
        uz.linear(x, w, act=act, ws=ws[:256])
    with pytest.raises(ValueError):
        uz.linear(x, w, act=act, ws=ws.view(torch.int16))
    with pytest.raises(ValueError):
        uz.linear(x.cpu(), w)


def test_stack_past_4_gib():
    """A packed stack of 4.8 GB: the last experts' tiles lie past 2^32 bytes."""
    e, n, k, m = 97, 4096, 8192, 40
    w = torch.empty(e, n, k, dtype=BF, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(100)
    for i in range(e):
        w[i] = torch.randn(n, k, generator=g, device=DEV) * 0.02
    p = uz.pack_weight(w)
    assert p.nbytes > 1 << 32
    last = w[e - 1].clone()
    back = uz.unpack_weight(p)
    assert torch.equal(back.view(torch.int16), w.view(torch.int16))
    del w, back
    x = normal(101, m, k)
    counts = [0] * e
    counts[0], counts[e - 1] = 3, m - 3
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    y = uz.grouped_linear(x, off, p)
    close(y[3:], *linear64(x[3:], last, None, "none", None, BF)[2:], "y")
    dy = normal(102, m, n)
    dx, _, _ = uz.grouped_linear_backward(dy, x, off, p, need_weight=False)
    close(dx[3:], *backward64(dy[3:], x[3:], last, None, "none", BF)["dx"], "dx")


@pytest.mark.parametrize("m", [20, 700])
def test_rows_far_apart(m):
    """Rows of x and y so far apart that their offsets pass 2^32 bytes."""
    n, k, stride = 48, 64, (1 << 22) + 8 if m < 100 else (1 << 21) + (1 << 20) + 8
    store = torch.zeros(((m - 1) * stride + 64,), dtype=BF, device=DEV)
    x = store.as_strided((m, k), (stride, 1))
    x.copy_(normal(110, m, k))
    w = normal(111, n, k, scale=0.1)
    p = uz.pack_weight(w)
    want = uz.linear(x.contiguous(), p)
    assert torch.equal(uz.linear(x, p), want)
    out = store.as_strided((m, n), (stride, 1), 8)
    xs = x.contiguous()
    uz.linear(xs, p, out=out)
    assert torch.equal(out, want)


def test_nothing_is_written_behind_a_workspace(monkeypatch):
    """Every workspace is exactly as large as its size function says, with a guard behind it."""
    import lossless_compression_float_amd.weights as ws
    held = []

    def guarded(need, device):
        t = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device=device)
        held.append((t, need))
        return t[:need]

    monkeypatch.setattr(ws, "workspace", guarded)
    x = normal(1, 17000, 20)
    p = uz.pack_weight(normal(2, 5000, 20, scale=0.1))
    t = torch.arange(17000, device=DEV) % 5000
    loss, lse = uz.linear_cross_entropy(x, p, t)
    uz.linear_cross_entropy_backward(torch.ones_like(loss), x, p, t, lse)  # two pieces, sums over them
    for m, n, k in ((100, 300, 1027), (70, 130, 4100), (777, 515, 330)):
        x = normal(3, m, k)
        p = uz.pack_weight(normal(4, n, k, scale=0.1))
        y, z = uz.linear(x, p, act="silu", return_preact=True)
        uz.linear_backward(y, x, p, preact=z, act="silu", need_bias=True)
        loss, lse = uz.linear_cross_entropy(x, p, torch.zeros(m, dtype=torch.int64, device=DEV))
        uz.linear_cross_entropy_backward(torch.ones_like(loss), x, p, torch.zeros(m, dtype=torch.int64, device=DEV), lse)
        p = uz.pack_weight(normal(5, 3, n // 2 * 2, k, scale=0.1), gated=True)
        off = torch.tensor([0, m // 3, m // 3, m], dtype=torch.int32, device=DEV)
        y, z = uz.grouped_linear(x, off, p, act="swiglu", return_preact=True)
        uz.grouped_linear_backward(y, x, off, p, preact=z, act="swiglu", need_bias=True)
    torch.cuda.synchronize()
    assert len(held) > 20
    for t, need in held:
        assert bool((t[need:] == 0xA5).all()), need


@pytest.mark.parametrize("m,n,k", [(1, 512, 256), (50, 4096, 2048), (100, 515, 4096), (300, 1030, 200), (2100, 8200, 64)])
def test_the_result_may_replace_its_residual(m, n, k):
    x, p = normal(1, m, k), uz.pack_weight(normal(2, n, k, scale=0.05))
    r = normal(3, m, n)
    want = uz.linear(x, p, residual=r)
    assert same(uz.linear(x, p, residual=r, out=r), want) and same(r, want)
    # and columns beside x in one buffer
    both = torch.zeros(m, n + k, dtype=BF, device=DEV)
    both[:, n:] = x
    uz.linear(both[:, n:], p, out=both[:, :n])
    assert same(both[:, :n], uz.linear(x, p)) and same(both[:, n:], x)


def small(seed, *shape):
    """-1, 0 and 1: sums of their products are exact."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device=DEV).to(BF)


WIDEST = (1 << 22) - 512


@pytest.mark.parametrize("m", [5, 300])
def test_the_most_rows_of_a_weight(m):
    w, x = small(1, WIDEST, 64), small(2, m, 64)
    p = uz.pack_weight(w)
    y, z = uz.linear(x, p, return_preact=True)
    for c in range(0, WIDEST, 1 << 20):
        assert torch.equal(y[:, c:c + (1 << 20)].float(), x.float() @ w[c:c + (1 << 20)].float().t())
    at = (torch.arange(m, device=DEV) * 13981) % WIDEST
    at[-1] = WIDEST - 1
    dy = torch.zeros(m, WIDEST, dtype=BF, device=DEV)
    dy[torch.arange(m), at] = 1
    del y
    for act in ("none", "relu"):  # dy as it is, and its product with the activation's gradient
        on = (z[torch.arange(m), at] > 0)[:, None] if act == "relu" else torch.ones(m, 1, dtype=torch.bool, device=DEV)
        dx, dw, _ = uz.linear_backward(dy, x, p, preact=z, act=act)
        assert torch.equal(dx, torch.where(on, w[at], 0))
        assert torch.equal(dw[at], torch.where(on, x, 0))
        assert int((dw != 0).sum()) == int((dw[at] != 0).sum())


@pytest.mark.parametrize("m", [5, 300])
def test_the_most_columns_of_a_weight(m):
    w, x = small(3, 16, WIDEST), small(4, m, WIDEST)
    p = uz.pack_weight(w)
    y = uz.linear(x, p, out_dtype=F32)
    want = torch.zeros(m, 16, dtype=torch.float64, device=DEV)
    for c in range(0, WIDEST, 1 << 20):
        s = slice(c, c + (1 << 20))
        want += (x[:, s].float() @ w[:, s].float().t()).double()  # (each exact: below 2^24)
    assert torch.equal(y.double(), want)
    dy = torch.zeros(m, 16, dtype=BF, device=DEV)
    dy[torch.arange(m), torch.arange(m) % 16] = 1
    dx, dw, _ = uz.linear_backward(dy, x, p)
    assert torch.equal(dx, w[torch.arange(m, device=DEV) % 16])
    for n in range(16):
        assert torch.equal(dw[n].float(), x[n::16].float().sum(0))


def test_the_largest_vocabulary():
    """Logits are exact here.  A token's sum passes through at most 32 additions in a lane, 10 in a tile and 262 over the
    16,382 tiles, each 2^-24 of it, and exponentials good to 2^-20: 1.9e-5 of the sum, and lse is rounded at 15."""
    m = 70
    w, x = small(5, WIDEST, 64), small(6, m, 64)
    t = (torch.arange(m, device=DEV) * 59999) % WIDEST
    p = uz.pack_weight(w)
    loss, lse = uz.linear_cross_entropy(x, p, t)
    total = torch.zeros(m, dtype=torch.float64, device=DEV)
    for c in range(0, WIDEST, 1 << 20):
        total += torch.exp((x.float() @ w[c:c + (1 << 20)].float().t()).double()).sum(1)
    want = torch.log(total)
    bound = 304 * 2.0 ** -24 + 2.0 ** -20 + 15 * 2.0 ** -23
    assert float((lse.double() - want).abs().max()) < bound
    picked = (x.float() * w[t].float()).sum(1).double()
    assert float((loss.double() - (want - picked)).abs().max()) < bound + 40 * 2.0 ** -24
    # with a dloss for one token only, dw's rows are multiples of its x: that of its target, and those of the softmax
    g = torch.zeros(m, device=DEV)
    g[9] = 1
    dx, dw = uz.linear_cross_entropy_backward(g, x, p, t, lse)
    soft = torch.exp(picked[9] - want[9]) - 1
    assert torch.allclose(dw[t[9]].double(), soft * x[9].double(), rtol=2.0 ** -7, atol=0)
    assert not bool(dx[:9].any()) and not bool(dx[10:].any()) and bool(dx[9].any())
