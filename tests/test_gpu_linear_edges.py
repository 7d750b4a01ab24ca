"""The products with packed weights where their contract has an edge: groups
out of order, rows of no group, the activations' tails, masked tokens, runs of
the contraction joined behind every epilogue.  The bounds are derived in
linear_testlib or beside the test."""
import pytest
import torch

import lossless_compression_float_amd as uz
from linear_testlib import backward64, close, linear64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


# ---- groups out of order --------------------------------------------------------

OUT_OF_ORDER = {
    # tokens, offsets: descending pairs are empty groups, the others may lie anywhere and leave gaps
    "behind the first": (12, [4, 2, 12]), "before the first": (12, [12, 0, 3]), "ends low": (12, [0, 10, 5]),
    "gap": (12, [5, 10, 0, 3]), "two gaps": (40, [30, 36, 12, 20, 2, 7]), "none": (9, [9, 5, 0]),
    "many rows": (900, [700, 900, 300, 520, 1, 290]), "runs": (150, [100, 150, 20, 75])}


@pytest.mark.parametrize("name", sorted(OUT_OF_ORDER))
@pytest.mark.parametrize("n,k,act,out", [(40, 64, "none", BF), (134, 72, "swiglu", F32), (272, 1024, "silu", BF)])
def test_groups_out_of_order_keep_their_rows(name, n, k, act, out):
    """Rows of a group are its results, whatever the order of the groups, and all other rows of a new output are zero."""
    t, offsets = OUT_OF_ORDER[name]
    g = gen(1)
    e, width = len(offsets) - 1, n // 2 if act == "swiglu" else n
    x, w, dy = normal(g, t, k), normal(g, e, n, k, scale=0.1), normal(g, t, width)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    p = uz.pack_weight(w, gated=act == "swiglu")
    for _ in range(3):
        junk = [torch.full((t, c), float("nan"), device=DEV) for c in (width, k)]  # what a new output's memory may hold
        torch.cuda.synchronize()
        del junk
        y = uz.grouped_linear(x, off, p, act=act, out_dtype=out)
        _, z = uz.grouped_linear(x, off, p, act=act, return_preact=True)
        dx, dw, _ = uz.grouped_linear_backward(dy, x, off, p, preact=z, act=act)
        rest = torch.ones(t, dtype=torch.bool, device=DEV)
        for i in range(e):
            s = slice(offsets[i], offsets[i + 1])
            if offsets[i + 1] <= offsets[i]:
                assert (dw[i] == 0).all()
                continue
            rest[s] = False
            _, _, y64, ey = linear64(x[s], w[i], None, act, None, out)
            close(y[s], y64, ey, "y of group %d" % i)
            want = backward64(dy[s], x[s], w[i], z[s], act, BF)
            close(dx[s], *want["dx"], "dx of group %d" % i)
            close(dw[i], *want["dw"], "dw of group %d" % i)
        assert (y[rest] == 0).all() and (dx[rest] == 0).all()


# ---- a stream of the call's own ----------------------------------------------------

def test_memory_of_a_call_on_another_stream_is_that_streams_own():
    """Blocks that the current stream's pending work still uses are not handed to a call on another stream."""
    m, n, k, act = 300, 320, 4096, "silu"
    g = gen(2)
    x, dy, wt = normal(g, m, k), normal(g, m, n), normal(g, n, k, scale=0.05)
    w, t, dl = uz.pack_weight(wt), torch.randint(0, n, (m,), generator=g).to(DEV), torch.ones(m, device=DEV)

    def calls(**kw):
        p = uz.pack_weight(wt, **kw)
        y, z = uz.linear(x, w, act=act, return_preact=True, **kw)
        dx, dw, db = uz.linear_backward(dy, x, w, preact=z, act=act, need_bias=True, **kw)
        loss, lse = uz.linear_cross_entropy(x, w, t, **kw)
        lx, lw = uz.linear_cross_entropy_backward(dl, x, w, t, lse, **kw)
        return [p.data, uz.unpack_weight(w, **kw), y, z, dx, dw, db, loss, lse, lx, lw]

    want = calls()
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = [torch.empty(s, dtype=torch.uint8, device=DEV) for s in (512, m * n * 2, m * n * 4, 1 << 21, 1 << 25, 1 << 25)]
    for b in busy:
        b.zero_()
    del b, busy  # free for the current stream's next work, and only for that
    side.wait_stream(main)
    got = calls(stream=side)
    blocks = [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
              if s["stream"] == side.cuda_stream]
    for r in got:
        assert any(a <= r.data_ptr() < e for a, e in blocks), (r.shape, r.dtype)
    main.wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
