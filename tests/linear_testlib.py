"""Plain 64-bit forms of the products with packed weights, and how far a
correct kernel's results may be from them.

Every bound below is arithmetic, for operands that are exact in bf16:
  * a sum of k products in fp32, in any order, is off by at most
    (k + 8) 2^-23 times the sum of the products' magnitudes (2^-24 a rounding;
    one bit is left for an accumulator that truncates);
  * a rounding to bf16 is off by at most 2^-8 of the value, to fp32 2^-24;
  * exp, erf and tanh of the device are within a few units in the last place:
    2^-20 relative covers the short formulas made of them.
"""
import math

import torch

ACC = 2.0 ** -23
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FUN = 2.0 ** -20


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "swiglu":
        h = z.shape[-1] // 2
        return z[:, :h] * torch.sigmoid(z[:, :h]) * z[:, h:]
    return z


def dz64(dy, z, act):
    """dy times the activation's derivative, by autograd in 64 bits."""
    z = z.detach().clone().requires_grad_(True)
    act64(z, act).backward(dy)
    return z.grad


def close(got, want, bound, what):
    """Every value of `got` within `bound` of `want`; names the worst if not.
    Infinities and NaNs have to be where they are in `want`."""
    got = got.detach().double().cpu()
    want, bound = want.double().cpu(), bound.double().cpu()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaNs elsewhere"
    special = ~fin & ~torch.isnan(want)
    assert torch.equal(got[special], want[special]), what + ": infinities elsewhere"
    assert torch.isfinite(got[fin]).all(), what + ": not finite"
    if not fin.any():
        return
    off = (got - want).abs()[fin]
    b = bound.expand_as(want)[fin]
    bad = off > b
    if bad.any():
        i = int((off / b.clamp(min=1e-300)).argmax())
        raise AssertionError("%s: %d of %d outside; worst off by %g with %g allowed, want %g" % (
            what, int(bad.sum()), off.numel(), float(off[i]), float(b[i]), float(want[fin][i])))


def linear64(x, w, bias, act, residual, out_dtype, preact_dtype=torch.float32):
    """(z, its bound, y, its bound) on the CPU in 64 bits."""
    x, w = x.double().cpu(), w.double().cpu()
    k = x.shape[1]
    z = x @ w.T
    ez = (k + 8) * ACC * (x.abs() @ w.abs().T)
    if bias is not None:
        z = z + bias.double().cpu()
        ez = ez + ACC * z.abs()
    y = act64(z, act)
    # the steepest slope of the activations is 1.13 (gelu)
    if act == "swiglu":
        h = z.shape[1] // 2
        a, b = z[:, :h], z[:, h:]
        ey = 1.13 * ez[:, :h] * (b.abs() + ez[:, h:]) + a.abs() * ez[:, h:] + FUN * (a * b).abs()
    else:
        ey = 1.13 * ez + (0 if act in ("none", "relu") else FUN * z.abs())
    if residual is not None:
        y = y + residual.double().cpu()
    ey = ey + 2.0 ** -24 * y.abs()
    return z, ez + HALF[preact_dtype] * (z.abs() + ez), y, ey + HALF[out_dtype] * (y.abs() + ey)


def backward64(dy, x, w, z, act, bias_dtype):
    """{name: (gradient, bound)} given the kept pre-activation."""
    dy, x, w = dy.double().cpu(), x.double().cpu(), w.double().cpu()
    dz = dy if act == "none" else dz64(dy, z.double().cpu(), act)
    # of the derivative: its own rounding and that of the formula's terms, which are below (1 + |z|)^2
    fun = torch.zeros_like(dz)
    if act not in ("none", "relu"):
        zz = z.double().cpu()
        if act == "swiglu":
            h = zz.shape[1] // 2
            fun[:, :h] = FUN * dy.abs() * zz[:, h:].abs() * (1 + zz[:, :h].abs())
            fun[:, h:] = FUN * dy.abs() * zz[:, :h].abs()
        else:
            fun = FUN * dy.abs() * (1 + zz.abs()) ** 2
    edz = fun + HALF[torch.bfloat16] * (dz.abs() + fun)
    m, n = dz.shape
    half = HALF[torch.bfloat16]
    dx = dz @ w
    ex = edz @ w.abs() + (n + 8) * ACC * ((dz.abs() + edz) @ w.abs())
    dw = dz.T @ x
    ew = edz.T @ x.abs() + (m + 8) * ACC * ((dz.abs() + edz).T @ x.abs())
    db = dz.sum(0)
    eb = fun.sum(0) + (m + 8) * ACC * (dz.abs() + fun).sum(0)
    return {"dx": (dx, ex + half * (dx.abs() + ex)), "dw": (dw, ew + half * (dw.abs() + ew)),
            "dbias": (db, eb + HALF[bias_dtype] * (db.abs() + eb))}


def loss64(x, w, target, ignore):
    """(loss, lse, their bounds, logits, the logits' bounds)."""
    x, w, t = x.double().cpu(), w.double().cpu(), target.cpu()
    k, v = x.shape[1], w.shape[0]
    z = x @ w.T
    ez = (k + 8) * ACC * (x.abs() @ w.abs().T)
    lse = torch.logsumexp(z, 1)
    kept = t != ignore
    at = torch.where(kept, t, 0)
    loss = torch.where(kept, lse - z.gather(1, at[:, None]).squeeze(1), torch.zeros_like(lse))
    # exp's argument is off by 2^-24 of it: weighted with the softmax that is at most log(v) 2^-24, three times for
    # its product with log2(e), exp's own rounding and the second exponential of the join; 64 roundings of sums
    el = ez.max(1).values + (3 * math.log(v + 1) + 64) * 2.0 ** -24 + 2 * 2.0 ** -24 * lse.abs()
    eloss = el + ez.max(1).values + 2.0 ** -24 * (loss.abs() + z.abs().max(1).values)
    return loss, lse, eloss, el, z, ez


def loss_backward64(dloss, x, w, target, ignore):
    loss, lse, eloss, el, z, ez = loss64(x, w, target, ignore)
    x, w, t = x.double().cpu(), w.double().cpu(), target.cpu()
    m, v = z.shape
    kept = (t != ignore).double()[:, None]
    p = torch.exp(z - lse[:, None])
    ep = p * (ez + el[:, None] + (z - lse[:, None]).abs() * 2.0 ** -23 + 2.0 ** -20)
    hot = torch.zeros_like(p)
    hot.scatter_(1, torch.where(t != ignore, t, 0)[:, None], 1.0)
    g = dloss.double().cpu()[:, None] * kept
    dz = g * (p - hot)
    e0 = g.abs() * (ep + 2.0 ** -24)
    half = HALF[torch.bfloat16]
    edz = e0 + half * (dz.abs() + e0)
    dx, dw = dz @ w, dz.T @ x
    ex = edz @ w.abs() + (v + 8) * ACC * ((dz.abs() + edz) @ w.abs())
    ew = edz.T @ x.abs() + (m + 8) * ACC * ((dz.abs() + edz).T @ x.abs())
    return (dx, ex + half * (dx.abs() + ex)), (dw, ew + half * (dw.abs() + ew))
