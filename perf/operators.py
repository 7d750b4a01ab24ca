"""Timed cases of the products that read packed weights: linear, grouped_linear and linear_cross_entropy, forward and
backward.

The weights of a model that arrived compressed stay in HBM losslessly packed (about 12 bits a bf16 value) and are
multiplied from there.  `run` with `own` false computes the same operators in their plain form: from the bf16 weights, in
fp32 with elementary torch operations, rounded once at the end.  Sizes are those of the package's own Llama-3-8B-shaped
weight set and of its small-message batch (hidden size 8192), with odd ones beside them.
"""
import math

import torch

own = False

DEV = "cuda"
IGNORE = -100
# Bits of one packed weight: 8 of sign and mantissa, 4 of exponent code, and a tile header of 64 bits per 1024 values.
PACKED_BITS = 8 + 4 + 64 / 1024


def listed():
    return [
        # one token through an attention output projection with its residual: the smallest call of a decode step
        dict(name="linear token", op="linear", m=1, n=4096, k=4096, act="none", bias=False, residual=True, out="bf16",
             backward=False),
        # a small serving batch through the fused gate and up projection
        dict(name="linear batch gated", op="linear", m=16, n=14336, k=4096, act="swiglu", bias=False, residual=False,
             out="bf16", backward=False),
        # a prompt of odd length through a layer with bias and odd sizes, result kept in fp32
        dict(name="linear odd prompt", op="linear", m=777, n=4099, k=1027, act="gelu", bias=True, residual=False,
             out="fp32", backward=False),
        # a long prompt through the down projection with its residual
        dict(name="linear long prompt", op="linear", m=8192, n=4096, k=14336, act="none", bias=False, residual=True,
             out="bf16", backward=False),
        # a training step through the gate and up projection: forward, then the gradients of input, weight and bias
        dict(name="linear step gated", op="linear", m=4096, n=14336, k=4096, act="swiglu", bias=True, residual=False,
             out="bf16", backward=True),
        # a decode batch over experts: a few tokens for each, some experts with none
        dict(name="experts batch", op="grouped", m=24, e=16, n=4096, k=4096, act="silu", bias=False, backward=False),
        # a prompt over experts of odd width, ragged groups
        dict(name="experts odd prompt", op="grouped", m=1999, e=7, n=1333, k=2050, act="gelu_tanh", bias=True,
             backward=False),
        # a long prompt over gated experts
        dict(name="experts long prompt", op="grouped", m=16384, e=8, n=4096, k=4096, act="swiglu", bias=False,
             backward=False),
        # a training step over experts
        dict(name="experts step", op="grouped", m=8192, e=8, n=4096, k=4096, act="silu", bias=True, backward=True),
        # the scores of a short rollout under weights that have just arrived
        dict(name="loss scoring", op="loss", m=64, n=128256, k=4096, backward=False),
        # the scores of a batch over an odd vocabulary
        dict(name="loss odd batch", op="loss", m=1001, n=32003, k=1024, backward=False),
        # a training step through the output head: loss, and the gradients of hidden states and weight
        dict(name="loss step", op="loss", m=4096, n=128256, k=4096, backward=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "loss"])
    backward = rng.random() < 0.35
    snap = rng.choice([1, 8, 16, 64])  # odd sizes, and sizes that are multiples of something

    def size(lo, hi):
        return max(snap, _log(rng, lo, hi) // snap * snap)

    if op == "linear":
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
        return dict(op=op, m=_log(rng, 1, 4096), n=size(64, 14336), k=size(64, 8192), act=act, bias=rng.random() < 0.5,
                    residual=act != "swiglu" and rng.random() < 0.5, out="bf16" if backward else rng.choice(["bf16", "fp32"]),
                    backward=backward)
    if op == "grouped":
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
        return dict(op=op, m=_log(rng, 2, 8192), e=_log(rng, 2, 32), n=size(64, 4096), k=size(64, 4096), act=act,
                    bias=rng.random() < 0.5, backward=backward)
    return dict(op=op, m=_log(rng, 1, 2048), n=size(512, 65536), k=size(64, 4096), backward=backward)


def _gated(case):
    return case.get("act") == "swiglu"


def _rows(case):
    return 2 * case["n"] if _gated(case) else case["n"]


def _counts(case, seed):
    """Ragged group sizes that add up to m: some experts are popular, some get nothing."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    pop = torch.rand(case["e"], generator=g, dtype=torch.float64) ** 2 + 0.05
    pick = torch.multinomial(pop, case["m"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["e"]).tolist()


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)

    m, n, k, rows = case["m"], case["n"], case["k"], _rows(case)
    # weights as in the package's weight set, N(0, 0.02^2); activations N(0, 1) with a log-normal scale for each token
    rms = torch.exp(0.5 * torch.randn((m, 1), generator=g, device=DEV))
    s = {"x": (torch.randn((m, k), generator=g, device=DEV) * rms).to(torch.bfloat16)}
    stack = (case["e"],) if case["op"] == "grouped" else ()
    s["w"] = normal(*stack, rows, k, scale=0.02)
    if case["op"] == "loss":
        s["target"] = torch.randint(0, n, (m,), generator=g, device=DEV)
        s["target"][torch.rand(m, generator=g, device=DEV) < 0.1] = IGNORE  # padding tokens
        s["dloss"] = torch.full((m,), 1.0 / m, device=DEV)
        return s
    s["bias"] = normal(*stack, rows, scale=0.1) if case["bias"] else None
    if case["op"] == "grouped":
        s["counts"] = _counts(case, seed)
        s["offsets"] = torch.tensor([0] + s["counts"]).cumsum(0).to(torch.int32).to(DEV)
    elif case["residual"]:
        s["residual"] = normal(m, n, dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    s["dy"] = normal(m, n) if case["backward"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        # A program that holds its weights packed has no bf16 copy of them; the plain form has the same values as bf16.
        import lossless_compression_float_amd as uz
        s["packed"] = uz.pack_weight(s.pop("w"), gated=_gated(case))
    return s


# ---- the plain forms: elementary torch operations in fp32 ----

def _act(z, act):
    """act(z); swiglu: the first half of z's columns gates the second."""
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        a, b = z.chunk(2, dim=-1)
        return a / (1 + torch.exp(-a)) * b
    return z


def _dact(dy, z, act):
    """The gradient of the pre-activation z, given that of act(z)."""
    if act == "relu":
        return dy * (z > 0)
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return dy * s * (1 + z * (1 - s))
    if act == "swiglu":
        a, b = z.chunk(2, dim=-1)
        s = 1 / (1 + torch.exp(-a))
        return torch.cat((dy * b * s * (1 + a * (1 - s)), dy * a * s), dim=-1)
    return dy


def _plain_linear(x, w, bias, act, residual, dy, backward, out):
    xf, wf = x.float(), w.float()
    z = xf @ wf.t()
    if bias is not None:
        z = z + bias.float()
    y = _act(z, act)
    if residual is not None:
        y = y + residual.float()
    r = {"y": y.to(torch.float32 if out == "fp32" else torch.bfloat16)}
    if backward:
        dz = _dact(dy.float(), z, act)
        r["dx"] = (dz @ wf).to(torch.bfloat16)
        r["dw"] = (dz.t() @ xf).to(torch.bfloat16)
        if bias is not None:
            r["dbias"] = dz.sum(0).to(torch.bfloat16)
    return r


def _plain_grouped(s, case):
    """The groups one after another (their sizes known on the host, which spares this form a wait)."""
    parts = []
    at = 0
    for e, c in enumerate(s["counts"]):
        rows = slice(at, at + c)
        at += c
        parts.append(_plain_linear(s["x"][rows], s["w"][e], None if s["bias"] is None else s["bias"][e], case["act"], None,
                                   None if s["dy"] is None else s["dy"][rows], case["backward"], "bf16"))
    r = {"y": torch.cat([p["y"] for p in parts])}
    if case["backward"]:
        r["dx"] = torch.cat([p["dx"] for p in parts])
        r["dw"] = torch.stack([p["dw"] for p in parts])
        if s["bias"] is not None:
            r["dbias"] = torch.stack([p["dbias"] for p in parts])
    return r


def _plain_loss(s, case):
    xf, wf, t = s["x"].float(), s["w"].float(), s["target"]
    z = xf @ wf.t()
    top = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    valid = t != IGNORE
    at = t.clamp(min=0).unsqueeze(1)
    r = {"loss": torch.where(valid, lse - z.gather(1, at).squeeze(1), 0.0), "lse": lse}
    if case["backward"]:
        g = torch.where(valid, s["dloss"], 0.0).unsqueeze(1)
        dz = e.mul_(g / total)
        dz.scatter_add_(1, at, -g)
        r["dx"] = (dz @ wf).to(torch.bfloat16)
        r["dw"] = (dz.t() @ xf).to(torch.bfloat16)
    return r


# ---- the framework's calls ----

def _own_linear(s, case):
    import lossless_compression_float_amd as uz
    w, act = s["packed"], case["act"]
    out = torch.float32 if case["out"] == "fp32" else torch.bfloat16
    if not case["backward"]:
        return {"y": uz.linear(s["x"], w, bias=s["bias"], act=act, residual=s.get("residual"), out_dtype=out)}
    y, z = uz.linear(s["x"], w, bias=s["bias"], act=act, residual=s.get("residual"), out_dtype=out, return_preact=True)
    dx, dw, db = uz.linear_backward(s["dy"], s["x"], w, preact=z, act=act, need_bias=s["bias"] is not None)
    r = {"y": y, "dx": dx, "dw": dw}
    if s["bias"] is not None:
        r["dbias"] = db
    return r


def _own_grouped(s, case):
    import lossless_compression_float_amd as uz
    w, act = s["packed"], case["act"]
    if not case["backward"]:
        return {"y": uz.grouped_linear(s["x"], s["offsets"], w, bias=s["bias"], act=act)}
    y, z = uz.grouped_linear(s["x"], s["offsets"], w, bias=s["bias"], act=act, return_preact=True)
    dx, dw, db = uz.grouped_linear_backward(s["dy"], s["x"], s["offsets"], w, preact=z, act=act,
                                            need_bias=s["bias"] is not None)
    r = {"y": y, "dx": dx, "dw": dw}
    if s["bias"] is not None:
        r["dbias"] = db
    return r


def _own_loss(s, case):
    import lossless_compression_float_amd as uz
    loss, lse = uz.linear_cross_entropy(s["x"], s["packed"], s["target"], ignore_index=IGNORE)
    r = {"loss": loss, "lse": lse}
    if case["backward"]:
        r["dx"], r["dw"] = uz.linear_cross_entropy_backward(s["dloss"], s["x"], s["packed"], s["target"], lse,
                                                            ignore_index=IGNORE)
    return r


def run(state):
    case = state["case"]
    if own:
        return {"linear": _own_linear, "grouped": _own_grouped, "loss": _own_loss}[case["op"]](state, case)
    if case["op"] == "linear":
        return _plain_linear(state["x"], state["w"], state["bias"], case["act"], state.get("residual"), state["dy"],
                             case["backward"], case["out"])
    return (_plain_grouped if case["op"] == "grouped" else _plain_loss)(state, case)


def work(case):
    """Each input read once and each output written once: the weights in their packed form (of the experts, those that
    can have a token), and the products' multiplications."""
    m, n, k, rows = case["m"], case["n"], case["k"], _rows(case)
    experts = min(case["e"], m) if case["op"] == "grouped" else 1
    wide = 4 if case.get("out") == "fp32" else 2
    product = 2.0 * m * rows * k
    size = experts * rows * k * PACKED_BITS / 8 + 2.0 * m * k
    if case["op"] == "loss":
        size += 8.0 * m + 8.0 * m
    else:
        size += wide * m * n * (2 if case.get("residual") else 1)
        size += 2.0 * experts * rows if case["bias"] else 0
    flops = product
    if case["backward"]:
        flops += 2 * product
        size += 2.0 * m * k + 2.0 * case.get("e", 1) * rows * k
        size += 4.0 * m if case["op"] == "loss" else 2.0 * m * n
        size += 2.0 * case.get("e", 1) * rows if case.get("bias") else 0
    return {"bytes": size, "flops": flops}


# ---- from the definitions, in 64 bits ----

def _exact_one(x, w, bias, act, residual, dy, backward):
    x, w = x.double(), w.double()
    n = w.shape[0]
    z = torch.matmul(x, w.T.contiguous())
    if bias is not None:
        z += bias.double()
    one = torch.ones((), dtype=torch.float64, device=DEV)
    if act == "swiglu":
        h = n // 2
        gate, up = z[:, :h], z[:, h:]
        sig = torch.sigmoid(gate)
        y = gate * sig * up
    elif act == "silu":
        sig = torch.sigmoid(z)
        y = z * sig
    elif act == "gelu":
        cdf = torch.special.ndtr(z)
        y = z * cdf
    elif act == "gelu_tanh":
        u = (2 / math.pi) ** 0.5 * z * (one + 0.044715 * z ** 2)
        y = z * torch.sigmoid(2 * u)
    elif act == "relu":
        y = torch.maximum(z, 0 * one)
    else:
        y = z
    r = {"y": y if residual is None else y + residual.double()}
    if not backward:
        return r
    dy = dy.double()
    if act == "swiglu":
        dz = torch.empty_like(z)
        dz[:, :h] = dy * up * (sig + gate * sig * (one - sig))
        dz[:, h:] = dy * gate * sig
    elif act == "silu":
        dz = dy * (sig + z * sig * (one - sig))
    elif act == "gelu":
        dz = dy * (cdf + z * torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5)
    elif act == "gelu_tanh":
        sg = torch.sigmoid(2 * u)
        dz = dy * (sg + z * 2 * sg * (one - sg) * (2 / math.pi) ** 0.5 * (one + 3 * 0.044715 * z ** 2))
    elif act == "relu":
        dz = torch.where(z > 0, dy, 0 * one)
    else:
        dz = dy
    r["dx"] = torch.matmul(dz, w)
    r["dw"] = torch.matmul(dz.T.contiguous(), x)
    if bias is not None:
        r["dbias"] = dz.sum(dim=0)
    return r


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear":
        return _exact_one(s["x"], s["w"], s["bias"], case["act"], s.get("residual"), s["dy"], case["backward"])
    if case["op"] == "grouped":
        ends = torch.tensor(s["counts"]).cumsum(0).tolist()
        each = [_exact_one(s["x"][b - c:b], s["w"][e], None if s["bias"] is None else s["bias"][e], case["act"], None,
                           None if s["dy"] is None else s["dy"][b - c:b], case["backward"])
                for e, (b, c) in enumerate(zip(ends, s["counts"]))]
        r = {"y": torch.cat([p["y"] for p in each])}
        if case["backward"]:
            r["dx"] = torch.cat([p["dx"] for p in each])
            r["dw"] = torch.stack([p["dw"] for p in each])
            if case["bias"]:
                r["dbias"] = torch.stack([p["dbias"] for p in each])
        return r
    x, w = s["x"].double(), s["w"].double()
    z = torch.matmul(x, w.T.contiguous())
    lse = torch.logsumexp(z, dim=1)
    kept = s["target"] != IGNORE
    idx = torch.where(kept, s["target"], 0)
    picked = z[torch.arange(z.shape[0], device=DEV), idx]
    r = {"loss": torch.where(kept, lse - picked, torch.zeros_like(lse)), "lse": lse}
    if case["backward"]:
        z.sub_(lse[:, None]).exp_()
        z[torch.arange(z.shape[0], device=DEV), idx] -= 1
        z.mul_((s["dloss"].double() * kept)[:, None])
        r["dx"] = torch.matmul(z, w)
        r["dw"] = torch.matmul(z.T.contiguous(), x)
    return r
