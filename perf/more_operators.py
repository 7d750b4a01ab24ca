"""Timed cases of the router, the expert layer for a few tokens and the sampler: moe_route with its gradient, moe, sample.

They are what a decode step with packed weights needs beside the products: the router's logits become experts and weights,
the experts are multiplied from their packed form, and the head's logits become tokens.  `run` with `own` false computes
the same in elementary torch operations: the expert layer in fp32 from the bf16 weights, what decides between neighbours
(a top-p border, a draw) in 64 bits.  Widths 4096 and 14336 and the vocabulary of 128256 are those of the package's own
Llama-3-8B-shaped weight set; the others are generic, odd ones among them.
"""
import math

import torch

own = False

DEV = "cuda"
# Bits of one packed weight: 8 of sign and mantissa, 4 of exponent code, and a tile header of 64 bits per 1024 values.
PACKED_BITS = 8 + 4 + 64 / 1024


def listed():
    return [
        # the router of one decode step with a few requests: the smallest call
        dict(name="route step", op="route", t=4, e=128, k=8, scores="softmax", bias=False, renorm=True, dtype="fp32",
             backward=False),
        # a prompt of odd length, an odd number of experts, logits in bf16 with many ties
        dict(name="route odd prompt", op="route", t=777, e=60, k=4, scores="softmax", bias=False, renorm=False, dtype="bf16",
             backward=False),
        # a training step: sigmoid scores with a balancing bias, and the gradient of the logits
        dict(name="route training", op="route", t=16384, e=64, k=6, scores="sigmoid", bias=True, renorm=True, dtype="fp32",
             backward=True),
        # one token through many small experts
        dict(name="experts token", op="moe", t=1, e=128, k=8, d=2048, f=768, act="swiglu", bias=False, residual=True),
        # a small batch of odd sizes, plain experts with biases
        dict(name="experts odd batch", op="moe", t=13, e=7, k=3, d=1027, f=1333, act="gelu", bias=True, residual=False),
        # a small batch over few large experts: nearly all weights are read
        dict(name="experts large", op="moe", t=16, e=8, k=2, d=4096, f=14336, act="swiglu", bias=False, residual=False),
        # a serving batch over many experts, about eight tokens each
        dict(name="experts batch", op="moe", t=64, e=64, k=8, d=2048, f=1024, act="swiglu", bias=False, residual=True),
        # a larger batch, short experts
        dict(name="experts wide batch", op="moe", t=200, e=128, k=4, d=1024, f=512, act="silu", bias=False, residual=False),
        # one request with the usual filters
        dict(name="sample token", op="sample", t=1, v=128256, dtype="fp32", temperature=0.7, top_k=50, top_p=0.9, min_p=0.0,
             mixed=False, spread=3.0),
        # a batch of rollouts at temperature 1 without filters, logits in bf16
        dict(name="sample rollout", op="sample", t=64, v=128256, dtype="bf16", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
             mixed=False, spread=2.5),
        # requests with parameters of their own, some greedy, an odd vocabulary
        dict(name="sample mixed", op="sample", t=33, v=32003, dtype="fp32", temperature=0.9, top_k=40, top_p=0.95, min_p=0.05,
             mixed=True, spread=3.0),
        # a large serving batch with top-p
        dict(name="sample batch", op="sample", t=256, v=128256, dtype="fp32", temperature=0.8, top_k=0, top_p=0.95, min_p=0.0,
             mixed=False, spread=3.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "sample", "sample"])
    if op == "route":
        e = _log(rng, 4, 256)
        scores = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, t=_log(rng, 1, 16384), e=e, k=rng.randint(1, min(8, e)), scores=scores,
                    bias=scores == "sigmoid" and rng.random() < 0.5, renorm=rng.random() < 0.5,
                    dtype=rng.choice(["fp32", "bf16"]), backward=rng.random() < 0.4)
    if op == "moe":
        snap = rng.choice([1, 8, 64])

        def size(lo, hi):
            return max(snap, _log(rng, lo, hi) // snap * snap)

        e, d = _log(rng, 4, 128), size(256, 4096)
        f = size(128, max(256, min(8192, 400_000_000 // (e * d))))
        act = rng.choice(["swiglu", "swiglu", "silu", "gelu", "relu"])
        return dict(op=op, t=_log(rng, 1, 256), e=e, k=rng.randint(1, min(8, e)), d=d, f=f, act=act,
                    bias=rng.random() < 0.3, residual=rng.random() < 0.5)
    return dict(op=op, t=_log(rng, 1, 256), v=_log(rng, 512, 128256), dtype=rng.choice(["fp32", "bf16"]),
                temperature=rng.choice([0.0, 0.5, 0.7, 1.0, 1.3]), top_k=rng.choice([0, 0, 1, 20, 50, 200, 1000]),
                top_p=rng.choice([1.0, 1.0, 0.5, 0.9, 0.95, 0.99]), min_p=rng.choice([0.0, 0.0, 0.02, 0.1]),
                mixed=rng.random() < 0.3, spread=rng.uniform(1.0, 4.0))


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)

    t, s = case["t"], {}
    if case["op"] == "sample":
        # a language model's logits: a broad bulk, a few tokens far above it
        v = case["v"]
        z = torch.randn((t, v), generator=g, device=DEV) * case["spread"]
        top = torch.randint(0, v, (t, 16), generator=g, device=DEV)
        z.scatter_add_(1, top, torch.rand((t, 16), generator=g, device=DEV) * 12.0 + 2.0)
        s["logits"] = z.to(_type(case))
        s["u"] = torch.rand(t, generator=g, device=DEV)
        if case["mixed"]:
            row = torch.rand((4, t), generator=g, device=DEV)
            s["temperature"] = torch.where(row[0] < 0.2, 0.0, case["temperature"] * (0.5 + row[0]))
            s["top_k"] = torch.where(row[1] < 0.5, 0, (case["top_k"] * 2 * row[1]).int()).to(torch.int32)
            s["top_p"] = torch.where(row[2] < 0.4, 1.0, 1 - (1 - case["top_p"]) * row[2])
            s["min_p"] = torch.where(row[3] < 0.4, 0.0, case["min_p"] * row[3])
        else:
            s.update({n: case[n] for n in ("temperature", "top_k", "top_p", "min_p")})
        return s
    e = case["e"]
    popular = torch.randn(e, generator=g, device=DEV) * 0.5  # some experts are asked for more often
    s["logits"] = torch.randn((t, e), generator=g, device=DEV) + popular
    if case["op"] == "route":
        s["logits"] = s["logits"].to(_type(case))
        s["bias"] = normal(e, scale=0.1, dtype=torch.float32) if case["bias"] else None
        if case["backward"]:
            s["dweights"] = normal(t, case["k"], dtype=torch.float32)
        return s
    d, f = case["d"], case["f"]
    rows = 2 * f if case["act"] == "swiglu" else f
    rms = torch.exp(0.5 * torch.randn((t, 1), generator=g, device=DEV))
    s["x"] = (torch.randn((t, d), generator=g, device=DEV) * rms).to(torch.bfloat16)
    # weights as in the package's weight set, N(0, 0.02^2), an expert at a time to spare memory
    s["up"] = torch.empty((e, rows, d), dtype=torch.bfloat16, device=DEV)
    s["down"] = torch.empty((e, d, f), dtype=torch.bfloat16, device=DEV)
    for i in range(e):
        s["up"][i] = normal(rows, d, scale=0.02)
        s["down"][i] = normal(d, f, scale=0.02)
    s["up_bias"] = normal(e, rows, scale=0.1) if case["bias"] else None
    s["down_bias"] = normal(e, d, scale=0.1) if case["bias"] else None
    s["residual"] = normal(t, d) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "moe":
        if own:
            # A program that holds its weights packed has no bf16 copy of them; the plain form has the same values as bf16.
            import lossless_compression_float_amd as uz
            s["up"] = uz.pack_weight(s["up"], gated=case["act"] == "swiglu")
            s["down"] = uz.pack_weight(s["down"])
        else:
            # the experts with a token, known on the host, which spares the plain form a wait
            s["active"] = torch.unique(_plain_route(s["logits"], case["k"], "softmax", None, True)[0]).tolist()
    return s


# ---- the plain forms ----

def _plain_route(logits, k, scores, bias, renorm):
    """(experts, weights, scores of all experts): the k best of each token, of equal ones the lowest first."""
    z = logits.float()
    if scores == "softmax":
        p = torch.exp(z - z.max(dim=1, keepdim=True).values)
        p = p / p.sum(dim=1, keepdim=True)
        by = z
    else:
        p = 1 / (1 + torch.exp(-z))
        by = z if bias is None else 1 / (1 + torch.exp(-z.double())) + bias.double()
    experts = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, experts)
    if renorm:
        w = w / w.sum(dim=1, keepdim=True)
    return experts, w, p


def _run_route(s, case):
    t, e, k = case["t"], case["e"], case["k"]
    experts, w, p = _plain_route(s["logits"], k, case["scores"], s["bias"], case["renorm"])
    flat = experts.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(e, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts.cumsum(0)
    r = {"experts": experts.int(), "weights": w, "order": order.int(), "offsets": offsets.int()}
    if case["backward"]:
        g = s["dweights"]
        chosen = p.gather(1, experts)
        if case["renorm"]:
            dp = (g - (g * w).sum(dim=1, keepdim=True)) / chosen.sum(dim=1, keepdim=True)
        else:
            dp = g
        if case["scores"] == "sigmoid":
            dz = torch.zeros_like(p).scatter_(1, experts, dp * chosen * (1 - chosen))
        else:
            dz = torch.zeros_like(p).scatter_(1, experts, dp * chosen) - p * (dp * chosen).sum(dim=1, keepdim=True)
        r["dlogits"] = dz.to(s["logits"].dtype)
    return r


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    a, b = z.chunk(2, dim=-1)
    return a / (1 + torch.exp(-a)) * b


def _run_moe(s, case):
    experts, w, _ = _plain_route(s["logits"], case["k"], "softmax", None, True)
    x = s["x"].float()
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].float()
    for i in s["active"]:
        z = x @ s["up"][i].float().t()
        if s["up_bias"] is not None:
            z = z + s["up_bias"][i].float()
        o = _act(z, case["act"]) @ s["down"][i].float().t()
        if s["down_bias"] is not None:
            o = o + s["down_bias"][i].float()
        y = y + (w * (experts == i)).sum(dim=1, keepdim=True) * o
    return {"y": y.to(torch.bfloat16), "experts": experts.int(), "weights": w}


def _parameters(s, case):
    """The parameters of each row in 64 bits, from their fp32 values, as columns."""
    def column(v):
        if not isinstance(v, torch.Tensor):
            v = torch.full((case["t"],), v, device=DEV, dtype=torch.float32)
        return v.double().unsqueeze(1)

    return [column(s[n]) for n in ("temperature", "top_k", "top_p", "min_p")]


def _run_sample(s, case):
    temperature, top_k, top_p, min_p = _parameters(s, case)
    z = s["logits"].double()
    greedy = temperature == 0
    y = (z - z.max(dim=1, keepdim=True).values) / torch.where(greedy, 1.0, temperature)
    e = torch.exp(y)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    es = e.gather(1, order)
    rank = torch.arange(case["v"], device=DEV).unsqueeze(0)
    keep = (rank < torch.where(top_k > 0, top_k, float(case["v"]))) & ~(greedy & (rank > 0))
    es = es * keep
    before = es.cumsum(dim=1) - es
    keep &= (before < top_p * es.sum(dim=1, keepdim=True)) | (top_p >= 1) | (rank == 0)
    keep &= (es >= min_p) | (rank == 0)
    kept = torch.zeros_like(e).scatter_(1, order, e.gather(1, order) * keep)  # back in the order of the vocabulary
    run = kept.cumsum(dim=1)
    token = (run <= s["u"].double().unsqueeze(1) * kept.sum(dim=1, keepdim=True)).sum(dim=1)
    logprob = y.gather(1, token.unsqueeze(1)).squeeze(1) - torch.log(e.sum(dim=1))
    return {"token": token, "logprob": logprob.float()}


# ---- the framework's calls ----

def _own(s, case):
    import lossless_compression_float_amd as uz
    if case["op"] == "route":
        r = uz.moe_route(s["logits"], case["k"], scores=case["scores"], bias=s["bias"], renormalize=case["renorm"])
        out = {"experts": r.experts, "weights": r.weights, "order": r.order, "offsets": r.offsets}
        if case["backward"]:
            out["dlogits"] = uz.moe_route_backward(s["dweights"], s["logits"], r)
        return out
    if case["op"] == "moe":
        r = uz.moe_route(s["logits"], case["k"])
        y = uz.moe(s["x"], r, s["up"], s["down"], act=case["act"], up_bias=s["up_bias"], down_bias=s["down_bias"],
                   residual=s["residual"])
        return {"y": y, "experts": r.experts, "weights": r.weights}
    token, logprob = uz.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"])
    return {"token": token, "logprob": logprob}


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"route": _run_route, "moe": _run_moe, "sample": _run_sample}[case["op"]](state, case)


def work(case):
    """Each input read once and each output written once.  Of the experts, the packed bytes of as many as have a token on
    average under an even router."""
    t = case["t"]
    wide = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "sample":
        return {"bytes": float(wide * t * case["v"] + 16 * t), "flops": 4.0 * t * case["v"]}
    e, k = case["e"], case["k"]
    if case["op"] == "route":
        size, flops = wide * t * e + 12.0 * t * k + 4.0 * e, 4.0 * t * e
        if case["backward"]:
            size, flops = size + 2 * wide * t * e + 4.0 * t * k, 2 * flops
        return {"bytes": size, "flops": flops}
    d, f = case["d"], case["f"]
    values = (3 if case["act"] == "swiglu" else 2) * d * f
    active = e * (1 - (1 - k / e) ** t)
    size = active * values * PACKED_BITS / 8 + 2.0 * t * d * (3 if case["residual"] else 2) + 4.0 * t * e + 8.0 * t * k
    if case["bias"]:
        size += active * 2.0 * (d + (2 * f if case["act"] == "swiglu" else f))
    return {"bytes": size, "flops": 2.0 * t * k * values}


# ---- from the definitions, in 64 bits ----

def _exact_route(z, k, scores, bias, renorm):
    """The experts one after another: the best of those left, the first of equal ones."""
    z = z.double()
    p = torch.softmax(z, dim=1) if scores == "softmax" else torch.sigmoid(z)
    left = z.clone() if bias is None else torch.sigmoid(z) + bias.double()
    picked = []
    column = torch.arange(z.shape[1], device=DEV)[None, :]
    for _ in range(k):
        top = left.amax(dim=1, keepdim=True)
        at = torch.where(left == top, column, z.shape[1]).amin(dim=1, keepdim=True)
        picked.append(at)
        left = left.scatter(1, at, float("-inf"))
    experts = torch.cat(picked, dim=1)
    return experts, p, (lambda p_: _weights(p_, experts, renorm))


def _weights(p, experts, renorm):
    w = torch.gather(p, 1, experts)
    return w / w.sum(dim=1)[:, None] if renorm else w


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "route":
        experts, p, weights = _exact_route(s["logits"], case["k"], case["scores"], s["bias"], case["renorm"])
        r = {"experts": experts.int(), "weights": weights(p)}
        flat = experts.flatten()
        # each pair's place: how many pairs go to lower experts, and how many earlier ones to its own
        hot = torch.nn.functional.one_hot(flat, case["e"])
        ends = hot.sum(dim=0).cumsum(dim=0)
        place = (ends - hot.sum(dim=0))[flat] + ((hot.cumsum(dim=0) - hot) * hot).sum(dim=1)
        r["order"] = torch.empty_like(flat).index_put_((place,), torch.arange(flat.numel(), device=DEV)).int()
        r["offsets"] = torch.cat([ends.new_zeros(1), ends]).int()
        if case["backward"]:
            # through the formulas by autograd, the choice held fixed
            z = s["logits"].double().requires_grad_(True)
            with torch.enable_grad():
                q = torch.softmax(z, dim=1) if case["scores"] == "softmax" else torch.sigmoid(z)
                r["dlogits"] = torch.autograd.grad(_weights(q, experts, case["renorm"]), z, s["dweights"].double())[0]
        return r
    if case["op"] == "moe":
        experts, p, weights = _exact_route(s["logits"], case["k"], "softmax", None, True)
        w = weights(p)
        x = s["x"].double()
        y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
        for i in range(case["e"]):
            token, slot = torch.nonzero(experts == i, as_tuple=True)
            if token.numel() == 0:
                continue
            z = torch.matmul(x[token], s["up"][i].double().T.contiguous())
            if case["bias"]:
                z += s["up_bias"][i].double()
            if case["act"] == "swiglu":
                gate, up = z[:, :case["f"]], z[:, case["f"]:]
                h = gate * torch.sigmoid(gate) * up
            elif case["act"] == "silu":
                h = z * torch.sigmoid(z)
            elif case["act"] == "gelu":
                h = z * torch.special.ndtr(z)
            else:
                h = torch.maximum(z, torch.zeros_like(z))
            o = torch.matmul(h, s["down"][i].double().T.contiguous())
            if case["bias"]:
                o += s["down_bias"][i].double()
            y.index_add_(0, token, o * w[token, slot][:, None])
        return {"y": y, "experts": experts.int(), "weights": w}
    # sample: the kept set by its border, the draw by the first running sum behind it; a few rows at a time
    temperature, top_k, top_p, min_p = [c.squeeze(1).tolist() for c in _parameters(s, case)]
    tokens, logprobs = [], []
    for i in range(case["t"]):
        z = s["logits"][i].double()
        heat = temperature[i] if temperature[i] > 0 else 1.0
        logp = torch.log_softmax(z / heat, dim=0)
        e = torch.exp((z - z.max()) / heat)
        rank = torch.argsort(-z, stable=True)
        count = int(top_k[i]) if 0 < top_k[i] < case["v"] else case["v"]
        if temperature[i] == 0:
            count = 1
        run = torch.cumsum(e[rank[:count]], dim=0)
        if top_p[i] < 1:
            count = min(count, 1 + int(torch.searchsorted(run, run[-1] * top_p[i])))
        count = max(1, min(count, int((e[rank[:count]] >= min_p[i]).sum())))
        kept = torch.sort(rank[:count]).values
        run = torch.cumsum(e[kept], dim=0)
        at = torch.searchsorted(run, run[-1] * s["u"][i].double(), right=True).clamp(max=count - 1)
        tokens.append(kept[at])
        logprobs.append(logp[kept[at]])
    return {"token": torch.stack(tokens), "logprob": torch.stack(logprobs)}
