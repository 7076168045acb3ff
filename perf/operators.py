"""The microscaled 4-bit and expert-routing operators, as cases that can be timed and checked.

A case is a dict of plain values.  ``prepare`` makes what a program holds before the call,
``run`` is one pass as a program makes it: in plain torch operations (``own`` false) or through
``addmm_implicit_im2col_gb300.binding`` (``own`` true).  ``exact`` gives the same results from the
operators' definitions in 64 bits, ``work`` the bytes and operations a pass cannot do without.

MXFP4: 32 consecutive values of a row share one scale 2^e, e = floor(log2(largest magnitude)) - 2
(clamped to -127 .. 127), and each is rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 times it
(ties to the even code, 6 at most).  A product of two such operands is taken along the rows' axis.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 32


def listed():
    return [
        # quantisation: the activations of one token before a decoding step's product
        {"name": "quantise token", "op": "quantise", "rows": 1, "cols": 4096, "both": False, "dtype": "bf16"},
        # quantisation: a training step's activations, as the operand of the forward product and,
        # transposed, of the weight's gradient
        {"name": "quantise both ways", "op": "quantise", "rows": 8192, "cols": 4096, "both": True, "dtype": "f32"},
        # product: one token through a square projection (decoding)
        {"name": "linear decode", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16", "relu": False, "bias": False},
        # product: a short prompt through a layer of odd sizes, with bias and ReLU
        {"name": "linear ragged", "op": "linear", "M": 77, "N": 1001, "K": 1100, "dtype": "f32", "relu": True, "bias": True},
        # product: a batch of long prompts, the benchmark's own 8192 x 4096 x 4096
        {"name": "linear prefill", "op": "linear", "M": 8192, "N": 4096, "K": 4096, "dtype": "bf16", "relu": False, "bias": True},
        # product and both gradients of a training step, everything quantised within it
        {"name": "linear training", "op": "train", "M": 8192, "N": 4096, "K": 1024, "dtype": "f32"},
        # routing of a few decoding tokens, softmax scores
        {"name": "route decode", "op": "route", "T": 4, "E": 64, "k": 4, "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renormalize": True, "dtype": "f32", "grad": False},
        # routing of a batch of prompts: sigmoid scores, balance bias, groups; and the rows in expert order
        {"name": "route prefill", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "renormalize": True, "dtype": "f32", "grad": False},
        # routing in a training step, with the gradient of the router's logits
        {"name": "route training", "op": "route", "T": 8191, "E": 128, "k": 8, "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renormalize": True, "dtype": "bf16", "grad": True},
        # experts' product for a few decoding tokens, and the sum over each token's experts
        {"name": "experts decode", "op": "experts", "T": 8, "E": 64, "k": 4, "N": 2048, "K": 1024, "dtype": "bf16", "sum": True, "grad": False},
        # experts' product for a batch of prompts: each token's row goes to its experts
        {"name": "experts prefill", "op": "experts", "T": 4096, "E": 64, "k": 8, "N": 1024, "K": 2048, "dtype": "bf16", "sum": False, "grad": False},
        # the second product of the experts' block, the weighted sum, and the sum's gradients
        {"name": "experts sum training", "op": "experts", "T": 2048, "E": 32, "k": 4, "N": 2048, "K": 1000, "dtype": "f32", "sum": True, "grad": True},
    ]


def _spread(rng, low, high):
    """A size spread over the logarithm of low .. high."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantise", "linear", "linear", "train", "route", "route", "experts", "experts"])
    dtype = rng.choice(["f32", "bf16", "f16"] if op in ("quantise", "linear") else ["f32", "bf16"])
    if op == "quantise":
        rows, cols = _spread(rng, 1, 8192), _spread(rng, 33, 4096)
        return {"op": op, "rows": rows, "cols": cols, "both": rng.random() < 0.5, "dtype": dtype}
    if op == "linear":
        return {"op": op, "M": _spread(rng, 1, 8192), "N": _spread(rng, 64, 4096), "K": _spread(rng, 64, 4096),
                "dtype": dtype, "relu": rng.random() < 0.3, "bias": rng.random() < 0.5}
    if op == "train":
        return {"op": op, "M": _spread(rng, 16, 8192), "N": _spread(rng, 64, 4096), "K": _spread(rng, 64, 1024), "dtype": dtype}
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(8, 256 // groups)
        k = rng.randint(1, 8)
        return {"op": op, "T": _spread(rng, 1, 16384), "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": max(1, groups // 2), "renormalize": k > 1,
                "dtype": dtype, "grad": rng.random() < 0.5}
    return {"op": op, "T": _spread(rng, 1, 4096), "E": rng.randint(8, 64), "k": rng.randint(1, 8), "N": _spread(rng, 64, 1024),
            "K": _spread(rng, 64, 2048), "dtype": dtype, "sum": rng.random() < 0.5, "grad": False}


# ------------------------------------------------------------------ inputs
def _activations(g, rows, cols, dtype):
    """Normal values with channels of different size, a few of them large, as activations have."""
    size = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    size = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8 * size, size)
    return (torch.randn(rows, cols, generator=g, device="cuda") * size).to(DT[dtype])


def _weight(g, *shape, dtype="f32"):
    return (torch.randn(*shape, generator=g, device="cuda") / math.sqrt(shape[-1])).to(DT[dtype])


def _near_ties(logits, bias, c):
    """Tokens whose choice is decided by less than 1e-6, which rounding of the scores could turn."""
    x = logits.double()
    s = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
    s = s if bias is None else s + bias.double()
    bad = torch.zeros(len(x), dtype=torch.bool, device=x.device)
    if c["groups"] > 1:
        best = s.view(len(x), c["groups"], -1).topk(2, -1).values.sum(-1).sort(dim=-1, descending=True)
        bad |= (best.values[:, c["top_groups"] - 1] - best.values[:, c["top_groups"]]) < 1e-6
        kept = torch.zeros_like(best.values, dtype=torch.bool).scatter_(1, best.indices[:, : c["top_groups"]], True)
        s = torch.where(kept.repeat_interleave(c["E"] // c["groups"], 1), s, float("-inf"))
    top = s.topk(min(c["k"] + 1, c["E"]), -1).values
    return bad | ((top[:, :-1] - top[:, 1:]) < 1e-6).any(-1)


def _experts_of(g, T, E, k):
    """k different experts for each token, some of them asked for more often, and their weights."""
    logits = 1.5 * torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    top = logits.topk(k, -1)
    return top.indices.to(torch.int32), torch.softmax(top.values, -1)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "quantise":
        return {"c": c, "x": _activations(g, c["rows"], c["cols"], c["dtype"])}
    if c["op"] == "train":
        return {"c": c, "x": _activations(g, c["M"], c["K"], c["dtype"]), "w": _weight(g, c["N"], c["K"], dtype=c["dtype"]),
                "dy": _activations(g, c["M"], c["N"], c["dtype"])}
    if c["op"] == "route":
        popular = 0.5 * torch.randn(c["E"], generator=g, device="cuda")
        bias = 0.1 * torch.randn(c["E"], generator=g, device="cuda") if c["bias"] else None
        logits = (1.5 * torch.randn(c["T"], c["E"], generator=g, device="cuda") + popular).to(DT[c["dtype"]])
        for _ in range(12):  # other values for tokens that rounding would decide
            bad = _near_ties(logits, bias, c)
            more = (1.5 * torch.randn(c["T"], c["E"], generator=g, device="cuda") + popular).to(DT[c["dtype"]])
            logits = torch.where(bad[:, None], more, logits)
        return {"c": c, "logits": logits, "bias": bias, "grad": torch.randn(c["T"], c["k"], generator=g, device="cuda")}
    if c["op"] == "linear":
        s = {"c": c, "x": _activations(g, c["M"], c["K"], c["dtype"])}
        w = _weight(g, c["N"], c["K"])
        s["bias"] = torch.randn(c["N"], generator=g, device="cuda") if c["bias"] else None
    else:
        rows = c["T"] * c["k"] if c["sum"] else c["T"]
        s = {"c": c, "x": _activations(g, rows, c["K"], c["dtype"]), "dout": _activations(g, c["T"], c["N"], c["dtype"])}
        s["experts"], s["weights"] = _experts_of(g, c["T"], c["E"], c["k"])
        w = _weight(g, c["E"], c["N"], c["K"])
    if own:  # the weight is quantised once, when a program loads it
        from addmm_implicit_im2col_gb300 import binding
        s["w"] = binding.quantize_mxfp4(w)
    else:
        s["w"] = _pack(w)
    return s


# -------------------------------------------------------------- plain forms
def _blocks(x):
    """Rows of x in 32 bits, cut into blocks of 32 (zeros after the last value)."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % BLOCK))
    return x.view(*x.shape[:-1], -1, BLOCK)


def _codes(x):
    """MXFP4 of the rows of x: (code magnitudes 0..7, negative?, scale's exponent + 127) of each block."""
    b = _blocks(x)
    exponent = (b.abs().amax(-1).view(torch.int32) >> 23) - 2
    exponent = exponent.clamp(min=0)
    a = b.abs() * _exp2(127 - exponent)[..., None]
    # halfway values go to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code, torch.signbit(b), exponent


def _exp2(n):
    """2^n for whole n in -127 .. 127, exactly."""
    return torch.where(n >= -126, (n.clamp(min=-126) + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _values(code, negative, exponent):
    """The values that MXFP4 codes stand for, rows without their blocks."""
    c = code.float()  # 0 .5 1 1.5, 2 3, 4 6
    level = torch.where(c < 4, 0.5 * c, torch.where(c < 6, c - 2, 2 * c - 8))
    v = torch.where(negative, -level, level) * _exp2(exponent - 127)[..., None]
    return v.flatten(-2)


def _pack(x):
    """MXFP4 of x as a program stores it: two codes to a byte, a byte for each scale."""
    code, negative, exponent = _codes(x)
    code = (code | (negative.to(torch.uint8) << 3)).flatten(-2)
    return {"codes": code[..., 0::2] | (code[..., 1::2] << 4), "scales": exponent.to(torch.uint8), "cols": x.shape[-1]}


def _unpack(p):
    code = torch.stack([p["codes"] & 15, p["codes"] >> 4], -1).flatten(-2)
    code = code.view(*code.shape[:-1], -1, BLOCK)
    return _values(code & 7, code > 7, p["scales"].int())[..., : p["cols"]]


def _rounded(x):
    """x as MXFP4 holds it, in 32 bits."""
    return _values(*_codes(x))[..., : x.shape[-1]]


def _plain_route(s):
    c, logits, bias = s["c"], s["logits"].float(), s["bias"]
    T, E, k = c["T"], c["E"], c["k"]
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    choice = score if bias is None else score + bias
    if c["groups"] > 1:
        best = choice.view(T, c["groups"], -1).topk(2, -1).values.sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, : c["top_groups"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(mask.repeat_interleave(E // c["groups"], 1), choice, float("-inf"))
    experts = choice.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    picked = score.gather(1, experts)
    total = picked.sum(-1, keepdim=True)
    weights = picked / total if c["renormalize"] else picked
    if c["grad"]:
        d = (s["grad"] - (s["grad"] * weights).sum(-1, keepdim=True)) / total if c["renormalize"] else s["grad"]
        d = torch.zeros_like(score).scatter_(1, experts, d)
        if c["score"] == "softmax":
            dlogits = score * (d - (d * score).sum(-1, keepdim=True))
        else:
            dlogits = d * score * (1 - score)
        return {"weights": weights, "experts": experts.int(), "dlogits": dlogits.to(s["logits"].dtype)}
    offsets, order = _plain_layout(experts, E)
    return {"weights": weights, "experts": experts.int(), "offsets": offsets, "order": order}


def _plain_layout(experts, E):
    """Where each expert's slots begin, and the slots (token * k + place) in expert order."""
    flat = experts.flatten()
    counts = torch.zeros(E, dtype=torch.int64, device=flat.device).scatter_add_(0, flat.long(), torch.ones_like(flat, dtype=torch.int64))
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    return offsets.int(), flat.sort(dim=0, stable=True).indices.int()


def _plain_experts(s):
    c = s["c"]
    T, E, k = c["T"], c["E"], c["k"]
    x, w = _rounded(s["x"]), _unpack(s["w"])
    offsets, order = _plain_layout(s["experts"], E)
    order = order.long()
    expert = s["experts"].flatten()[order].long()
    place = torch.arange(T * k, device=x.device) - offsets[expert]
    most = int((offsets[1:] - offsets[:-1]).max())
    batch = torch.zeros(E, most, c["K"], device=x.device)
    batch[expert, place] = x[order if c["sum"] else order // k]
    y = torch.empty(T * k, c["N"], device=x.device)
    y[order] = torch.bmm(batch, w.transpose(1, 2))[expert, place]
    if not c["sum"]:
        return {"y": y.to(s["x"].dtype)}
    y = y.to(s["x"].dtype)  # the product's own result type
    yk = y.float().view(T, k, -1)
    got = {"out": (s["weights"][..., None] * yk).sum(1).to(y.dtype)}
    if c["grad"]:
        d = s["dout"].float()
        got["dy"] = (s["weights"][..., None] * d[:, None, :]).to(y.dtype).view(T * k, -1)
        got["dweights"] = (d[:, None, :] * yk).sum(-1)
    return got


def _plain(s):
    c = s["c"]
    if c["op"] == "quantise":
        x = s["x"]
        got = {"rows": _rounded(x).to(x.dtype)}
        if c["both"]:
            got["columns"] = _rounded(x.t().contiguous()).to(x.dtype)
        return got
    if c["op"] == "linear":
        y = _rounded(s["x"]) @ _unpack(s["w"]).t()
        y = y if s["bias"] is None else y + s["bias"]
        y = torch.where(y > 0, y, 0.0) if c["relu"] else y
        return {"y": y.to(s["x"].dtype)}
    if c["op"] == "train":
        x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
        y = _rounded(x) @ _rounded(w).t()
        dx = _rounded(dy) @ _rounded(w.t().contiguous()).t()
        dw = _rounded(dy.t().contiguous()) @ _rounded(x.t().contiguous()).t()
        return {"y": y.to(s["x"].dtype), "dx": dx.to(s["x"].dtype), "dw": dw.to(s["x"].dtype)}
    return _plain_route(s) if c["op"] == "route" else _plain_experts(s)


def run(state):
    if not own:
        return _plain(state)
    from addmm_implicit_im2col_gb300 import binding
    s, c = state, state["c"]
    if c["op"] == "quantise":
        x = s["x"]
        got = {"rows": binding.dequantize_mxfp4(binding.quantize_mxfp4(x), dtype=x.dtype)}
        if c["both"]:
            got["columns"] = binding.dequantize_mxfp4(binding.quantize_mxfp4(x, transpose=True), dtype=x.dtype)
        return got
    if c["op"] == "linear":
        return {"y": binding.linear_mxfp4(s["x"], s["w"], s["bias"], relu=c["relu"])}
    if c["op"] == "train":
        y = binding.linear_mxfp4(s["x"], s["w"])
        dx, dw = binding.linear_mxfp4_backward(s["dy"], s["x"], s["w"])
        return {"y": y, "dx": dx, "dw": dw}
    if c["op"] == "route":
        weights, experts = binding.route_experts(s["logits"], c["k"], s["bias"], score=c["score"], groups=c["groups"],
                                                 top_groups=c["top_groups"], renormalize=c["renormalize"])
        got = {"weights": weights, "experts": experts}
        if c["grad"]:
            got["dlogits"] = binding.route_experts_backward(s["grad"], s["logits"], experts, score=c["score"],
                                                               renormalize=c["renormalize"])
        else:
            layout = binding.experts_layout(experts, c["E"])
            got["offsets"], got["order"] = layout.offsets, layout.order
        return got
    layout = binding.experts_layout(s["experts"], c["E"])
    y = binding.experts_linear_mxfp4(s["x"], s["w"], layout)
    if not c["sum"]:
        return {"y": y}
    got = {"out": binding.experts_combine(y, s["weights"])}
    if c["grad"]:
        got["dy"], got["dweights"] = binding.experts_combine_backward(s["dout"], y, s["weights"])
    return got


# ------------------------------------------------------------------- work
def _mx_bytes(rows, cols):
    return rows * -(-cols // BLOCK) * 17


def work(case):
    c, b = case, SIZE[case["dtype"]]
    if c["op"] == "quantise":
        n = c["rows"] * c["cols"]
        return {"bytes": n * b * (3 if c["both"] else 2), "flops": 0}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M * K + M * N) * b + _mx_bytes(N, K) + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    if c["op"] == "train":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * (M * K + N * K + M * N) * b, "flops": 6 * M * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "route":
        # weights and experts, and the order or the gradient of the weights: 12 bytes a slot
        return {"bytes": T * E * b * (2 if c["grad"] else 1) + 12 * T * k, "flops": 0}
    N, K = c["N"], c["K"]
    used = E * (1 - (1 - k / E) ** T)  # experts that some token asks for
    size = T * K * b * (k if c["sum"] else 1) + used * _mx_bytes(N, K) + T * k * 4
    size += T * N * b if c["sum"] else T * k * N * b
    if c["sum"]:
        size += T * k * 4
    if c["grad"]:
        size += T * N * b + T * k * N * b + T * k * 4
    return {"bytes": size, "flops": 2 * T * k * N * K}


# ------------------------------------------------------------------ exact
def _mx64(x):
    """x as MXFP4 holds it, from the definition in 64 bits: round to a multiple of the step at the
    value's own power of two (half a unit below 1), 6 at most."""
    x = x.double()
    cols = x.shape[-1]
    y = torch.zeros(*x.shape[:-1], -(-cols // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    y[..., :cols] = x
    y = y.reshape(*x.shape[:-1], -1, BLOCK)
    top = y.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 1 - 2).clamp(-127, 127)
    e = torch.where(top > 0, e, -127)
    v = torch.ldexp(y, -e)
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v).exponent - 1).clamp(min=0) - 1)
    v = (torch.round(v / step) * step).clamp(-6, 6)
    return torch.ldexp(v, e).reshape(*x.shape[:-1], -1)[..., :cols]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
        g = torch.Generator(device="cuda")
    finally:
        own = was
    c = case
    if c["op"] == "quantise":
        got = {"rows": _mx64(s["x"])}
        if c["both"]:
            got["columns"] = _mx64(s["x"].t())
        return got
    if c["op"] == "train":
        x, w, dy = s["x"], s["w"], s["dy"]
        return {"y": _mx64(x) @ _mx64(w).T, "dx": _mx64(dy) @ _mx64(w.t()).T, "dw": _mx64(dy.t()) @ _mx64(x.t()).T}
    if c["op"] == "route":
        x = s["logits"].double()
        p = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
        key = p.clone() if s["bias"] is None else p + s["bias"].double()
        if c["groups"] > 1:
            per = c["E"] // c["groups"]
            two = key.reshape(-1, c["groups"], per).sort(-1).values[..., -2:].sum(-1)
            limit = two.sort(-1).values[:, -c["top_groups"]]
            key[(two < limit[:, None]).repeat_interleave(per, 1)] = -math.inf
        experts = key.topk(c["k"], -1).indices
        x.requires_grad_(True)
        p = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
        weights = p.gather(1, experts)
        if c["renormalize"]:
            weights = weights / weights.sum(-1, keepdim=True)
        got = {"weights": weights.detach(), "experts": experts.int()}
        if c["grad"]:
            got["dlogits"] = torch.autograd.grad(weights, x, s["grad"].double())[0]
        else:
            flat = experts.flatten()
            got["offsets"] = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=c["E"]).cumsum(0)]).int()
            got["order"] = torch.argsort(flat, stable=True).int()
        return got
    # the weight's values, made again from the seed as prepare() makes them
    g.manual_seed(seed)
    if c["op"] == "linear":
        _activations(g, c["M"], c["K"], c["dtype"])
        y = _mx64(s["x"]) @ _mx64(_weight(g, c["N"], c["K"])).T
        y = y if s["bias"] is None else y + s["bias"].double()
        return {"y": y.clamp(min=0) if c["relu"] else y}
    T, k = c["T"], c["k"]
    _activations(g, len(s["x"]), c["K"], c["dtype"])
    _activations(g, T, c["N"], c["dtype"])
    _experts_of(g, T, c["E"], k)
    w = _weight(g, c["E"], c["N"], c["K"])
    x, flat = _mx64(s["x"]), s["experts"].flatten()
    y = torch.zeros(T * k, c["N"], dtype=torch.float64, device=x.device)
    for e in range(c["E"]):
        at = (flat == e).nonzero().flatten()
        if len(at):
            y[at] = x[at if c["sum"] else at // k] @ _mx64(w[e]).T
    if not c["sum"]:
        return {"y": y}
    y = y.view(T, k, -1)
    p, d = s["weights"].double(), s["dout"].double()
    got = {"out": (p[..., None] * y).sum(1)}
    if c["grad"]:
        got["dy"] = (p[..., None] * d[:, None, :]).reshape(T * k, -1)
        got["dweights"] = (d[:, None, :] * y).sum(-1)
    return got
