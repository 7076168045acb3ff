"""Low-rank adapters beside a shared projection and the routers' balance loss, as measured cases.

A case is a dict of plain values.  ``prepare`` makes what a program holds before the call,
``run`` is one pass as a program makes it: in plain torch operations (``own`` false) or through
``addmm_implicit_im2col_gb300.binding`` (``own`` true).  ``exact`` gives the same results from the
operators' definitions in 64 bits, ``work`` the bytes and operations a pass cannot do without.

Adapters.  Row t of x [T, K] has an adapter l = which[t] of L (or none); a [L, r, K], b [L, N, r]:
    out[t] = base[t] + scale[l] * (x[t] a[l]^T) b[l]^T                (base[t] where it has none)
with g[t] = scale[l] * (grad[t] b[l]), the gradients
    grad_x[t] = base[t] + g[t] a[l],  grad_a[l] = sum_t g[t]^T x[t],
    grad_b[l] = sum_t grad[t]^T (scale[l] * x[t] a[l]^T).

Balance loss.  p = softmax(logits), or sigmoid(logits) divided by its sum over the E experts; a
sequence s holds n tokens offsets[s] .. offsets[s + 1], of which c[s, e] chosen slots went to e:
    loss[s] = E / (k n^2) * sum_e c[s, e] * sum_t p[t, e]             (0 where n = 0)
Its gradient takes the counts as constant.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one token of one request through a projection and its adapter (decoding)
        {"name": "adapters token", "op": "adapters", "T": 1, "L": 8, "r": 16, "K": 4096, "N": 4096, "dtype": "bf16", "mix": "each"},
        # a decoding batch, each request with its own adapter, some with none
        {"name": "adapters decode", "op": "adapters", "T": 64, "L": 64, "r": 16, "K": 4096, "N": 1024, "dtype": "bf16", "mix": "each"},
        # short prompts at odd sizes in fp32
        {"name": "adapters ragged", "op": "adapters", "T": 777, "L": 5, "r": 9, "K": 1100, "N": 1001, "dtype": "f32", "mix": "runs"},
        # prompts and decoding tokens of many requests in one batch
        {"name": "adapters mixed", "op": "adapters", "T": 2048, "L": 32, "r": 64, "K": 2048, "N": 4096, "dtype": "f16", "mix": "runs"},
        # a batch of long prompts
        {"name": "adapters prefill", "op": "adapters", "T": 8192, "L": 8, "r": 32, "K": 4096, "N": 4096, "dtype": "bf16", "mix": "runs"},
        # gradients of one adapter that the whole batch trains
        {"name": "adapters training", "op": "adapters backward", "T": 8192, "L": 1, "r": 16, "K": 4096, "N": 4096, "dtype": "bf16", "mix": "runs"},
        # gradients of several adapters trained at once, fp32, odd sizes
        {"name": "adapters training ragged", "op": "adapters backward", "T": 2047, "L": 4, "r": 8, "K": 1000, "N": 2048, "dtype": "f32", "mix": "runs"},
        # the loss and the counts of a small batch
        {"name": "balance small", "op": "balance", "T": 512, "S": 1, "E": 64, "k": 4, "score": "softmax", "dtype": "f32", "grad": "none"},
        # a training step: the loss, the counts and the logits' gradient of the loss
        {"name": "balance training", "op": "balance", "T": 8191, "S": 1, "E": 128, "k": 8, "score": "softmax", "dtype": "bf16", "grad": "loss"},
        # the same by sequences, with the gradient of the routing weights in the same pass
        {"name": "balance sequences", "op": "balance", "T": 16384, "S": 8, "E": 256, "k": 8, "score": "sigmoid", "dtype": "f32", "grad": "both"},
    ]


def _spread(rng, low, high):
    """A size spread over the logarithm of low .. high."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters", "adapters backward", "adapters backward", "balance", "balance"])
    if op == "balance":
        E = rng.choice([rng.randint(4, 32), 8 * rng.randint(4, 32)])
        T = _spread(rng, 16, 16384)
        return {"op": op, "T": T, "S": min(T, rng.choice([1, 1, rng.randint(2, 16), _spread(rng, 1, 256)])), "E": E,
                "k": rng.randint(1, min(8, E // 2)), "score": rng.choice(["softmax", "sigmoid"]), "dtype": rng.choice(["f32", "bf16"]),
                "grad": rng.choice(["none", "loss", "both"])}
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    T = _spread(rng, 1 if op == "adapters" else 16, 8192)
    r = rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 64)])
    K, N = (_spread(rng, 64, 4096) for _ in range(2))
    if op != "adapters" or dtype == "f32":  # no more work than the largest listed case
        r, K, N = min(r, 16), min(K, 2048) if dtype == "f32" else K, min(N, 2048) if dtype == "f32" else N
    elif T * r > 8192 * 32:
        r = 32
    if rng.random() < 0.5:
        K, N = K + -K % 8, N + -N % 8
    return {"op": op, "T": T, "L": _spread(rng, 1, 64), "r": r, "K": K, "N": N, "dtype": dtype, "mix": rng.choice(["each", "runs"])}


# ------------------------------------------------------------------ inputs
def _activations(g, rows, cols, dtype):
    """Normal values with channels of different size, a few of them large, as activations have."""
    size = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    size = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8 * size, size)
    return (torch.randn(rows, cols, generator=g, device="cuda") * size).to(DT[dtype])


def _adapter_inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    back = c["op"] != "adapters"
    T, L, r, K, N = c["T"], c["L"], c["r"], c["K"], c["N"]
    s = {"c": c, "x": _activations(g, T, K, c["dtype"])}
    if back:
        s["grad"] = _activations(g, T, N, c["dtype"])
    s["base"] = _activations(g, T, K if back else N, c["dtype"])
    s["a"] = (torch.randn(L, r, K, generator=g, device="cuda") / math.sqrt(K)).to(DT[c["dtype"]])
    s["b"] = (torch.randn(L, N, r, generator=g, device="cuda") / math.sqrt(r)).to(DT[c["dtype"]])
    s["scale"] = 0.25 + 1.75 * torch.rand(L, generator=g, device="cuda")
    if c["mix"] == "each":  # every row a request of its own, one in ten without an adapter
        which = torch.randint(0, L, (T,), generator=g, device="cuda")
        which = torch.where(torch.rand(T, generator=g, device="cuda") < (0.1 if T > 1 else 0.0), -1, which)
    else:  # requests of different lengths one after the other; in serving one in ten without an adapter
        n = min(T, 2 * L + 3)
        cuts = torch.randint(0, T, (n,), generator=g, device="cuda")
        of = torch.randint(0, L, (n + 1,), generator=g, device="cuda")
        none = torch.rand(n + 1, generator=g, device="cuda") < (0.0 if back else 0.1)
        run = (torch.arange(T, device="cuda")[:, None] >= cuts[None, :]).sum(1)
        which = torch.where(none, -1, of)[run]
    s["which"] = which.to(torch.int32)
    return s


def _balance_inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, S, E, k = c["T"], c["S"], c["E"], c["k"]
    popular = 0.5 * torch.randn(E, generator=g, device="cuda")
    logits = (1.5 * torch.randn(T, E, generator=g, device="cuda") + popular).to(DT[c["dtype"]])
    s = {"c": c, "logits": logits, "experts": logits.float().topk(k, -1).indices.to(torch.int32)}
    if S == 1:
        s["offsets"] = None
    else:  # sequences of different lengths, behind the last one a few rows of padding
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        ends = torch.tensor([0, T - T // 50], device="cuda")
        s["offsets"] = torch.cat([ends[:1], cuts.clamp(max=T - T // 50), ends[1:]]).to(torch.int32)
    # a loss's weight of a hundredth, times the loss scale of a training step in 16 bits
    s["grad_loss"] = (0.01 * 65536) * (0.5 + torch.rand(S, generator=g, device="cuda"))
    s["grad_weights"] = torch.randn(T, k, generator=g, device="cuda")
    return s


def prepare(case, seed):
    if case["op"] == "balance":
        return _balance_inputs(case, seed)
    s = _adapter_inputs(case, seed)
    # the rows in adapter order: made once a step, used by every projection of every layer
    if own:
        from addmm_implicit_im2col_gb300 import binding
        s["layout"] = binding.experts_layout(s["which"][:, None].contiguous(), case["L"])
    else:
        which = s["which"].long()
        rows = which.sort(stable=True).indices
        rows = rows[which[rows] >= 0]
        adapter = which[rows]
        counts = torch.bincount(adapter, minlength=case["L"])
        s["rows"], s["adapter"], s["most"] = rows, adapter, max(1, int(counts.max()))
        s["place"] = torch.arange(len(rows), device="cuda") - (counts.cumsum(0) - counts)[adapter]
    return s


# -------------------------------------------------------------- plain forms
def _by_adapter(s, x):
    """Rows of x in 32 bits, [L, most, columns], zeros where an adapter has fewer rows."""
    batch = torch.zeros(s["c"]["L"], s["most"], x.shape[1], device=x.device)
    batch[s["adapter"], s["place"]] = x[s["rows"]].float()
    return batch


def _added(s, batch):
    out = s["base"].float()
    out = out.index_add(0, s["rows"], batch[s["adapter"], s["place"]])
    return out.to(s["base"].dtype)


def _plain_adapters(s):
    x, a, b, scale = _by_adapter(s, s["x"]), s["a"].float(), s["b"].float(), s["scale"][:, None, None]
    h = scale * torch.bmm(x, a.transpose(1, 2))
    if s["c"]["op"] == "adapters":
        return {"out": _added(s, torch.bmm(h, b.transpose(1, 2)))}
    d = _by_adapter(s, s["grad"])
    g = scale * torch.bmm(d, b)
    dtype = s["x"].dtype
    return {"grad_x": _added(s, torch.bmm(g, a)), "grad_a": torch.bmm(g.transpose(1, 2), x).to(dtype),
            "grad_b": torch.bmm(d.transpose(1, 2), h).to(dtype)}


def _plain_balance(s):
    c, logits = s["c"], s["logits"].float()
    T, S, E, k = c["T"], c["S"], c["E"], c["k"]
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = p = e / e.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
        total = score.sum(-1, keepdim=True)
        p = score / total
    t = torch.arange(T, device=logits.device)
    if s["offsets"] is None:
        seq, n = torch.zeros_like(t), torch.full((S,), float(T), device=logits.device)
    else:
        seq = torch.searchsorted(s["offsets"][1:].long(), t, right=True)  # S: behind the last one
        n = (s["offsets"][1:] - s["offsets"][:-1]).float()
    sums = torch.zeros(S + 1, E, dtype=torch.float64, device=logits.device).index_add_(0, seq, p.double())[:S]
    slots = (seq[:, None] * E + s["experts"]).flatten()
    counts = torch.zeros((S + 1) * E, dtype=torch.int64, device=logits.device).scatter_add_(0, slots, torch.ones_like(slots))
    counts = counts.view(S + 1, E)[:S]
    per = torch.where(n > 0, E / (k * n * n), 0.0)
    got = {"loss": (per * (counts * sums).sum(-1)).float(), "counts": counts.int()}
    if c["grad"] != "none":
        coef = torch.zeros(S + 1, E, device=logits.device)
        coef[:S] = (s["grad_loss"] * per)[:, None] * counts
        coef = coef[seq]
        d = coef - (coef * p).sum(-1, keepdim=True)
        if c["score"] == "sigmoid":
            d = d / total
        if c["grad"] == "both":  # weights = the chosen scores divided by their sum
            experts = s["experts"].long()
            picked = score.gather(1, experts)
            chosen = picked.sum(-1, keepdim=True)
            w = (s["grad_weights"] - (s["grad_weights"] * picked / chosen).sum(-1, keepdim=True)) / chosen
            w = torch.zeros_like(score).scatter_(1, experts, w)
            d = d + (w - (w * score).sum(-1, keepdim=True) if c["score"] == "softmax" else w)
        got["grad_logits"] = (d * score if c["score"] == "softmax" else d * score * (1 - score)).to(s["logits"].dtype)
    return got


def run(state):
    s, c = state, state["c"]
    if not own:
        return _plain_balance(s) if c["op"] == "balance" else _plain_adapters(s)
    from addmm_implicit_im2col_gb300 import binding
    if c["op"] == "adapters":
        return {"out": binding.adapters_linear(s["x"], s["a"], s["b"], s["layout"], s["base"], scale=s["scale"])}
    if c["op"] == "adapters backward":
        grad_x, grad_a, grad_b = binding.adapters_linear_backward(s["grad"], s["x"], s["a"], s["b"], s["layout"], s["base"],
                                                                  scale=s["scale"])
        return {"grad_x": grad_x, "grad_a": grad_a, "grad_b": grad_b}
    loss, counts = binding.balance_loss(s["logits"], s["experts"], score=c["score"], offsets=s["offsets"])
    got = {"loss": loss, "counts": counts}
    if c["grad"] == "loss":
        got["grad_logits"] = binding.balance_loss_backward(s["grad_loss"], s["logits"], s["experts"], counts, score=c["score"],
                                                           offsets=s["offsets"])
    elif c["grad"] == "both":
        got["grad_logits"] = binding.balance_loss_backward(s["grad_loss"], s["logits"], s["experts"], counts, score=c["score"],
                                                           offsets=s["offsets"], grad_weights=s["grad_weights"])
    return got


# ------------------------------------------------------------------- work
def work(case):
    c, b = case, SIZE[case["dtype"]]
    T = c["T"]
    if c["op"] == "balance":
        E, k, S = c["E"], c["k"], c["S"]
        size = T * E * b + T * k * 4 + S * (E + 1) * 4
        if c["grad"] != "none":
            size += T * E * b
        if c["grad"] == "both":
            size += T * k * 4
        return {"bytes": size, "flops": 0}
    L, r, K, N = c["L"], c["r"], c["K"], c["N"]
    used = L * (1 - (1 - 1 / L) ** T) if c["mix"] == "each" else min(L, T)  # adapters that some row has
    if c["op"] == "adapters":
        return {"bytes": (T * (K + 2 * N) + used * r * (K + N)) * b + 8 * T, "flops": 2 * T * r * (K + N)}
    return {"bytes": (T * (3 * K + N) + 2 * used * r * (K + N)) * b + 8 * T, "flops": 2 * T * r * (3 * K + 2 * N)}


# ------------------------------------------------------------------ exact
def _exact_adapters(s):
    c = s["c"]
    x, a, b = s["x"].double(), s["a"].double(), s["b"].double()
    base = s["base"].double()
    if c["op"] == "adapters":
        out = base.clone()
    else:
        grad = s["grad"].double()
        got = {"grad_x": base.clone(), "grad_a": torch.zeros_like(a), "grad_b": torch.zeros_like(b)}
    for l in range(c["L"]):
        at = (s["which"] == l).nonzero().flatten()
        if len(at) == 0:
            continue
        xs, scale = x[at], s["scale"][l].double()
        h = scale * (xs @ a[l].T)
        if c["op"] == "adapters":
            out[at] += h @ b[l].T
            continue
        ds = grad[at]
        g = scale * (ds @ b[l])
        got["grad_x"][at] += g @ a[l]
        got["grad_a"][l] = g.T @ xs
        got["grad_b"][l] = ds.T @ h
    return {"out": out} if c["op"] == "adapters" else got


def _exact_balance(s):
    c = s["c"]
    T, S, E, k = c["T"], c["S"], c["E"], c["k"]
    x = s["logits"].double().requires_grad_(True)
    score = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
    p = score if c["score"] == "softmax" else score / score.sum(-1, keepdim=True)
    offsets = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    chosen = torch.zeros(T, E, dtype=torch.float64, device=x.device).scatter_(1, s["experts"].long(), 1.0)
    losses, counts = [], []
    for q in range(S):
        part = slice(offsets[q], offsets[q + 1])
        n = offsets[q + 1] - offsets[q]
        counts.append(chosen[part].sum(0))
        share = counts[-1] / max(1, k * n)
        losses.append(E * (share * p[part].sum(0) / max(1, n)).sum())
    loss = torch.stack(losses)
    got = {"loss": loss.detach(), "counts": torch.stack(counts).int()}
    if c["grad"] != "none":
        total = (loss * s["grad_loss"].double()).sum()
        if c["grad"] == "both":
            picked = score.gather(1, s["experts"].long())
            total = total + (picked / picked.sum(-1, keepdim=True) * s["grad_weights"].double()).sum()
        got["grad_logits"] = torch.autograd.grad(total, x)[0]
    return got


def exact(case, seed):
    if case["op"] == "balance":
        return _exact_balance(_balance_inputs(case, seed))
    return _exact_adapters(_adapter_inputs(case, seed))
