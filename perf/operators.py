"""Operators at the end of a training step whose rank buffers lie in one GPU's HBM, as cases that can be timed.

Four operators, each in a plain form of elementary torch operations and as the library's own calls:

- ``norm_fwd``: the sum of N rank buffers and a residual, and its layer norm (``mrr_layernorm_fwd``);
- ``norm_bwd``: that norm's gradient, with the reduction of the weight's and the bias's (``mrr_layernorm_bwd``);
- ``xent_fwd``: cross entropy of a linear layer whose vocabulary rows lie in N rank shards (``mrr_linear_xent_fwd``);
- ``xent_bwd``: its gradient for the hidden states and for every shard (``mrr_linear_xent_bwd``).

``own`` chooses: False computes the plain forms, True calls the library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100  # the target of a token that has no loss
EPS = 1e-5


def _norm(op, rows, cols, ranks, dtype, wdtype, residual, name=None):
    c = {"op": op, "rows": rows, "cols": cols, "ranks": ranks, "dtype": dtype, "wdtype": wdtype, "residual": residual}
    return dict(c, name=name) if name else c


def _xent(op, tokens, vocab, cols, ranks, dtype, name=None):
    c = {"op": op, "tokens": tokens, "vocab": vocab, "cols": cols, "ranks": ranks, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of a model sharded over 8 ranks: only the call's latency counts
        _norm("norm_fwd", 1, 4096, 8, "bf16", "bf16", True, "norm_fwd 1 token 8 ranks"),
        # a training batch after the row-parallel product of 4 ranks, norm weights kept in 32 bits
        _norm("norm_fwd", 4096, 8192, 4, "bf16", "f32", True, "norm_fwd batch 4 ranks"),
        # a norm with nothing to sum, odd rows and columns: no vector of a row is aligned
        _norm("norm_fwd", 2047, 1023, 1, "f16", "f16", False, "norm_fwd odd f16"),
        # the same training batch size backwards, with the gradient that the residual path brings
        _norm("norm_bwd", 16384, 4096, 1, "bf16", "f32", True, "norm_bwd batch"),
        # a small 32-bit model's batch
        _norm("norm_bwd", 513, 1600, 1, "f32", "f32", False, "norm_bwd small f32"),
        # few long rows: the reduction over rows has next to nothing to reduce
        _norm("norm_bwd", 8, 16384, 1, "bf16", "bf16", True, "norm_bwd long rows"),
        # the score of a single token against a vocabulary in 8 shards: the weights are read once
        _xent("xent_fwd", 1, 32000, 4096, 8, "bf16", "xent_fwd 1 token"),
        # a training batch over a large vocabulary in 8 shards
        _xent("xent_fwd", 4096, 128256, 4096, 8, "bf16", "xent_fwd batch"),
        # a vocabulary that no shard count or tile divides, a ragged batch
        _xent("xent_fwd", 700, 50257, 1600, 4, "f16", "xent_fwd ragged f16"),
        # the large batch backwards: the logits are computed again, then both gradients
        _xent("xent_bwd", 4096, 128256, 4096, 8, "bf16", "xent_bwd batch"),
        # odd everything: no row of the hidden states or of the weights is aligned
        _xent("xent_bwd", 1001, 32003, 1023, 2, "f16", "xent_bwd odd f16"),
        # a small 32-bit model
        _xent("xent_bwd", 130, 3003, 520, 3, "f32", "xent_bwd small f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _to(rng, n, to):
    """n as it is drawn, or next to it a multiple of `to`, as most models have it."""
    return n if rng.random() < 0.4 else max(to, (n + to // 2) // to * to)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "xent_fwd", "xent_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("norm"):
        cols = _to(rng, _log(rng, 64, 16384), 64)
        rows = min(_log(rng, 1, 16384), 16384 * 4096 // cols)
        ranks = rng.choice([1, 2, 3, 4, 8]) if op == "norm_fwd" else 1
        return _norm(op, rows, cols, ranks, dtype, rng.choice(["f32", dtype]), rng.random() < 0.6)
    cols = _to(rng, _log(rng, 64, 4096), 64)
    vocab = _to(rng, _log(rng, 500, 128256), 64)
    most = 4096 * 4096 * 128256 // (16 if dtype == "f32" else 1)  # 32-bit products run at a sixteenth of the rate
    tokens = max(1, min(_log(rng, 1, 4096), most // (cols * vocab)))
    return _xent(op, tokens, vocab, cols, rng.choice([1, 2, 3, 4, 8]), dtype)


def _shards(vocab, ranks):
    """Rows of each shard: as even as they get, the first ones larger."""
    return [vocab // ranks + (1 if r < vocab % ranks else 0) for r in range(ranks)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, cols, ranks = case["rows"], case["cols"], case["ranks"]
        wdt = TYPES[case["wdtype"]]
        # a few channels far larger than the others and off zero, as in the residual stream of a trained model
        channel = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 12.0, 1.0)
        offset = 0.3 * normal(cols)
        s["weight"] = (1 + 0.1 * normal(cols)).to(wdt)
        s["bias"] = (0.1 * normal(cols)).to(wdt)
        s["mean"], s["rstd"] = empty(rows, dtype=torch.float32), empty(rows, dtype=torch.float32)
        if case["op"] == "norm_fwd":
            s["inputs"] = [((normal(rows, cols) * channel + offset) / ranks ** 0.5).to(dt) for _ in range(ranks)]
            s["residual"] = (2 * normal(rows, cols) * channel).to(dt) if case["residual"] else None
            s["sum"] = empty(rows, cols) if ranks > 1 or case["residual"] else None
            s["out"] = empty(rows, cols)
        else:
            s["sum"] = (2 * normal(rows, cols) * channel + offset).to(dt)
            x = s["sum"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
            s["dout"] = (0.1 * normal(rows, cols)).to(dt)
            s["dresidual"] = (0.1 * normal(rows, cols)).to(dt) if case["residual"] else None
            s["dsum"], s["dweight"], s["dbias"] = empty(rows, cols), empty(cols, dtype=wdt), empty(cols, dtype=wdt)
        return s
    tokens, vocab, cols = case["tokens"], case["vocab"], case["cols"]
    s["rows"] = _shards(vocab, case["ranks"])
    s["weights"] = [(normal(n, cols) * (1.2 / cols ** 0.5)).to(dt) for n in s["rows"]]
    s["targets"] = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    # half of the tokens are ones that the model is sure of: their hidden state leans to the target's row
    lean = torch.where(torch.rand(tokens, generator=g, device="cuda") < 0.5, 6.0, 0.0)
    # (rows of all shards without a joint copy of them)
    row = torch.zeros(tokens, cols, device="cuda")
    first = 0
    for w in s["weights"]:
        mine = (s["targets"] >= first) & (s["targets"] < first + w.shape[0])
        at = (s["targets"] - first).clamp(0, max(0, w.shape[0] - 1))
        row += torch.where(mine[:, None], w[at].float(), 0.0)
        first += w.shape[0]
    s["hidden"] = (normal(tokens, cols) + lean[:, None] * row).to(dt)
    del row
    if tokens > 1:
        s["targets"][torch.rand(tokens, generator=g, device="cuda") < 0.1] = IGNORE
    s["loss"], s["lse"] = empty(tokens, dtype=torch.float32), empty(tokens, dtype=torch.float32)
    if case["op"] == "xent_bwd":
        s["lse"] = torch.logsumexp(torch.cat([s["hidden"].float() @ w.float().T for w in s["weights"]], 1), 1)
        scale = 1024.0 if case["dtype"] == "f16" else 1.0  # 16-bit floats are trained with a scaled loss
        s["dloss"] = (0.5 + torch.rand(tokens, generator=g, device="cuda")) * (scale / tokens)
        s["dhidden"] = empty(tokens, cols)
        s["dweights"] = [empty(n, cols) for n in s["rows"]]
    return s


def _plain_norm_fwd(s):
    dt = s["out"].dtype
    x = torch.stack(s["inputs"]).float().sum(0)
    if s["residual"] is not None:
        x = x + s["residual"].float()
    x = x.to(dt)
    h = x.float()
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(1) + EPS)
    out = {"out": (d * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(dt), "mean": mean, "rstd": rstd}
    if s["sum"] is not None:
        out["sum"] = x
    return out


def _plain_norm_bwd(s):
    dt, wdt = s["sum"].dtype, s["weight"].dtype
    dy = s["dout"].float()
    xhat = (s["sum"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dsum": dx.to(dt), "dweight": (dy * xhat).sum(0).to(wdt), "dbias": dy.sum(0).to(wdt)}


def _plain_xent_fwd(s):
    z = s["hidden"].float() @ torch.cat(s["weights"]).float().T
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    valid = s["targets"] != IGNORE
    zt = z.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(valid, lse - zt, 0.0), "lse": lse}


def _plain_xent_bwd(s):
    dt = s["hidden"].dtype
    h, w = s["hidden"].float(), torch.cat(s["weights"]).float()
    valid = s["targets"] != IGNORE
    p = torch.exp(h @ w.T - s["lse"][:, None])
    p.scatter_add_(1, s["targets"].clamp(min=0)[:, None], torch.full_like(s["lse"], -1.0)[:, None])
    p *= torch.where(valid, s["dloss"], 0.0)[:, None]
    return {"dhidden": (p @ w).to(dt), "dweights": list((p.T @ h).to(dt).split(s["rows"]))}


def _workspace(s, nbytes):
    """The workspace that a training program keeps from one step to the next."""
    if s.get("workspace") is None:
        s["workspace"] = torch.empty(max(256, nbytes), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import allreduce_reduction_nranks_amd as mrr
    c = s["case"]
    op, dtype = c["op"], c["dtype"]
    if op == "norm_fwd":
        mrr.check(mrr.mrr_layernorm_fwd(s["inputs"], c["ranks"], s["residual"], s["weight"], s["bias"], s["sum"], s["out"],
                                        s["mean"], s["rstd"], c["rows"], c["cols"], c["cols"], c["cols"], EPS, dtype,
                                        c["wdtype"]), op)
        return {k: s[k] for k in ("out", "mean", "rstd", "sum") if s[k] is not None}
    if op == "norm_bwd":
        n = mrr.mrr_layernorm_bwd_workspace_bytes(c["rows"], c["cols"])
        mrr.check(mrr.mrr_layernorm_bwd(s["dout"], s["sum"], s["weight"], s["mean"], s["rstd"], s["dresidual"], s["dsum"],
                                        s["dweight"], s["dbias"], c["rows"], c["cols"], c["cols"], c["cols"], dtype,
                                        c["wdtype"], _workspace(s, n), n), op)
        return {k: s[k] for k in ("dsum", "dweight", "dbias")}
    tokens, cols, ranks = c["tokens"], c["cols"], c["ranks"]
    n = mrr.mrr_linear_xent_workspace_bytes(tokens, cols, s["rows"], ranks, dtype, op == "xent_bwd")
    if op == "xent_fwd":
        mrr.check(mrr.mrr_linear_xent_fwd(s["hidden"], s["weights"], s["rows"], ranks, s["targets"], IGNORE, s["loss"],
                                          s["lse"], tokens, cols, cols, cols, dtype, _workspace(s, n), n), op)
        return {"loss": s["loss"], "lse": s["lse"]}
    mrr.check(mrr.mrr_linear_xent_bwd(s["hidden"], s["weights"], s["rows"], ranks, s["targets"], IGNORE, s["lse"],
                                      s["dloss"], 1, s["dhidden"], s["dweights"], tokens, cols, cols, cols, dtype,
                                      _workspace(s, n), n), op)
    return {"dhidden": s["dhidden"], "dweights": s["dweights"]}


def run(state):
    if own:
        return _own(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "xent_fwd": _plain_xent_fwd,
            "xent_bwd": _plain_xent_bwd}[state["case"]["op"]](state)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        n, cols = case["rows"] * case["cols"], case["cols"]
        wsize = 4 if case["wdtype"] == "f32" else 2
        res = 1 if case["residual"] else 0
        if case["op"] == "norm_fwd":
            tensors = case["ranks"] + res + 1 + (1 if case["ranks"] > 1 or res else 0)
            return {"bytes": n * size * tensors + 2 * cols * wsize + 8 * case["rows"], "flops": n * (case["ranks"] + res + 8)}
        return {"bytes": n * size * (3 + res) + 3 * cols * wsize + 8 * case["rows"], "flops": n * 14}
    tokens, vocab, cols = case["tokens"], case["vocab"], case["cols"]
    once = (tokens + vocab) * cols * size
    if case["op"] == "xent_fwd":
        return {"bytes": once + 16 * tokens, "flops": 2 * tokens * vocab * cols + 4 * tokens * vocab}
    return {"bytes": 2 * once + 16 * tokens, "flops": 6 * tokens * vocab * cols + 4 * tokens * vocab}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_fwd":
        x = sum((t.double() for t in s["inputs"]), torch.zeros((), device="cuda", dtype=torch.float64))
        if s["residual"] is not None:
            x = x + s["residual"].double()
        rounded = x.to(s["out"].dtype).double()  # the norm is that of the stored sum
        var, mean = torch.var_mean(rounded, dim=1, unbiased=False)
        y = (rounded - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * s["weight"].double() + s["bias"].double()
        out = {"out": y, "mean": mean, "rstd": 1 / torch.sqrt(var + EPS)}
        if s["sum"] is not None:
            out["sum"] = x
        return out
    if case["op"] == "norm_bwd":
        x = s["sum"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
        sd = torch.sqrt(var + EPS)
        xhat = (x - mean) / sd
        dy = s["dout"].double()
        dxhat = dy * s["weight"].double()
        n = x.shape[1]
        dx = (n * dxhat - dxhat.sum(1, keepdim=True) - xhat * (dxhat * xhat).sum(1, keepdim=True)) / (n * sd)
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].double()
        return {"dsum": dx, "dweight": torch.einsum("ij,ij->j", dy, xhat), "dbias": dy.sum(0)}
    h = s["hidden"].double()
    z = torch.cat([h @ w.double().T for w in s["weights"]], 1)
    lse = torch.logsumexp(z, 1)
    counted = (s["targets"] != IGNORE).nonzero()[:, 0]
    t = s["targets"][counted]
    if case["op"] == "xent_fwd":
        loss = torch.zeros_like(lse)
        loss[counted] = lse[counted] - z[counted, t]
        return {"loss": loss, "lse": lse}
    z.sub_(lse[:, None]).exp_()
    z[counted, t] -= 1
    weight = torch.zeros_like(lse)
    weight[counted] = s["dloss"][counted].double()
    z.mul_(weight[:, None])
    parts = z.split(s["rows"], 1)
    dh = torch.zeros_like(h)
    for part, w in zip(parts, s["weights"]):
        dh += part @ w.double()
    return {"dhidden": dh, "dweights": [part.T @ h for part in parts]}
