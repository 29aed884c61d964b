"""Operators of a training step around its attention and its weights' update, with every rank's buffers in one GPU's HBM,
as cases that can be timed.

Four operators, each in a plain form of elementary torch operations and as the library's own calls:

- ``qk_fwd``: the sum of N rank buffers of a projection to queries, keys and values, the norm of each head of the queries
  and keys, and their rotation by position (``mrr_qknorm_rope_fwd``);
- ``qk_bwd``: its gradient, with those of the two norms' weights (``mrr_qknorm_rope_bwd``);
- ``orth``: matrices made orthogonal by Newton-Schulz products (``mrr_orthogonalize``);
- ``muon``: the weights' update by them: the sum of N rank gradients, momentum, the products, and the new weights for every
  rank (``mrr_muon_step``).

``own`` chooses: False computes the plain forms, True calls the library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6          # of the heads' norms
TINY = 1e-7         # added to a matrix's norm
BASE = 500000.0     # of the rotation's frequencies
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
MOMENTUM, RATE, DECAY = 0.95, 0.02, 0.002


def _qk(op, tokens, heads, dim, rot, pairs, ranks, dtype, wdtype, pad, name=None):
    """heads: of the queries, keys and values; rot: rotated elements of a head; pairs: neighbours rotate together, not halves;
    pad: the share of tokens that fill up a padded batch."""
    c = {"op": op, "tokens": tokens, "heads_q": heads[0], "heads_k": heads[1], "heads_v": heads[2], "dim": dim, "rot": rot,
         "pairs": pairs, "ranks": ranks, "dtype": dtype, "wdtype": wdtype, "pad": pad}
    return dict(c, name=name) if name else c


def _mat(op, rows, cols, batch, ranks, dtype, wdtype, nesterov, name=None):
    """dtype: of the gradients (orth: of the matrices), wdtype: of the weights."""
    c = {"op": op, "rows": rows, "cols": cols, "batch": batch, "ranks": ranks, "dtype": dtype, "wdtype": wdtype, "nesterov": nesterov}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of a model sharded over 8 ranks: only the call's latency counts
        _qk("qk_fwd", 1, (32, 8, 8), 128, 128, False, 8, "bf16", "bf16", 0.0, "qk_fwd 1 token 8 ranks"),
        # a training batch, grouped heads, norm weights kept in 32 bits
        _qk("qk_fwd", 16384, (32, 8, 8), 128, 128, False, 1, "bf16", "f32", 0.0, "qk_fwd batch"),
        # odd counts, a head that is no power of two and rotates in part, neighbours in pairs, a padded batch, 4 partial sums
        _qk("qk_fwd", 2047, (5, 3, 1), 80, 32, True, 4, "f16", "f16", 0.2, "qk_fwd odd f16 4 ranks"),
        # the training batch backwards
        _qk("qk_bwd", 16384, (32, 8, 8), 128, 128, False, 1, "bf16", "f32", 0.0, "qk_bwd batch"),
        # a small 32-bit model's batch, as many key heads as query heads
        _qk("qk_bwd", 513, (12, 12, 12), 64, 64, False, 1, "f32", "f32", 0.0, "qk_bwd small f32"),
        # one key head for all queries, a padded batch
        _qk("qk_bwd", 701, (7, 1, 1), 96, 48, True, 1, "f16", "f16", 0.3, "qk_bwd odd f16"),
        # a large model's square weight
        _mat("orth", 4096, 4096, 1, 1, "bf16", "bf16", False, "orth 4096 x 4096"),
        # the output weights of 12 layers of a small 32-bit model, one matrix a head
        _mat("orth", 64, 768, 12, 1, "f32", "f32", False, "orth 12 heads f32"),
        # more rows than columns, odd both, every product in two parts
        _mat("orth", 1600, 1023, 1, 1, "f16", "f16", False, "orth odd f16"),
        # the update of a small model's weight in 32 bits, 2 ranks
        _mat("muon", 520, 1600, 1, 2, "f32", "f32", True, "muon small f32 2 ranks"),
        # the update of four layers' weights at once, kept in 32 bits beside 16-bit gradients of 4 ranks
        _mat("muon", 1024, 1024, 4, 4, "bf16", "f32", True, "muon 4 layers 4 ranks"),
        # the update of a large model's wide weight, 8 ranks
        _mat("muon", 4096, 16384, 1, 8, "bf16", "bf16", True, "muon 4096 x 16384 8 ranks"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _to(rng, n, to):
    """n as it is drawn, or next to it a multiple of `to`, as most models have it."""
    return n if rng.random() < 0.4 else max(to, (n + to // 2) // to * to)


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "orth", "muon"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("qk"):
        dim = rng.choice([64, 128, 2 * _log(rng, 8, 128)])
        rot = rng.choice([dim, dim // 4 * 2])
        kv = _log(rng, 1, 16)
        heads = (kv * rng.choice([1, 2, 4, 7]), kv, rng.choice([kv, kv, 0]))
        ranks = rng.choice([1, 2, 4, 8]) if op == "qk_fwd" else 1
        tokens = _log(rng, 1, max(1, min(16384, 16384 * 48 * 128 // (sum(heads) * dim * ranks))))
        return _qk(op, tokens, heads, dim, rot, rng.random() < 0.4, ranks, dtype, rng.choice(["f32", dtype]),
                   rng.choice([0.0, 0.0, 0.25]))
    rows, cols = (_to(rng, _log(rng, 32, 8192), 64) for _ in range(2))
    ranks = rng.choice([1, 2, 4, 8]) if op == "muon" else 1
    wdtype = rng.choice(["f32", dtype]) if op == "muon" else dtype
    # 32-bit products cost more, small matrices have batches
    most = 4096 * 4096 * 16384 // (1 if wdtype == "bf16" else 8)
    while rows * cols * min(rows, cols) > most or rows * cols * ranks > 4096 * 16384 * 8:
        rows, cols = (rows + 1) // 2, (cols + 1) // 2
    batch = _log(rng, 1, max(1, min(16, 4096 * 4096 // (rows * cols))))
    return _mat(op, rows, cols, batch, ranks, dtype, wdtype, rng.random() < 0.7)


def _table(case, rows):
    """Cosines and sines of the positions below `rows`, computed in 64 bits."""
    half = case["rot"] // 2
    f = BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, wdt = TYPES[case["dtype"]], TYPES[case["wdtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"].startswith("qk"):
        tokens, dim, ranks = case["tokens"], case["dim"], case["ranks"]
        heads = [case["heads_q"], case["heads_k"], case["heads_v"]]
        width = sum(heads) * dim
        # heads of different sizes, a few elements of each far larger than the others, as in a trained model
        scale = torch.where(torch.rand(width, generator=g, device="cuda") < 0.02, 8.0, 1.0) * torch.exp(
            0.5 * normal(sum(heads), 1)).expand(-1, dim).reshape(-1)
        s["heads"], s["width"] = heads, width
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * normal(dim)).to(wdt) for _ in range(2))
        # sequences side by side, each from a position of its own on; a fifth or so of a padded batch's tokens are none
        first = torch.randint(0, 4096, (64,), generator=g, device="cuda")
        t = torch.arange(tokens, device="cuda")
        each = max(1, tokens // 5)
        s["positions"] = first[(t // each) % 64] + t % each
        if case["pad"]:
            s["positions"][t % each >= int(each * (1 - case["pad"]))] = -1
        s["table"] = _table(case, 4096 + each)
        if case["op"] == "qk_fwd":
            s["inputs"] = [(normal(tokens, width) * scale / ranks ** 0.5).to(dt) for _ in range(ranks)]
            s["sum"] = torch.zeros(tokens, width, device="cuda", dtype=dt) if ranks > 1 else None
            s["outs"] = [torch.zeros(tokens, n, dim, device="cuda", dtype=dt) if n else None for n in heads]
        else:
            s["sum"] = (normal(tokens, width) * scale).to(dt)
            s["douts"] = [(0.1 * normal(tokens, n, dim)).to(dt) if n else None for n in heads]
            s["dsum"] = empty(tokens, width)
            s["dq_weight"], s["dk_weight"] = empty(dim, dtype=wdt), empty(dim, dtype=wdt)
        return s
    rows, cols, batch, ranks = case["rows"], case["cols"], case["batch"], case["ranks"]

    def gradient(noise):
        """A few directions that stand out of noise, rows of different sizes."""
        k = 1 + min(rows, cols) // 16
        low = torch.bmm(normal(batch, rows, k), normal(batch, k, cols)) / k ** 0.5
        return (low + noise * normal(batch, rows, cols)) * torch.exp(0.3 * normal(batch, rows, 1))

    if case["op"] == "orth":
        s["in"] = (1e-3 * gradient(0.5)).to(dt)
        s["out"] = empty(batch, rows, cols)
        return s
    common = gradient(0.2)
    scale = 256.0 if case["dtype"] == "f16" else 1.0  # 16-bit floats are trained with a scaled loss
    s["grad_scale"] = 1.0 / (ranks * scale)
    s["grads"] = [(1e-3 * scale * (common + normal(batch, rows, cols))).to(dt) for _ in range(ranks)]
    s["momentum"] = 1e-2 * (common + gradient(0.3))
    s["weight"] = (normal(batch, rows, cols) / cols ** 0.5).to(wdt)
    s["momentum_out"] = empty(batch, rows, cols, dtype=torch.float32)
    s["weights_out"] = [empty(batch, rows, cols, dtype=wdt) for _ in range(ranks)]
    return s


def _rotate(x, cos, sin, case, back):
    """x: [tokens, heads, dim]; cos, sin: [tokens, 1, rot / 2]."""
    rot = case["rot"]
    if back:
        sin = -sin
    if case["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _angles(s):
    half = s["case"]["rot"] // 2
    row = s["table"][s["positions"].clamp(min=0)][:, None]
    return row[..., :half], row[..., half:]


def _plain_qk_fwd(s):
    c = s["case"]
    dt = s["inputs"][0].dtype
    live = s["positions"] >= 0
    h = torch.stack(s["inputs"]).float().sum(0).to(dt)
    q, k, v = h.view(c["tokens"], -1, c["dim"]).split(s["heads"], 1)
    cos, sin = _angles(s)

    def normed(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        return _rotate(y, cos, sin, c, False).to(dt)

    outs = [normed(q, s["q_weight"]), normed(k, s["k_weight"]), v]
    out = {n: torch.where(live[:, None, None], o, 0.0) for n, o, have in zip("qkv", outs, s["heads"]) if have}
    if s["sum"] is not None:
        out["sum"] = torch.where(live[:, None], h, 0.0)
    return out


def _plain_qk_bwd(s):
    c = s["case"]
    dt, wdt = s["sum"].dtype, s["q_weight"].dtype
    live = (s["positions"] >= 0)[:, None, None]
    parts = s["sum"].view(c["tokens"], -1, c["dim"]).split(s["heads"], 1)
    cos, sin = _angles(s)
    d, out = [], {}
    for n, x, w in zip("qk", parts, (s["q_weight"], s["k_weight"])):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xhat = x * r
        u = torch.where(live, _rotate(s["douts"]["qk".index(n)].float(), cos, sin, c, True), 0.0)
        g = u * w.float()
        d.append((r * (g - xhat * (g * xhat).mean(-1, keepdim=True))).to(dt))
        out["d%s_weight" % n] = (u * xhat).sum((0, 1)).to(wdt)
    if s["heads"][2]:
        d.append(torch.where(live, s["douts"][2], 0.0))
    out["dsum"] = torch.cat(d, 1).flatten(1)
    return out


def _products(x, batch, rows, cols):
    """Newton-Schulz products of [batch, rows, cols]."""
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + TINY)
    if rows > cols:
        x = x.transpose(1, 2).contiguous()
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        m = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * m + c * torch.bmm(m, m), x)
    return x.transpose(1, 2) if rows > cols else x


def _plain_orth(s):
    c = s["case"]
    return {"out": _products(s["in"].float(), c["batch"], c["rows"], c["cols"]).to(s["out"].dtype).contiguous()}


def _plain_muon(s):
    c = s["case"]
    g = torch.stack(s["grads"]).float().sum(0) * s["grad_scale"]
    m = MOMENTUM * s["momentum"] + g
    u = g + MOMENTUM * m if c["nesterov"] else m
    w = (1 - DECAY) * s["weight"].float() - RATE * _products(u, c["batch"], c["rows"], c["cols"])
    w = w.to(s["weight"].dtype)
    return {"momentum": m, "weights": [w.clone() for _ in range(c["ranks"])]}


def _workspace(s, nbytes):
    """The workspace that a training program keeps from one step to the next."""
    if s.get("workspace") is None:
        s["workspace"] = torch.empty(max(256, nbytes), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import allreduce_reduction_nranks_amd as mrr
    c = s["case"]
    op, dtype, wdtype = c["op"], c["dtype"], c["wdtype"]
    if op.startswith("qk"):
        tokens, dim, heads, width = c["tokens"], c["dim"], s["heads"], s["width"]
        lds, strides = [n * dim for n in heads], [dim] * 3
        if op == "qk_fwd":
            mrr.check(mrr.mrr_qknorm_rope_fwd(s["inputs"], c["ranks"], s["q_weight"], s["k_weight"], s["table"], s["table"].shape[0],
                                              s["positions"], s["sum"], s["outs"], tokens, heads, dim, c["rot"], c["pairs"], width,
                                              lds, strides, EPS, dtype, wdtype), op)
            out = {n: o for n, o in zip("qkv", s["outs"]) if o is not None}
            if s["sum"] is not None:
                out["sum"] = s["sum"]
            return out
        n = mrr.mrr_qknorm_rope_bwd_workspace_bytes(tokens, heads, dim)
        mrr.check(mrr.mrr_qknorm_rope_bwd(s["douts"], s["sum"], s["q_weight"], s["k_weight"], s["table"], s["table"].shape[0],
                                          s["positions"], s["dsum"], s["dq_weight"], s["dk_weight"], tokens, heads, dim, c["rot"],
                                          c["pairs"], width, lds, strides, EPS, dtype, wdtype, _workspace(s, n), n), op)
        return {k: s[k] for k in ("dsum", "dq_weight", "dk_weight")}
    rows, cols, batch = c["rows"], c["cols"], c["batch"]
    if op == "orth":
        n = mrr.mrr_orthogonalize_workspace_bytes(rows, cols, batch, dtype)
        mrr.check(mrr.mrr_orthogonalize(s["in"], s["out"], rows, cols, cols, cols, batch, rows * cols, rows * cols, STEPS,
                                        COEFFICIENTS * STEPS, TINY, dtype, "auto", _workspace(s, n), n), op)
        return {"out": s["out"]}
    n = mrr.mrr_muon_workspace_bytes(rows, cols, batch, wdtype)
    mrr.check(mrr.mrr_muon_step(s["grads"], c["ranks"], s["grad_scale"], s["momentum"], s["momentum_out"], MOMENTUM, c["nesterov"],
                                s["weight"], s["weights_out"], RATE, DECAY, rows, cols, cols, cols, batch, rows * cols, rows * cols,
                                STEPS, COEFFICIENTS * STEPS, TINY, dtype, wdtype, "auto", _workspace(s, n), n), op)
    return {"momentum": s["momentum_out"], "weights": s["weights_out"]}


def run(state):
    if own:
        return _own(state)
    return {"qk_fwd": _plain_qk_fwd, "qk_bwd": _plain_qk_bwd, "orth": _plain_orth, "muon": _plain_muon}[state["case"]["op"]](state)


def work(case):
    size, wsize = (4 if case[k] == "f32" else 2 for k in ("dtype", "wdtype"))
    if case["op"].startswith("qk"):
        normed = case["tokens"] * (case["heads_q"] + case["heads_k"]) * case["dim"]
        n = normed + case["tokens"] * case["heads_v"] * case["dim"]
        # a table row of each position: that of a sequence's place is read by all heads
        table = case["tokens"] * (4 * case["rot"] + 8)
        if case["op"] == "qk_fwd":
            ranks = case["ranks"]
            return {"bytes": n * size * (ranks + 1 + (1 if ranks > 1 else 0)) + table + 2 * case["dim"] * wsize,
                    "flops": n * (ranks - 1) + normed * 7}
        return {"bytes": n * size * 2 + normed * size + table + 4 * case["dim"] * wsize, "flops": normed * 13}
    rows, cols, ranks = case["rows"], case["cols"], case["ranks"]
    n, m, k = case["batch"] * rows * cols, min(rows, cols), max(rows, cols)
    # two of a step's three products are symmetric: half of each is enough
    flops = case["batch"] * STEPS * (m * (m + 1) * k + m * m * (m + 1) + 2 * m * m * k)
    if case["op"] == "orth":
        return {"bytes": 2 * n * size, "flops": flops + 2 * n}
    return {"bytes": n * (ranks * size + 8 + (ranks + 1) * wsize), "flops": flops + n * (ranks + 8)}


def _exact_products(x):
    """The same polynomial of the singular values, by products in 64 bits from the other side than the plain form's where the
    matrix is square."""
    x = x / (torch.linalg.vector_norm(x) + TINY)
    a, b, c = COEFFICIENTS
    if x.shape[0] >= x.shape[1]:
        eye = torch.eye(x.shape[1], dtype=x.dtype, device=x.device)
        for _ in range(STEPS):
            m = x.T @ x
            x = x @ (a * eye + m @ (b * eye + c * m))
        return x
    eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    for _ in range(STEPS):
        m = x @ x.T
        x = (a * eye + m @ (b * eye + c * m)) @ x
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orth":
        return {"out": torch.stack([_exact_products(x) for x in s["in"].double()])}
    if case["op"] == "muon":
        g = sum((t.double() for t in s["grads"]), torch.zeros((), device="cuda", dtype=torch.float64)) * s["grad_scale"]
        m = s["momentum"].double() * MOMENTUM + g
        del s["grads"]
        u = m * MOMENTUM + g if case["nesterov"] else m
        w = s["weight"].double() * (1 - DECAY) - torch.stack([_exact_products(x) for x in u]) * RATE
        return {"momentum": m, "weights": [w] * case["ranks"]}
    dim, rot, heads = case["dim"], case["rot"], s["heads"]
    half = rot // 2
    # the rotation as a product of complex numbers, of the angles that the table's values stand for
    row = s["table"].double()[s["positions"].clamp(min=0)]
    turn = torch.complex(row[:, :half], row[:, half:])[:, None]
    live = (s["positions"] >= 0)[:, None, None]

    def turned(x, by):
        p = x[..., :rot].unflatten(-1, (half, 2)) if case["pairs"] else x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(p.contiguous()) * by)
        z = z if case["pairs"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., rot:]], -1)

    if case["op"] == "qk_fwd":
        total = sum((t.double() for t in s["inputs"]), torch.zeros((), device="cuda", dtype=torch.float64))
        h = total.to(s["inputs"][0].dtype).double().view(case["tokens"], -1, dim)  # the norm is that of the stored sum
        out = {}
        for i, n in enumerate("qkv"):
            if not heads[i]:
                continue
            x = h[:, sum(heads[:i]):sum(heads[:i + 1])]
            if i < 2:
                x = turned(x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + EPS) * s[n + "_weight"].double(), turn)
            out[n] = x * live
        if s["sum"] is not None:
            out["sum"] = total * live[:, :, 0]
        return out
    h = s["sum"].double().view(case["tokens"], -1, dim)
    d, out = torch.zeros_like(h), {}
    for i, n in enumerate("qk"):
        at = slice(sum(heads[:i]), sum(heads[:i + 1]))
        x, w = h[:, at], s[n + "_weight"].double()
        rms = torch.sqrt((x * x).sum(-1, keepdim=True) / dim + EPS)
        u = turned(s["douts"][i].double(), turn.conj()) * live
        out["d%s_weight" % n] = (u * x / rms).flatten(0, 1).sum(0)
        d[:, at] = u * w / rms - x * (u * w * x).sum(-1, keepdim=True) / (dim * rms ** 3)
    if heads[2]:
        d[:, heads[0] + heads[1]:] = s["douts"][2].double() * live
    out["dsum"] = d.flatten(1)
    return out
