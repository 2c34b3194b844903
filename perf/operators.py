"""The training-step operators, as they are measured: cases, inputs, plain forms.

A model around the convolution begins with an embedding of atom species or
tokens, passes its features through norms with a gate and a scaled residual
around every block, and ends a training step with the clipping of all
gradients by their global norm.  Each direction is a path of its own:

    embed_fwd   out[t] = scale * table[token[t]]; a token outside [0, rows) is padding, a zero row
    embed_bwd   d_table[v] = scale * sum of grad_out[t] over the t with token[t] = v
    norm_fwd    r' = r + alpha * gate * N(h; w_post),  u = N(r'; w_pre)
    norm_bwd    its gradients (d_r, d_h, d_w_post, d_w_pre[, d_gate]) for grad_r (of r') and grad_u (of u)
    clip        every gradient times min(1, max_norm / (norm + 1e-6)), norm over all of them

Features are [nodes, D, C] with D = (lmax + 1)^2 components of the degrees
0..lmax; lmax = 0 is the ordinary [rows, C].  N(x; w) = w[l(d), c] * x * s with
s = (eps + mean over c and l of (sum_m x[l m, c]^2 / (2l + 1)))^(-1/2), one s a
row: for lmax = 0 the root-mean-square norm.  `gate` is absent ("none"), one
value a degree and channel ("channel"), or that for every row ("row").
"""
import math
import random

import torch

own = False     # False: the plain forms below; True: the framework's operators

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6          # of the norms
CLIP_EPS = 1e-6     # of the clipping factor
MOST_BYTES = 1.2e9  # a drawn case moves at most this


def listed():
    return [
        # the smallest lookup: 64 nodes of 16 channels (the tiny graph), where the call's latency is all there is
        dict(name="embed_fwd tiny f32", op="embed_fwd", rows=100, channels=16, tokens=64, index="i32", dtype="f32",
             skew=1.0, pad=0.0, scale=1.0),
        # a text-sized vocabulary under a long batch, the usual sqrt(C) scale
        dict(name="embed_fwd vocab bf16", op="embed_fwd", rows=65536, channels=1024, tokens=32768, index="i64",
             dtype="bf16", skew=3.0, pad=0.0, scale=32.0),
        # the water box: 1503 atoms of few species, the table of the elements
        dict(name="embed_bwd water f32", op="embed_bwd", rows=100, channels=128, tokens=1503, index="i32", dtype="f32",
             skew=6.0, pad=0.1, scale=1.0),
        # a large batch of structures: every row of the small table is hit thousands of times
        dict(name="embed_bwd species f32", op="embed_bwd", rows=100, channels=128, tokens=131072, index="i32",
             dtype="f32", skew=2.0, pad=0.1, scale=1.0),
        # a large vocabulary: most rows of the gradient are zero, a few are hot
        dict(name="embed_bwd vocab bf16", op="embed_bwd", rows=131072, channels=2048, tokens=16384, index="i64",
             dtype="bf16", skew=4.0, pad=0.0, scale=1.0),
        # the water box's features between two convolutions: 1503 atoms, 128 channels, degrees 0..3
        dict(name="norm_fwd water l3 f32", op="norm_fwd", rows=1503, lmax=3, channels=128, dtype="f32", gate="channel",
             alpha=0.5),
        # long batches of plain rows, gated row by row
        dict(name="norm_fwd rows bf16", op="norm_fwd", rows=8192, lmax=0, channels=4096, dtype="bf16", gate="row",
             alpha=0.5),
        # odd everything: rows that do not start on 16 bytes
        dict(name="norm_bwd odd f16", op="norm_bwd", rows=5001, lmax=0, channels=1003, dtype="f16", gate="none",
             alpha=1.0),
        # rows of the usual width, gated row by row
        dict(name="norm_bwd rows bf16", op="norm_bwd", rows=8192, lmax=0, channels=4096, dtype="bf16", gate="row",
             alpha=0.5),
        # the features of the large graph: 16384 nodes, 128 channels, degrees 0..3
        dict(name="norm_bwd nodes l3 f32", op="norm_bwd", rows=16384, lmax=3, channels=128, dtype="f32",
             gate="channel", alpha=0.5),
        # the parameters of a small potential: few matrices, vectors, single numbers
        dict(name="clip small f32", op="clip", width=128, layers=4, dtype="f32", spread=1.0, max_norm=10.0),
        # a large model's gradients
        dict(name="clip large bf16", op="clip", width=2048, layers=24, dtype="bf16", spread=0.01, max_norm=10.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    while True:
        op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "clip"])
        c = dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]))
        if op in ("embed_fwd", "embed_bwd"):
            c.update(rows=_log(rng, 2, 200000), channels=_log(rng, 8, 4096), tokens=_log(rng, 16, 262144),
                     index=rng.choice(["i32", "i64"]), skew=rng.choice([1.0, 2.0, 4.0, 6.0]),
                     pad=rng.choice([0.0, 0.0, 0.1, 0.5]), scale=rng.choice([1.0, 0.125, 11.3]))
        elif op in ("norm_fwd", "norm_bwd"):
            lmax = rng.choice([0, 0, 0, 1, 2, 3])
            c.update(rows=_log(rng, 1, 32768), lmax=lmax, channels=_log(rng, 8, 16384 // (lmax + 1) ** 2),
                     gate=rng.choice(["none", "channel", "row"]), alpha=rng.choice([1.0, 0.5, 0.17]))
        else:
            c.update(width=_log(rng, 8, 2048), layers=_log(rng, 1, 100), spread=rng.choice([1.0, 0.01]),
                     max_norm=rng.choice([1.0, 10.0]))
        if work(c)["bytes"] <= MOST_BYTES:
            return c


def _sizes(case):
    """Elements of every gradient: per layer two matrices, a table, a vector and a single number."""
    k = case["width"]
    return [100 * k] + [s for _ in range(case["layers"]) for s in (2 * k * k, k * k, 4 * k, k, 1)]


def _slots(sizes):
    """Where each tensor begins in the flat output (256-byte steps for 4-byte values), and the flat length."""
    at, starts = 0, []
    for s in sizes:
        starts.append(at)
        at += -(-s // 64) * 64
    return starts, at


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op in ("embed_fwd", "embed_bwd"):
        n, v, c = case["tokens"], case["rows"], case["channels"]
        ids = n * (4 if case["index"] == "i32" else 8)
        rows = min(n, v) if op == "embed_fwd" else v
        return {"bytes": ids + b * c * (n + rows), "flops": n * c}
    if op in ("norm_fwd", "norm_bwd"):
        n, d = case["rows"], (case["lmax"] + 1) ** 2
        w, lc = d * case["channels"], (case["lmax"] + 1) * case["channels"]
        gate = {"none": 0, "channel": lc, "row": n * lc}[case["gate"]]
        if op == "norm_fwd":
            return {"bytes": b * (4 * n * w + 2 * lc + gate), "flops": 10 * n * w}
        return {"bytes": b * (6 * n * w + 4 * lc + 2 * gate), "flops": 24 * n * w}
    total = sum(_sizes(case))
    return {"bytes": 2 * b * total, "flops": 3 * total}


def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case, dtype=dt)
    if op in ("embed_fwd", "embed_bwd"):
        n, v, c = case["tokens"], case["rows"], case["channels"]
        # ids fall off as a power law from 0, then are scattered over the table
        ids = (torch.rand(n, generator=gen, device="cuda").pow(case["skew"]) * v).long().clamp_(max=v - 1)
        ids = torch.randperm(v, generator=gen, device="cuda")[ids]
        ids[torch.rand(n, generator=gen, device="cuda") < case["pad"]] = -1
        s["tokens"] = ids.to(torch.int32 if case["index"] == "i32" else torch.int64)
        if op == "embed_fwd":
            s["table"] = _normal(gen, (v, c), dt)
        else:
            s["grad_out"] = _normal(gen, (n, c), dt)
    elif op in ("norm_fwd", "norm_bwd"):
        n, nl, c = case["rows"], case["lmax"] + 1, case["channels"]
        row = (n, c) if nl == 1 else (n, nl * nl, c)
        per = (c,) if nl == 1 else (nl, c)
        s["w_post"] = _normal(gen, per, dt, 0.2, 1.0)
        s["w_pre"] = _normal(gen, per, dt, 0.2, 1.0)
        s["gate"] = {"none": lambda: None, "channel": lambda: _normal(gen, per, dt, 0.5, 0.5),
                     "row": lambda: _normal(gen, (n,) + per, dt, 0.5, 0.5)}[case["gate"]]()
        s["h"] = _normal(gen, row, dt, 3.0)
        s["r"] = _normal(gen, row, dt)
        if op == "norm_bwd":        # r is then the stored r' of the forward pass
            s["grad_r"] = _normal(gen, row, dt)
            s["grad_u"] = _normal(gen, row, dt)
    else:
        sizes = _sizes(case)
        starts, length = _slots(sizes)
        s["grads"] = [_normal(gen, (k,), dt, case["spread"]) for k in sizes]
        s["flat"] = torch.zeros(length, dtype=dt, device="cuda")
        s["out"] = [s["flat"][a:a + k] for a, k in zip(starts, sizes)]
        ends = starts[1:] + [length]
        s["pieces"] = [p for g, a, k, e in zip(s["grads"], starts, sizes, ends)
                       for p in (g, torch.zeros(e - a - k, dtype=dt, device="cuda"))]
    return s


def _degree_of(lmax, device):
    """l(d) of every component, and the weight 1 / ((lmax + 1) (2l + 1)) of its square in the row's mean."""
    l = torch.arange((lmax + 1) ** 2, device=device).add(0.5).sqrt().floor().long()
    return l, 1.0 / ((lmax + 1) * (2 * l + 1).float())


def _plain_embed(s):
    case, tokens = s["case"], s["tokens"].long()
    valid = ((tokens >= 0) & (tokens < case["rows"]))[:, None]
    at = tokens.clamp(0, case["rows"] - 1)
    if case["op"] == "embed_fwd":
        return torch.where(valid, s["table"][at].float() * case["scale"], 0.0).to(s["dtype"])
    g = torch.where(valid, s["grad_out"].float(), 0.0)
    d = torch.zeros(case["rows"], case["channels"], device="cuda").index_add_(0, at, g)
    return (d * case["scale"]).to(s["dtype"])


def _plain_norm(s):
    case, dt = s["case"], s["dtype"]
    n, nl, c, alpha = case["rows"], case["lmax"] + 1, case["channels"], case["alpha"]
    l, b = _degree_of(case["lmax"], "cuda")
    b = b[:, None] / c

    def rows(name):
        return s[name].float().view(n, nl * nl, c)

    def per_degree(name):
        return s[name].float().view(-1, nl, c)[:, l]        # [1 or n, D, C]

    def scale(x):
        return torch.rsqrt((x.square() * b).sum((1, 2), keepdim=True) + EPS)

    def by_degree(x):       # [k, D, C] summed over the components of each degree
        return torch.zeros(x.shape[0], nl, c, device="cuda").index_add_(1, l, x)

    h, r, w_post, w_pre = rows("h"), rows("r"), per_degree("w_post"), per_degree("w_pre")
    gate = alpha if s["gate"] is None else alpha * per_degree("gate")
    s1 = scale(h)
    if case["op"] == "norm_fwd":
        r = r + gate * (h * s1 * w_post)
        u = r * scale(r) * w_pre
        return {"r": r.to(dt).view(s["r"].shape), "u": u.to(dt).view(s["r"].shape)}
    s2 = scale(r)
    a = rows("grad_u")
    d_pre = by_degree((a * r * s2).sum(0, keepdim=True))
    a = a * w_pre
    d = rows("grad_r") + s2 * a - r * b * (s2 ** 3 * (a * r).sum((1, 2), keepdim=True))
    dy = gate * d
    d_post = by_degree((dy * h * s1).sum(0, keepdim=True))
    a = dy * w_post
    dh = s1 * a - h * b * (s1 ** 3 * (a * h).sum((1, 2), keepdim=True))
    out = {"d_r": d.to(dt).view(s["r"].shape), "d_h": dh.to(dt).view(s["r"].shape),
           "d_w_post": d_post.to(dt).view(s["w_post"].shape), "d_w_pre": d_pre.to(dt).view(s["w_pre"].shape)}
    if s["gate"] is not None:
        dg = alpha * d * (h * s1 * w_post)
        dg = by_degree(dg.sum(0, keepdim=True) if case["gate"] == "channel" else dg)
        out["d_gate"] = dg.to(dt).view(s["gate"].shape)
    return out


def _plain_clip(s):
    flat = torch.cat(s["pieces"]).float()
    norm = flat.square().sum().sqrt()
    factor = (s["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return {"grads": (flat * factor).to(s["dtype"]), "norm": norm}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"embed_fwd": _plain_embed, "embed_bwd": _plain_embed, "norm_fwd": _plain_norm,
                "norm_bwd": _plain_norm, "clip": _plain_clip}[op](s)
    import tensor_product_message_amd as ctp
    if op == "embed_fwd":
        return ctp.embed_fwd(s["table"], s["tokens"], scale=case["scale"])
    if op == "embed_bwd":
        return ctp.embed_bwd(s["grad_out"], s["tokens"], case["rows"], scale=case["scale"])
    if op == "norm_fwd":
        r, u = ctp.norm_residual_fwd(s["h"], s["r"], s["w_post"], s["w_pre"], gate=s["gate"], alpha=case["alpha"],
                                     eps=EPS, lmax=case["lmax"])
        return {"r": r, "u": u}
    if op == "norm_bwd":
        names = ("d_h", "d_r", "d_w_post", "d_w_pre", "d_gate")
        got = ctp.norm_residual_bwd(s["grad_r"], s["grad_u"], s["h"], s["r"], s["w_post"], s["w_pre"],
                                    gate=s["gate"], alpha=case["alpha"], eps=EPS, lmax=case["lmax"])
        return {k: v for k, v in zip(names, got) if v is not None}
    _, norm = ctp.clip_grad_norm(s["grads"], case["max_norm"], eps=CLIP_EPS, out=s["out"])
    return {"grads": s["flat"], "norm": norm}


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions: gradients by differentiating the definition itself."""
    s = prepare(case, seed)
    if case["op"] in ("embed_fwd", "embed_bwd"):
        ids = s["tokens"].long()
        real = ((ids >= 0) & (ids < case["rows"])).nonzero()[:, 0]
        if case["op"] == "embed_fwd":
            out = torch.zeros(case["tokens"], case["channels"], dtype=torch.float64, device="cuda")
            out[real] = case["scale"] * torch.index_select(s["table"], 0, ids[real]).double()
            return out
        order = real[torch.argsort(ids[real])]
        count = torch.bincount(ids[real], minlength=case["rows"])
        # sums of the sorted rows by a running total would cancel: added one by one, in 64 bits
        where = torch.repeat_interleave(torch.arange(case["rows"], device="cuda"), count)
        d = torch.zeros(case["rows"], case["channels"], dtype=torch.float64, device="cuda")
        return d.index_put_((where,), s["grad_out"][order].double(), accumulate=True) * case["scale"]
    if case["op"] in ("norm_fwd", "norm_bwd"):
        lmax = case["lmax"]

        def leaf(name):
            return None if s[name] is None else s[name].double().requires_grad_(case["op"] == "norm_bwd")

        def norm(x, w):     # degree by degree
            if lmax == 0:
                return w * x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
            mean = sum(x[:, l * l:(l + 1) ** 2].pow(2).mean((1, 2)) for l in range(lmax + 1)) / (lmax + 1)
            x = x / (mean + EPS).sqrt()[:, None, None]
            return torch.cat([x[:, l * l:(l + 1) ** 2] * w[l] for l in range(lmax + 1)], 1)

        def gated(y, g):
            if g is None:
                return y
            if lmax == 0:
                return y * g
            g = g.view(-1, lmax + 1, case["channels"])
            return torch.cat([y[:, l * l:(l + 1) ** 2] * g[:, l:l + 1] for l in range(lmax + 1)], 1)

        h, r, w_post, w_pre, gate = leaf("h"), leaf("r"), leaf("w_post"), leaf("w_pre"), leaf("gate")
        add = case["alpha"] * gated(norm(h, w_post), gate)
        if case["op"] == "norm_fwd":
            return {"r": r + add, "u": norm(r + add, w_pre)}
        # r is r' as the forward pass stored it: what reaches it also reaches the old r and the addend
        (d_r, d_pre) = torch.autograd.grad(norm(r, w_pre), (r, w_pre), s["grad_u"].double())
        d_r = d_r + s["grad_r"].double()
        wants = [h, w_post] + ([gate] if gate is not None else [])
        got = torch.autograd.grad(add, wants, d_r)
        out = {"d_r": d_r, "d_h": got[0], "d_w_post": got[1], "d_w_pre": d_pre}
        return out if gate is None else {**out, "d_gate": got[2]}
    starts, length = _slots(_sizes(case))
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
    flat = torch.zeros(length, dtype=torch.float64, device="cuda")
    for g, a in zip(s["grads"], starts):
        flat[a:a + g.numel()] = g.double() * min(1.0, case["max_norm"] / (norm + CLIP_EPS))
    return {"grads": flat, "norm": norm}
