"""The dense operators around the convolution, as they are measured: cases, inputs, plain forms.

Radial networks make the convolution's weights, channels are mixed degree by degree before and after it, node
scalars pass through a gated feed-forward block, and behind the clipping of gradients an optimiser may
orthogonalise its updates.  Each direction is a path of its own:

    linear_fwd     z = x w^T + bias,  y = act(z) + residual
    linear_bwd     s = grad act'(z): d_x = s w, d_w = s^T x, d_bias = sum of s
    gated_fwd      z = x w^T + bias for both halves of w [2, F, C],  h = act(z[0]) z[1]
    gated_bwd      its gradients (d_x, d_w, d_bias), for the z that the forward pass stored
    orthogonalise  X = M / (|M| + eps), then steps times X <- a X + (b A + c A A) X with A = X X^T

For lmax > 0 rows are [D, C], D = (lmax + 1)^2 components of the degrees 0..lmax, w is [lmax + 1, out, in], one matrix
a degree, the bias is the scalars' (degree 0) and there is no activation.
"""
import math
import random

import torch

own = False     # False: the plain forms below; True: the framework's operators

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
ACTS = ["none", "relu", "silu", "gelu", "sigmoid", "tanh"]
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7              # of the norm that the iteration begins with
MOST_BYTES = 1.45e9     # a drawn case moves at most this,
MOST_FLOPS = 1.0e12     # and computes at most this


def listed():
    return [
        # 64 nodes of 16 channels (the tiny graph): the call's latency is all there is
        dict(name="linear_fwd tiny l1 f32", op="linear_fwd", rows=64, lmax=1, inner=16, outer=16, act="none", bias=True,
             residual=True, z=False, dtype="f32"),
        # a hidden layer of the water box's radial network: 83325 edges, 64 -> 64, in training
        dict(name="linear_fwd hidden f32", op="linear_fwd", rows=83325, lmax=0, inner=64, outer=64, act="silu",
             bias=True, residual=False, z=True, dtype="f32"),
        # that network's last layer, which writes the convolution's weights: 34 paths of 128 channels an edge
        dict(name="linear_fwd weights f32", op="linear_fwd", rows=83325, lmax=0, inner=64, outer=4352, act="none",
             bias=False, residual=False, z=False, dtype="f32"),
        # channel mixing of the large graph's features: 16384 nodes, degrees 0..3, added to the residual
        dict(name="linear_fwd nodes l3 f32", op="linear_fwd", rows=16384, lmax=3, inner=128, outer=128, act="none",
             bias=True, residual=True, z=False, dtype="f32"),
        # the same mixing's gradients on the water box: 1503 atoms
        dict(name="linear_bwd water l3 f32", op="linear_bwd", rows=1503, lmax=3, inner=128, outer=128, act="none",
             bias=True, dtype="f32"),
        # the hidden radial layer's gradients
        dict(name="linear_bwd hidden f32", op="linear_bwd", rows=83325, lmax=0, inner=64, outer=64, act="silu",
             bias=True, dtype="f32"),
        # odd everything: rows that do not start on 16 bytes
        dict(name="linear_bwd odd f16", op="linear_bwd", rows=5001, lmax=0, inner=1003, outer=777, act="gelu",
             bias=True, dtype="f16"),
        # one row: a single structure's or token's pass, where the weights' bytes are all there is
        dict(name="gated_fwd one row bf16", op="gated_fwd", rows=1, inner=4096, outer=16384, act="silu", bias=False,
             z=False, dtype="bf16"),
        # long batches, in training
        dict(name="gated_fwd rows bf16", op="gated_fwd", rows=8192, inner=2048, outer=8192, act="silu", bias=False,
             z=True, dtype="bf16"),
        dict(name="gated_bwd rows bf16", op="gated_bwd", rows=8192, inner=2048, outer=8192, act="silu", bias=False,
             dtype="bf16"),
        # the matrices of a small potential: mixing of each degree, feed-forward blocks, radial layers
        dict(name="orthogonalise small f32", op="orthogonalise", width=128, ratio=4, degrees=4, layers=2, extra=4352,
             low_rank=False, dtype="f32"),
        # a wide model's, gradients of few directions among noise
        dict(name="orthogonalise large bf16", op="orthogonalise", width=2048, ratio=4, degrees=1, layers=1, extra=0,
             low_rank=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    while True:
        op = rng.choice(["linear_fwd", "linear_bwd", "gated_fwd", "gated_bwd", "orthogonalise"])
        c = dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]))
        if op == "orthogonalise":
            c.update(width=_log(rng, 16, 2048), ratio=rng.choice([1, 2, 4]), degrees=rng.choice([1, 2, 4]),
                     layers=_log(rng, 1, 12), extra=rng.choice([0, 0, _log(rng, 8, 4352)]),
                     low_rank=rng.choice([True, False]))
        else:
            linear = op in ("linear_fwd", "linear_bwd")
            lmax = rng.choice([0, 0, 1, 2, 3]) if linear else 0
            top = 1024 if lmax else 8192
            c.update(rows=_log(rng, 1, 131072), inner=_log(rng, 8, top), outer=_log(rng, 8, top),
                     bias=rng.choice([True, False]), act=rng.choice(ACTS))
            if linear:
                c.update(lmax=lmax)
                if lmax:
                    c.update(act="none")
            if op == "linear_fwd":
                c.update(residual=rng.choice([True, False]))
            if op in ("linear_fwd", "gated_fwd"):
                c.update(z=rng.choice([True, False]))
        w = work(c)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return c


def _shapes(case):
    """Matrices of every layer: the degrees' square ones in one tensor, a tall one, a wide one; one more in all."""
    k, r = case["width"], case["ratio"]
    shapes = [s for _ in range(case["layers"]) for s in ((case["degrees"], k, k), (r * k, k), (k, r * k))]
    return shapes + ([(case["extra"], 64)] if case["extra"] else [])


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op == "orthogonalise":
        size = flops = 0
        for shape in _shapes(case):
            n, (s, l) = (shape[0] if len(shape) == 3 else 1), sorted(shape[-2:])
            size += n * s * l
            flops += n * STEPS * (3 * s * s * l + s ** 3)     # A and A A are symmetric: half of each is enough
        return {"bytes": 2 * b * size, "flops": flops}
    m, i, o = case["rows"], case["inner"], case["outer"]
    if op in ("linear_fwd", "linear_bwd"):
        d, nl = (case["lmax"] + 1) ** 2, case["lmax"] + 1
        w, bias, act = nl * i * o, o * case["bias"], case["act"] != "none"
        if op == "linear_fwd":
            return {"bytes": b * (m * d * (i + o * (1 + case["residual"] + case["z"])) + w + bias),
                    "flops": 2 * m * d * i * o}
        return {"bytes": b * (m * d * (2 * i + o * (1 + act)) + 2 * w + bias), "flops": 4 * m * d * i * o}
    w, bias = 2 * i * o, 2 * o * case["bias"]
    if op == "gated_fwd":
        return {"bytes": b * (m * (i + o * (1 + 2 * case["z"])) + w + bias), "flops": 4 * m * i * o}
    return {"bytes": b * (m * (2 * i + 3 * o) + 2 * w + bias), "flops": 8 * m * i * o}


def _normal(gen, shape, dtype, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case, dtype=dt)
    if op == "orthogonalise":
        s["updates"] = []
        for shape in _shapes(case):
            u = _normal(gen, shape, torch.float32, 1e-3)
            if case["low_rank"]:
                rank = max(1, min(shape[-2:]) // 16)
                u *= 0.1
                u += _normal(gen, shape[:-1] + (rank,), torch.float32, 1e-3) @ _normal(gen, shape[:-2] + (rank, shape[-1]),
                                                                                      torch.float32)
            s["updates"].append(u.to(dt))
        s["out"] = [torch.empty_like(u) for u in s["updates"]]
        return s
    m, i, o = case["rows"], case["inner"], case["outer"]
    if op in ("linear_fwd", "linear_bwd"):
        d, nl = (case["lmax"] + 1) ** 2, case["lmax"] + 1
        comps, per = (() if nl == 1 else (d,)), (() if nl == 1 else (nl,))
        s["x"] = _normal(gen, (m, *comps, i), dt)
        s["w"] = _normal(gen, (*per, o, i), dt, i ** -0.5)
        s["bias"] = _normal(gen, (o,), dt, 0.5) if case["bias"] else None
        if op == "linear_fwd":
            s["residual"] = _normal(gen, (m, *comps, o), dt) if case["residual"] else None
        else:
            s["grad"] = _normal(gen, (m, *comps, o), dt)
            s["z"] = _normal(gen, (m, o), dt, 1.1) if case["act"] != "none" else None
        return s
    s["x"] = _normal(gen, (m, i), dt)
    s["w"] = _normal(gen, (2, o, i), dt, i ** -0.5)
    s["bias"] = _normal(gen, (2, o), dt, 0.5) if case["bias"] else None
    if op == "gated_bwd":
        s["grad"] = _normal(gen, (m, o), dt)
        s["z"] = _normal(gen, (m, 2, o), dt, 1.1)
    return s


def _act(name, z):
    """act(z) and act'(z)."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).to(z.dtype)
    if name == "tanh":
        t = 1.0 - 2.0 / (1.0 + torch.exp(2.0 * z))
        return t, 1.0 - t * t
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    g = 1.0 / (1.0 + torch.exp(-z))
    if name == "sigmoid":
        return g, g * (1.0 - g)
    return z * g, g * (1.0 + z * (1.0 - g))


def _degrees(lmax):
    """(l, first component, one past the last) of every degree."""
    return [(l, l * l, (l + 1) ** 2) for l in range(lmax + 1)]


def _plain_linear_fwd(s):
    case, dt = s["case"], s["dtype"]
    x, w = s["x"].float(), s["w"].float()
    if case["lmax"]:
        z = torch.cat([(x[:, a:b].reshape(-1, case["inner"]) @ w[l].t()).view(-1, b - a, case["outer"])
                       for l, a, b in _degrees(case["lmax"])], 1)
        if case["bias"]:
            z[:, 0] += s["bias"].float()
    else:
        z = x @ w.t()
        if case["bias"]:
            z = z + s["bias"].float()
    y = _act(case["act"], z)[0]
    if case["residual"]:
        y = y + s["residual"].float()
    return {"y": y.to(dt), "z": z.to(dt)} if case["z"] else {"y": y.to(dt)}


def _plain_linear_bwd(s):
    case, dt = s["case"], s["dtype"]
    x, w, g = s["x"].float(), s["w"].float(), s["grad"].float()
    if case["lmax"]:
        d_x, d_w = torch.empty_like(x), torch.empty_like(w)
        for l, a, b in _degrees(case["lmax"]):
            gl = g[:, a:b].reshape(-1, case["outer"])
            d_x[:, a:b] = (gl @ w[l]).view(-1, b - a, case["inner"])
            d_w[l] = gl.t() @ x[:, a:b].reshape(-1, case["inner"])
        d_b = g[:, 0].sum(0)
    else:
        if case["act"] != "none":
            g = g * _act(case["act"], s["z"].float())[1]
        d_x, d_w, d_b = g @ w, g.t() @ x, g.sum(0)
    out = {"d_x": d_x.to(dt), "d_w": d_w.to(dt)}
    return {**out, "d_bias": d_b.to(dt)} if case["bias"] else out


def _plain_gated(s):
    case, dt, o = s["case"], s["dtype"], s["case"]["outer"]
    x, w = s["x"].float(), s["w"].float().view(2 * o, -1)
    if case["op"] == "gated_fwd":
        z = x @ w.t()
        if case["bias"]:
            z = z + s["bias"].float().view(-1)
        z = z.view(-1, 2, o)
        h = (_act(case["act"], z[:, 0])[0] * z[:, 1]).to(dt)
        return {"h": h, "z": z.to(dt)} if case["z"] else {"h": h}
    g, z = s["grad"].float(), s["z"].float()
    f, df = _act(case["act"], z[:, 0])
    d_z = torch.stack([g * z[:, 1] * df, g * f], 1).view(-1, 2 * o)
    out = {"d_x": (d_z @ w).to(dt), "d_w": (d_z.t() @ x).to(dt).view(s["w"].shape)}
    return {**out, "d_bias": d_z.sum(0).to(dt).view(2, o)} if case["bias"] else out


def _plain_orthogonalise(s):
    a, b, c = QUINTIC
    for u, out in zip(s["updates"], s["out"]):
        x = u.float()
        tall = x.shape[-2] > x.shape[-1]
        if tall:
            x = x.transpose(-1, -2).contiguous()
        x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + EPS)
        for _ in range(STEPS):
            p = x @ x.transpose(-1, -2).contiguous()
            x = a * x + (b * p + c * (p @ p)) @ x
        out.copy_(x.transpose(-1, -2) if tall else x)
    return s["out"]


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"linear_fwd": _plain_linear_fwd, "linear_bwd": _plain_linear_bwd, "gated_fwd": _plain_gated,
                "gated_bwd": _plain_gated, "orthogonalise": _plain_orthogonalise}[op](s)
    import tensor_product_message_amd as ctp
    if op == "linear_fwd":
        y, z = ctp.linear_fwd(s["x"], s["w"], s["bias"], s["residual"], act=case["act"], lmax=case["lmax"],
                              keep_z=case["z"])
        return {"y": y, "z": z} if case["z"] else {"y": y}
    if op == "gated_fwd":
        h, z = ctp.gated_linear_fwd(s["x"], s["w"], s["bias"], act=case["act"], keep_z=case["z"])
        return {"h": h, "z": z} if case["z"] else {"h": h}
    if op == "orthogonalise":
        return ctp.orthogonalise(s["updates"], steps=STEPS, eps=EPS, out=s["out"])
    needs = (True, True, case["bias"])
    if op == "linear_bwd":
        got = ctp.linear_bwd(s["grad"], s["x"], s["w"], s["z"], act=case["act"], lmax=case["lmax"], needs=needs)
    else:
        got = ctp.gated_linear_bwd(s["grad"], s["x"], s["w"], s["z"], act=case["act"], needs=needs)
    return {k: v for k, v in zip(("d_x", "d_w", "d_bias"), got) if v is not None}


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions: gradients by differentiating the definition itself."""
    s = prepare(case, seed)
    op = case["op"]
    nn = torch.nn.functional
    act = {"none": lambda z: z, "relu": nn.relu, "silu": nn.silu, "gelu": nn.gelu, "sigmoid": torch.sigmoid,
           "tanh": torch.tanh}
    if op == "orthogonalise":
        # every iterate is (a polynomial of the first A) times the first X: two products with the long side in all
        results = []
        for u in s["updates"]:
            stack = []
            for one in u.double().view(-1, *u.shape[-2:]):
                m = one.mT.contiguous() if one.shape[0] > one.shape[1] else one
                m = m / (torch.linalg.matrix_norm(m) + EPS)
                gram, total = m @ m.mT, None
                eye = torch.eye(m.shape[0], dtype=torch.float64, device="cuda")
                for _ in range(STEPS):
                    q = QUINTIC[0] * eye + gram @ (QUINTIC[1] * eye + QUINTIC[2] * gram)
                    total = q if total is None else q @ total
                    gram = q @ gram @ q
                m = total @ m
                stack.append(m.mT if one.shape[0] > one.shape[1] else m)
            results.append(torch.stack(stack).view(u.shape))
        return results
    x, w = s["x"].double(), s["w"].double()
    bias = None if s["bias"] is None else s["bias"].double()
    if op == "linear_fwd":
        if case["lmax"]:
            of = torch.tensor([l for l, a, b in _degrees(case["lmax"]) for _ in range(a, b)])
            z = torch.stack([x[:, d] @ w[int(l)].mT for d, l in enumerate(of)], 1)
            if bias is not None:
                z[:, 0] += bias
        else:
            z = nn.linear(x, w, bias)
        y = act[case["act"]](z)
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if case["z"] else {"y": y}
    if op == "gated_fwd":
        z = torch.stack([nn.linear(x, w[k], None if bias is None else bias[k]) for k in (0, 1)], 1)
        h = act[case["act"]](z[:, 0]) * z[:, 1]
        return {"h": h, "z": z} if case["z"] else {"h": h}
    grad = s["grad"].double()
    if op == "linear_bwd" and case["lmax"]:
        # component by component
        d_x, d_w = torch.zeros_like(x), torch.zeros_like(w)
        for l, a, b in _degrees(case["lmax"]):
            for d in range(a, b):
                d_x[:, d] = grad[:, d] @ w[l]
                d_w[l] += grad[:, d].mT @ x[:, d]
        d_b = grad[:, 0].sum(0)
    else:
        # the stored z is what the activation's derivative is taken at
        s_z = grad
        if s["z"] is not None:
            z = s["z"].double().requires_grad_()
            f = act[case["act"]](z) if op == "linear_bwd" else act[case["act"]](z[:, 0]) * z[:, 1]
            s_z, = torch.autograd.grad(f, z, grad)
        s_z = s_z.reshape(case["rows"], -1)
        w2 = w.view(-1, case["inner"])
        d_x, d_w, d_b = s_z @ w2, (s_z.mT @ x).view(w.shape), s_z.sum(0)
        if op == "gated_bwd":
            d_b = d_b.view(2, -1)
    out = {"d_x": d_x, "d_w": d_w}
    return {**out, "d_bias": d_b} if case["bias"] else out
