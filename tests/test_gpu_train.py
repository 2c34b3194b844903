"""The training-step operators (include/convtp_train.h) on the GPU against plain
float64 forms on the CPU.

Tolerances are derived, not fitted.  An output is rounded once to its type
(unit roundoff U: 2^-24, 2^-8, 2^-11 for float32, bfloat16, float16; half the
smallest subnormal below the normal range) from a value computed in float32.
That value's error is at most K 2^-24 S, where S is the same expression with
every term replaced by its absolute value, and K counts the roundings a value
passes through:

* a lookup: one product (K = 2);
* a sum over tokens or rows: one rounding a term at most (K = terms + 8);
* a norm: a lane sums up to 64 squares, then a tree of at most 6 + 16 steps;
  the gradient passes through two such sums and some 20 products (K = 256).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
EPS32 = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def ctp(dev):
    import tensor_product_message_amd as t
    return t


def close(name, got, ref, S, K, dtype=None):
    dtype = dtype or got.dtype
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    tol = U[dtype] * ref.abs() * (1 + 2.0 ** -10) + TINY[dtype] + K * EPS32 * S * (1 + U[dtype])
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst ratio "
                           f"{float((err / tol.clamp(min=1e-300)).max()):.3f}, err {float(err.max()):.3e}")


def tell(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


# ---------------------------------------------------------------- embedding


def draw_tokens(g, n, v, skew, pad):
    t = (torch.rand(n, generator=g).pow(skew) * v).long().clamp(max=max(v - 1, 0))
    if pad:
        bad = torch.tensor([-1, v, v + 7, -2 ** 31 + 5, 2 ** 31 - 1])
        where = torch.rand(n, generator=g) < pad
        t = torch.where(where, bad[torch.randint(0, 5, (n,), generator=g)], t)
    return t


EMBED_SHAPES = [  # tokens, rows, channels, skew, share of padding
    (0, 5, 8, 1, 0), (1, 1, 1, 1, 0), (7, 3, 1, 1, 0.3), (64, 100, 16, 1, 0.1), (257, 1000, 33, 2, 0.2),
    (1503, 100, 128, 6, 0.1), (1025, 1023, 7, 1, 0), (3000, 70001, 130, 3, 0.05), (130, 5, 2051, 1, 0.1),
    (5, 9, 4099, 1, 0), (64, 2, 64, 1, 1.0), (2049, 1024, 24, 1, 0.01),
]


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,c,skew,pad", EMBED_SHAPES)
def test_embed_fwd(ctp, dev, n, v, c, skew, pad, dtype, index):
    g = gen(n + v + c)
    table, tok, scale = normal(g, (v, c), dtype), draw_tokens(g, n, v, skew, pad), 1.7
    tell("embed_fwd", n, v, c, dtype, index)
    out = ctp.embed_fwd(table.to(dev), tok.to(index).to(dev), scale)
    valid = (tok >= 0) & (tok < v)
    ref = torch.zeros(n, c, dtype=torch.float64)
    ref[valid] = float(np.float32(scale)) * table.double()[tok[valid]]
    assert out.dtype == dtype
    close("out", out, ref, ref.abs(), 2)


def embed_bwd_ref(grad, tok, v, scale):
    valid = (tok >= 0) & (tok < v)
    ref, S = (torch.zeros(v, grad.shape[1], dtype=torch.float64) for _ in range(2))
    ref.index_add_(0, tok[valid], grad.double()[valid])
    S.index_add_(0, tok[valid], grad.double()[valid].abs())
    scale = float(np.float32(scale))
    most = int(torch.bincount(tok[valid], minlength=1).max()) if valid.any() else 0
    return ref * scale, S * abs(scale), most + 8


EMBED_BWD_SHAPES = EMBED_SHAPES + [
    (5000, 1, 40, 1, 0), (5000, 70000, 36, 40, 0), (20000, 3, 8, 1, 0.3), (140001, 119, 20, 3, 0.1),
    (70001, 66000, 12, 4, 0), (3000, 1100001, 3, 1, 0), (66000, 2000, 9, 2, 0), (16, 1, 8, 1, 0), (17, 1, 8, 1, 0),
    (33, 2, 8, 9, 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,c,skew,pad", EMBED_BWD_SHAPES)
def test_embed_bwd(ctp, dev, n, v, c, skew, pad, dtype):
    g = gen(n + v + c)
    grad, tok, scale = normal(g, (n, c), dtype), draw_tokens(g, n, v, skew, pad), -0.6
    index = torch.int32 if n % 2 else torch.int64
    tell("embed_bwd", n, v, c, dtype, index)
    ref, S, K = embed_bwd_ref(grad, tok, v, scale)
    grad_d, tok_d = grad.to(dev), tok.to(index).to(dev)
    got = ctp.embed_bwd(grad_d, tok_d, v, scale)
    assert got.dtype == dtype
    close("d_table", got, ref, S, K)
    again = ctp.embed_bwd(grad_d, tok_d, v, scale)
    assert torch.equal(got, again), "not the same bits twice"
    if dtype != torch.float32:
        close("d_table f32", ctp.embed_bwd(grad_d, tok_d, v, scale, dtype=torch.float32), ref, S, K)


def test_embed_strides_shapes_and_outputs(ctp, dev):
    g = gen(5)
    wide = normal(g, (50, 41), torch.float32).to(dev)
    table = wide[:, 3:36]                       # 33 of 41 values a row, from an odd place
    tok = torch.randint(-1, 51, (4, 9), generator=g)
    out = torch.full((4, 9, 33), float("nan"), device=dev)
    assert ctp.embed_fwd(table, tok.to(dev), 1.0, out=out) is out
    ref = table.cpu()[tok.clamp(0, 49)] * ((tok >= 0) & (tok < 50))[..., None]
    assert torch.equal(out.cpu(), ref)
    grads = normal(g, (36, 50), torch.float32).to(dev)
    gout = grads[:, 5:38]
    dwide = torch.full((50, 64), 7.0, device=dev)
    d = dwide[:, 1:34]
    ctp.embed_bwd(gout, tok.reshape(-1).to(dev), 50, out=d)
    ref, S, K = embed_bwd_ref(gout.cpu(), tok.reshape(-1), 50, 1.0)
    close("d", d, ref, S, K)
    assert bool((dwide[:, 0] == 7).all()) and bool((dwide[:, 34:] == 7).all())


def test_embed_autograd_twice(ctp, dev):
    g = gen(6)
    table = normal(g, (11, 5), torch.float32).to(dev).requires_grad_()
    tok = torch.tensor([0, 3, 3, -1, 10, 11], device=dev)
    a = normal(g, (6, 5), torch.float32).to(dev)
    out = ctp.embed(table, tok, 2.0)
    (d,) = torch.autograd.grad((out.square() * a).sum(), table, create_graph=True)
    valid = ((tok >= 0) & (tok < 11)).cpu()
    t64 = table.detach().cpu().double().requires_grad_()
    o64 = 2.0 * t64[tok.cpu()[valid]]
    (d64,) = torch.autograd.grad((o64.square() * a.cpu().double()[valid]).sum(), t64, create_graph=True)
    close("d", d, d64.detach(), d64.detach().abs(), 40)
    (dd,) = torch.autograd.grad(d.square().sum(), table)
    (dd64,) = torch.autograd.grad(d64.square().sum(), t64)
    assert torch.allclose(dd.cpu().double(), dd64, rtol=1e-5, atol=1e-5 * float(dd64.abs().max()))


# ---------------------------------------------------------------- norms


def degrees(lmax):
    return torch.tensor([l for l in range(lmax + 1) for _ in range(2 * l + 1)])


def norm_ref(h, r, w_post, w_pre, gate, alpha, eps, lmax, grad_r=None, grad_u=None):
    """float64 forward (grad_* None) or backward from the formulas, with the absolute-term bounds S: everything as
    [n, D, C] / [1 or n, L, C].  For the backward r is r'."""
    l = degrees(lmax)
    D, C = r.shape[1:]
    b = (1.0 / ((lmax + 1) * (2 * l + 1).double() * C))[:, None]
    per = lambda w: torch.ones(1, D, C, dtype=torch.float64) if w is None else w[:, l]  # noqa: E731
    stat = lambda x: ((x.square() * b).sum((1, 2), keepdim=True) + eps).rsqrt()  # noqa: E731
    fold = lambda x: torch.zeros(x.shape[0], lmax + 1, C, dtype=torch.float64).index_add_(1, l, x)  # noqa: E731
    W1, W2, G = per(w_post), per(w_pre), alpha * per(gate)
    s1 = None if h is None else (stat(h) if w_post is not None else torch.ones(len(h), 1, 1, dtype=torch.float64))
    if grad_r is None and grad_u is None:
        add = torch.zeros_like(r) if h is None else G * W1 * h * s1
        rp, Sr = r + add, r.abs() + add.abs()
        s2 = stat(rp)
        return dict(r=(rp, Sr), u=(rp * s2 * W2, W2.abs() * s2 * (Sr + rp.abs())))
    z = torch.zeros_like(r)
    gr, gu = (z if grad_r is None else grad_r), (z if grad_u is None else grad_u)
    s2 = stat(r) if w_pre is not None else torch.zeros(len(r), 1, 1, dtype=torch.float64)
    A = W2 * gu
    pull = lambda s, a, x: s ** 3 * (a * x).sum((1, 2), keepdim=True) * b * x  # noqa: E731
    d = gr + s2 * A - pull(s2, A, r)
    Sd = gr.abs() + s2 * A.abs() + pull(s2, A.abs(), r.abs())
    out = dict(d_r=(d, Sd))
    if w_pre is not None:
        t = gu * r * s2
        out["d_w_pre"] = (fold(t).sum(0), fold(t.abs()).sum(0))
    if h is None:
        return out
    dy, Sdy = G * d, G.abs() * Sd
    B, SB = dy * W1, Sdy * W1.abs()
    if w_post is not None:
        out["d_h"] = (s1 * B - pull(s1, B, h), s1 * SB + pull(s1, SB, h.abs()))
        out["d_w_post"] = (fold(dy * h * s1).sum(0), fold(Sdy * h.abs() * s1).sum(0))
    else:
        out["d_h"] = (B, SB)
    if gate is not None:
        dg, Sdg = fold(alpha * d * h * s1 * W1), fold(abs(alpha) * Sd * h.abs() * s1 * W1.abs())
        shared = gate.shape[0] == 1
        out["d_gate"] = (dg.sum(0), Sdg.sum(0)) if shared else (dg, Sdg)
    return out


NORM_SHAPES = [  # rows, lmax, channels
    (0, 0, 8), (1, 0, 1), (3, 0, 7), (5, 0, 64), (129, 0, 33), (65, 0, 250), (1100, 0, 130), (40, 0, 1003),
    (33, 0, 2048), (9, 0, 4096), (7, 0, 8191), (5, 0, 16384), (64, 1, 16), (31, 1, 5), (70, 2, 33), (1503, 3, 8),
    (90, 3, 128), (3, 3, 1024), (4, 2, 1820), (17, 3, 301),
]


def norm_case(rows, lmax, c, dtype, param, kind, seed):
    g = gen(seed)
    D, L = (lmax + 1) ** 2, lmax + 1
    row = (rows, c) if lmax == 0 else (rows, D, c)
    per = (c,) if lmax == 0 else (L, c)
    t = dict(h=normal(g, row, dtype, 3.0), r=normal(g, row, dtype), grad_r=normal(g, row, dtype),
             grad_u=normal(g, row, dtype), w_post=normal(g, per, param, 0.2, 1.0), w_pre=normal(g, per, param, 0.2, 1.0),
             gate={"none": None, "channel": normal(g, per, param, 0.5, 0.5),
                   "row": normal(g, (rows, *per), dtype, 0.5, 0.5)}[kind])
    wide = {k: None if v is None else v.double().reshape(-1, D if k in ("h", "r", "grad_r", "grad_u") else L, c)
            for k, v in t.items()}
    return t, wide


@pytest.mark.parametrize("kind", ["none", "channel", "row"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,lmax,c", NORM_SHAPES)
def test_norm_residual(ctp, dev, rows, lmax, c, dtype, kind):
    param = torch.float32 if (rows + c) % 2 else dtype
    t, w = norm_case(rows, lmax, c, dtype, param, kind, rows + lmax + c)
    tell("norm", rows, lmax, c, dtype, param, kind)
    alpha, eps = 0.5, 1e-6
    d = {k: None if v is None else v.to(dev) for k, v in t.items()}
    r_out, u = ctp.norm_residual_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], alpha, eps, lmax)
    ref = norm_ref(w["h"], w["r"], w["w_post"], w["w_pre"], w["gate"], alpha, eps, lmax)
    for name, got in (("r", r_out), ("u", u)):
        assert got.shape == t["r"].shape and got.dtype == dtype
        close(name, got.reshape(ref[name][0].shape), *ref[name], 256)
    args = (d["grad_r"], d["grad_u"], d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], alpha, eps, lmax)
    got = dict(zip(("d_h", "d_r", "d_w_post", "d_w_pre", "d_gate"), ctp.norm_residual_bwd(*args)))
    ref = norm_ref(w["h"], w["r"], w["w_post"], w["w_pre"], w["gate"], alpha, eps, lmax, w["grad_r"], w["grad_u"])
    assert (got["d_gate"] is None) == (kind == "none")
    for name, (x, S) in ref.items():
        assert got[name].dtype == (param if name.startswith("d_w") or (name == "d_gate" and kind == "channel") else dtype)
        close(name, got[name].reshape(x.shape), x, S, 256 + (rows * (2 * lmax + 1) if x.shape[0] != rows or name.startswith("d_w") else 0))
    again = dict(zip(got, ctp.norm_residual_bwd(*args)))
    assert all(got[k] is None or torch.equal(got[k], again[k]) for k in got), "not the same bits twice"


@pytest.mark.parametrize("lmax,c", [(0, 72), (2, 19)])
@pytest.mark.parametrize("parts", ["no h", "no w_post", "no w_pre", "no w_post gate", "no grad_r", "no grad_u"])
def test_norm_parts(ctp, dev, parts, lmax, c):
    rows, dtype = 77, torch.bfloat16
    kind = "row" if "gate" in parts else "channel"
    t, w = norm_case(rows, lmax, c, dtype, dtype, "none" if parts == "no h" else kind, 3)
    gone = {"no h": ["h", "w_post"], "no w_post": ["w_post"], "no w_pre": ["w_pre", "grad_u"],
            "no w_post gate": ["w_post"], "no grad_r": ["grad_r"], "no grad_u": ["grad_u"]}[parts]
    for k in gone:
        t[k] = w[k] = None
    tell("norm parts", parts, lmax, c)
    d = {k: None if v is None else v.to(dev) for k, v in t.items()}
    if "grad" not in parts:
        r_out, u = ctp.norm_residual_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 0.7, 1e-5, lmax)
        ref = norm_ref(w["h"], w["r"], w["w_post"], w["w_pre"], w["gate"], 0.7, 1e-5, lmax)
        if parts == "no h":
            assert r_out is d["r"]
        else:
            close("r", r_out.reshape(ref["r"][0].shape), *ref["r"], 256)
        if parts == "no w_pre":
            assert u is None
        else:
            close("u", u.reshape(ref["u"][0].shape), *ref["u"], 256)
    got = dict(zip(("d_h", "d_r", "d_w_post", "d_w_pre", "d_gate"),
                   ctp.norm_residual_bwd(d["grad_r"], d["grad_u"], d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"],
                                         0.7, 1e-5, lmax)))
    ref = norm_ref(w["h"], w["r"], w["w_post"], w["w_pre"], w["gate"], 0.7, 1e-5, lmax, w["grad_r"], w["grad_u"])
    for name in got:
        assert (got[name] is None) == (name not in ref), name
    for name, (x, S) in ref.items():
        close(name, got[name].reshape(x.shape), x, S, 256 + rows * (2 * lmax + 1))


def test_norm_strides_and_in_place(ctp, dev):
    g = gen(9)
    rows, c = 50, 37
    t, w = norm_case(rows, 0, c, torch.float16, torch.float16, "row", 9)
    d = {k: v.to(dev) for k, v in t.items()}

    def spread(x, width, at):       # the same rows inside a wider array
        big = torch.full((rows, width), 3.0, dtype=x.dtype, device=dev)
        big[:, at:at + c] = x
        return big[:, at:at + c]
    s = {k: spread(d[k], 41 + 2 * i, i) for i, k in enumerate(("h", "r", "gate", "grad_r", "grad_u"))}
    r_out, u = ctp.norm_residual_fwd(s["h"], s["r"], d["w_post"], d["w_pre"], s["gate"], 0.5)
    r2, u2 = ctp.norm_residual_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 0.5)
    assert torch.equal(r_out, r2) and torch.equal(u, u2)
    a = ctp.norm_residual_bwd(s["grad_r"], s["grad_u"], s["h"], s["r"], d["w_post"], d["w_pre"], s["gate"], 0.5)
    b = ctp.norm_residual_bwd(d["grad_r"], d["grad_u"], d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 0.5)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    own = d["r"].clone()
    r3, u3 = ctp.norm_residual_fwd(d["h"], own, d["w_post"], d["w_pre"], d["gate"], 0.5, out=(own, None))
    assert r3 is own and torch.equal(own, r2) and torch.equal(u3, u2)


def test_norm_special_rows(ctp, dev):
    """Rows of zeros, of very large values and with a NaN: finite where the formula is, and no row touches another."""
    rows, c = 6, 96
    t, w = norm_case(rows, 0, c, torch.float32, torch.float32, "none", 4)
    t["h"][1] = 0.0
    t["r"][1] = 0.0
    t["h"][2] *= 1e15
    t["r"][2] *= 1e15
    for k in t:
        w[k] = None if t[k] is None else t[k].double().reshape(-1, 1, c)
    t["h"][4, 7] = float("nan")
    d = {k: None if v is None else v.to(dev) for k, v in t.items()}
    r_out, u = ctp.norm_residual_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], None, 1.0)
    ref = norm_ref(w["h"], w["r"], w["w_post"], w["w_pre"], None, 1.0, 1e-6, 0)
    keep = [0, 1, 2, 3, 5]
    for name, got in (("r", r_out), ("u", u)):
        close(name, got[keep], *(x[keep, 0] for x in ref[name]), 256)
        assert got[4].isnan().all()
    d_h, d_r, *_ = ctp.norm_residual_bwd(d["grad_r"], d["grad_u"], d["h"], d["r"], d["w_post"], d["w_pre"], None, 1.0)
    ref = norm_ref(w["h"], w["r"], w["w_post"], w["w_pre"], None, 1.0, 1e-6, 0, w["grad_r"], w["grad_u"])
    close("d_h", d_h[keep], *(x[keep, 0] for x in ref["d_h"]), 256)
    close("d_r", d_r, *(x[:, 0] for x in ref["d_r"]), 256)
    assert d_h[4].isnan().all()


@pytest.mark.parametrize("lmax,c,kind", [(0, 40, "row"), (2, 12, "channel"), (1, 9, "row"), (3, 6, "none")])
def test_norm_gradient_against_differences(ctp, dev, lmax, c, kind):
    """Directional derivatives of <p, r'> + <q, u> by central differences of the float64 forward (step 1e-5: their
    error is of order 1e-9) against the kernel's float32 gradients (some 1e-5 at these sizes)."""
    rows = 23
    t, w = norm_case(rows, lmax, c, torch.float32, torch.float32, kind, 12)
    d = {k: None if v is None else v.to(dev).requires_grad_(k not in ("grad_r", "grad_u")) for k, v in t.items()}
    r_out, u = ctp.norm_residual(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 0.5, 1e-6, lmax)
    loss = (r_out * d["grad_r"]).sum() + (u * d["grad_u"]).sum()
    names = [k for k in ("h", "r", "w_post", "w_pre", "gate") if d[k] is not None]
    grads = dict(zip(names, torch.autograd.grad(loss, [d[k] for k in names])))
    g = gen(13)

    def value(x):
        o = norm_ref(x["h"], x["r"], x["w_post"], x["w_pre"], x["gate"], 0.5, 1e-6, lmax)
        return float((o["r"][0] * w["grad_r"]).sum() + (o["u"][0] * w["grad_u"]).sum())
    for k in names:
        way = torch.randn(w[k].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        diff = (value({**w, k: w[k] + step * way}) - value({**w, k: w[k] - step * way})) / (2 * step)
        got = grads[k].double().cpu().reshape(way.shape)
        size = float(got.norm() * way.norm())
        assert abs(float((got * way).sum()) - diff) <= 1e-5 * size, (k, float((got * way).sum()), diff)


# ---------------------------------------------------------------- clipping


def clip_ref(ts, max_norm, eps=1e-6):
    norm = float(torch.cat([t.double().reshape(-1) for t in ts]).norm()) if ts else 0.0
    f = min(1.0, max_norm / (norm + eps))
    return norm, [t.double() * f for t in ts]


SIZES = [0, 1, 3, 7, 8, 255, 256, 16383, 16384, 16385, 100003]


@pytest.mark.parametrize("max_norm", [0.0, 0.25, 1e9])
@pytest.mark.parametrize("dtype", DTYPES + ["mixed"])
def test_clip(ctp, dev, dtype, max_norm):
    g = gen(21)
    kinds = DTYPES if dtype == "mixed" else [dtype]
    ts = [normal(g, (s,), kinds[i % len(kinds)], 0.3) for i, s in enumerate(SIZES)] + [normal(g, (3, 5, 7), kinds[0])]
    tell("clip", dtype, max_norm)
    norm, ref = clip_ref(ts, max_norm)
    d = [t.to(dev) for t in ts]
    out, got = ctp.clip_grad_norm(d, max_norm)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(float(got) - norm) <= 2 ** -23 * norm
    assert abs(float(ctp.grad_norm(d)) - norm) <= 2 ** -23 * norm
    for k, (o, x) in enumerate(zip(out, ref)):
        close(f"out {k}", o, x, x.abs(), 8)
        assert torch.equal(d[k].cpu(), ts[k]), "an input changed"
    again, got2 = ctp.clip_grad_norm(d, max_norm)
    assert torch.equal(got, got2) and all(torch.equal(a, b) for a, b in zip(out, again))
    ctp.clip_grad_norm(d, max_norm, out=d)
    assert all(torch.equal(a, b) for a, b in zip(d, out))


def test_clip_many_tensors_and_odd_places(ctp, dev):
    g = gen(22)
    sizes = [int(x) for x in torch.randint(0, 900, (300,), generator=g)]
    ts = [normal(g, (s,), torch.bfloat16) for s in sizes]
    norm, ref = clip_ref(ts, 3.0)
    total = sum(sizes) + 1
    flat_in, flat_out = (torch.zeros(total, dtype=torch.bfloat16, device=dev) for _ in range(2))
    d, out, at = [], [], 1                # neither side begins on 16 bytes
    for t in ts:
        d.append(flat_in[at:at + t.numel()].copy_(t))
        out.append(flat_out[at:at + t.numel()])
        at += t.numel()
    got, n = ctp.clip_grad_norm(d, 3.0, out=out)
    assert abs(float(n) - norm) <= 2 ** -23 * norm
    for o, x in zip(got, ref):
        close("out", o, x, x.abs(), 8)
    assert float(flat_out[0]) == 0.0


def test_clip_special_values(ctp, dev):
    big = torch.full((5000,), 1e30, device=dev)          # squares leave float32, not float64
    out, n = ctp.clip_grad_norm([big], 1.0)
    ref = 1e30 * 5000 ** 0.5
    assert abs(float(n) - ref) <= 2e-7 * ref
    close("big", out[0], big.double().cpu() / ref, big.double().cpu() / ref, 8)
    small = torch.full((5000,), 1e-30, device=dev)
    out, n = ctp.clip_grad_norm([small], 1.0)
    assert torch.equal(out[0], small) and abs(float(n) - 1e-30 * 5000 ** 0.5) <= 2e-7 * 1e-28
    zero = [torch.zeros(0, device=dev), torch.zeros(9, device=dev)]
    out, n = ctp.clip_grad_norm(zero, 1.0)
    assert float(n) == 0.0 and float(out[1].abs().sum()) == 0.0
    assert float(ctp.grad_norm(zero[:1])) == 0.0
    for bad, factor in ((float("inf"), 0.0), (float("nan"), float("nan"))):
        x = torch.ones(300, device=dev)
        x[17] = bad
        out, n = ctp.clip_grad_norm([x], 1.0)
        want = x * factor
        assert torch.equal(n.isnan(), torch.tensor(bad != bad, device=dev)) and (bad != bad or float(n) == bad)
        assert torch.equal(out[0].isnan(), want.isnan()) and torch.equal(out[0].nan_to_num(5.0), want.nan_to_num(5.0))


# ---------------------------------------------------------------- streams, graphs, refusals


def test_on_another_stream_and_in_a_graph(ctp, dev):
    g = gen(31)
    tok = torch.randint(-1, 60, (400,), generator=g).to(dev)
    grad = normal(g, (400, 48), torch.float32).to(dev)
    table = normal(g, (60, 48), torch.float32).to(dev)
    t, _ = norm_case(200, 0, 48, torch.float32, torch.float32, "channel", 31)
    n = {k: v.to(dev) for k, v in t.items()}

    def step():
        x = ctp.embed_fwd(table, tok, 2.0)
        d = ctp.embed_bwd(grad, tok, 60, 2.0)
        f = ctp.norm_residual_fwd(n["h"], n["r"], n["w_post"], n["w_pre"], n["gate"], 0.5)
        b = ctp.norm_residual_bwd(n["grad_r"], n["grad_u"], n["h"], f[0], n["w_post"], n["w_pre"], n["gate"], 0.5)
        c, norm = ctp.clip_grad_norm([d, *b], 0.5)
        return [x, d, *f, *b, *c, norm]
    eager = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for k in range(4):
        tok.copy_(torch.randint(-1, 60, (400,), generator=g))
        grad.normal_()
        n["h"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        fresh = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, fresh)), k


def test_refusals(ctp, dev):
    f = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
    ids = torch.zeros(4, dtype=torch.int64, device=dev)
    for call, err in (
            (lambda: ctp.embed_fwd(f(3, 4, dtype=torch.float64), ids), ValueError),
            (lambda: ctp.embed_fwd(f(3, 4), f(4)), ValueError),
            (lambda: ctp.embed_fwd(f(3), ids), ValueError),
            (lambda: ctp.embed_fwd(f(4, 3).t(), ids), ValueError),
            (lambda: ctp.embed_fwd(f(3, 4), ids.cpu()), ValueError),
            (lambda: ctp.embed_fwd(f(3, 4), f(8).long()[::2]), ValueError),
            (lambda: ctp.embed_fwd(f(3, 4), ids, out=f(4, 5)), ValueError),
            (lambda: ctp.embed_bwd(f(5, 4), ids, 3), ValueError),
            (lambda: ctp.embed_bwd(f(1, 4).expand(4, 4), ids, 3), ValueError),
            (lambda: ctp.embed_bwd(f(4, 4), ids, 3, dtype=torch.bfloat16), ctp.ConvTPError),
            (lambda: ctp.embed_bwd(f(4, 4), ids, 3, workspace=f(1)), ctp.ConvTPError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 9), f(8), f(8)), ValueError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 8), f(9), f(8)), ValueError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 8), f(8).half(), f(8).half()), ValueError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 8), f(8), f(8).half()), ValueError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 8), f(8), f(8), f(3, 8)), ValueError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 8), f(8), f(8), lmax=1), ValueError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 8), f(8), f(8), lmax=4), ValueError),
            (lambda: ctp.norm_residual_fwd(f(2, 8), f(2, 8), f(8), f(8), eps=-1.0), ctp.ConvTPError),
            (lambda: ctp.norm_residual_fwd(None, f(2, 8), None, None), ctp.ConvTPError),
            (lambda: ctp.norm_residual_fwd(None, f(2, 8), f(8), f(8)), ctp.ConvTPError),
            (lambda: ctp.norm_residual_fwd(f(1, 16385), f(1, 16385), None, f(16385)), ctp.ConvTPError),
            (lambda: ctp.norm_residual_bwd(None, None, f(2, 8), f(2, 8), f(8), f(8)), TypeError),
            (lambda: ctp.norm_residual_bwd(f(2, 8), f(2, 8), f(2, 8), f(2, 8), f(8), None), ValueError),
            (lambda: ctp.clip_grad_norm([], 1.0), ValueError),
            (lambda: ctp.clip_grad_norm([f(4), f(4).double()], 1.0), ValueError),
            (lambda: ctp.clip_grad_norm([f(4, 4).t()], 1.0), ValueError),
            (lambda: ctp.clip_grad_norm([f(4)], 1.0, out=[f(5)]), ValueError),
            (lambda: ctp.clip_grad_norm([f(4)], -1.0), ctp.ConvTPError),
            (lambda: ctp.clip_grad_norm([f(4)], float("nan")), ctp.ConvTPError)):
        with pytest.raises(err):
            call()


# ---------------------------------------------------------------- long runs, long arrays, the example


@pytest.mark.parametrize("n,v,c,dtype,same", [
    (9000, 2, 2048, torch.bfloat16, 0.7),       # one row a workgroup, a run over hundreds of spans
    (30000, 2000, 64, torch.float32, 1.0),      # one token in a large table
    (40000, 3, 5, torch.float16, 0.5),          # many rows a workgroup
    (20000, 900, 260, torch.float32, 0.02),     # runs that end and begin all over the spans
])
def test_embed_bwd_long_runs(ctp, dev, n, v, c, dtype, same):
    g = gen(n)
    tok = torch.randint(0, v, (n,), generator=g)
    tok[torch.rand(n, generator=g) < same] = v - 1
    grad = normal(g, (n, c), dtype)
    tell("embed_bwd runs", n, v, c, dtype)
    ref, S, K = embed_bwd_ref(grad, tok, v, 1.0)
    got = ctp.embed_bwd(grad.to(dev), tok.to(dev), v)
    close("d_table", got, ref, S, K)


def test_embed_bwd_every_run_length(ctp, dev):
    """Runs of 1, 2, 3 .. tokens: every place of a run's ends in chunks and spans."""
    for c, dtype in ((24, torch.float32), (200, torch.float32), (1030, torch.bfloat16)):
        lengths = torch.arange(1, 180)
        tok = torch.repeat_interleave(torch.arange(len(lengths)), lengths)
        g = gen(c)
        tok = tok[torch.randperm(len(tok), generator=g)]
        grad = normal(g, (len(tok), c), dtype)
        ref, S, K = embed_bwd_ref(grad, tok, len(lengths) + 3, 1.0)
        close("d_table", ctp.embed_bwd(grad.to(dev), tok.to(dev), len(lengths) + 3), ref, S, K)


def test_offsets_beyond_32_bits(ctp, dev):
    """Tables, features and gradients of more than 2^31 elements: sampled rows against the definition."""
    v, c = 1_100_000, 2048
    table = torch.empty((v, c), dtype=torch.bfloat16, device=dev)
    for k in range(0, v, 100_000):
        table[k:k + 100_000].normal_()
    tok = torch.tensor([0, v - 1, v // 2, 1_048_577, -1], device=dev)
    tell("large embed")
    out = ctp.embed_fwd(table, tok, 1.0)
    assert torch.equal(out[:4], table[tok[:4]]) and float(out[4].abs().sum()) == 0.0
    grad = torch.randn((5, c), device=dev).to(torch.bfloat16)
    ctp.embed_bwd(grad, tok, v, out=table)
    assert torch.equal(table[tok[:4]], grad[:4])
    assert int((table != 0).any(1).sum()) == 4
    del out
    rows = table.view(137_500, 16384)                 # the same memory as wide rows
    rows.normal_()
    h = rows.clone()
    w = torch.ones(16384, dtype=torch.bfloat16, device=dev)
    tell("large norm")
    r_out, u = ctp.norm_residual_fwd(h, rows, w, w)
    at = [0, 70_000, 131_073, 137_499]
    one = ctp.norm_residual_fwd(h[at], rows[at], w, w)
    assert torch.equal(r_out[at], one[0]) and torch.equal(u[at], one[1])
    d_h, d_r, *_ = ctp.norm_residual_bwd(u, h, h, r_out, w, w)
    one = ctp.norm_residual_bwd(u[at], h[at], h[at], r_out[at], w, w)
    assert torch.equal(d_h[at], one[0]) and torch.equal(d_r[at], one[1])
    del d_h, d_r, u, r_out
    tell("large clip")
    flat = h.view(-1)
    (clipped,), norm = ctp.clip_grad_norm([flat], 1.0)
    total = sum(float(flat[k:k + 2 ** 28].double().square().sum()) for k in range(0, flat.numel(), 2 ** 28)) ** 0.5
    assert abs(float(norm) - total) <= 1e-6 * total
    factor = np.float32(1.0) / (np.float32(float(norm)) + np.float32(1e-6))
    for k in (0, 2 ** 31 - 5, 2 ** 31 + 3, flat.numel() - 9):
        assert torch.equal(clipped[k:k + 9], (flat[k:k + 9].float() * float(factor)).to(torch.bfloat16))


def test_example_trains(dev):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_energy
    losses, norms = train_energy.train(steps=30, atoms=200, channels=16, lmax=2, log=None)
    assert all(np.isfinite(losses)) and all(np.isfinite(norms))
    assert losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])


# ---------------------------------------------------------------- the norms' second backward pass


def norm_forward64(h, r, w_post, w_pre, gate, alpha, eps, lmax):
    """The definition, differentiable: (r', u) of [n, D, C] features and [1 or n, L, C] parameters."""
    l = degrees(lmax)
    b = (1.0 / ((lmax + 1) * (2 * l + 1).double() * r.shape[2]))[:, None]
    stat = lambda x: ((x.square() * b).sum((1, 2), keepdim=True) + eps).rsqrt()  # noqa: E731
    if h is not None:
        y = h if w_post is None else h * stat(h) * w_post[:, l]
        r = r + alpha * (y if gate is None else y * gate[:, l])
    return r, None if w_pre is None else r * stat(r) * w_pre[:, l]


SECOND = ("g_grad_r", "g_grad_u", "g_h", "g_r", "g_w_post", "g_w_pre", "g_gate")


def second_ref(w, alpha, eps, lmax, Q, P):
    """float64 gradients of <Q, d_h> + <P, d_r> in the first backward's inputs, by differentiating the definition
    twice: r' is a leaf, reached by grad_r directly and by grad_u through the second norm."""
    leaf = {k: None if v is None else v.clone().requires_grad_() for k, v in w.items()}
    keys = ("grad_r", "grad_u", "h", "r", "w_post", "w_pre", "gate")
    rp = leaf["r"]
    zero = torch.zeros_like(rp)
    d = zero if leaf["grad_r"] is None else leaf["grad_r"]
    if leaf["w_pre"] is not None and leaf["grad_u"] is not None:
        u = norm_forward64(None, rp, None, leaf["w_pre"], None, alpha, eps, lmax)[1]
        d = d + torch.autograd.grad(u, rp, leaf["grad_u"], create_graph=True)[0]
    total = (d * P).sum() if P is not None else 0.0 * d.sum()
    if leaf["h"] is not None and Q is not None:
        out = norm_forward64(leaf["h"], zero, leaf["w_post"], None, leaf["gate"], alpha, eps, lmax)[0]
        d_h, = torch.autograd.grad(out, leaf["h"], d, create_graph=True)
        total = total + (d_h * Q).sum()
    wants = [leaf[k] for k in keys if leaf[k] is not None]
    got = iter(torch.autograd.grad(total, wants, allow_unused=True))
    res = {}
    for k, name in zip(keys, SECOND):
        if leaf[k] is not None:
            g = next(got)
            res[name] = torch.zeros_like(leaf[k]) if g is None else g
    return res


def second_bounds(w, alpha, eps, lmax, Q, P):
    """S of every output: the formulas with every term replaced by its absolute value."""
    l = degrees(lmax)
    some = next(w[k] for k in ("h", "grad_r", "r") if w[k] is not None)
    n, D, C = some.shape
    zero = torch.zeros(n, D, C, dtype=torch.float64)
    b = (1.0 / ((lmax + 1) * (2 * l + 1).double() * C))[:, None]
    mag = lambda x: zero if x is None else x.abs()  # noqa: E731
    per = lambda x: torch.ones(1, D, C, dtype=torch.float64) if x is None else x.abs()[:, l]  # noqa: E731
    dot = lambda x, y: (x * y).sum((1, 2), keepdim=True)  # noqa: E731
    stat = lambda x: ((x.square() * b).sum((1, 2), keepdim=True) + eps).rsqrt()  # noqa: E731
    fold = lambda x: torch.zeros(x.shape[0], lmax + 1, C, dtype=torch.float64).index_add_(1, l, x)  # noqa: E731
    P, Q, h, r, gr, gu = (mag(x) for x in (P, Q, w["h"], w["r"], w["grad_r"], w["grad_u"]))
    w1, w2, g = per(w["w_post"]), per(w["w_pre"]), abs(alpha) * per(w["gate"])
    s1 = stat(h) if w["w_post"] is not None else torch.ones(n, 1, 1, dtype=torch.float64)
    s2 = stat(r) if w["w_pre"] is not None else torch.zeros(n, 1, 1, dtype=torch.float64)
    hs, rs, A = s1 * h, s2 * r, w2 * gu
    ar, qh = dot(A, rs), dot(b * Q, hs) if w["w_post"] is not None else torch.zeros(n, 1, 1, dtype=torch.float64)
    d, EB = gr + s2 * (A + b * rs * ar), s1 * (Q + hs * qh)
    Ed, q = P + g * w1 * EB, d * g
    B = w1 * q
    bh, er = dot(B, hs), dot(b * Ed, rs)
    EA = s2 * (Ed + rs * er)
    dg = fold(abs(alpha) * d * w1 * EB)
    shared = w["gate"] is None or w["gate"].shape[0] == 1
    return dict(g_grad_r=Ed, g_grad_u=w2 * EA, g_h=s1 ** 2 * (b * (hs * (dot(Q, B) + 3 * qh * bh) + Q * bh) + B * qh),
                g_r=s2 ** 2 * (b * (rs * (dot(Ed, A) + 3 * er * ar) + Ed * ar) + A * er),
                g_w_post=fold(EB * q).sum(0, keepdim=True), g_w_pre=fold(gu * EA).sum(0, keepdim=True),
                g_gate=dg.sum(0, keepdim=True) if shared else dg)


@pytest.mark.parametrize("kind", ["none", "channel", "row"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,lmax,c", [(3, 0, 7), (65, 0, 250), (1100, 0, 130), (33, 0, 2048), (5, 0, 8191),
                                         (3, 0, 16384), (64, 1, 16), (70, 2, 33), (90, 3, 128), (3, 3, 1024)])
def test_norm_second_backward(ctp, dev, rows, lmax, c, dtype, kind):
    """Against double differentiation in float64.  K = 512: a value passes through the first pass's sums and products
    and as many again; sums over rows add one rounding a row."""
    param = torch.float32 if (rows + c) % 2 else dtype
    t, w = norm_case(rows, lmax, c, dtype, param, kind, rows + lmax + c + 7)
    g = gen(rows)
    Q, P = normal(g, t["h"].shape, dtype), normal(g, t["h"].shape, dtype)
    tell("norm second", rows, lmax, c, dtype, param, kind)
    d = {k: None if v is None else v.to(dev) for k, v in t.items()}
    Q64, P64 = (x.double().reshape(w["h"].shape) for x in (Q, P))
    ref, S = second_ref(w, 0.5, 1e-6, lmax, Q64, P64), second_bounds(w, 0.5, 1e-6, lmax, Q64, P64)
    args = (Q.to(dev), P.to(dev), d["grad_r"], d["grad_u"], d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 0.5, 1e-6, lmax)
    got = dict(zip(SECOND, ctp.norm_residual_bwd_bwd(*args)))
    assert (got["g_gate"] is None) == (kind == "none")
    for name, x in ref.items():
        terms = rows * (2 * lmax + 1) if name.startswith("g_w") or (name == "g_gate" and kind == "channel") else 0
        close(name, got[name].reshape(x.shape), x, S[name], 512 + terms)
    again = dict(zip(SECOND, ctp.norm_residual_bwd_bwd(*args)))
    assert all(got[k] is None or torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("parts", ["no h", "no w_post", "no w_pre", "no grad_r", "no grad_u", "no P", "no Q"])
def test_norm_second_backward_parts(ctp, dev, parts):
    rows, lmax, c = 41, 1, 21
    t, w = norm_case(rows, lmax, c, torch.float32, torch.float32, "none" if parts == "no h" else "channel", 8)
    g = gen(8)
    Q, P = (normal(g, t["h"].shape, torch.float32) for _ in range(2))
    for k in {"no h": ["h", "w_post"], "no w_post": ["w_post"], "no w_pre": ["w_pre", "grad_u"],
              "no grad_r": ["grad_r"], "no grad_u": ["grad_u"]}.get(parts, []):
        t[k] = w[k] = None
    Q = None if parts in ("no h", "no Q") else Q
    P = None if parts == "no P" else P
    wide = lambda x: None if x is None else x.double()  # noqa: E731
    ref, S = second_ref(w, 0.7, 1e-5, lmax, wide(Q), wide(P)), second_bounds(w, 0.7, 1e-5, lmax, wide(Q), wide(P))
    d = {k: None if v is None else v.to(dev) for k, v in t.items()}
    to = lambda x: None if x is None else x.to(dev)  # noqa: E731
    got = dict(zip(SECOND, ctp.norm_residual_bwd_bwd(to(Q), to(P), d["grad_r"], d["grad_u"], d["h"], d["r"],
                                                     d["w_post"], d["w_pre"], d["gate"], 0.7, 1e-5, lmax)))
    for name, x in ref.items():
        if parts == "no w_pre" and name == "g_r":
            assert got[name] is None        # r' is not an input then
            continue
        close(name, got[name].reshape(x.shape), x, S[name], 512 + rows * 3)


def test_norm_trains_on_first_gradients(ctp, dev):
    """A loss on the gradient of an energy, differentiated again through autograd, against float64."""
    rows, lmax, c = 30, 2, 10
    t, w = norm_case(rows, lmax, c, torch.float32, torch.float32, "row", 15)
    keys = ("h", "r", "w_post", "w_pre", "gate")

    def loss_grads(x, forward, a, b):
        r_out, u = forward(x["h"], x["r"], x["w_post"], x["w_pre"], x["gate"])
        energy = (u.sin() * a).sum() + (r_out.square() * b).sum()
        f_h, f_r = torch.autograd.grad(energy, (x["h"], x["r"]), create_graph=True)
        return torch.autograd.grad(f_h.square().sum() + (f_r * a).sum(), [x[k] for k in keys])
    x32 = {k: t[k].to(dev).requires_grad_() for k in keys}
    x64 = {k: w[k].clone().requires_grad_() for k in keys}
    got = loss_grads(x32, lambda *p: ctp.norm_residual(*p, 0.5, 1e-6, lmax), t["grad_r"].to(dev), t["grad_u"].to(dev))
    ref = loss_grads(x64, lambda *p: norm_forward64(*p, 0.5, 1e-6, lmax), w["grad_r"], w["grad_u"])
    for k, g, r in zip(keys, got, ref):
        assert float((g.double().cpu().reshape(r.shape) - r).abs().max()) <= 2e-5 * float(r.abs().max()), k
    u = ctp.norm_residual(x32["h"], x32["r"], x32["w_post"], x32["w_pre"], x32["gate"], 0.5, 1e-6, lmax)[1]
    d_w, = torch.autograd.grad(u.sum(), x32["w_pre"], create_graph=True)
    with pytest.raises(NotImplementedError):
        d_w.sum().backward()


def test_second_backward_refusals(ctp, dev):
    f = lambda *s: torch.zeros(s, device=dev)  # noqa: E731
    x, w = f(2, 8), f(8)
    for call, err in ((lambda: ctp.norm_residual_bwd_bwd(None, None, x, x, x, x, w, w), TypeError),
                      (lambda: ctp.norm_residual_bwd_bwd(x, x, x, x, None, x, None, w), ValueError),
                      (lambda: ctp.norm_residual_bwd_bwd(f(2, 9), x, x, x, x, x, w, w), ValueError),
                      (lambda: ctp.norm_residual_bwd_bwd(f(2, 16)[:, ::2], x, x, x, x, x, w, w), ValueError),
                      (lambda: ctp.norm_residual_bwd_bwd(x, x, None, None, x, x, w, w), TypeError)):
        with pytest.raises(err):
            call()


def test_wide_rows_in_a_graph(ctp, dev):
    """Kernels that ask for more than 64 KB of LDS are launched in a capture too."""
    t, _ = norm_case(12, 3, 1024, torch.float32, torch.float32, "row", 2)
    n = {k: v.to(dev) for k, v in t.items()}

    def step():
        args = (n["grad_r"], n["grad_u"], n["h"], n["r"], n["w_post"], n["w_pre"], n["gate"], 0.5, 1e-6, 3)
        return [*ctp.norm_residual_bwd(*args), *ctp.norm_residual_bwd_bwd(n["r"], n["h"], *args)]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        n["h"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,c,skew,pad", [
    (8192, 5000, 40, 3, 0.1), (8192, 200001, 12, 30, 0.0), (8191, 3000, 300, 1, 0.5), (300, 150000, 64, 1, 0.1),
    (8000, 2100, 1100, 60, 0.0), (8193, 5000, 40, 3, 0.1), (100, 2049, 4100, 1, 0.0), (4097, 70000, 9, 2, 0.0),
    (5, 0, 16, 1, 0.0),
])
def test_embed_bwd_few_tokens_large_tables(ctp, dev, n, v, c, skew, pad, dtype):
    g = gen(n + v)
    grad, tok = normal(g, (n, c), dtype), draw_tokens(g, n, v, skew, pad)
    tell("embed_bwd few", n, v, c, dtype)
    ref, S, K = embed_bwd_ref(grad, tok, v, 2.0)
    got = ctp.embed_bwd(grad.to(dev), tok.to(dev), v, 2.0)
    close("d_table", got, ref, S, K)
    assert torch.equal(got, ctp.embed_bwd(grad.to(dev), tok.to(torch.int32).to(dev), v, 2.0))
