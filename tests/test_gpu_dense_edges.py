"""The dense operators on the GPU at sizes and values of which the documentation says something; forms and tolerances
as in test_gpu_dense.py."""
import pytest
import torch

from tests.test_gpu_dense import EPS32, act, close, newton_schulz, normal, sum_error, tell

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def ctp(dev):
    import tensor_product_message_amd as t
    return t


@pytest.mark.parametrize("dtype,rows,inner,outer", [(torch.bfloat16, 70, 16384, 65536), (torch.float16, 200, 32768, 32768)])
def test_gated_matrices_of_2_30_values(ctp, dev, dtype, rows, inner, outer):
    """A column's partner lies 2^31 bytes on: columns of both halves, in the forward and the second backward pass."""
    tell("large gated", dtype, rows, inner, outer)
    g = torch.Generator().manual_seed(1)
    x, u, grad = (normal(g, (rows, n), dtype) for n in (inner, inner, outer))
    bias = normal(g, (2, outer), dtype, 0.5)
    w = torch.empty(2, outer, inner, dtype=dtype, device=dev).normal_(0, inner ** -0.5, generator=torch.Generator(dev).manual_seed(2))
    cols = torch.tensor([0, 1, 31, 32, 63, 64, 127, 128, outer // 2 + 5, outer - 64, outer - 33, outer - 1])
    W = w[:, cols.to(dev)].double().cpu()
    h, z = ctp.gated_linear_fwd(x.to(dev), w, bias.to(dev), keep_z=True)
    e = sum_error(dtype, inner)
    Z = [x.double() @ W[k].T + bias[k, cols].double() for k in (0, 1)]
    ez = [e * (x.double().abs() @ W[k].abs().T + bias[k, cols].double().abs()) for k in (0, 1)]
    f = act("silu", Z[0])[0]
    ef = 1.13 * ez[0] + 16 * EPS32 * (1 + Z[0].abs())
    for k in (0, 1):
        close(f"z[{k}]", z[:, k][:, cols.to(dev)], Z[k], ez[k])
    close("h", h[:, cols.to(dev)], f * Z[1], ef * Z[1].abs() + f.abs() * ez[1] + ef * ez[1] + 4 * EPS32 * (f * Z[1]).abs())
    g_grad = ctp.gated_linear_bwd_bwd(u.to(dev), grad.to(dev), x.to(dev), w, z, needs=(True, False, False, False))[0]
    a, b = (z[:, k][:, cols.to(dev)].double().cpu() for k in (0, 1))
    f, d1, _ = act("silu", a)
    va, vb = (u.double() @ W[k].T for k in (0, 1))
    ea, eb = (e * (u.double().abs() @ W[k].abs().T) for k in (0, 1))
    one = 32 * EPS32 * (1 + a.abs()) ** 2
    close("g_grad", g_grad[:, cols.to(dev)], va * b * d1 + vb * f,
          ea * (b * d1).abs() + eb * f.abs() + one * (va.abs() + ea) * b.abs() + one * (vb.abs() + eb))
    del w, h, z, g_grad
    torch.cuda.empty_cache()


def test_gradients_of_matrices_beyond_2_gib(ctp, dev):
    """d_w's parts, one a component, of 4 GiB; the second pass's, one of each of its products, of 2 GiB each."""
    tell("large parts")
    g = torch.Generator().manual_seed(3)
    inner = outer = 16384
    rows, dtype = 20, torch.bfloat16
    cols = torch.tensor([0, 1, 63, 64, 8191, 16383])
    x, grad = normal(g, (rows, 4, inner), dtype), normal(g, (rows, 4, outer), dtype)
    w = torch.empty(2, outer, inner, dtype=dtype, device=dev).normal_(0, inner ** -0.5, generator=torch.Generator(dev).manual_seed(4))
    d_w = ctp.linear_bwd(grad.to(dev), x.to(dev), w, lmax=1, needs=(False, True, False))[1]
    for degree, comps in ((0, slice(0, 1)), (1, slice(1, 4))):
        X, G = x[:, comps].double().reshape(-1, inner), grad[:, comps][..., cols].double().reshape(-1, len(cols))
        close(f"d_w[{degree}]", d_w[degree][cols.to(dev)], G.T @ X, sum_error(dtype, 3 * rows * 7) * (G.abs().T @ X.abs()))
    del d_w
    x, u, grad, z = (normal(g, (rows, n), dtype) for n in (inner, inner, outer, outer))
    g_w = ctp.linear_bwd_bwd(u.to(dev), grad.to(dev), x.to(dev), w[0], z.to(dev), act="silu", needs=(False, False, True, False))[2]
    W, X, V, G, Z = (t.double() for t in (w[0][cols.to(dev)].cpu(), x, u, grad[:, cols], z[:, cols]))
    _, d1, d2 = act("silu", Z)
    v, ev = V @ W.T, sum_error(dtype, inner) * (V.abs() @ W.abs().T)
    one, half = 32 * EPS32 * (1 + Z.abs()) ** 2, 2.0 ** -8
    gz, s = v * G * d2, G * d1
    ez = ev * (G * d2).abs() + one * (v.abs() + ev) * G.abs()
    ez, es = ez + half * (gz.abs() + ez), half * s.abs() + one * G.abs()
    e = sum_error(dtype, 2 * rows * 7)
    close("g_w", g_w[cols.to(dev)], gz.T @ X + s.T @ V,
          (ez + e * (gz.abs() + ez)).T @ X.abs() + (es + e * (s.abs() + es)).T @ V.abs())
    del w, g_w
    torch.cuda.empty_cache()


def test_orthogonalise_beyond_2_gib(ctp, dev):
    """A workspace of more than 2^31 bytes; the bound is test_gpu_dense.py's."""
    tell("large list")
    m = torch.randn(150, 1024, 1024, device=dev, generator=torch.Generator(dev).manual_seed(5))
    out, = ctp.orthogonalise([m])
    for k in (0, 149):
        ref, e = newton_schulz(m[k].cpu())
        assert float((out[k].double().cpu() - ref).norm()) <= e + EPS32 * float(ref.norm()), k
    assert torch.isfinite(out).all()
    del m, out
    torch.cuda.empty_cache()


def test_orthogonalise_empty_matrices(ctp, dev):
    """Matrices without rows, without columns or without either, by themselves and beside others."""
    shapes = [(0, 0), (0, 5), (5, 0), (2, 0, 0), (0, 5, 5), (3, 0, 7)]
    empty = [torch.empty(s, device=dev) for s in shapes]
    for one, s in zip(empty, shapes):
        assert ctp.orthogonalise([one])[0].shape == s
    m = torch.randn(40, 70, device=dev)
    want, = ctp.orthogonalise([m])
    outs = ctp.orthogonalise([*empty, m, *empty])
    assert torch.equal(outs[len(empty)], want) and [tuple(o.shape) for o in outs] == [*shapes, (40, 70), *shapes]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,inner,outer", [(3000, 64, 64), (81, 100, 128), (600, 24, 7), (3000, 200, 300), (900, 1003, 1000)])
@pytest.mark.parametrize("gated", [False, True])
def test_bias_sums_before_any_rounding(ctp, dev, dtype, rows, inner, outer, gated):
    """Terms that cancel: what they are rounded to would not (each up to half a step of some 20, thousands of them)."""
    tell("bias", dtype, rows, inner, outer, gated)
    g = torch.Generator().manual_seed(6)
    a, b = (torch.randint(-60, 61, (rows // 3, outer), generator=g).double() for _ in range(2))
    grad = torch.cat([a, b, -(a + b)])[torch.randperm(rows, generator=g)].to(dtype)     # whole numbers below 128
    z = normal(g, (2, outer) if gated else (outer,), dtype)
    zs = z.expand(rows, *z.shape).contiguous()
    x, w = normal(g, (rows, inner), dtype), normal(g, (2, outer, inner) if gated else (outer, inner), dtype, inner ** -0.5)
    for name in ("silu", "gelu", "tanh"):
        back = ctp.gated_linear_bwd if gated else ctp.linear_bwd
        d_bias = back(grad.to(dev), x.to(dev), w.to(dev), zs.to(dev), act=name, needs=(True, True, True))[2]
        Z, S = z.double(), grad.double().abs().sum(0)
        f, d1, _ = act(name, Z[0] if gated else Z)
        # a row's derivative is the same number in all rows, a term one rounding (gated: two) and the additions follow
        slope = torch.stack([(Z[1] * d1).abs(), f.abs()]) if gated else d1.abs()
        close(name, d_bias, torch.zeros_like(slope), (rows + 8) * EPS32 * S * slope * (1 + 2.0 ** -10))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,inner,outer", [(24, 64, 40), (81, 100, 128), (600, 24, 7), (90, 2100, 33), (900, 512, 500)])
@pytest.mark.parametrize("gated", [False, True])
def test_second_bias_sums_before_any_rounding(ctp, dev, dtype, rows, inner, outer, gated):
    """As above for the second pass: every row has the same cotangent and z, so only grad's values differ, and cancel."""
    tell("second bias", dtype, rows, inner, outer, gated)
    g = torch.Generator().manual_seed(7)
    a, b = (torch.randint(-60, 61, (rows // 3, outer), generator=g).double() for _ in range(2))
    grad = torch.cat([a, b, -(a + b)])[torch.randperm(rows, generator=g)].to(dtype)
    z = normal(g, (2, outer) if gated else (outer,), dtype)
    u, w = normal(g, (inner,), dtype), normal(g, (2, outer, inner) if gated else (outer, inner), dtype, inner ** -0.5)
    x = normal(g, (rows, inner), dtype)
    args = [t.to(dev) for t in (u.expand(rows, inner).contiguous(), grad, x, w, z.expand(rows, *z.shape).contiguous())]
    second = ctp.gated_linear_bwd_bwd if gated else ctp.linear_bwd_bwd
    for name in ("silu", "gelu", "tanh"):
        g_bias = second(*args, act=name)[3]
        Z, V, S = z.double(), w.double() @ u.double(), grad.double().abs().sum(0)
        f, d1, d2 = act(name, Z[0] if gated else Z)
        # v, its error in it, is the same in all rows
        V = V.abs() + sum_error(dtype, inner) * (w.double().abs() @ u.double().abs())
        slope = (torch.stack([V[0] * (Z[1] * d2).abs() + V[1] * d1.abs(), V[0] * d1.abs()]) if gated else V * d2.abs())
        # act' and act'' off by some roundings of 1 + |z|
        slope = slope + 32 * EPS32 * (1 + Z.abs()) ** 2 * (V.sum(0) * (1 + Z[1].abs()) if gated else V)
        close(name, g_bias, torch.zeros_like(slope), (rows + 8) * EPS32 * S * slope * (1 + 2.0 ** -10))
        assert torch.equal(second(*args, act=name, needs=(False, False, False, True))[3], g_bias)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_activations_far_out(ctp, dev, dtype):
    """z whose square is beyond float's range: slopes 0 or 1, curvature 0, and what a row gets from it."""
    z = torch.tensor([-3e38, -1e25, -1e20, -2e19, -1.8e19, 0.0, 1.8e19, 2e19, 1e20, 1e25, 3e38]).to(dtype)[:, None]
    one = torch.ones(len(z), 1, dtype=dtype, device=dev)
    far = (z != 0).double()
    for name in ("relu", "silu", "gelu", "sigmoid", "tanh"):
        d_x, d_w, d_bias = ctp.linear_bwd(one, one, one[:1], z.to(dev), act=name)
        slope = act(name, z.double())[1]
        close(name, d_x, slope, 64 * EPS32 * (1 + slope.abs()))
        assert torch.isfinite(d_w).all() and torch.isfinite(d_bias).all()
        curve = act(name, z.double().clamp(-1e3, 1e3))[2]       # (beyond, the formula's own terms overflow)
        g_grad, g_x, g_w, g_bias = ctp.linear_bwd_bwd(one, one, one, one[:1], z.to(dev), act=name)
        assert not (curve * far).any()
        close(name, g_x, curve, 256 * EPS32 * (1 + curve.abs()))
        assert all(torch.isfinite(t).all() for t in (g_grad, g_w, g_bias))
        y, _ = ctp.linear_fwd(z.to(dev), one[:1], act=name)
        ref = act(name, z.double())[0]
        close(name, y, ref, 16 * EPS32 * (1 + ref.abs()))
        zz = torch.stack([z, torch.ones_like(z)], 1).to(dev)
        got = [*ctp.gated_linear_bwd(one, one, one[:2, None], zz, act=name), *ctp.gated_linear_bwd_bwd(one, one, one, one[:2, None], zz, act=name)]
        # act(z) itself is a slope of these, and sums of it pass the type's range: no NaN
        assert not any(torch.isnan(t).any() for t in got)


LAYERS = [  # few rows; tiles of 64 and of 128; rows in registers, plain and with an epilogue; cut sums; odd sizes
    (20, 64, 40, {}), (100, 64, 64, dict(bias=True)), (1500, 600, 1400, {}), (5000, 64, 1024, {}), (5000, 100, 1040, dict(act="relu", bias=True)),
    (200, 2100, 90, {}), (77, 33, 129, dict(residual=True)), (300, 2, 5, {}), (3000, 40, 520, dict(gated=True)), (90, 70, 33, dict(gated=True)),
    (64, 1500, 200, dict(gated=True)),
]


@pytest.mark.parametrize("rows,inner,outer,how", LAYERS)
def test_infinities_of_floats(ctp, dev, rows, inner, outer, how):
    """What is not finite in a float layer comes out as the formula has it, whatever kernel forms it: infinities of either
    sign, NaN, products beyond the range; the other results are not touched."""
    tell("infinities", rows, inner, outer, how)
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(9)
    gated, name = how.get("gated", False), how.get("act", "none")
    x = torch.randn(rows, inner, generator=g)
    w = torch.randn(2, outer, inner, generator=g) if gated else torch.randn(outer, inner, generator=g)
    w = torch.where(w.abs() < 0.05, 0.5, w)
    bias = torch.randn(w.shape[:-1], generator=g) if how.get("bias") else None
    residual = torch.randn(rows, outer, generator=g) if how.get("residual") else None
    clean, _ = ctp.gated_linear_fwd(*(to_dev(dev, x, w, bias)), act=name) if gated else ctp.linear_fwd(*to_dev(dev, x, w, bias, residual), act=name)
    odd = {1: (0, inf), 7: (inner - 1, -inf), rows - 1: (inner // 2, nan)}
    if inner > 3:
        odd[rows - 3] = (1, 3e38)
    for r, (k, v) in odd.items():
        x[r, k] = v
    x[5, 0], x[5, inner // 2] = inf, inf
    w.view(-1, inner)[3, 1] = 4.0                                   # times 3e38: beyond the range, without infinities beside it
    w.view(-1, inner)[-1, 0] = -inf
    w.view(-1, inner)[2, inner // 2] = 0.0
    X, W = x.double(), w.double()

    def product(x, w):      # one term of a sum at most is beyond float's range: its sum is
        return (x[:, None, :] * w[None]).sum(-1)

    Z = [torch.cat([product(X[i:i + 50], m) for i in range(0, rows, 50)]) for m in (W if gated else W[None])]
    if bias is not None:
        Z = [z + b.double() for z, b in zip(Z, bias.view(len(Z), -1))]
    f = act(name, Z[0])[0]
    want = f * Z[1] if gated else f
    if residual is not None:
        want = want + residual.double()
    y, _ = ctp.gated_linear_fwd(*to_dev(dev, x, w, bias), act=name) if gated else ctp.linear_fwd(*to_dev(dev, x, w, bias, residual), act=name)
    y = y.double().cpu()
    want = want.float().double()        # beyond the range: infinities
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    beyond = torch.isinf(want)
    assert torch.equal(y[beyond], want[beyond]) and not torch.isinf(y[~beyond]).any()
    # rows and columns without any of it: the same bits
    rest, cols = torch.ones(rows, dtype=torch.bool), torch.ones(outer, dtype=torch.bool)
    rest[[*odd, 5, rows - 3]] = False
    cols[[2, 3, outer - 1]] = False
    assert torch.equal(y[rest][:, cols], clean.double().cpu()[rest][:, cols])
    if gated:
        return
    # the gradients, of which d_w sums over the rows
    grad = torch.randn(rows, outer, generator=g)
    grad[2, 1], grad[9, 0] = inf, -inf
    grad[rows - 3, :2] = 0
    z = torch.randn(rows, outer, generator=g)
    d_x, d_w, _ = ctp.linear_bwd(*to_dev(dev, grad, x, w), to_dev(dev, z)[0] if name != "none" else None, act=name)
    s = (grad * act(name, z.double())[1].float()).double()
    for got, a, b in ((d_x, s, W.T), (d_w, s.T, X.T)):
        ref = torch.cat([product(a[i:i + 50], b) for i in range(0, len(a), 50)]).float()
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(ref))
        beyond = torch.isinf(ref)
        assert torch.equal(got.cpu()[beyond], ref[beyond]) and not torch.isinf(got.cpu()[~beyond]).any()


def to_dev(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalise_same_bits_in_any_list(ctp, dev, dtype):
    """A matrix alone, in lists that are computed in tiles of 128 or of 64 and whose sums are cut or not: the same bits."""
    g = torch.Generator().manual_seed(10)
    shapes = [(2048, 2048), (520, 3000), (3, 300, 1100), (64, 5000), (1100, 130), (130, 130), (1, 700, 700), (257, 1030)]
    ms = [normal(g, s, dtype).to(dev) for s in shapes]
    alone = [ctp.orthogonalise([m])[0] for m in ms]
    wide = torch.randn(40, 400, 900, generator=g).to(dev)       # enough tiles of 128 for the card
    for k, company in enumerate(([wide], [ms[5]], [wide, wide, wide[:, :, :130].contiguous()], [])):
        tell("company", k)
        for m, o, a in zip(ms, ctp.orthogonalise([*ms, *company]), alone):
            assert torch.equal(o, a), (k, tuple(m.shape))
        for m, a in zip(ms, alone):
            assert torch.equal(ctp.orthogonalise([*company, m])[-1], a), (k, tuple(m.shape))
    # one matrix of a batch, and by itself
    out, = ctp.orthogonalise([wide])
    for k in (0, 17, 39):
        assert torch.equal(out[k], ctp.orthogonalise([wide[k]])[0]), k


def test_infinities_in_long_sums(ctp, dev):
    """One infinity among 200000 rows: its column of d_w, and of d_bias's terms; what has none of it keeps its bits."""
    g = torch.Generator(dev).manual_seed(11)
    rows, inner, outer = 200000, 200, 300
    x, grad = (torch.randn(rows, n, device=dev, generator=g) for n in (inner, outer))
    w, z = torch.randn(outer, inner, device=dev, generator=g), torch.randn(rows, outer, device=dev, generator=g)
    clean = ctp.linear_bwd(grad, x, w, z, act="silu")
    x[123456, 7] = float("inf")
    d_x, d_w, d_bias = ctp.linear_bwd(grad, x, w, z, act="silu")
    s = grad[123456].double() * act("silu", z[123456].double())[1]
    assert torch.equal(d_w[:, 7].double(), s.sign() * float("inf"))
    keep = torch.arange(inner, device=dev) != 7
    assert torch.equal(d_x, clean[0]) and torch.equal(d_w[:, keep], clean[1][:, keep]) and torch.equal(d_bias, clean[2])
