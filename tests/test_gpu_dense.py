"""The dense operators (include/convtp_dense.h) on the GPU against plain float64
forms on the CPU.

Tolerances are derived, not fitted.  U is an output type's unit roundoff (2^-24,
2^-8, 2^-11), S an expression with every term replaced by its absolute value.

* A product of k terms: 16-bit factors have exact fp32 products, and a term
  passes through at most k + 8 additions, each off by at most 2^-23 (half a
  step, or a whole one where a matrix core cuts): SUM16 = 2 (k + 8) 2^-24 S.  Floats are
  taken apart into three parts and the products below 2^-24 of the whole left
  out; a term is six products, so SUM32 = (1 + 12 (k + 8)) 2^-24 S.
* An activation: its slope is at most 1.13 and its own evaluation a few roundings
  of values up to 1 + |z|: 16 2^-24 (1 + |z|); its derivative, whose slope is at
  most 1 (silu 0.5, gelu 0.8, tanh 0.77), likewise.
* s = grad act'(z), and what the second pass multiplies, is rounded to the type
  before the product: U S more.
"""
import itertools
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}
EPS32 = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "silu", "gelu", "sigmoid", "tanh"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def ctp(dev):
    import tensor_product_message_amd as t
    return t


def tell(*a):
    print(*a, flush=True)


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def close(name, got, ref, bound):
    got_cpu = got.detach().double().cpu()
    assert got_cpu.shape == ref.shape, (name, got_cpu.shape, ref.shape)
    u = U[got.dtype]
    tol = u * ref.abs() * (1 + 2.0 ** -10) + TINY[got.dtype] + bound * (1 + u)
    # a value beyond the type's largest is rounded to an infinity: two terms of 3.4e38 are 6.8e38, the largest 3.403e38
    beyond = ref.abs() > torch.finfo(got.dtype).max * (1 + u)
    bad = torch.where(beyond, got_cpu != ref.sign() * math.inf, ~((got_cpu - ref).abs() <= tol))
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst ratio "
                           f"{float(((got_cpu - ref).abs() / tol).max()):.3f}")


def sum_error(dtype, k):
    return (1 + 12 * (k + 8)) * EPS32 if dtype == torch.float32 else 2 * (k + 8) * EPS32


def act(name, z):
    """act, act', act'' in float64."""
    if name == "none":
        return z, torch.ones_like(z), torch.zeros_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double(), torch.zeros_like(z)
    if name == "tanh":
        t = torch.tanh(z)
        return t, 1 - t * t, -2 * t * (1 - t * t)
    if name == "gelu":
        c, p = 0.5 * torch.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * c, c + z * p, p * (2 - z * z)
    s = torch.sigmoid(z)
    if name == "sigmoid":
        return s, s * (1 - s), s * (1 - s) * (1 - 2 * s)
    return z * s, s + z * s * (1 - s), s * (1 - s) * (2 + z * (1 - 2 * s))


def degrees(lmax):
    return [int(math.isqrt(d)) for d in range((lmax + 1) ** 2)]


class Case:
    """A layer's inputs on the CPU in their type, and everything about it in float64."""

    def __init__(self, rows, inner, outer, dtype, name="none", lmax=0, gated=False, bias=True, residual=False, seed=0):
        g = torch.Generator().manual_seed(seed + rows + 7 * inner + 31 * outer)
        comps, self.lmax, self.name, self.gated, self.dtype = (lmax + 1) ** 2, lmax, name, gated, dtype
        lead = (rows, comps) if lmax else (rows,)
        self.x = normal(g, (*lead, inner), dtype)
        shape = (2, outer, inner) if gated else (lmax + 1, outer, inner) if lmax else (outer, inner)
        self.w = normal(g, shape, dtype, inner ** -0.5)
        self.bias = normal(g, (2, outer) if gated else (outer,), dtype, 0.5) if bias else None
        self.residual = normal(g, (*lead, outer), dtype) if residual else None
        self.grad = normal(g, (*lead, outer), dtype)
        self.u = normal(g, (*lead, inner), dtype)
        self.rows, self.inner, self.outer, self.comps = rows, inner, outer, comps
        self.curved = gated or name != "none"
        # [rows, comps, .] and one matrix a component (a gated layer's halves beside each other)
        w = self.w.double()
        self.W = w.view(1, 2 * outer, inner) if gated else w.view(lmax + 1, outer, inner)[degrees(lmax)]
        self.X, self.G, self.Uu = (t.double().view(rows, comps, -1) for t in (self.x, self.grad, self.u))

    def forward(self):
        e = sum_error(self.dtype, self.inner)
        z = torch.einsum("ndi,doi->ndo", self.X, self.W)
        S = torch.einsum("ndi,doi->ndo", self.X.abs(), self.W.abs())
        if self.bias is not None:
            z[:, 0] += self.bias.double().view(-1)
            S[:, 0] += self.bias.double().view(-1).abs()
        ez = e * S
        if self.gated:
            a, b = z[:, 0, :self.outer], z[:, 0, self.outer:]
            ea, eb = ez[:, 0, :self.outer], ez[:, 0, self.outer:]
            f = act(self.name, a)[0]
            ef = 1.13 * ea + 16 * EPS32 * (1 + a.abs())
            return z.view(self.rows, 2, self.outer), ez.view(self.rows, 2, self.outer), f * b, ef * b.abs() + f.abs() * eb + ef * eb + 4 * EPS32 * (f * b).abs()
        y = act(self.name, z)[0]
        ey = 1.13 * ez + (16 * EPS32 * (1 + z.abs()) if self.curved else 0)
        if self.residual is not None:
            r = self.residual.double().view(y.shape)
            y, ey = y + r, ey + 4 * EPS32 * (y.abs() + r.abs())
        shape = self.grad.shape
        return z.view(shape), ez.view(shape), y.view(shape), ey.view(shape)

    def s(self, z):
        """(s, its error bound), [rows, comps, outer or 2 outer], at a stored z."""
        if not self.curved:
            return self.G, torch.zeros_like(self.G)
        u = U[self.dtype]
        if self.gated:
            a, b = z[:, 0], z[:, 1]
            f, d1, _ = act(self.name, a)
            g = self.G[:, 0]
            s = torch.cat([g * b * d1, g * f], 1)
            e = torch.cat([16 * EPS32 * (g * b).abs() * (1 + a.abs()), 16 * EPS32 * g.abs() * (1 + a.abs())], 1)
            return s[:, None], (e + u * s.abs() + TINY[self.dtype])[:, None]
        d1 = act(self.name, z)[1].view(self.G.shape)
        s = self.G * d1
        return s, u * s.abs() + 16 * EPS32 * self.G.abs() * (1 + z.abs().view(s.shape)) + TINY[self.dtype]

    def weight_sum(self, s, es, x, rows=None):
        """d_w = sum of s^T x by degree, and its bound."""
        per = torch.einsum("ndo,ndi->doi", s, x)
        S = torch.einsum("ndo,ndi->doi", s.abs(), x.abs())
        E = torch.einsum("ndo,ndi->doi", es, x.abs())
        degs = degrees(self.lmax)
        n = 1 if self.gated else self.lmax + 1
        d, b = (torch.zeros(n, *per.shape[1:], dtype=torch.float64) for _ in range(2))
        for k in range(self.comps):
            d[degs[k]] += per[k]
            b[degs[k]] += sum_error(self.dtype, rows or self.rows * 7) * (S[k] + E[k]) + E[k]
        return d.view(self.w.shape), b.view(self.w.shape)

    def backward(self, z):
        s, es = self.s(z)
        k = s.shape[-1]
        d_x = torch.einsum("ndo,doi->ndi", s, self.W)
        e_x = torch.einsum("ndo,doi->ndi", es + sum_error(self.dtype, k) * (s.abs() + es), self.W.abs())
        d_w, e_w = self.weight_sum(s, es, self.X)
        # the bias sums s before its rounding, in fp32: its own error and the additions'
        d_b = s[:, 0].sum(0)
        e_b = (es[:, 0] + (self.rows + 8) * EPS32 * (s.abs() + es)[:, 0]).sum(0)
        shape = self.w.shape[:-1] if self.gated else (self.outer,)
        return (d_x.view(self.x.shape), e_x.view(self.x.shape)), (d_w, e_w), (d_b.view(shape), e_b.view(shape))

    def second(self, z):
        v = torch.einsum("ndi,doi->ndo", self.Uu, self.W)
        ev = sum_error(self.dtype, self.inner) * torch.einsum("ndi,doi->ndo", self.Uu.abs(), self.W.abs())
        s, es = self.s(z)
        u, zero = U[self.dtype], None
        if not self.curved:
            d_w, e_w = self.weight_sum(s, es, self.Uu)
            return (v.view(self.grad.shape), ev.view(self.grad.shape)), zero, (d_w, e_w), zero
        if self.gated:
            a, b, g = z[:, 0], z[:, 1], self.G[:, 0]
            f, d1, d2 = act(self.name, a)
            va, vb = v[:, 0, :self.outer], v[:, 0, self.outer:]
            ea, eb = ev[:, 0, :self.outer], ev[:, 0, self.outer:]
            one = 32 * EPS32 * (1 + a.abs()) ** 2        # of act, act', act'': few roundings each
            gG = va * b * d1 + vb * f
            eG = ea * (b * d1).abs() + eb * f.abs() + one * (va.abs() + ea) * b.abs() + one * (vb.abs() + eb)
            gz = torch.cat([va * g * b * d2 + vb * g * d1, va * g * d1], 1)
            ez = torch.cat([ea * (g * b * d2).abs() + eb * (g * d1).abs() + one * ((va.abs() + ea) * (g * b).abs() + (vb.abs() + eb) * g.abs()),
                            ea * (g * d1).abs() + one * (va.abs() + ea) * g.abs()], 1)
            gz, ez = gz[:, None], ez[:, None]
        else:
            zz = z.view(v.shape)
            _, d1, d2 = act(self.name, zz)
            one = 32 * EPS32 * (1 + zz.abs()) ** 2
            gG, gz = v * d1, v * self.G * d2
            eG = ev * d1.abs() + one * (v.abs() + ev)
            ez = ev * (self.G * d2).abs() + one * (v.abs() + ev) * self.G.abs()
        ez = ez + u * (gz.abs() + ez) + TINY[self.dtype]
        k = gz.shape[-1]
        g_x = torch.einsum("ndo,doi->ndi", gz, self.W)
        e_x = torch.einsum("ndo,doi->ndi", ez + sum_error(self.dtype, k) * (gz.abs() + ez), self.W.abs())
        w1, e1 = self.weight_sum(gz, ez, self.X)
        w2, e2 = self.weight_sum(s, es, self.Uu)
        g_b = gz[:, 0].sum(0)
        e_b = (ez[:, 0] + (self.rows + 8) * EPS32 * (gz.abs() + ez)[:, 0]).sum(0)
        shape = self.w.shape[:-1] if self.gated else (self.outer,)
        return ((gG.view(self.grad.shape), eG.view(self.grad.shape)), (g_x.view(self.x.shape), e_x.view(self.x.shape)),
                (w1 + w2, e1 + e2 + 4 * EPS32 * (w1.abs() + w2.abs())), (g_b.view(shape), e_b.view(shape)))


def to(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


SHAPES = [  # rows, inner, outer: single rows, odd sizes, tiles and their edges, sums longer than a tile
    (1, 1, 1), (1, 8, 5), (1, 333, 77), (3, 64, 64), (5, 7, 9), (16, 512, 40), (17, 520, 33), (31, 100, 130),
    (1, 4099, 37), (20, 3000, 50), (9, 2600, 1000),
    (33, 600, 70), (64, 2048, 100), (200, 1030, 90), (90, 70, 1100), (2, 100, 2000), (5000, 64, 64), (3001, 100, 128), (900, 127, 3),
    (64, 16, 16), (65, 63, 129), (130, 65, 66), (257, 130, 257), (1503, 8, 64), (300, 1003, 77), (40, 2051, 24),
    (2000, 24, 3), (129, 192, 320), (513, 256, 264), (700, 264, 520),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", SHAPES)
def test_linear(ctp, dev, rows, inner, outer, dtype):
    for name, residual in ((ACTS[(rows + inner) % 6], outer % 2 == 0), ("none", outer % 2 == 1)):
        c = Case(rows, inner, outer, dtype, name, residual=residual, bias=(rows + outer) % 3 != 0)
        tell("linear", rows, inner, outer, dtype, name)
        x, w, b, r, grad, u = to(dev, c.x, c.w, c.bias, c.residual, c.grad, c.u)
        y, z = ctp.linear_fwd(x, w, b, r, act=name, keep_z=True)
        z_ref, ez, y_ref, ey = c.forward()
        close("z", z, z_ref, ez)
        close("y", y, y_ref, ey)
        y2, none = ctp.linear_fwd(x, w, b, r, act=name)
        assert none is None and torch.equal(y, y2), "not the same bits twice"
        zs = z.double().cpu()
        got = ctp.linear_bwd(grad, x, w, z, act=name)
        for n, a, (ref, bound) in zip(("d_x", "d_w", "d_bias"), got, c.backward(zs)):
            close(n, a, ref, bound)
        assert all(torch.equal(a, b2) for a, b2 in zip(got, ctp.linear_bwd(grad, x, w, z, act=name)))
        second = ctp.linear_bwd_bwd(u, grad, x, w, z, act=name)
        for n, a, ref in zip(("g_grad", "g_x", "g_w", "g_bias"), second, c.second(zs)):
            if ref is None:
                assert a is None, n
            else:
                close(n, a, *ref)


WIDE = [  # enough tiles of 256 and of 128 for the card, in each direction's product; sums that end inside a tile
    (3400, 72, 3600, False), (1500, 80, 1400, False), (3400, 3600, 40, False), (2600, 2608, 40, False), (40, 3400, 3600, False),
    (72, 1400, 1504, False), (3400, 72, 1800, True), (1500, 136, 712, True), (40, 3400, 1800, True),
    (1500, 1003, 777, False), (2000, 1000, 777, False), (2000, 1003, 776, False), (1300, 1003, 512, True), (1300, 1001, 511, True),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer,gated", WIDE)
def test_wide(ctp, dev, rows, inner, outer, gated, dtype):
    c = Case(rows, inner, outer, dtype, "silu", gated=gated)
    tell("wide", rows, inner, outer, gated, dtype)
    x, w, b, grad = to(dev, c.x, c.w, c.bias, c.grad)
    f, back = (ctp.gated_linear_fwd, ctp.gated_linear_bwd) if gated else (ctp.linear_fwd, ctp.linear_bwd)
    y, z = f(x, w, b, act="silu", keep_z=True)
    z_ref, ez, y_ref, ey = c.forward()
    close("z", z, z_ref, ez)
    close("y", y, y_ref, ey)
    got = back(grad, x, w, z, act="silu")
    for n, a, (ref, bound) in zip(("d_x", "d_w", "d_bias"), got, c.backward(z.double().cpu())):
        close(n, a, ref, bound)
    assert all(torch.equal(a, b2) for a, b2 in zip(got, back(grad, x, w, z, act="silu")))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lmax,rows,inner,outer,gap", [(0, 1501, 1001, 779, 0), (0, 1501, 1000, 776, 3), (1, 700, 333, 1111, 0),
                                                       (1, 700, 336, 1104, 5), (2, 300, 600, 645, 0), (0, 1501, 1000, 777, 0)])
def test_wide_without_activation(ctp, dev, lmax, rows, inner, outer, gap, dtype):
    """Odd rows and odd strides (gap values behind each row), sizes at which 16-bit rows are laid out anew."""
    c = Case(rows, inner, outer, dtype, lmax=lmax)
    tell("wide, no activation", lmax, rows, inner, outer, gap, dtype)
    x, w, b, grad = to(dev, c.x, c.w, c.bias, c.grad)

    def with_gap(t):
        wide = torch.full((t.shape[0], t[0].numel() + gap), float("nan"), dtype=dtype, device=dev)
        wide[:, :t[0].numel()] = t.view(t.shape[0], -1)
        return wide[:, :t[0].numel()].unflatten(1, t.shape[1:])

    x, grad = with_gap(x), with_gap(grad)
    y, _ = ctp.linear_fwd(x, w, b, lmax=lmax)
    _, _, y_ref, ey = c.forward()
    close("y", y, y_ref, ey)
    got = ctp.linear_bwd(grad, x, w, lmax=lmax)
    for n, a, (ref, bound) in zip(("d_x", "d_w", "d_bias"), got, c.backward(None)):
        close(n, a, ref, bound)
    part = ctp.linear_bwd(grad, x, w, lmax=lmax, needs=(False, True, False))
    assert part[0] is None and torch.equal(part[1], got[1])
    assert torch.equal(ctp.linear_bwd(grad, x, w, lmax=lmax, needs=(True, False, False))[0], got[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lmax,rows,inner,outer", [(1, 1, 16, 16), (1, 64, 16, 16), (2, 77, 33, 20), (3, 100, 128, 128),
                                                   (3, 301, 9, 65), (2, 700, 64, 136), (1, 50, 640, 40), (1, 40, 40, 700), (3, 1503, 24, 32)])
def test_linear_degrees(ctp, dev, lmax, rows, inner, outer, dtype):
    c = Case(rows, inner, outer, dtype, lmax=lmax, residual=True)
    tell("linear degrees", lmax, rows, inner, outer, dtype)
    x, w, b, r, grad, u = to(dev, c.x, c.w, c.bias, c.residual, c.grad, c.u)
    y, z = ctp.linear_fwd(x, w, b, r, lmax=lmax, keep_z=True)
    z_ref, ez, y_ref, ey = c.forward()
    close("z", z, z_ref, ez)
    close("y", y, y_ref, ey)
    for n, a, (ref, bound) in zip(("d_x", "d_w", "d_bias"), ctp.linear_bwd(grad, x, w, lmax=lmax), c.backward(None)):
        close(n, a, ref, bound)
    g_grad, g_x, g_w, g_b = ctp.linear_bwd_bwd(u, grad, x, w, lmax=lmax)
    refs = c.second(None)
    close("g_grad", g_grad, *refs[0])
    close("g_w", g_w, *refs[2])
    assert g_x is None and g_b is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", [(1, 8, 1), (1, 257, 96), (2, 64, 33), (15, 100, 64), (64, 40, 31), (65, 129, 65),
                                              (300, 72, 136), (1503, 129, 17), (513, 256, 264), (33, 1029, 8), (50, 2048, 48), (41, 1100, 33)])
def test_gated(ctp, dev, rows, inner, outer, dtype):
    for k, bias in ((0, True), (3, False)):
        name = ACTS[(rows + outer + k) % 6]
        c = Case(rows, inner, outer, dtype, name, gated=True, bias=bias)
        tell("gated", rows, inner, outer, dtype, name)
        x, w, b, grad, u = to(dev, c.x, c.w, c.bias, c.grad, c.u)
        h, z = ctp.gated_linear_fwd(x, w, b, act=name, keep_z=True)
        z_ref, ez, h_ref, eh = c.forward()
        close("z", z, z_ref, ez)
        close("h", h, h_ref, eh)
        assert torch.equal(h, ctp.gated_linear_fwd(x, w, b, act=name)[0])
        zs = z.double().cpu()
        for n, a, (ref, bound) in zip(("d_x", "d_w", "d_bias"), ctp.gated_linear_bwd(grad, x, w, z, act=name), c.backward(zs)):
            close(n, a, ref, bound)
        for n, a, (ref, bound) in zip(("g_grad", "g_x", "g_w", "g_bias"),
                                      ctp.gated_linear_bwd_bwd(u, grad, x, w, z, act=name), c.second(zs)):
            close(n, a, ref, bound)


@pytest.mark.parametrize("k", [1, 2, 5])
def test_float_products_keep_24_bits(ctp, dev, k):
    """Few terms, all significands in use: a part of a float that got lost would show."""
    g = torch.Generator().manual_seed(k)
    x = torch.randn(200, k, generator=g) * torch.exp2(torch.randint(-30, 30, (200, 1), generator=g).float())
    x[0], x[1], x[2] = torch.finfo(torch.float32).max, 1.0 + 2.0 ** -23, 3.3999999e38
    w = torch.randn(50, k, generator=g)
    w[0], w[1] = 0.5 / k, 1.0 - 2.0 ** -24
    w[2:] *= 1.0 / k / w[2:].abs().amax()
    y, _ = ctp.linear_fwd(x.to(dev), w.to(dev))
    S = x.double().abs() @ w.double().abs().T
    # terms of one product: the part left out, six additions
    close("y", y, x.double() @ w.double().T, (1 + 2 * 6 * k) * EPS32 * S)
    d_x, d_w, _ = ctp.linear_bwd(y[:0].to(dev), x[:0].to(dev), w.to(dev))
    assert d_x.shape == (0, k) and not d_w.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_shapes_outputs_and_empty(ctp, dev, dtype):
    g = torch.Generator().manual_seed(3)
    wide = normal(g, (6, 11, 61), dtype).to(dev)
    x = wide[..., 3:40]                                   # 37 of 61 values a row, from an odd place
    w, b = to(dev, normal(g, (29, 37), dtype, 0.2), normal(g, (29,), dtype))
    r = normal(g, (6, 11, 35), dtype).to(dev)[..., 1:30]
    y, z = ctp.linear_fwd(x, w, b, r, act="silu", keep_z=True)
    xc, rc = x.contiguous(), r.contiguous()
    want = ctp.linear_fwd(xc, w, b, rc, act="silu", keep_z=True)
    assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    into = rc.clone()
    got, _ = ctp.linear_fwd(x, w, b, into, act="silu", out=into)        # over the residual
    assert got is into or got.data_ptr() == into.data_ptr()
    assert torch.equal(into, y)
    grad = normal(g, (6, 11, 50), dtype).to(dev)[..., 7:36]
    a, c = ctp.linear_bwd(grad, x, w, z, act="silu"), ctp.linear_bwd(grad.contiguous(), xc, w, z, act="silu")
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    for needs in itertools.product((True, False), repeat=3):
        part = ctp.linear_bwd(grad, x, w, z, act="silu", needs=needs)
        for need, p, q in zip(needs, part, c):
            assert torch.equal(p, q) if need else p is None
    u = normal(g, (6, 11, 37), dtype).to(dev)
    full = ctp.linear_bwd_bwd(u, grad, x, w, z, act="silu")
    for needs in itertools.product((True, False), repeat=4):
        for need, p, q in zip(needs, ctp.linear_bwd_bwd(u, grad, x, w, z, act="silu", needs=needs), full):
            assert torch.equal(p, q) if need else p is None
    for lead in ((0,), (3, 0)):
        e = torch.empty(*lead, 37, dtype=dtype, device=dev)
        y, z = ctp.linear_fwd(e, w, b, act="relu", keep_z=True)
        assert y.shape == z.shape == (*lead, 29)
        d_x, d_w, d_b = ctp.linear_bwd(y, e, w, z, act="relu")
        assert d_x.shape == e.shape and not d_w.any() and not d_b.any()
        gs = ctp.linear_bwd_bwd(e, y, e, w, z, act="relu")
        assert not gs[2].any() and not gs[3].any()
    one = torch.zeros(37, dtype=dtype, device=dev)
    assert ctp.linear_fwd(one, w, b)[0].shape == (29,) and torch.equal(ctp.linear_fwd(one, w, b)[0], b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", [(7, 64, 40), (200, 64, 64), (300, 512, 512), (1600, 1000, 1000), (30000, 64, 320)])
def test_storage_at_any_element(ctp, dev, rows, inner, outer, dtype):
    """Every array one element behind a 16-byte place: the results of arrays at such places."""
    c = Case(rows, inner, outer, dtype, "silu", residual=True)
    tell("odd places", rows, inner, outer, dtype)
    even = to(dev, c.x, c.w, c.bias, c.residual, c.grad, c.u)

    def odd(t):
        s = torch.empty(t.numel() + 1, dtype=dtype, device=dev)[1:].view(t.shape)
        return s.copy_(t)

    results = []
    for place in (lambda t: t, odd):
        x, w, b, r, grad, u = (place(t) for t in even)
        out = place(torch.zeros(rows, outer, dtype=dtype, device=dev))
        y, z = ctp.linear_fwd(x, w, b, r, act="silu", keep_z=True, out=out)
        assert y is out or y.data_ptr() == out.data_ptr()
        z = place(z)
        results.append([y, z, *ctp.linear_bwd(grad, x, w, z, act="silu"), *ctp.linear_bwd_bwd(u, grad, x, w, z, act="silu")])
    k = max(inner, outer, rows)
    for a, b in zip(*results):
        # other tiles may sum in another order
        assert float((a - b).abs().max()) <= (2 * U[dtype] + 12 * k ** 0.5 * EPS32) * float(b.abs().max()) * 2


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
def test_extreme_values(ctp, dev, dtype, gated):
    """Values outside one row do not reach another; derivatives far out are 0 or 1."""
    x = torch.zeros(70, 16, dtype=dtype, device=dev)
    x[:, 0] = 1
    x[3, 5], x[69, 0], x[7, 2] = float("nan"), float("inf"), float("-inf")
    w = torch.ones(2, 24, 16, dtype=dtype, device=dev) if gated else torch.ones(24, 16, dtype=dtype, device=dev)
    y = (ctp.gated_linear_fwd(x, w) if gated else ctp.linear_fwd(x, w, act="silu"))[0].float()
    bad = torch.zeros(70, dtype=torch.bool, device=dev)
    bad[[3, 69, 7]] = True
    assert torch.isfinite(y[~bad]).all() and not torch.isfinite(y[[3, 69]]).any()
    z = torch.tensor([-6e4, -300.0, -88.0, -20.0, 0.0, 20.0, 88.0, 300.0, 6e4], device=dev).to(dtype)[:, None]
    one = torch.ones(9, 1, dtype=dtype, device=dev)
    for name in ACTS:
        d_x, _, _ = ctp.linear_bwd(one, one, one[:1], z, act=name)
        ref = act(name, z.double().cpu())[1]
        close(name, d_x, ref, 64 * EPS32 * (1 + ref.abs()))
        g = ctp.linear_bwd_bwd(one, one, one, one[:1], z, act=name)
        ref2 = act(name, z.double().cpu())[2].nan_to_num(0.0)
        if name != "none":
            close(name, g[1], ref2, 256 * EPS32 * (1 + ref2.abs()))


def test_autograd_once_and_twice(ctp, dev):
    """Gradients and gradients of gradients against torch's on the same formula in float64."""
    g = torch.Generator().manual_seed(11)
    for gated, name, lmax in ((False, "silu", 0), (False, "gelu", 0), (True, "silu", 0), (True, "tanh", 0), (False, "none", 2)):
        c = Case(37, 20, 24, torch.float32, name, lmax=lmax, gated=gated, residual=not gated)
        x, w, b, r = (t.detach().clone().requires_grad_() if t is not None else None for t in to(dev, c.x, c.w, c.bias, c.residual))
        X, W, B, R = (t.detach().double().cpu().clone().requires_grad_() if t is not None else None for t in (x, w, b, r))
        y = ctp.gated_linear(x, w, b, act=name) if gated else ctp.linear(x, w, b, r, act=name, lmax=lmax)
        if gated:
            Z = [X @ W[k].T + B[k] for k in (0, 1)]
            Y = act(name, Z[0])[0] * Z[1]
        elif lmax:
            Y = torch.einsum("ndi,doi->ndo", X, W[degrees(lmax)])
            Y = torch.cat([Y[:, :1] + B, Y[:, 1:]], 1) + R
        else:
            Y = act(name, X @ W.T + B)[0] + R
        cot, cot2 = torch.randn(Y.shape, generator=g).double(), torch.randn(X.shape, generator=g).double()

        def both(y, x, w, b, r, cot, cot2):
            leaves = [t for t in (w, b, r) if t is not None]
            first = torch.autograd.grad((y * cot + 0.1 * y * y).sum(), [x, *leaves], create_graph=True)
            second = torch.autograd.grad((first[0] * cot2).sum(), [x, *leaves], allow_unused=True)
            return [*first, *second]

        got = both(y, x, w, b, r, cot.float().to(dev), cot2.float().to(dev))
        want = both(Y, X, W, B, R, cot, cot2)
        for k, (a, ref) in enumerate(zip(got, want)):
            if ref is None or a is None:
                assert (ref is None or not ref.any()) and (a is None or not a.any()), (name, k)
                continue
            # some 100 roundings of terms whose sum of absolute values is at most 100 times the largest value
            tol = 1e4 * EPS32 * float(ref.abs().max())
            assert float((a.double().cpu() - ref).abs().max()) <= tol, (name, gated, k)
        x2 = x.detach().requires_grad_()
        first = torch.autograd.grad(ctp.linear(x2, w[0] if w.dim() == 3 else w).square().sum(), [x2, w], create_graph=True)
        with pytest.raises(NotImplementedError):
            first[1].sum().backward()


def test_gradients_against_differences(ctp, dev):
    c = Case(9, 12, 10, torch.float32, "gelu", gated=True)
    x, w, b, grad = to(dev, c.x, c.w, c.bias, c.grad)
    _, z = ctp.gated_linear_fwd(x, w, b, act="gelu", keep_z=True)
    got = ctp.gated_linear_bwd(grad, x, w, z, act="gelu")

    def loss(x, w, b):
        Z = [x @ w[k].T + b[k] for k in (0, 1)]
        return float((act("gelu", Z[0])[0] * Z[1] * c.grad.double()).sum())

    at = [t.double().cpu() for t in (x, w, b)]
    g = torch.Generator().manual_seed(1)
    for k in range(3):
        d = torch.randn(at[k].shape, generator=g).double()
        step = 1e-5
        ends = [loss(*(t + s * step * d if j == k else t for j, t in enumerate(at))) for s in (1, -1)]
        diff, mine = (ends[0] - ends[1]) / (2 * step), float((got[k].double().cpu() * d).sum())
        assert abs(diff - mine) <= 1e-4 * (1 + abs(diff)), k


def test_block_run_together(ctp, dev):
    """Embedding, norm, gated block, output layer with the residual, clipping, orthogonalised step: as a model uses them."""
    g = torch.Generator().manual_seed(2)
    n, c, f = 90, 24, 40
    species = torch.randint(0, 10, (n,), generator=g).to(dev)
    std = lambda *s: torch.randn(*s, generator=g) * 0.3  # noqa: E731
    params = [std(10, c), 1 + 0.1 * std(c), std(2, f, c), std(c, f), std(4, c), std(4)]
    p = [t.to(dev).requires_grad_() for t in params]
    q = [t.double().requires_grad_() for t in params]
    r = ctp.embed(p[0], species)
    _, u = ctp.norm_residual(None, r, None, p[1])
    out = ctp.linear(ctp.linear(ctp.gated_linear(u, p[2]), p[3], residual=r), p[4], p[5], act="tanh")
    R = q[0][species.cpu()]
    Uu = R / (R.square().mean(1, keepdim=True) + 1e-6).sqrt() * q[1]
    H = torch.nn.functional.silu(Uu @ q[2][0].T) * (Uu @ q[2][1].T)
    OUT = torch.tanh((H @ q[3].T + R) @ q[4].T + q[5])
    assert float((out.double().cpu() - OUT).abs().max()) <= 1e-5
    got, want = torch.autograd.grad(out.square().sum(), p), torch.autograd.grad(OUT.square().sum(), q)
    for a, b in zip(got, want):
        assert float((a.double().cpu() - b).abs().max()) <= 1e-5 * (1 + float(b.abs().max()))
    clipped, norm = ctp.clip_grad_norm(got, 1.0)
    total = math.sqrt(sum(float(b.square().sum()) for b in want))
    assert abs(float(norm) - total) <= 1e-5 * total
    steps = ctp.orthogonalise([clipped[0], clipped[2], clipped[3]])
    for s, b in zip(steps, (want[0], want[2], want[3])):
        ref = newton_schulz(b)[0]
        assert float((s.double().cpu() - ref).norm()) <= 1e-3 * float(ref.norm())


def test_example_runs_with_orthogonalised_steps(dev):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_energy
    losses, norms = train_energy.train(steps=6, atoms=120, channels=16, lmax=1, log=None, orthogonal=True)
    assert len(losses) == 6 and all(math.isfinite(x) for x in losses + norms)


def test_example_gradients(ctp, dev):
    """The example's gradients through its radial networks: as with torch's own layers in them."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_energy
    species, vec, _, graph, batch, energy, _ = train_energy.structures(60, 2, dev, 0)
    torch.manual_seed(0)
    model = train_energy.Potential(8, 1, dev)
    vec.requires_grad_()
    params = [p for p in model.parameters()]

    def gradients():
        e = model(species, vec, graph, batch, 2)
        f, = torch.autograd.grad(e.sum(), vec, create_graph=True)
        return torch.autograd.grad((e - energy).square().sum() + f.square().sum(), params)

    got = gradients()
    own, ctp.linear = ctp.linear, lambda x, w, b, act="none": (
        torch.nn.functional.silu(torch.nn.functional.linear(x, w, b)) if act == "silu" else torch.nn.functional.linear(x, w, b))
    try:
        want = gradients()
    finally:
        ctp.linear = own
    # fp32 on both sides: some hundred roundings of terms up to a hundred times the result
    for a, b in zip(got, want):
        assert float((a - b).abs().max()) <= 1e4 * EPS32 * float(b.abs().max()) + 1e-6


# ---------------------------------------------------------------- orthogonalising

QUINTIC = (3.4445, -4.7750, 2.0315)


def newton_schulz(m, steps=5, eps=1e-7):
    """(result, bound of the kernels' error in the Frobenius norm) of one matrix or a batch of them, in float64.

    The step is an odd polynomial p of the singular values, so it carries an error e of X (Frobenius norm) to at most
    g e, g the largest |p(s) -+ p(t)| / |s -+ t| over the singular values (0 among them where sides differ).  What a step
    adds: X, A and B = b A + c A A are rounded to 22 bits and their products summed in fp32 in three parts, each sum of k
    terms off by at most (3 k + 8) 2^-23 of the sum of absolute values, which has at most the product of the factors'
    Frobenius norms as its own; B's rounding and A's reach X through products with it."""
    if m.dim() > 2:
        parts = [newton_schulz(x, steps, eps) for x in m.reshape(-1, *m.shape[-2:])]
        return torch.stack([p[0] for p in parts]).view(m.shape), max((p[1] for p in parts), default=0.0)
    m = m.double()
    x = m.T if m.shape[0] > m.shape[1] else m
    a, b, c = QUINTIC
    x = x / (x.norm() + eps)
    e = 2.0 ** -21
    for _ in range(steps):
        s = torch.cat([torch.linalg.svdvals(x), torch.zeros(1, dtype=torch.float64)])
        p = a * s + b * s ** 3 + c * s ** 5
        up = (p[:, None] + p[None]).abs() / (s[:, None] + s[None]).clamp(min=1e-300)
        gap = (s[:, None] - s[None]).abs()
        near = gap < 1e-9
        down = torch.where(near, (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs()[:, None].expand_as(gap),
                           (p[:, None] - p[None]).abs() / gap.clamp(min=1e-300))
        grow = float(torch.maximum(up.where((s[:, None] + s[None]) > 1e-12, torch.tensor(a, dtype=torch.float64)), down).max())
        A = x @ x.T
        B = b * A + c * (A @ A)
        k_s, k_l = min(x.shape), max(x.shape)
        fro, two = float(x.norm()), float(s.max())
        # additions come in blocks of 16 terms a matrix instruction and the terms' signs and roundings are not all alike:
        # errors add up like the root of their number
        r = lambda k: (2.0 ** -22) + 2.0 ** -23 * math.sqrt(3 * k + 8)  # noqa: E731
        dA = r(k_l) * fro * fro
        dB = abs(b) * dA + 2 * abs(c) * float(A.norm()) * dA + r(k_s) * float(A.norm()) ** 2 * abs(c) + 2.0 ** -22 * float(B.norm())
        e = grow * e + dB * two + r(k_s) * float(B.norm()) * fro + 2.0 ** -22 * a * fro
        x = a * x + B @ x
    return (x.T if m.shape[0] > m.shape[1] else x), e


ORTHO = [(1, 1), (40, 2500), (3001, 130), (1, 7), (9, 1), (5, 5), (16, 16), (33, 65), (64, 64), (128, 128), (130, 64), (63, 200), (64, 700), (519, 70),
         (200, 257), (3, 40, 40), (2, 3, 20, 50), (4, 70, 33), (0, 5, 5), (300, 300)]


@pytest.mark.parametrize("dtype", DTYPES)
def test_orthogonalise(ctp, dev, dtype):
    g = torch.Generator().manual_seed(4)
    ms = [normal(g, s, dtype, 0.01) for s in ORTHO]
    tell("orthogonalise", len(ms), dtype)
    ins = [m.to(dev) for m in ms]
    outs = ctp.orthogonalise(ins)
    for m, i, o in zip(ms, ins, outs):
        assert torch.equal(i.cpu(), m) and o.dtype == dtype and o.shape == m.shape
        if m.numel() == 0:
            continue
        ref, e = newton_schulz(m)
        n = 1 if m.dim() == 2 else m[..., 0, 0].numel()
        err = float((o.double().cpu() - ref).norm())
        assert err <= (e * math.sqrt(n) + U[dtype] * float(ref.norm())) * (1 + 2.0 ** -10), (m.shape, err, e)
    again = ctp.orthogonalise(ins, out=ins)
    assert all(torch.equal(a, b) for a, b in zip(again, outs)), "in place, not the same bits"
    # alone, and as one of many: the same result
    for k in (1, 2, 5, 10, 14):
        alone, = ctp.orthogonalise([ms[k].to(dev)])
        assert torch.equal(alone, outs[k])


@pytest.mark.parametrize("shape", [(96, 96), (80, 320), (260, 100)])
def test_orthogonalise_few_directions(ctp, dev, shape):
    """Few strong directions among noise, where rounding noise grows with the weak ones."""
    g = torch.Generator().manual_seed(5)
    m = torch.randn(shape[0], 4, generator=g) @ torch.randn(4, shape[1], generator=g) + 0.01 * torch.randn(shape, generator=g)
    for dtype in DTYPES:
        t = m.to(dtype)
        o, = ctp.orthogonalise([t.to(dev)], scale=0.5)
        ref, e = newton_schulz(t)
        assert float((o.double().cpu() - 0.5 * ref).norm()) <= 0.5 * e + U[dtype] * float(0.5 * ref.norm())


def test_orthogonalise_edges(ctp, dev):
    z = torch.zeros(70, 40, device=dev)
    assert not ctp.orthogonalise([z])[0].any()
    big = torch.full((20, 30), 3e38, device=dev)
    big[0, 0] = -3e38
    small = big * 1e-38 * 1e-30
    a, b = ctp.orthogonalise([big, small], eps=0.0)
    ref = newton_schulz(big.cpu(), eps=0.0)
    assert float((a.double().cpu() - ref[0]).norm()) <= ref[1] + EPS32 * float(ref[0].norm())
    assert torch.isfinite(b).all()
    x = torch.randn(3, 40, 50, device=dev)
    x[1, 3, 4] = float("nan")
    o, = ctp.orthogonalise([x])
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all() and not torch.isfinite(o[1]).any()
    for steps in (1, 2, 8):
        m = torch.randn(50, 60)
        o, = ctp.orthogonalise([m.to(dev)], steps=steps)
        ref, e = newton_schulz(m, steps)
        assert float((o.double().cpu() - ref).norm()) <= e + EPS32 * float(ref.norm())
    # more tensors than one launch takes, of mixed types
    many = [torch.randn(5 + k, 70 - k, device=dev).to(DTYPES[k % 3]) for k in range(70)]
    for m, o in zip(many, ctp.orthogonalise(many)):
        assert torch.equal(o, ctp.orthogonalise([m])[0])


def test_streams_and_graphs(ctp, dev):
    """On another stream, and captured and replayed: the eager result each time."""
    g = torch.Generator().manual_seed(6)
    c = Case(200, 72, 100, torch.bfloat16, "silu", gated=True)
    x, w, b, grad = to(dev, c.x, c.w, c.bias, c.grad)
    m = normal(g, (100, 72), torch.float32).to(dev)

    def step():
        h, z = ctp.gated_linear_fwd(x, w, b, keep_z=True)
        return [h, *ctp.gated_linear_bwd(grad, x, w, z), *ctp.orthogonalise([m, w])]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b2) for a, b2 in zip(other, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(normal(g, x.shape, torch.bfloat16).to(dev))
        m.mul_(1.5).add_(0.1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b2) for a, b2 in zip(out, step())), k


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_far_apart(ctp, dev, dtype):
    """Row strides at which a tile's offsets pass 32 bits."""
    rows, inner, outer, stride = 260, 64, 8320, 9_000_000
    base = torch.empty(rows * stride, dtype=dtype, device=dev)
    far = base.as_strided((rows, inner), (stride, 1))
    g = torch.Generator().manual_seed(8)
    x = normal(g, (rows, inner), dtype).to(dev)
    far.copy_(x)
    w = normal(g, (outer, inner), dtype, 0.1).to(dev)
    assert torch.equal(ctp.linear_fwd(far, w)[0], ctp.linear_fwd(x, w)[0])
    grad = normal(g, (rows, outer), dtype).to(dev)
    for a, b in zip(ctp.linear_bwd(grad, far, w), ctp.linear_bwd(grad, x, w)):
        assert float((a - b).abs().max()) <= 8 * U[dtype] * float(b.abs().max())
    del far, base
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", DTYPES)
def test_stride_of_a_single_row_is_not_looked_at(ctp, dev, dtype):
    """Through the C ABI, where the stride of one row may be anything."""
    import ctypes

    from tensor_product_message_amd import _capi
    L = _capi.dense_lib()
    c = Case(1, 1024, 2048, dtype, "silu")
    x, w, grad = to(dev, c.x, c.w, c.grad)
    z = torch.zeros(1, 2048, dtype=dtype, device=dev)
    want = ctp.linear_bwd(grad, x, w, z, act="silu")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for stride in (0, 8, -64):
        prob = _capi.LinearProblem(1, stride, stride, stride, 0, 1024, 2048, DTYPES.index(dtype), 2, 0)
        n = ctypes.c_int64()
        assert L.conv_tp_linear_bwd_workspace(ctypes.byref(prob), ctypes.byref(n)) == 0
        ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
        got = [torch.empty_like(t) for t in want]
        st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert L.conv_tp_linear_bwd(ctypes.byref(prob), p(grad), p(x), p(w), p(z), *map(p, got), p(ws), n.value, st) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want)), stride


def test_no_grad_and_frozen(ctp, dev):
    x, w, b = torch.randn(5, 8, device=dev), torch.randn(6, 8, device=dev), torch.randn(6, device=dev)
    want = torch.nn.functional.silu(x @ w.T + b)
    for req in (False, True):
        w.requires_grad_(req)
        with torch.no_grad():
            y = ctp.linear(x, w, b, act="silu")
        assert not y.requires_grad and float((y - want).abs().max()) <= 1e-5
    y = ctp.linear(x, w, b, act="silu")
    y.sum().backward()
    assert x.grad is None and b.grad is None and w.grad.shape == w.shape
    with torch.inference_mode():
        assert float((ctp.gated_linear(x, w.detach().view(2, 3, 8)) - torch.nn.functional.silu(x @ w[:3].T) * (x @ w[3:].T)).abs().max()) <= 1e-4


def test_refusals(ctp, dev):
    x, w = torch.randn(4, 8, device=dev), torch.randn(6, 8, device=dev)
    bad = [
        (lambda: ctp.linear_fwd(x, w, act="swish"), ValueError), (lambda: ctp.linear_fwd(x, w.half()), ValueError),
        (lambda: ctp.linear_fwd(x, w[:, :7]), ValueError), (lambda: ctp.linear_fwd(x, w.t()), ValueError),
        (lambda: ctp.linear_fwd(x.t(), w), ValueError), (lambda: ctp.linear_fwd(x, w, w[0]), ValueError),
        (lambda: ctp.linear_fwd(x, w, residual=x), ValueError), (lambda: ctp.linear_fwd(x, w.cpu()), ValueError),
        (lambda: ctp.linear_fwd(x.double(), w.double()), ValueError), (lambda: ctp.linear_fwd(x, w, lmax=1), ValueError),
        (lambda: ctp.linear_fwd(x[:, None], w[None], act="silu", lmax=0), ValueError),
        (lambda: ctp.linear_fwd(torch.randn(4, 4, 8, device=dev), torch.randn(2, 6, 8, device=dev), act="silu", lmax=1), ValueError),
        (lambda: ctp.linear_fwd(x, w, out=x), ValueError), (lambda: ctp.linear_fwd(None, w), TypeError),
        (lambda: ctp.linear_bwd(x, x, w), ValueError), (lambda: ctp.linear_bwd(torch.ones(4, 6, device=dev), x, w, act="silu"), TypeError),
        (lambda: ctp.linear_bwd(torch.ones(4, 6, device=dev), x, w, workspace=torch.empty(8, device=dev)), ctp.ConvTPError),
        (lambda: ctp.gated_linear_fwd(x, w), ValueError), (lambda: ctp.gated_linear_fwd(x, w.view(2, 3, 8), act=3), ValueError),
        (lambda: ctp.orthogonalise([]), ValueError), (lambda: ctp.orthogonalise([x[0]]), ValueError),
        (lambda: ctp.orthogonalise([x.t()]), ValueError), (lambda: ctp.orthogonalise([x], steps=0), ValueError),
        (lambda: ctp.orthogonalise([x], eps=-1.0), ctp.ConvTPError), (lambda: ctp.orthogonalise([x], out=[w]), ValueError),
        (lambda: ctp.orthogonalise([x.double()]), ValueError), (lambda: ctp.orthogonalise([x, w.cpu()]), ValueError),
    ]
    for k, (call, error) in enumerate(bad):
        with pytest.raises(error):
            call()
            tell("accepted", k)
