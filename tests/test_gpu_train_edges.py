"""The training-step operators at the ends of their documented ranges.  Forms,
bounds and their derivation are test_gpu_train.py's."""
import pytest
import torch

from tests.test_gpu_train import (SECOND, close, ctp, dev, draw_tokens, embed_bwd_ref, gen, norm_case,  # noqa: F401
                                  norm_ref, normal, second_bounds, second_ref, tell)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rows that a workgroup has too many


# Rows of up to 16, 64 and 128 vectors share a workgroup, 16, 4 and 2 at once; wider ones have it to themselves.
UNEVEN = [  # rows, lmax, channels
    (1, 0, 8), (5, 0, 64), (17, 0, 40), (3, 0, 250), (5, 0, 500), (1, 0, 1003), (3, 0, 1100), (3, 0, 2048), (5, 1, 5),
    (17, 2, 9), (7, 3, 8), (31, 3, 16), (1, 2, 33),
]


@pytest.mark.parametrize("kind", ["none", "channel", "row"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,lmax,c", UNEVEN)
def test_norm_gradients_without_eps(ctp, dev, rows, lmax, c, dtype, kind):
    """eps = 0 and no row of zeros: everything is finite, whatever a workgroup's places without a row hold."""
    t, w = norm_case(rows, lmax, c, dtype, torch.float32 if c % 2 else dtype, kind, rows + lmax + c + 1)
    tell("norm eps 0", rows, lmax, c, dtype, kind)
    d = {k: None if v is None else v.to(dev) for k, v in t.items()}
    args = (d["grad_r"], d["grad_u"], d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 0.5, 0.0, lmax)
    terms = rows * (2 * lmax + 1)

    def shared(name):
        return "_w_" in name or (name.endswith("gate") and kind == "channel")
    got = dict(zip(("d_h", "d_r", "d_w_post", "d_w_pre", "d_gate"), ctp.norm_residual_bwd(*args)))
    ref = norm_ref(w["h"], w["r"], w["w_post"], w["w_pre"], w["gate"], 0.5, 0.0, lmax, w["grad_r"], w["grad_u"])
    for name, (x, S) in ref.items():
        close(name, got[name].reshape(x.shape), x, S, 256 + terms * shared(name))
    g = gen(rows + c)
    Q, P = normal(g, t["h"].shape, dtype), normal(g, t["h"].shape, dtype)
    Q64, P64 = (x.double().reshape(w["h"].shape) for x in (Q, P))
    got = dict(zip(SECOND, ctp.norm_residual_bwd_bwd(Q.to(dev), P.to(dev), *args)))
    ref, S = second_ref(w, 0.5, 0.0, lmax, Q64, P64), second_bounds(w, 0.5, 0.0, lmax, Q64, P64)
    for name, x in ref.items():
        close(name, got[name].reshape(x.shape), x, S[name], 512 + terms * shared(name))


@pytest.mark.parametrize("c", [8, 250, 500])
def test_norm_gradients_of_infinite_parameters(ctp, dev, c):
    """One row in a workgroup of 16, 4 or 2: an infinite parameter gives the other one's gradient infinity in its
    channel, as the formula does, and not NaN."""
    t, w = norm_case(1, 0, c, torch.float32, torch.float32, "channel", c)
    tell("norm infinite", c)
    g = gen(c + 1)
    Q, P = normal(g, (1, c), torch.float32), normal(g, (1, c), torch.float32)
    for param, first, second in (("gate", "d_w_post", "g_w_post"), ("w_post", "d_gate", "g_gate")):
        x, x64 = dict(t), dict(w)
        x[param] = t[param].clone()
        x[param][3] = float("inf")
        x64[param] = x[param].double().reshape(w[param].shape)
        d = {k: v.to(dev) for k, v in x.items()}
        args = (d["grad_r"], d["grad_u"], d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 0.5, 1e-6, 0)
        got = dict(zip(("d_h", "d_r", "d_w_post", "d_w_pre", "d_gate"), ctp.norm_residual_bwd(*args)))
        ref, S = norm_ref(x64["h"], x64["r"], x64["w_post"], x64["w_pre"], x64["gate"], 0.5, 1e-6, 0, x64["grad_r"],
                          x64["grad_u"])[first]
        rest = [k for k in range(c) if k != 3]
        assert bool(ref[0, 3].isinf())
        assert float(got[first][3]) == float(ref[0, 3])
        close(first, got[first][rest], ref[0, rest], S[0, rest], 257)
        # the second pass: EB alpha d times the other parameter, EB = s1 (Q - h^ <b Q, h^>)
        d64 = norm_ref(None, x64["r"], None, x64["w_pre"], None, 0.5, 1e-6, 0, x64["grad_r"], x64["grad_u"])["d_r"][0]
        h = x64["h"] * (x64["h"].square().mean() + 1e-6).rsqrt()
        eb = (x64["h"].square().mean() + 1e-6).rsqrt() * (Q.double() - h * (Q.double() * h).mean())
        ref = (eb * 0.5 * d64 * x64[param])[0, 0]
        got = dict(zip(SECOND, ctp.norm_residual_bwd_bwd(Q.to(dev), P.to(dev), *args)))
        assert float(got[second][3]) == float(ref[3])
        assert bool(got[second].isfinite()[rest].all())


# ---------------------------------------------------------------- more than one launch


def test_norm_rows_beyond_a_launch(ctp, dev):
    """2^28 + 21 rows of one value, 16 lanes each: more than the 2^32 - 1 threads of a launch."""
    n = 2 ** 28 + 21
    g = torch.Generator(device=dev).manual_seed(3)
    h, r, gate = (torch.randn((n, 1), generator=g, device=dev, dtype=torch.float16) for _ in range(3))
    w = torch.tensor([1.5], dtype=torch.float16, device=dev)
    out = tuple(torch.full((n, 1), float("nan"), dtype=torch.float16, device=dev) for _ in range(2))
    tell("norm rows", n)
    ctp.norm_residual_fwd(h, r, w, w, gate, 0.5, out=out)
    assert not any(bool(x.isnan().any()) for x in out)
    at = torch.cat([torch.arange(n - 40, n, device=dev), torch.arange(40, device=dev),
                    torch.arange(2 ** 28 - 60, 2 ** 28 + 20, device=dev),
                    torch.randint(0, n, (4096,), generator=g, device=dev)])
    part = ctp.norm_residual_fwd(h[at], r[at], w, w, gate[at], 0.5)
    assert all(torch.equal(x[at], y) for x, y in zip(out, part))


def test_table_rows_beyond_a_launch(ctp, dev):
    """The gradient of a table of 2^29 + 77 rows: the workgroups that write its zero rows."""
    v = 2 ** 29 + 77
    tok = torch.tensor([0, v - 1, 2 ** 29, 5, -1], device=dev)
    grad = torch.arange(1, 6, dtype=torch.float16, device=dev)[:, None]
    table = torch.full((v, 1), float("nan"), dtype=torch.float16, device=dev)
    tell("table rows", v)
    ctp.embed_bwd(grad, tok, v, out=table)
    assert torch.equal(table[tok[:4]], grad[:4])
    assert int((table != 0).sum()) == 4


def test_lookups_beyond_a_launch(ctp, dev):
    """2^26 + 3 tokens of 1025 channels, a quarter of a workgroup of 256 each."""
    n, c = 2 ** 26 + 3, 1025
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160 * 2 ** 30:
        pytest.skip("needs 160 GiB of GPU memory")
    g = torch.Generator(device=dev).manual_seed(5)
    table = torch.randn((50, c), generator=g, device=dev, dtype=torch.float16)
    tok = torch.randint(0, 50, (n,), generator=g, device=dev, dtype=torch.int32)
    out = torch.full((n, c), float("nan"), dtype=torch.float16, device=dev)
    tell("lookups", n)
    ctp.embed_fwd(table, tok, out=out)
    for k in range(0, n, 2 ** 20):
        assert torch.equal(out[k:k + 2 ** 20], table[tok[k:k + 2 ** 20].long()]), k
    del out
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- outputs that autograd watches


def test_given_outputs_count_as_written(ctp, dev):
    """Every output that the caller gives gets a new version, so that a backward pass which saved it refuses it."""
    f = lambda *s: torch.ones(s, device=dev)  # noqa: E731
    ids = torch.zeros(4, dtype=torch.int64, device=dev)
    outs = [f(4, 8), f(3, 8), f(4, 8), f(4, 8), f(4, 8), torch.ones((), device=dev)]
    before = [x._version for x in outs]
    ctp.embed_fwd(f(3, 8), ids, out=outs[0])
    ctp.embed_bwd(f(4, 8), ids, 3, out=outs[1])
    ctp.norm_residual_fwd(f(4, 8), f(4, 8), f(8), f(8), out=(outs[2], outs[3]))
    ctp.clip_grad_norm([f(4, 8)], 1.0, out=[outs[4]])
    ctp.grad_norm([f(4, 8)], out=outs[5])
    assert all(x._version > v for x, v in zip(outs, before)), [x._version - v for x, v in zip(outs, before)]
    x, w = f(4, 8), f(8)
    for call in (lambda ws: ctp.embed_bwd(x, ids, 3, workspace=ws),
                 lambda ws: ctp.norm_residual_bwd(x, x, x, x, w, w, workspace=ws),
                 lambda ws: ctp.norm_residual_bwd_bwd(x, x, x, x, x, x, w, w, workspace=ws)):
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
        call(ws)
        assert ws._version > 0


@pytest.mark.parametrize("how", ["clip", "norm", "embed_fwd", "embed_bwd", "grad_norm"])
def test_a_saved_tensor_that_is_written_is_refused(ctp, dev, how):
    x = torch.randn((4, 8) if how != "grad_norm" else (), device=dev, requires_grad=True)
    y = 2 * x
    loss = y.square().sum()                 # saves y
    to, one, ids = y.detach(), torch.ones(8, device=dev), torch.arange(4, device=dev)
    {"clip": lambda: ctp.clip_grad_norm([to], 0.1, out=[to]),
     "norm": lambda: ctp.norm_residual_fwd(torch.ones_like(to), to, one, one, out=(to, None)),
     "embed_fwd": lambda: ctp.embed_fwd(torch.ones(4, 8, device=dev), ids, out=to),
     "embed_bwd": lambda: ctp.embed_bwd(torch.ones(4, 8, device=dev), ids, 4, out=to),
     "grad_norm": lambda: ctp.grad_norm([torch.ones(4, device=dev)], out=to)}[how]()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_written(ctp, dev):
    """They have no version; writing them needs none."""
    ids = torch.arange(4, device=dev)
    with torch.inference_mode():
        table, out = torch.randn(4, 8, device=dev), torch.zeros(4, 8, device=dev)
        ctp.embed_fwd(table, ids, out=out)
        assert torch.equal(out, table)
    out2 = ctp.embed_fwd(table, ids, 2.0, out=out)
    assert out2 is out and torch.equal(out, 2 * table)


# ---------------------------------------------------------------- norms and factors outside float32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value,n,max_norm", [
    (3e38, 4, 1.0),             # the norm is above float32's largest number
    (3e38, 5003, 0.125),        # so is the norm, and the factor below its smallest
    (1e37, 100, 0.5),           # the norm fits, the factor is subnormal
    (1e30, 20000, 1e-9), (2e38, 2, 1e-3),
])
def test_clip_norms_beyond_float32(ctp, dev, value, n, max_norm, dtype):
    """The squares are summed in 64 bits, so the clipped gradients are the formula's although the norm, one float,
    overflows or the factor is no normal one.  Two products and a sum of 64 bits: K = 8."""
    x = torch.full((n,), value).to(dtype)
    x[::3] *= -0.5
    small = torch.linspace(-1e-3, 1e3, 77).to(dtype)
    tell("clip", value, n, max_norm, dtype)
    norm = float(torch.cat([x.double(), small.double()]).norm())
    max64 = float(torch.tensor(max_norm, dtype=torch.float32))
    for in_place in (False, True):
        d = [x.to(dev), small.to(dev)]
        out, got = ctp.clip_grad_norm(d, max_norm, out=d if in_place else None)
        ref = torch.tensor(norm, dtype=torch.float64).float()
        assert float(got) == float(ref) if ref.isinf() else abs(float(got) - norm) <= 2 ** -23 * norm
        for o, i in zip(out, (x, small)):
            want = i.double() * (max64 / (norm + 1e-6))
            close("out", o, want, want.abs(), 8)


# ---------------------------------------------------------------- the embedding gradient's choices


@pytest.mark.parametrize("dtype,out,c,rows", [  # a workgroup a row and 8 vectors: both sides of 2 and 4 rounds
    (torch.float32, None, 32, 1024), (torch.float32, None, 32, 1025), (torch.float32, None, 30, 2048),
    (torch.float32, None, 30, 2049), (torch.float32, None, 1000, 64), (torch.float32, None, 1000, 65),
    (torch.bfloat16, None, 64, 512), (torch.bfloat16, None, 64, 513), (torch.float16, None, 61, 1024),
    (torch.float16, torch.float32, 61, 1025), (torch.bfloat16, torch.float32, 250, 256),
])
@pytest.mark.parametrize("n", [4096, 4097, 8192, 8193])
def test_embed_bwd_at_the_ends_of_the_one_launch_form(ctp, dev, n, dtype, out, c, rows):
    g = gen(n + rows)
    grad, tok = normal(g, (n, c), dtype), draw_tokens(g, n, rows, 2, 0.1)
    tell("embed_bwd ends", n, dtype, out, c, rows)
    ref, S, K = embed_bwd_ref(grad, tok, rows, 0.7)
    close("d_table", ctp.embed_bwd(grad.to(dev), tok.to(dev), rows, 0.7, dtype=out), ref, S, K)


@pytest.mark.parametrize("n,v,c,dtype", [  # both sides of 2^21 and 2^23 vectors
    (2 ** 20 - 1, 700, 8, torch.float32), (2 ** 20, 700, 8, torch.float32), (4095, 900, 2048, torch.float32),
    (4096, 900, 2045, torch.float32), (16383, 300, 2048, torch.float32), (16384, 300, 2047, torch.float32),
    (131071, 5000, 121, torch.bfloat16), (131072, 5000, 121, torch.bfloat16), (2 ** 19, 60000, 126, torch.float16),
])
def test_embed_bwd_of_every_chunk_length(ctp, dev, n, v, c, dtype):
    g = gen(n + c)
    grad, tok = normal(g, (n, c), dtype), draw_tokens(g, n, v, 2, 0.05)
    tell("embed_bwd chunks", n, v, c, dtype)
    ref, S, K = embed_bwd_ref(grad, tok, v, -1.5)
    got = ctp.embed_bwd(grad.to(dev), tok.to(dev), v, -1.5)
    close("d_table", got, ref, S, K)
    assert torch.equal(got, ctp.embed_bwd(grad.to(dev), tok.to(dev), v, -1.5))


# ---------------------------------------------------------------- one row without a batch


@pytest.mark.parametrize("lmax,c", [(0, 24), (2, 7)])
@pytest.mark.parametrize("kind", ["float32", "own"])
def test_norm_of_a_single_row(ctp, dev, lmax, c, kind):
    """[C] or [D, C] alone: a gate of the parameters' shape may have their type or the features', as in a batch."""
    t, _ = norm_case(1, lmax, c, torch.bfloat16, torch.float32, "channel", 6)
    if kind == "own":
        t["gate"] = t["gate"].bfloat16()
    d = {k: v.to(dev) for k, v in t.items()}
    one = {k: v[0] if k in ("h", "r", "grad_r", "grad_u") else v for k, v in d.items()}
    in_batch = d["gate"] if kind == "float32" else d["gate"][None]      # in the features' type it is a gate of every row

    def passes(x, gate):
        fwd = ctp.norm_residual_fwd(x["h"], x["r"], x["w_post"], x["w_pre"], gate, 0.5, 1e-6, lmax)
        bwd = ctp.norm_residual_bwd(x["grad_r"], x["grad_u"], x["h"], x["r"], x["w_post"], x["w_pre"], gate, 0.5, 1e-6, lmax)
        return [*fwd, *bwd]
    for got, want in zip(passes(one, d["gate"]), passes(d, in_batch)):
        assert got.dtype == want.dtype and torch.equal(got, want.reshape(got.shape))
