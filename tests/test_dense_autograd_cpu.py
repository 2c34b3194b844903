"""What the dense operators' wrappers leave to autograd, without a GPU: a stub stands for the native calls."""
import pytest
import torch
from torch.autograd import forward_ad

from tensor_product_message_amd import dense


class Stub:
    calls = 0

    def linear_fwd(self, x, w, bias, residual, act, lmax, gated, keep_z, out):
        self.calls += 1
        z = x @ w.flatten(0, -2).T
        return (z[..., :w.shape[-2]] * z[..., w.shape[-2]:] if gated else z), (z if keep_z else None)


@pytest.fixture
def stub(monkeypatch):
    s = Stub()
    monkeypatch.setattr(dense, "dense_native", lambda: s)
    return s


CALLS = [lambda x, w: dense.linear(x, w[0]), lambda x, w: dense.gated_linear(x, w),
         lambda x, w: dense.linear(x.detach(), w[0], residual=x[:, :3])]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("grad_mode", [False, True])
def test_forward_mode_is_refused(stub, call, grad_mode):
    """A tangent must not get lost: forward mode works under no_grad too."""
    x, w = torch.randn(4, 8), torch.randn(2, 3, 8)
    with torch.set_grad_enabled(grad_mode), forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        assert forward_ad.unpack_dual(dual @ w[0].T).tangent is not None
        with pytest.raises((RuntimeError, NotImplementedError)):
            call(dual, w)
        # nothing asked of these
        y = call(x, w)
        assert forward_ad.unpack_dual(y).tangent is None
    assert call(x, w).shape == (4, 3)


@pytest.mark.parametrize("call", CALLS)
def test_forward_mode_by_transform_is_refused(stub, call):
    x, w = torch.randn(4, 8), torch.randn(2, 3, 8)
    with torch.no_grad(), pytest.raises((RuntimeError, NotImplementedError)):
        torch.func.jvp(lambda x: call(x, w), (x,), (torch.ones_like(x),))


def test_without_derivatives_the_call_goes_past_autograd(stub, monkeypatch):
    x, w = torch.randn(4, 8), torch.randn(2, 3, 8, requires_grad=True)
    monkeypatch.setattr(dense.LinearFunction, "apply", lambda *a: pytest.fail("through autograd"))
    with torch.no_grad():
        assert not dense.linear(x, w[0]).requires_grad and not dense.gated_linear(x, w).requires_grad
    with torch.inference_mode():
        dense.linear(x, w[0])
    assert stub.calls == 3
