"""Derivatives that the calls over the whole vocabulary and the gradient norm do not give are refused, not dropped."""
import pytest

import top_support_capture_gb300 as sfc

torch = pytest.importorskip("torch")
fwAD = torch.autograd.forward_ad


@pytest.mark.gpu
def test_calls_over_the_whole_vocabulary():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B, V = 2, 100
    x, T = torch.randn(B, V, device="cuda"), torch.ones(B, device="cuda")
    tok = torch.zeros(B, dtype=torch.int32, device="cuda")
    f = lambda x=x, T=T: sfc.token_logprobs(x, T, tok, top=2).logprobs
    grad = lambda t: t.clone().requires_grad_()
    plain = f()
    with pytest.raises(sfc.SfcError, match="temperature requires a gradient"):
        f(grad(x), grad(T))
    with fwAD.dual_level():
        for kw in (dict(x=fwAD.make_dual(x, torch.ones_like(x))), dict(T=fwAD.make_dual(T, torch.ones_like(T)))):
            with pytest.raises(sfc.SfcError, match="forward-mode"):
                f(**kw)
        with pytest.raises(sfc.SfcError, match="forward-mode"):
            sfc.grad_norm([fwAD.make_dual(x, torch.ones_like(x))])
        assert torch.equal(f(), plain)
    y = grad(x)
    assert torch.equal(f(y), plain) and f(y).requires_grad
    (first,) = torch.autograd.grad(f(y).sum(), y, create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        torch.autograd.grad(first.sum(), y)
    with torch.no_grad():
        assert torch.equal(f(grad(x), grad(T)), plain) and not f(y).requires_grad
    with pytest.raises(sfc.SfcError, match="keep_stats"):
        sfc.token_logprobs(y, T, tok, keep_stats=True)
    out = f(y)
    with torch.no_grad():
        y.mul_(2.0)  # changed before its gradient is taken
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()
