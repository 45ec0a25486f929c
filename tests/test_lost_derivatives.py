"""Derivatives that distillation and replay do not give are refused, not dropped."""
import pytest

import top_support_capture_gb300 as sfc
from top_support_capture_gb300 import training

torch = pytest.importorskip("torch")
fwAD = torch.autograd.forward_ad


def test_check():
    x, T, y = torch.zeros(3, 10, requires_grad=True), torch.ones(3), torch.zeros(3, 4)
    f = lambda x=x, T=T, y=y: training.check_derivatives(x, temperature=T, teacher_values=y)
    f()
    for kw, name in (({"T": T.clone().requires_grad_()}, "temperature"), ({"y": y.clone().requires_grad_()}, "teacher_values")):
        with pytest.raises(sfc.SfcError, match=name):
            f(**kw)
        with torch.no_grad():
            f(**kw)
    with fwAD.dual_level():
        f()
        for name, key, t in (("logits", "x", x.detach()), ("temperature", "T", T), ("teacher_values", "y", y)):
            with pytest.raises(sfc.SfcError, match=f"{name}.*forward-mode"):
                f(**{key: fwAD.make_dual(t, torch.ones_like(t))})
            with torch.no_grad(), pytest.raises(sfc.SfcError, match="forward-mode"):
                f(**{key: fwAD.make_dual(t, torch.ones_like(t))})
    f()


@pytest.mark.gpu
def test_calls():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B, V, W = 2, 100, 4
    x, T = torch.randn(B, V, device="cuda"), torch.ones(B, device="cuda")
    ids = torch.arange(W, dtype=torch.int32, device="cuda").expand(B, W).contiguous()
    y, n = torch.full((B, W), -1.4, device="cuda"), torch.full((B,), W, dtype=torch.int32, device="cuda")
    tok = torch.zeros(B, dtype=torch.int32, device="cuda")
    calls = (lambda x=x, T=T, y=y: sfc.distill_loss(x, T, ids, y, n).loss, lambda x=x, T=T, y=y: sfc.replay_logprob(x, T, ids, n, tok).token_logprob)
    grad = lambda t: t.clone().requires_grad_()
    for f in calls:
        plain = f()
        with pytest.raises(sfc.SfcError, match="temperature requires a gradient"):
            f(grad(x), grad(T))
        with fwAD.dual_level():
            with pytest.raises(sfc.SfcError, match="forward-mode"):
                f(fwAD.make_dual(x, torch.ones_like(x)))
            with pytest.raises(sfc.SfcError, match="forward-mode"):
                f(T=fwAD.make_dual(T, torch.ones_like(T)))
            assert torch.equal(f(), plain)
        assert torch.equal(f(grad(x)), plain) and f(grad(x)).requires_grad
        with torch.no_grad():
            assert torch.equal(f(grad(x), grad(T)), plain)
    with pytest.raises(sfc.SfcError, match="teacher_values requires a gradient"):
        calls[0](y=grad(y))
    # a temperature that requires a gradient beside logits that do not: a constant, as ever
    assert not calls[1](T=grad(T)).requires_grad
