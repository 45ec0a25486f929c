"""The example program: distillation lowers the loss, and a trained draft yields more tokens per call of the target."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_draft_and_verify(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_and_verify.py")
    spec = importlib.util.spec_from_file_location("draft_and_verify", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses, before, after, tuned, dense = module.main()
    assert torch.isfinite(losses).all() and float(losses[-1]) < 0.5 * float(losses[0])
    assert 1.0 <= before < after <= module.DRAFTS + 1 and tuned > before and dense > 1.0
