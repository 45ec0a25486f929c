"""Log-probabilities of finite logits that lie further below the row's largest than the largest float32: at T > 1 they are
numbers. Tolerances as in test_token_logprobs_gpu and test_policy_gpu."""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import _cuda, as_input  # noqa: F401 (the fixture)
from test_policy_gpu import call, check
from test_token_logprobs_gpu import args, check_values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("V", [5, 2053, 100003])
def test_logits_at_both_ends(dtype, V):
    import top_support_capture_gb300 as sfc

    K = 5
    l = np.full((4, V), -3.3e38, np.float32)
    l[0, 1:3] = [3e38, 2e38]
    l[1, 1:3] = [4e37, -1e38]
    l[2, 1:3] = [1.0, -3e38]
    l[3, 1:3] = [2e38, -np.inf]
    c = dict(l=as_input(l, dtype), dtype=dtype, T=np.array([10.0, 3.0, 2.0, 1.0], np.float32), tokens=np.array([[0, 1], [0, 2], [0, 2], [0, 2]], np.int32))
    ref = oracle.token_logprobs(c["l"], dtype, c["T"], c["tokens"], K)
    assert np.isfinite(ref.logprobs).sum() == 7 and np.abs(ref.logprobs[3, 0]) > 3.5e38  # (the last row's is not a float32)
    out = sfc.token_logprobs(*args(c), top=K)
    assert torch.isfinite(out.logprobs[:3]).all() and torch.isfinite(out.top_logprobs[:3]).all()
    check_values(c, ref, out, K)
    for column in (0, 1):
        some = dict(c, l=c["l"][:3], T=c["T"][:3], tokens=c["tokens"][:3, column], A=np.full(3, 0.25, np.float32), g=np.ones(3, np.float32), old=None,
                    weight=0.01)
        assert torch.isfinite(call(some).loss).all()
        check(some, call(some))
