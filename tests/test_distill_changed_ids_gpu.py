"""The gradient's own call with teacher entries that are not those of the forward call: nothing outside the rows is
written."""
import pytest

import top_support_capture_gb300 as sfc

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,B", [(5, 1), (1003, 3), (50021, 2), (20001, 320)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ids_outside_the_row(V, B, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W, pad, dev = 4, 64, "cuda"
    lib, code = sfc.load_library(), sfc.SFC_BF16 if dtype == torch.bfloat16 else sfc.SFC_F32
    logits = torch.randn(B, V, device=dev).to(dtype)
    T, up = torch.ones(B, device=dev), torch.ones(B, device=dev)
    ids = torch.arange(W, dtype=torch.int32, device=dev).expand(B, W).contiguous()
    y, n = torch.full((B, W), -1.4, device=dev), torch.full((B,), W, dtype=torch.int32, device=dev)
    loss, stats, status = torch.empty(B, device=dev), torch.empty(B, 4, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    rows = (logits.data_ptr(), code, B, V, V, T.data_ptr())
    assert lib.sfc_distill_forward(*rows, ids.data_ptr(), y.data_ptr(), n.data_ptr(), W, 0, loss.data_ptr(), stats.data_ptr(),
                                   status.data_ptr(), stream) == 0
    buf = torch.full((B, V + pad), 7.0, dtype=dtype, device=dev)

    def backward(ids):
        assert lib.sfc_distill_backward(*rows, ids.data_ptr(), y.data_ptr(), n.data_ptr(), W, 0, stats.data_ptr(), up.data_ptr(),
                                        buf.data_ptr(), V + pad, stream) == 0
        assert (buf[:, V:] == 7).all()
        return buf[:, :V].clone()

    right = backward(ids)
    other = ids.clone()
    other[:, 1], other[:, 2], other[:, 3] = V, V + pad - 1, -1
    got, want = backward(other), right.clone()
    x = logits.float()
    lse = x.double().logsumexp(1, keepdim=True)
    tau = 4 * y[:, :1].double().exp()
    dense = (tau * (x.double() - lse).exp())[:, 1:W]
    # the entries that lie outside have left their places to the dense values; all others are what they were
    want[:, 1:W] = got[:, 1:W]
    assert torch.equal(got, want)
    eps = torch.finfo(dtype).eps / 2
    assert ((got[:, 1:W].double() - dense).abs() <= eps * dense + 128 * 2.0 ** -24 * dense).all()
