"""The workspaces that the binding keeps, on the streams and in the graphs that use them."""
import numpy as np
import pytest

from top_support_capture_gb300 import workloads as wl

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import top_support_capture_gb300 as sfc

    sfc.load_library()


def decode_args(seed=0, B=2, V=151936, W=1024):
    """Logits of a short batch, whose rows are split into slices that meet in the workspace, and its parameters."""
    import top_support_capture_gb300 as sfc

    assert sfc.workspace_size(B, V, W, wl.DT_BF16) > 0
    gen = torch.Generator("cuda").manual_seed(seed)
    logits = (3 * torch.randn((B, V), generator=gen, device="cuda")).to(torch.bfloat16)
    full = lambda v, dt: torch.full((B,), v, dtype=dt, device="cuda")
    return (logits, full(0.9, torch.float32), full(100, torch.int32), full(0.95, torch.float32), full(0.0, torch.float32)), full(1, torch.uint8)


def same(a, b):
    n = a.lengths.tolist()
    assert n == b.lengths.tolist() and torch.equal(a.tokens, b.tokens) and torch.equal(a.row_status, b.row_status)
    for r, k in enumerate(n):
        assert torch.equal(a.support_ids[r, :k], b.support_ids[r, :k]) and torch.equal(a.support_logprobs[r, :k], b.support_logprobs[r, :k])


def test_made_on_the_stream_that_uses_it(monkeypatch):
    """A call on a stream that is not the current one: its workspace is zero-filled on that stream, not behind what
    the current one still has to do."""
    import top_support_capture_gb300 as sfc

    made, allocate = [], sfc.allocate_workspace
    monkeypatch.setattr(sfc, "allocate_workspace", lambda n, dev: (made.append(torch.cuda.current_stream()), allocate(n, dev))[1])
    args, capture = decode_args()
    ref = sfc.sample_filter_capture(*args, 3, 4, capture)
    side = torch.cuda.Stream()
    sfc._step_workspaces.current.pop((0, side.cuda_stream), None)  # the pool may have given its handle out before
    out = sfc.allocate_outputs(2, 1024, "cuda")
    side.wait_stream(torch.cuda.current_stream())
    del made[:]
    sfc.sample_filter_capture_into(out, *args, 3, 4, capture, stream=side)
    side.synchronize()
    assert made == [side]
    assert torch.cuda.current_stream() != side
    same(ref, out)
