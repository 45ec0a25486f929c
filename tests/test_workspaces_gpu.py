"""The workspaces that the binding keeps, on the streams and in the graphs that use them."""
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
    if not hasattr(a, "lengths"):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        return
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


def test_capture_ids():
    """Its own for each capture, the same on every stream that joined it, 0 outside."""
    import top_support_capture_gb300 as sfc

    lib, ids = sfc.load_library(), []
    here = lambda: lib.sfc_capture_id(torch.cuda.current_stream().cuda_stream)
    assert here() == 0 and lib.sfc_capture_id(None) == 0
    x = torch.zeros(8, device="cuda")
    for _ in range(2):
        side, other = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            ids.append(here())
            assert ids[-1] != 0 and lib.sfc_capture_id(other.cuda_stream) == 0
            other.wait_stream(side)
            assert lib.sfc_capture_id(other.cuda_stream) == ids[-1]
            x.add_(1)
            side.wait_stream(other)
    assert ids[0] != ids[1] and here() == 0


@pytest.mark.parametrize("kind", ["decode", "verify"])
def test_graphs_of_one_stream_replayed_beside_each_other(kind):
    """Two graphs captured on one stream after one warm-up there, replayed at once on two streams, beside eager calls on
    the stream they were captured on: each result is that of a call by itself."""
    import top_support_capture_gb300 as sfc
    from top_support_capture_gb300 import speculative

    if kind == "decode":
        inputs = [decode_args(seed) for seed in range(3)]
        call = lambda i: sfc.sample_filter_capture(*inputs[i][0], 3, 4 + i, inputs[i][1])
    else:
        def one(seed, B=2, D=3, V=50021):
            gen = torch.Generator("cuda").manual_seed(seed)
            t = 2 * torch.randn((B, D + 1, V), generator=gen, device="cuda")
            d = t[:, :D] + 0.5 * torch.randn((B, D, V), generator=gen, device="cuda")
            return t, d.contiguous(), d.argmax(2).int(), torch.rand((B, D), generator=gen, device="cuda"), torch.ones(B, device="cuda")

        inputs = [one(seed) for seed in range(3)]
        call = lambda i: sfc.verify_drafts(*inputs[i], 3, 4 + i)
    alone = [call(i) for i in range(3)]
    torch.cuda.synchronize()
    side, replay = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    with torch.cuda.stream(side):
        call(2)
    graphs, held = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=side):
            held.append([call(i) for _ in range(8)])
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(replay[i]):
                graphs[i].replay()
        with torch.cuda.stream(side):
            eager = call(2)
    torch.cuda.synchronize()
    same(alone[2], eager)
    for i in range(2):
        for out in held[i]:
            same(alone[i], out)
    for kept in (sfc._step_workspaces, speculative._workspaces):  # each left as it has to be
        for ws in (*kept.current.values(), *(w for had in kept.captured.values() for w in had)):
            assert not ws.any()
