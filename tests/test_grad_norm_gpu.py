"""GPU parity of the global gradient norm and of clipping against float64.

Tolerances, counted from the roundings before the first run: a batch of at most 32 squares is summed in 32 bits (32 half steps
of 2^-24), the rest in 64: the norm is within 16 half steps and its own rounding. A clipped element takes the scale (the
norm's 16, its rounding), a product and a rounding to the output's type. Results below the smallest normal number are
within half of the smallest one.
"""
import math

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import top_support_capture_gb300 as sfc

    sfc.load_library()


def make(sizes, types, seed=0, offset=0, scale=1.0):
    """Tensors of those sizes and types (cycled), starting `offset` times their place elements into their buffers."""
    gen = torch.Generator("cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        at = offset * i % 7
        buf = torch.randn(n + at, generator=gen, device="cuda") * scale * 4.0 ** (i % 5 - 2)
        out.append(buf.to(TYPES[types[i % len(types)]])[at:])
    return out


def f64(tensors):
    return [t.detach().double().cpu().numpy().ravel() for t in tensors]


def check_norm(want, norm):
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= 18 * HALF * want + 2.0 ** -149


def check_clipped(before, out, max_norm):
    want = oracle.grad_norm(before)
    scale = oracle.clip_scale(want, max_norm)
    for b, o in zip(before, out):
        bf16 = o.dtype == torch.bfloat16
        got = o.detach().double().cpu().numpy().ravel()
        limit = (20 * HALF + (2.0 ** -8 if bf16 else HALF)) * np.abs(b * scale) + (2.0 ** -134 if bf16 else 2.0 ** -149)
        assert np.all(np.abs(got - b * scale) <= limit)


SIZES = [[1], [0], [3, 0, 5], [8], [4096], [64000, 64000], [1, 2, 3, 7, 8, 9, 15, 16, 17], [1] * 16, [16384 * 32], [16384 * 32 + 1], [8192 * 32 + 3], [20000] * 15, [131072], [131073, 5], [16384 * 3 + 1, 16383, 16384 * 2],
         [3000001], [5000, 1] * 30, [40000, 7, 0, 300] * 64, [700] * 1001, [3] * 2500, [12_000_001, 1_000_003, 5]]


@pytest.mark.parametrize("types", [["bf16"], ["f32"], ["bf16", "f32"]])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip(sizes, types):
    import top_support_capture_gb300 as sfc

    grads = make(sizes, types, offset=1)
    before = f64(grads)
    want = oracle.grad_norm(before)
    norm = sfc.grad_norm(grads)
    check_norm(want, norm)
    for to in ("bf16", "f32"):
        for max_norm in (0.3 * want, 3 * want):
            bufs = [torch.full((t.numel() + 9,), 7.0, dtype=TYPES[to], device="cuda") for t in grads]
            out = [b[i % 5:][:t.numel()] for i, (b, t) in enumerate(zip(bufs, grads))]
            assert torch.equal(sfc.clip_grad_norm(grads, max_norm, out=out), norm)  # the same bits
            check_clipped(before, out, max_norm)
            for i, (b, t) in enumerate(zip(bufs, grads)):  # nothing beside them
                assert (b[:i % 5] == 7).all() and (b[i % 5 + t.numel():] == 7).all()
    assert all(np.array_equal(a, b) for a, b in zip(before, f64(grads)))
    same = sfc.clip_grad_norm(grads, 3 * want)  # in place, nothing to do
    assert torch.equal(same, norm) and all(np.array_equal(a, b) for a, b in zip(before, f64(grads)))
    assert torch.equal(sfc.clip_grad_norm(grads, 0.3 * want), norm)
    check_clipped(before, grads, 0.3 * want)


def test_the_whole_range_of_the_types():
    """Squares that overflow or vanish in 32 bits, zeros, subnormal numbers, infinities and NaN."""
    import top_support_capture_gb300 as sfc

    rng = np.random.default_rng(0)
    for dtype in TYPES.values():
        for scale in (1e-37, 1e-25, 1e-19, 1e-16, 1e15, 1e19, 1e30):
            t = [torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32)).cuda().to(dtype) for n in (5000, 33)]
            check_norm(oracle.grad_norm(f64(t)), sfc.grad_norm(t))
        # zeros among numbers, and nothing but zeros
        t = torch.zeros(70000, dtype=dtype, device="cuda")
        assert float(sfc.grad_norm([t])) == 0.0
        assert float(sfc.clip_grad_norm([t], 1.0)) == 0.0 and not t.any()
        t[69999] = 1e-30
        t[3] = -2e-30
        check_norm(oracle.grad_norm(f64([t])), sfc.grad_norm([t]))
        t[40000] = 1e25
        check_norm(oracle.grad_norm(f64([t])), sfc.grad_norm([t]))
    tiny = torch.full((100,), 2.0 ** -149, device="cuda")
    check_norm(10 * 2.0 ** -149, sfc.grad_norm([tiny]))
    big = torch.full((4,), 3e38, device="cuda")
    assert float(sfc.grad_norm([big])) == math.inf  # above float32's range
    # what is not finite scales as the formula has it
    for bad, expect in ((math.inf, (math.nan, 0.0)), (-math.inf, (math.nan, 0.0)), (math.nan, (math.nan, math.nan))):
        t = torch.ones(50000, device="cuda")
        t[12345] = bad
        norm = sfc.clip_grad_norm([t], 1.0)
        assert float(norm) == math.inf or math.isnan(bad) and math.isnan(float(norm))
        got = (float(t[12345]), float(t[0]))
        assert all(g == e or math.isnan(g) and math.isnan(e) for g, e in zip(got, expect))
    t = torch.ones(100, device="cuda")
    t[3] = math.inf
    assert float(sfc.clip_grad_norm([t], math.inf)) == math.inf and float(t[0]) == 1.0 and float(t[3]) == math.inf
    assert float(sfc.clip_grad_norm(t[4:], 0.0)) == np.float32(math.sqrt(96)) and not t[4:].any()


def test_layouts_and_lists():
    """Transposed tensors, scalars, entries None, a single tensor, an iterator; a norm that repeats to the bit."""
    import top_support_capture_gb300 as sfc

    a = torch.randn(300, 70, device="cuda").t()
    b = torch.randn(4, 5, 6, device="cuda", dtype=torch.bfloat16).permute(2, 0, 1)
    s = torch.tensor(3.0, device="cuda")
    grads = [a, None, b, s]
    before = f64([a, b, s])
    norm = sfc.grad_norm(iter(grads))
    check_norm(oracle.grad_norm(before), norm)
    out = [torch.empty_like(t) for t in (a, b, s)]
    assert out[0].stride() == a.stride()
    sfc.clip_grad_norm(grads, 1.0, out=out)
    check_clipped(before, out, 1.0)
    version = a._version
    assert torch.equal(sfc.clip_grad_norm(grads, 1.0), norm) and a._version > version
    check_clipped(before, [a, b, s], 1.0)
    check_norm(float(s), sfc.grad_norm(s))


def test_inference_tensors():
    import top_support_capture_gb300 as sfc

    with torch.inference_mode():
        t = torch.full((16,), 3.0, device="cuda")
        assert float(sfc.clip_grad_norm([t], 6.0)) == 12.0 and abs(float(t[0]) - 1.5) < 1e-6
    assert float(sfc.clip_grad_norm([t, torch.zeros(3, device="cuda")], 3.0)) == pytest.approx(6.0, abs=1e-5) and abs(float(t[0]) - 0.75) < 1e-6


def test_refused():
    import top_support_capture_gb300 as sfc

    t = lambda *shape, **kw: torch.ones(*shape, device="cuda", **kw)
    x = t(100)
    leaf = t(10, requires_grad=True)
    for grads in ([x, x], [x[:60], x[50:]], [x, x.view(10, 10)]):  # in place: the same memory twice
        with pytest.raises(sfc.SfcError, match="overlap"):
            sfc.clip_grad_norm(grads, 1.0)
    assert float(sfc.grad_norm([x, x])) == pytest.approx(math.sqrt(200))  # only read
    with pytest.raises(sfc.SfcError, match="overlap"):
        sfc.clip_grad_norm([x, t(5)], 1.0, out=[t(100), x[:5]])
    with pytest.raises(sfc.SfcError, match="overlap"):
        sfc.clip_grad_norm([t(50), t(50)], 1.0, out=[x[:50], x[49:99]])
    with pytest.raises(sfc.SfcError, match="overlap"):  # its own place in another type
        sfc.clip_grad_norm([x], 1.0, out=[x.view(torch.bfloat16)[:100]])
    assert (x == 1).all()
    with pytest.raises(sfc.SfcError, match="requires a gradient"):
        sfc.clip_grad_norm([leaf], 1.0)
    with torch.no_grad():
        sfc.clip_grad_norm([leaf], 1.0)
    assert float(sfc.grad_norm(leaf.detach())) == pytest.approx(1.0, abs=1e-5)
    with pytest.raises(sfc.SfcError, match="shape"):
        sfc.clip_grad_norm([x], 1.0, out=[t(99)])
    with pytest.raises(sfc.SfcError, match="strides"):
        sfc.clip_grad_norm([t(4, 6)], 1.0, out=[t(6, 4).t()])


def test_streams_and_graphs():
    """Two captured graphs that run side by side and share no memory; a replay sees new gradients in the same place."""
    import top_support_capture_gb300 as sfc

    sets = [make([300001, 77, 4096], ["bf16", "f32"], seed=s) for s in (1, 2)]
    outs = [[torch.empty(t.numel(), device="cuda") for t in s] for s in sets]
    first = [sfc.clip_grad_norm(s, 1.0, out=o) for s, o in zip(sets, outs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sfc.grad_norm(sets[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, first[0])
    moved = [torch.zeros_like(o) for o in outs[0]]
    side.wait_stream(torch.cuda.current_stream())
    other = sfc.clip_grad_norm(sets[0], 1.0, out=moved, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, first[0]) and all(torch.equal(p, q) for p, q in zip(moved, outs[0]))
    graphs = []
    for s, o in zip(sets, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = sfc.clip_grad_norm(s, 1.0, out=o)
            again = sfc.clip_grad_norm(o, 0.5)  # in place, after it
        graphs.append((graph, norm, again))
    for s in sets:
        for t in s:
            t.mul_(2.0)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for st, (graph, *_) in zip(streams, graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for s, o, (_, norm, again) in zip(sets, outs, graphs):
        before = f64(s)
        check_norm(oracle.grad_norm(before), norm)
        assert abs(float(again) - 1.0) < 1e-3  # bf16 elements' roundings aside
        want = [b * oracle.clip_scale(oracle.grad_norm(before), 1.0) * 0.5 for b in before]
        for w, t in zip(want, o):
            assert np.all(np.abs(t.double().cpu().numpy() - w) <= 64 * HALF * np.abs(w) + 1e-6 * np.abs(w) + 1e-30)


def test_a_tensor_past_32_bit_offsets():
    import top_support_capture_gb300 as sfc

    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    n = 2 ** 31 + 12345
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-3:] = torch.tensor([3.0, 4.0, 12.0])
    t[5] = 84.0
    assert float(sfc.grad_norm([t])) == 85.0
    assert float(sfc.clip_grad_norm([t], 42.5)) == 85.0
    assert t[-3:].tolist() == [1.5, 2.0, 6.0] and float(t[5]) == 42.0 and int(t.count_nonzero()) == 4
