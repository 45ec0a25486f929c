"""GPU parity of the verification of drafted tokens (full rows and captured supports) against the float64 oracle.

Tokens, counts and statuses are compared exactly on requests whose decisions clear float32 rounding (the oracle's
``clear``: 2^-15 relative, several times what the exponents' roundings, 8 |z| half steps, and the mass's give);
nearly all do. Log-probabilities are computed in 64 bits from a mass in 32: within 64 half steps, rounded once.
"""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import as_input, cuda

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import top_support_capture_gb300 as sfc

    sfc.load_library()


def dev(x, dtype):
    x = np.ascontiguousarray(x)
    return torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16) if dtype == wl.DT_BF16 else torch.from_numpy(x).cuda()


def make(B, D, V, dtype, seed, spread=2.0, near=0.7, mode="logits", ragged=False):
    """Target rows, draft rows near them, drafts drawn from the draft rows."""
    rng = np.random.default_rng(seed)
    t = (rng.standard_normal((B, D + 1, V)) * spread).astype(np.float32)
    d = (t[:, :D] + near * rng.standard_normal((B, D, V))).astype(np.float32)
    T, Td = rng.uniform(0.6, 1.4, B).astype(np.float32), rng.uniform(0.6, 1.4, B).astype(np.float32)
    drafted = np.argmax(d / Td[:, None, None] + rng.gumbel(size=d.shape), axis=2).astype(np.int32)
    n = rng.integers(0, D + 1, B).astype(np.int32) if ragged else None
    return dict(t=as_input(t, dtype), d=as_input(d, dtype) if mode == "logits" else None, dtype=dtype, drafted=drafted,
                u=rng.random((B, D), dtype=np.float32), T=T, Td=Td if mode == "logits" else None, n=n, seed=seed + (5 << 33),
                step=(3 << 32) + seed)


def run(c, target=None, draft=None, **kw):
    import top_support_capture_gb300 as sfc

    opt = lambda a, dt: None if a is None else cuda(a, dt)
    target = dev(c["t"], c["dtype"]) if target is None else target
    draft = (None if c["d"] is None else dev(c["d"], c["dtype"])) if draft is None else draft
    return sfc.verify_drafts(target, draft, cuda(c["drafted"], np.int32), cuda(c["u"], np.float32), cuda(c["T"], np.float32), c["seed"],
                             c["step"], draft_temperature=opt(c["Td"], np.float32), num_drafts=opt(c["n"], np.int32), **kw)


def ref_of(c, **kw):
    return oracle.verify_drafts(c["t"], c["d"], c["dtype"], c["drafted"], c["u"], c["T"], c["seed"], c["step"], c["Td"], c["n"], **kw)


def check(ref, out, most_unclear=0.02):
    ok = ref.clear
    assert (~ok).mean() <= most_unclear or (~ok).sum() <= 1
    got = {k: v.cpu().numpy() for k, v in out._asdict().items()}
    np.testing.assert_array_equal(got["row_status"][ok], ref.row_status[ok])
    np.testing.assert_array_equal(got["accepted"][ok], ref.accepted[ok])
    np.testing.assert_array_equal(got["tokens"][ok], ref.tokens[ok])
    a, b = got["token_logprobs"][ok].astype(np.float64), ref.token_logprobs[ok]
    np.testing.assert_array_equal(np.isnan(a), np.isnan(b))
    assert np.all(np.abs(a - b)[~np.isnan(b)] <= 64 * HALF * (1 + np.abs(b[~np.isnan(b)])))


SHAPES = [(1, 1, 1), (3, 2, 2), (5, 3, 7), (16, 4, 33), (40, 7, 1000), (9, 3, 4099), (300, 2, 257), (4, 5, 50021), (1, 4, 151936),
          (3, 2, 262144), (2, 64, 130)]


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,D,V", SHAPES)
@pytest.mark.parametrize("mode", ["logits", "lookup"])
def test_verify(dtype, B, D, V, mode):
    c = make(B, D, V, dtype, B + D + V, mode=mode, ragged=B > 2, spread=2.0 if V > 10 else 0.5)
    check(ref_of(c), run(c))


@pytest.mark.parametrize("near", [0.0, 0.05, 5.0])
def test_identical_near_and_far_drafts(near):
    """Drafts from the target itself are all accepted; from far away, nearly none."""
    c = make(64, 4, 3001, wl.DT_F32, 8, near=near)
    if near == 0.0:
        c["Td"] = c["T"]
    ref, out = ref_of(c), run(c)
    if near == 0.0:
        assert (out.accepted == 4).all()
    check(ref, out, most_unclear=1.0 if near == 0.0 else 0.1)  # u q = p u is a clear decision only for u < 1 - margin


def test_layouts():
    """Padded rows, unaligned starts, position-major rows, rows shared by every request."""
    c = make(6, 3, 1001, wl.DT_BF16, 4)
    ref = ref_of(c)
    check(ref, run(c))
    t, d = dev(c["t"], c["dtype"]), dev(c["d"], c["dtype"])
    B, D, V = 6, 3, 1001
    wide = torch.full((B, D + 1, V + 13), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :, 5:5 + V] = t
    major = t.transpose(0, 1).contiguous().transpose(0, 1)
    dmajor = d.transpose(0, 1).contiguous().transpose(0, 1)
    for target, draft in ((wide[:, :, 5:5 + V], d), (major, dmajor)):  # (where a row starts sets the order of its sums)
        check(ref, run(c, target, draft))
    c["t"], c["d"] = np.repeat(c["t"][:1], B, 0), np.repeat(c["d"][:1], B, 0)
    shared = run(c, t[:1].expand(B, D + 1, V), d[:1].expand(B, D, V))
    check(ref_of(c), shared)


def test_greedy_rows_among_sampled_ones():
    c = make(24, 3, 2000, wl.DT_BF16, 6, ragged=True)
    c["T"][::3] = 0
    c["Td"][::4] = 0
    c["drafted"][0, 0] = int(np.argmax(oracle.widen_logits(c["t"][0, :1], c["dtype"])[0]))
    check(ref_of(c, greedy_t0=True), run(c, greedy_t0=True))
    ref = ref_of(c)  # without the flag those requests are refused
    assert (ref.row_status[::3] == -1).all()
    check(ref, run(c))


def test_bad_requests_and_masked_rows():
    """Each fault refuses its request only, and only where the walk reaches it; -inf logits are just improbable."""
    B, D, V = 12, 3, 515
    c = make(B, D, V, wl.DT_F32, 10)
    c["n"] = np.full(B, D, np.int32)
    c["u"][:] = 0.999999
    c["u"][4:6] = 0.0
    t, d = c["t"], c["d"]
    t[0, 0, 3] = np.nan
    t[1, 0] = -np.inf
    d[2, 0, 9] = np.inf
    c["drafted"][3, 0] = V
    t[4, 1, 0] = np.nan  # reached: u = 0 accepts the first draft
    t[5, 0, 100:] = -np.inf
    c["drafted"][5, 0] = 50
    d[5, 0, 50] = 3.0
    c["n"][6] = D + 1
    c["n"][7] = -1
    c["T"][8] = np.nan
    c["Td"][9] = 0
    c["drafted"][10] = -1
    c["n"][10] = 0  # no drafts: the drafted tokens are not looked at
    t[11, 1:] = np.nan  # past the first refusal
    c["drafted"][11, 0] = int(np.argmin(t[11, 0]))
    d[11, 0, c["drafted"][11, 0]] = 20.0
    ref = ref_of(c)
    assert list(ref.row_status) == [-1, -1, -1, -1, -1, 0, -1, -1, -1, -1, 0, 0]
    assert ref.accepted[5] >= 1 and ref.accepted[11] == 0
    check(ref, run(c), most_unclear=0.1)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_steep_rows(dtype):
    """Logits that rise hundreds of units over what comes first in the row, and differ by as much: the masses are
    held against a reference that has to be given up; rows that start with masked entries."""
    c = make(12, 3, 6007, dtype, 21, spread=200.0, near=2.0)
    t, d = (np.array(oracle.widen_logits(c[k].reshape(-1, 6007), dtype), np.float32).reshape(c[k].shape) for k in "td")
    t[:4, :, :3000] -= 1000.0
    d[:4, :, :3000] -= 1000.0
    t[4:6, :, :5000] = -np.inf
    d[6:8, :, :2500] = -3.3895313892515355e38
    c["drafted"] = np.argmax(np.where(np.isfinite(d), d, -np.inf), axis=2).astype(np.int32)
    c["t"], c["d"] = as_input(t.reshape(-1, 6007), dtype).reshape(t.shape), as_input(d.reshape(-1, 6007), dtype).reshape(d.shape)
    ref = ref_of(c)
    assert (ref.row_status == 0).all()
    check(ref, run(c), most_unclear=0.1)


def test_rows_past_32_bit_offsets():
    V, D = 262144, 2
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    c = make(2, D, V, wl.DT_BF16, 9)
    t, d = dev(c["t"], c["dtype"]), dev(c["d"], c["dtype"])
    far = torch.empty(2 ** 31 + 8 * V, dtype=torch.bfloat16, device="cuda")
    target = far.as_strided((2, D + 1, V), (2 ** 31 + 3, V, 1), 5)
    target.copy_(t)
    check(ref_of(c), run(c, target, d))


def test_no_residual_mass():
    """A refused certain draft that has all of the target's mass leaves nothing: the draw is from the target."""
    c = make(4, 1, 9, wl.DT_F32, 3, mode="lookup")
    c["t"][:, 0] = -np.inf
    c["t"][:, 0, 4] = 1.0
    c["drafted"][:] = 4
    c["u"][:] = 1.0  # just past the range: 1 < 1 refuses
    out = run(c)
    assert (out.accepted == 0).all() and (out.tokens[:, 0] == 4).all() and (out.row_status == 0).all()


def test_emitted_tokens_follow_the_target():
    rng = np.random.default_rng(1)
    B, D, V = 40000, 2, 6
    t, d = rng.standard_normal((1, D + 1, V)).astype(np.float32), rng.standard_normal((1, D, V)).astype(np.float32)
    drafted = np.argmax(d + rng.gumbel(size=(B, D, V)), axis=2).astype(np.int32)
    c = dict(drafted=drafted, u=rng.random((B, D), dtype=np.float32), T=np.ones(B, np.float32), Td=None, n=None, seed=77, step=5,
             dtype=wl.DT_F32, t=t, d=d)
    out = run(c, dev(t, wl.DT_F32).expand(B, D + 1, V), dev(d, wl.DT_F32).expand(B, D, V))
    tokens, accepted = out.tokens.cpu().numpy(), out.accepted.cpu().numpy()
    for j in range(D + 1):
        seen = tokens[accepted >= j, j]
        p = np.exp(t[0, j].astype(np.float64))
        p /= p.sum()
        got = np.bincount(seen, minlength=V)
        assert ((got - seen.size * p) ** 2 / (seen.size * p)).sum() < 25.8  # 5 degrees of freedom, 1e-4


def test_repeats_streams_graphs_and_workspaces():
    """The same bits on every call: after calls of other sizes over the same workspace, on another stream, replayed
    from a graph, and for a batch cut into shards."""
    import top_support_capture_gb300 as sfc

    c, other = make(20, 4, 5000, wl.DT_BF16, 1, ragged=True), make(3, 9, 777, wl.DT_F32, 2)
    size = max(sfc.verify_workspace_size(20, 4, 5000, 0), sfc.verify_workspace_size(3, 9, 777, 1))
    ws = sfc.allocate_workspace(size, "cuda")
    first = run(c, workspace=ws)
    check(ref_of(c), first)
    check(ref_of(other), run(other, workspace=ws), most_unclear=0.4)
    for again in (run(c, workspace=ws), run(c)):
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        there = run(c)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, there))
    t, d = dev(c["t"], c["dtype"]), dev(c["d"], c["dtype"])
    rest = (cuda(c["drafted"], np.int32), cuda(c["u"], np.float32), cuda(c["T"], np.float32))
    kw = dict(draft_temperature=cuda(c["Td"], np.float32), num_drafts=cuda(c["n"], np.int32))
    own = t.clone()  # goes out of scope while the other stream may still read it
    side.wait_stream(torch.cuda.current_stream())
    there = sfc.verify_drafts(own, d, *rest, c["seed"], c["step"], stream=side, **kw)
    del own
    junk = [torch.full_like(t, 9.0) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, there)) and len(junk) == 4
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = sfc.verify_drafts(t, d, *rest, c["seed"], c["step"], workspace=ws, **kw)
    for _ in range(3):
        for o in held:
            o.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held))
    for lo, hi in ((0, 7), (7, 20)):
        part = sfc.verify_drafts(t[lo:hi], d[lo:hi], *(x[lo:hi] for x in rest), c["seed"], c["step"], row_offset=lo,
                                 **{k: v[lo:hi] for k, v in kw.items()})
        assert torch.equal(part.tokens, first.tokens[lo:hi]) and torch.equal(part.accepted, first.accepted[lo:hi])


# ------------------------------------------------------------------------------------------------ supports


def supports(rng, rows, V, W, logits=None):
    """Packed supports of `rows` rows: ids in any order, logprobs renormalised, ragged lengths."""
    ids, lps, n = np.full((rows, W), -1, np.int32), np.full((rows, W), np.nan, np.float32), np.zeros(rows, np.int32)
    for r in range(rows):
        n[r] = rng.integers(1, min(W, V) + 1)
        ids[r, :n[r]] = rng.choice(V, n[r], replace=False)
        z = rng.standard_normal(n[r]) * 2
        lps[r, :n[r]] = z - np.log(np.exp(z).sum())
    return ids, lps, n


def support_case(B, D, V, W, Wd, seed, ragged=False):
    rng = np.random.default_rng(seed)
    ids, lps, n = supports(rng, B * (D + 1), V, W)
    dids, dlps, dn = supports(rng, B * D, V, Wd)
    drafted = np.array([dids[r, rng.integers(dn[r])] for r in range(B * D)], np.int32).reshape(B, D)
    return dict(ids=ids.reshape(B, D + 1, W), lps=lps.reshape(B, D + 1, W), lens=n.reshape(B, D + 1), dids=dids.reshape(B, D, Wd),
                dlps=dlps.reshape(B, D, Wd), dlens=dn.reshape(B, D), drafted=drafted, u=rng.random((B, D), dtype=np.float32) * 0.5,
                n=rng.integers(0, D + 1, B).astype(np.int32) if ragged else None, seed=(7 << 40) + seed, step=seed)


def run_supports(c):
    import top_support_capture_gb300 as sfc

    i = lambda k: None if c[k] is None else cuda(c[k], np.int32)
    f = lambda k: None if c[k] is None else cuda(c[k], np.float32)
    return sfc.verify_supports(i("ids"), f("lps"), i("lens"), i("dids"), f("dlps"), i("dlens"), i("drafted"), f("u"), c["seed"], c["step"],
                               num_drafts=i("n"))


def ref_supports(c):
    return oracle.verify_supports(c["ids"], c["lps"], c["lens"], c["dids"], c["dlps"], c["dlens"], c["drafted"], c["u"], c["seed"],
                                  c["step"], c["n"])


@pytest.mark.parametrize("B,D,V,W,Wd", [(1, 1, 1, 1, 1), (5, 3, 6, 4, 3), (40, 4, 50, 33, 50), (9, 7, 2000, 1024, 512), (3, 2, 40000, 8192, 100),
                                        (2, 2, 40000, 100, 16384), (2, 1, 2 ** 31 - 1, 77, 50), (30, 64, 12, 8, 8)])
def test_supports(B, D, V, W, Wd):
    if V > 10 ** 6:  # ids up to the largest
        c = support_case(B, D, 1000, W, Wd, 5)
        for k in ("ids", "dids", "drafted"):
            c[k] = np.where(c[k] >= 0, c[k] + (V - 1000), -1).astype(np.int32)
    else:
        c = support_case(B, D, V, W, Wd, B + W, ragged=B > 4)
    check(ref_supports(c), run_supports(c))


def test_supports_certain_drafts():
    c = support_case(20, 3, 40, 20, 10, 3)
    c["dlens"][:, 1] = 0
    check(ref_supports(c), run_supports(c))
    c["dids"] = c["dlps"] = c["dlens"] = None
    check(ref_supports(c), run_supports(c))


def test_supports_faults():
    c = support_case(10, 2, 30, 16, 8, 12)
    c["n"] = np.full(10, 2, np.int32)
    c["lens"][0, 0] = 0
    c["lens"][1, 0] = 17
    c["dlens"][2, 0] = 9
    c["dlens"][3, 0] = -1
    c["drafted"][4, 0] = -5
    c["lps"][5, :, :] = np.nan
    c["n"][6] = 3
    c["n"][7] = -2
    c["lps"][8, :, :] = -np.inf
    ref = ref_supports(c)
    assert list(ref.row_status) == [-1, 1, 1, -1, -1, -1, -1, -1, -1, 0]
    check(ref, run_supports(c))


def test_captured_supports_end_to_end():
    """Draft and target rows through the decode step's capture, then verified: what the oracle makes of the same
    captured supports; and the tokens that follow are members of the target's supports."""
    import top_support_capture_gb300 as sfc

    B, D, V, W = 8, 3, 3000, 256
    rng = np.random.default_rng(5)
    t = (rng.standard_normal((B * (D + 1), V)) * 2).astype(np.float32)
    d = (t.reshape(B, D + 1, V)[:, :D].reshape(-1, V) + 0.5 * rng.standard_normal((B * D, V))).astype(np.float32)

    def capture(x, seed):
        rows = len(x)
        full = lambda v, dt: torch.full((rows,), v, dtype=dt, device="cuda")
        return sfc.sample_filter_capture(cuda(x, np.float32), full(0.9, torch.float32), full(50, torch.int32), full(0.95, torch.float32),
                                         full(0.0, torch.float32), seed, 1, full(1, torch.uint8), packed_width=W)

    dr, ta = capture(d, 3), capture(t, 4)
    u = cuda(rng.random((B, D)), np.float32)
    three = lambda x, k: x.view(B, k, -1)
    out = sfc.verify_supports(three(ta.support_ids, D + 1), three(ta.support_logprobs, D + 1), ta.lengths.view(B, D + 1),
                              three(dr.support_ids, D), three(dr.support_logprobs, D), dr.lengths.view(B, D), dr.tokens.view(B, D), u, 3, 1)
    n = lambda x: x.cpu().numpy()
    ref = oracle.verify_supports(n(three(ta.support_ids, D + 1)), n(three(ta.support_logprobs, D + 1)), n(ta.lengths.view(B, D + 1)),
                                 n(three(dr.support_ids, D)), n(three(dr.support_logprobs, D)), n(dr.lengths.view(B, D)),
                                 n(dr.tokens.view(B, D)), n(u), 3, 1)
    check(ref, out)
    assert out.accepted.sum() > 0
