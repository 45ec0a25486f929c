"""GPU parity of the verification over full rows whose masses lie far from the rows' first logits: grammar masks over
most of a row, low temperatures, peaks far apart. Compared as in test_verify_gpu, at its tolerances.

Each row's true maximum is the reference of its sums, so no mass is lost to a reference that lies above it; a sum that
is taken against 0 (for a masked start) or against each thread's own first logits loses some or all of it on these rows.
"""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import as_input
from test_verify_gpu import _cuda, check, make, ref_of, run  # noqa: F401 (the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LOWEST = -3.3895313892515355e38  # of bfloat16


def masked(B, D, V, dtype, seed, T, level, first, allowed=50, fill=-np.inf, sides="td", mode="logits"):
    """Rows whose `allowed` finite logits lie at random places from `first` on, about `level`; the draft's near the
    target's; drafts drawn from the draft's rows."""
    rng = np.random.default_rng(seed)
    t, d = (np.full((B, k, V), fill, np.float32) for k in (D + 1, D))
    for b in range(B):
        for j in range(D + 1):
            ids = rng.choice(np.arange(first, V), min(allowed, V - first), replace=False)
            live = level + 1.5 * T * rng.standard_normal(ids.size)
            t[b, j, ids] = live
            if j < D:
                d[b, j, ids] = live + 0.5 * T * rng.standard_normal(ids.size)
    if "t" not in sides:
        t = (3 * rng.standard_normal(t.shape)).astype(np.float32)
    if "d" not in sides:
        d = (3 * rng.standard_normal(d.shape)).astype(np.float32)
    drafted = np.argmax(np.where(d > -1e30, d.astype(np.float64) / T, -np.inf) + rng.gumbel(size=d.shape), axis=2)
    lookup = mode == "lookup"
    return dict(t=as_input(t.reshape(-1, V), dtype).reshape(t.shape), d=None if lookup else as_input(d.reshape(-1, V), dtype).reshape(d.shape),
                dtype=dtype, drafted=drafted.astype(np.int32), u=rng.random((B, D), dtype=np.float32) * 0.9,
                T=np.full(B, T, np.float32), Td=None, n=None, seed=seed + 11, step=seed)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("fill", [-np.inf, LOWEST])
@pytest.mark.parametrize("level,T", [(-20.0, 0.02), (-20.0, 0.2), (-17.5, 0.2), (-8.6, 0.1), (-6.0, 0.05), (-100.0, 1.0), (-200.0, 0.3),
                                     (-200.0, 1.0)])
def test_masked_rows(dtype, fill, level, T):
    """The allowed tokens past the first 20000 or 4100: rows in several slices, of which the first are wholly masked, and
    rows in one."""
    for B, V, first in ((3, 32003, 20000), (70, 9001, 4100)):
        c = masked(B, 4, V, dtype, int(-level) + B, T, level, first, fill=fill)
        ref = ref_of(c)
        assert (ref.row_status == 0).all()
        check(ref, run(c), most_unclear=0.1)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("sides,mode", [("t", "logits"), ("d", "logits"), ("t", "lookup")])
def test_one_masked_side(dtype, sides, mode):
    c = masked(6, 3, 20011, dtype, 4, 0.25, -30.0, 5000, sides=sides, mode=mode)
    check(ref_of(c), run(c), most_unclear=0.2)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_a_single_allowed_token(dtype):
    """The last token of the row, in its ragged tail or its last vector, or the first, before the first boundary."""
    for V, at in ((4099, 4098), (4096, 4095), (50021, 0)):
        c = make(5, 2, V, dtype, 3)
        for k in "td":
            x = np.full(c[k].shape, -np.inf, np.float32)
            x[:, :, at] = -90.0
            c[k] = as_input(x.reshape(-1, V), dtype).reshape(x.shape)
        c["drafted"][:] = at
        out = run(c)
        assert (out.accepted == 2).all() and (out.tokens == at).all() and (out.token_logprobs == 0).all()


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_rows_of_the_lowest_value(dtype):
    """Finite everywhere, so a uniform distribution: no mass may be lost, and it is no bad row."""
    V = 5003
    c = make(4, 2, V, dtype, 8)
    for k in "td":
        c[k] = as_input(np.full((c[k][..., 0].size, V), LOWEST, np.float32), dtype).reshape(c[k].shape)
    ref = ref_of(c)
    assert (ref.row_status == 0).all()
    check(ref, run(c), most_unclear=1.0)


@pytest.mark.parametrize("V,peaks", [(32768, (0, 12328)), (32768, (8, 20520)), (65536, (0, 12328, 40000))])
@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_peaks_far_above_the_rest(dtype, V, peaks):
    """Equal peaks 87.5 T above all others share the mass: each has it in equal parts."""
    B, D = 40, 8
    c = make(B, D, V, dtype, 2, mode="lookup")
    x = np.full((B * (D + 1), V), 1.25, np.float32)
    x[:, list(peaks)] = 10.0
    c["t"] = as_input(x, dtype).reshape(c["t"].shape)
    c["T"] = np.full(B, 0.1, np.float32)
    c["drafted"] = np.full((B, D), peaks[-1], np.int32)
    c["u"] = np.where(np.arange(B)[:, None] % 2, 0.98, 1.02).astype(np.float32) / len(peaks) * np.ones((B, D), np.float32)
    ref, out = ref_of(c), run(c)
    check(ref, out)
    assert (out.accepted.cpu().numpy() == np.where(np.arange(B) % 2, D, 0)).all()


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("T", [0.02, 0.1, 0.3])
def test_low_temperatures(dtype, T):
    c = make(40, 4, 20011, dtype, 13, spread=3.0, near=0.1)
    c["T"] = c["Td"] = np.full(40, T, np.float32)
    rows = np.array(oracle.widen_logits(c["d"].reshape(-1, 20011), dtype), np.float64).reshape(c["d"].shape)
    c["drafted"] = np.argmax(rows / T + np.random.default_rng(1).gumbel(size=rows.shape), axis=2).astype(np.int32)
    check(ref_of(c), run(c), most_unclear=0.2)
