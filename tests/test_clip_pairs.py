"""Lists of gradients with entries None beside lists of outputs: each output belongs to the gradient in its place."""
import pytest

import top_support_capture_gb300 as sfc
from top_support_capture_gb300 import gradients

torch = pytest.importorskip("torch")


def test_pairs():
    a, b, x, y = (torch.full((3,), float(i)) for i in range(4))
    same = lambda got, *want: all(p is q for g, w in zip(got, want) for p, q in zip(g, w)) and [len(g) for g in got] == [len(w) for w in want]
    assert same(gradients.pair([a, b], [x, y]), [a, b], [x, y])
    assert same(gradients.pair([None, b], [x, y]), [b], [y])  # x belongs to no gradient
    assert same(gradients.pair([a, None], [x, None]), [a], [x])
    assert same(gradients.pair([a, None, b], [x, y]), [a, b], [x, y])  # one for each gradient there is
    assert same(gradients.pair(a, x), [a], [x]) and same(gradients.pair(iter([a]), iter([x])), [a], [x])
    for grads, out in (([None, b], [x, None]), ([a, b], [x, None]), ([a, None, b], [x, None]), ([a, b], [x]), ([a], [x, y]),
                       ([a, None, b], [x, y, x, y]), ([a, None, b], [None, x, y])):
        with pytest.raises(sfc.SfcError, match="out"):
            gradients.pair(grads, out)


@pytest.mark.gpu
def test_outputs_of_lists_with_gaps():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    full = lambda v: torch.full((5,), v, device="cuda")
    b, x, y = full(2.0), full(7.0), full(8.0)
    with pytest.raises(sfc.SfcError, match=r"out\[1\]"):
        sfc.clip_grad_norm([None, b], 1.0, out=[x, None])
    assert (x == 7).all()
    norm = sfc.clip_grad_norm([None, b], 1.0, out=[x, y])
    assert (x == 7).all() and torch.allclose(y, b / norm)
    sfc.clip_grad_norm([None, b, None], 1.0, out=[x])
    assert torch.equal(x, y)
