"""The operators together, as a training step uses them: tokens drawn by the decode step, their log-probabilities under the
sampling policy, clipped policy updates of a small model's tables, gradients clipped into the optimizer's type; eager and as
one captured graph, against the same step in float64."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
V, R, B, MAX_NORM = 5003, 48, 96, 0.02


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import top_support_capture_gb300 as sfc

    sfc.load_library()


def start():
    gen = torch.Generator("cuda").manual_seed(0)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    rows, cols = rand(V, R) * 0.3, rand(R, V)
    context = torch.randint(0, V, (B,), generator=gen, device="cuda")
    return rows, cols, context, rand(B), torch.full((B,), 0.9, device="cuda")


def drawn(logits, T):
    import top_support_capture_gb300 as sfc

    full = lambda v, dt: torch.full((B,), v, dtype=dt, device="cuda")
    out = sfc.sample_filter_capture(logits, T, full(0, torch.int32), full(1.0, torch.float32), full(0.0, torch.float32), 7, 1)
    tokens = out.tokens.clone()
    tokens[5::17] = -1  # padding
    return tokens


def update(rows, cols, context, tokens, advantages, T, old, scratch, rate):
    """One step with the library; returns its norm and losses."""
    import top_support_capture_gb300 as sfc

    picked = rows[context]
    logits = picked @ cols
    out = sfc.policy_loss_and_grad(logits, T, tokens, advantages, torch.full_like(T, 1 / B), old_logprobs=old, clip_low=0.1, clip_high=0.1,
                                   entropy_weight=0.02)
    g_cols = picked.t() @ out.grad_logits
    g_rows = torch.zeros_like(rows).index_add_(0, context, out.grad_logits @ cols.t())
    norm = sfc.clip_grad_norm([g_rows, g_cols], MAX_NORM, out=scratch)
    rows.sub_(scratch[0], alpha=rate)
    cols.sub_(scratch[1], alpha=rate)
    return norm, out.loss


def update64(rows, cols, context, tokens, advantages, T, old, rate):
    rows, cols = rows.requires_grad_(), cols.requires_grad_()
    ln_p = torch.log_softmax(rows[context] @ cols / T.double()[:, None], 1)
    there = tokens >= 0
    lp = ln_p.gather(1, tokens.clamp_min(0).long()[:, None])[:, 0]
    rho, A = (lp - old.double()).exp(), advantages.double()
    loss = -torch.minimum(rho * A, rho.clamp(0.9, 1.1) * A) + 0.02 * (ln_p.exp() * ln_p).sum(1)
    loss = torch.where(there, loss, 0.0)
    g = torch.autograd.grad(loss.sum() / B, [rows, cols])
    norm = torch.stack([x.square().sum() for x in g]).sum().sqrt()
    scale = (MAX_NORM / (norm + 1e-6)).clamp_max(1.0)
    return norm, loss.detach(), rows.detach() - rate * scale * g[0], cols.detach() - rate * scale * g[1], lp.detach(), rho.detach()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rate", [0.5, 200.0])  # ratios that hardly move, and some that leave the range
def test_training_steps(captured, rate, steps=4):
    import top_support_capture_gb300 as sfc

    torch.backends.cuda.matmul.allow_tf32 = False
    rows, cols, context, advantages, T = start()
    rows64, cols64 = rows.double(), cols.double()
    logits = rows[context] @ cols
    tokens = drawn(logits, T)
    old = sfc.token_logprobs(logits, T, tokens).logprobs
    scratch = [torch.empty_like(rows), torch.empty_like(cols)]
    args = (rows, cols, context, tokens, advantages, T, old, scratch, rate)
    if captured:
        update(*(a.clone() for a in args[:-2]), [s.clone() for s in scratch], rate)  # warm, on copies
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = update(*args)
    clipped = 0
    for step in range(steps):
        if captured:
            graph.replay()
            norm, loss = held
        else:
            norm, loss = update(*args)
        norm64, loss64, rows64, cols64, lp, rho = update64(rows64, cols64, context, tokens, advantages, T, old, rate)
        if step == 0:  # nothing has moved yet: every ratio is 1, and the losses are the advantages
            assert float((rho - 1)[tokens >= 0].abs().max()) < 1e-5
        near = torch.minimum((rho - 0.9).abs(), (rho - 1.1).abs()) < 1e-4
        if step > 1 and near[tokens >= 0].any():  # a side is a matter of rounding, here and in what follows
            break
        clipped += int(((rho < 0.9) | (rho > 1.1))[tokens >= 0].sum())
        assert (step > 0 or float(norm64) > MAX_NORM) and abs(float(norm) / float(norm64) - 1) < 1e-4
        assert float((loss.double() - loss64).abs().max()) < 1e-4 and not loss[tokens < 0].any()
        # what the parameters have moved by, in all steps so far, is right to a thousandth and the roundings of the
        # parameters themselves, half a step of each a time
        for p, q, first in ((rows, rows64, start()[0]), (cols, cols64, start()[1])):
            moved = q - first.double()
            assert float((p.double() - q).norm()) < 1e-3 * float(moved.norm()) + (step + 1) * 2.0 ** -24 * float(q.norm())
    assert (clipped > 0) == (rate > 1)


def test_scores_of_captured_supports():
    """A token's log-probability over the whole row, over its captured support (replay), and the support's mass agree; the
    top alternatives are the support of a top-k capture."""
    import top_support_capture_gb300 as sfc

    K = 20
    rows, cols, context, _, T = start()
    logits = rows[context] @ cols
    full = lambda v, dt: torch.full((B,), v, dtype=dt, device="cuda")
    out = sfc.sample_filter_capture(logits, T, full(K, torch.int32), full(1.0, torch.float32), full(0.0, torch.float32), 3, 0,
                                    full(1, torch.uint8), packed_width=64)
    assert (out.lengths == K).all()  # (no ties at the cut among these)
    score = sfc.token_logprobs(logits, T, out.tokens, top=K)
    assert torch.equal(score.top_ids, out.support_ids[:, :K])
    mass = score.top_logprobs.double().exp().sum(1).log()
    replay = sfc.replay_logprob(logits, T, out.support_ids, out.lengths, out.tokens)
    np.testing.assert_allclose((replay.token_logprob.double() + mass).cpu().numpy(), score.logprobs.double().cpu().numpy(), atol=1e-5)
    lps = score.top_logprobs - mass[:, None]
    np.testing.assert_allclose(lps.cpu().numpy(), out.support_logprobs[:, :K].cpu().numpy(), atol=1e-5)
