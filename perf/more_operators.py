"""What is measured of the operators beside a policy's whole vocabulary: the log-probabilities of given tokens with the
entropy and the top alternatives (and their gradient), the clipped policy loss with its gradient, and the global norm of a
model's gradients with their clipping.

Each operator has its plain form here, in elementary torch operations, beside the call that a user makes.
"""
import math
import random

import torch

own = False

# ----------------------------------------------------------------------------------------------
# Cases. Vocabularies (32000, 151936, 129280, 262144) and row counts are those of this repository's decode workloads;
# 50021 is its tests' odd vocabulary. The gradients are those of its example's draft model (two tables of 2000 x 32)
# and of a generic decoder stack.
# ----------------------------------------------------------------------------------------------


def listed():
    bf16, f32 = "bfloat16", "float32"
    return [
        # one user's decode step with the alternatives shown beside the token: the smallest, where latency counts
        dict(name="score_1x151936_bf16_top20", kind="score", N=1, V=151936, pad=0, M=1, K=20, dtype=bf16, masked=False),
        # a serving batch's decode step
        dict(name="score_64x151936_bf16_top5", kind="score", N=64, V=151936, pad=0, M=1, K=5, dtype=bf16, masked=False),
        # a prompt scored token by token, or the rollouts of a reinforcement-learning batch
        dict(name="score_2048x151936_bf16_top1", kind="score", N=2048, V=151936, pad=0, M=1, K=1, dtype=bf16, masked=False),
        # multiple-choice scoring: several tokens a row, rows that a grammar masks down to a few tokens, odd rows
        dict(name="score_33x50021_f32_top64_masked", kind="score", N=33, V=50021, pad=3, M=7, K=64, dtype=f32, masked=True),
        # a training micro-batch through autograd, with gradients of the log-probabilities and the entropies
        dict(name="score_grad_64x32000_bf16", kind="score_grad", N=64, V=32000, pad=0, M=1, K=0, dtype=bf16, masked=False),
        # the same in f32 over several tokens a row
        dict(name="score_grad_256x129280_f32_m4", kind="score_grad", N=256, V=129280, pad=0, M=4, K=0, dtype=f32, masked=False),
        # a small fine-tuning step: weighted cross-entropy, rows of padding among them
        dict(name="policy_64x32000_bf16_plain", kind="policy", N=64, V=32000, pad=0, dtype=bf16, clipped=False, entropy=0.0),
        # a full reinforcement-learning batch of tokens: the largest
        dict(name="policy_2048x151936_bf16", kind="policy", N=2048, V=151936, pad=0, dtype=bf16, clipped=True, entropy=0.01),
        # a short batch with odd rows
        dict(name="policy_33x50021_f32", kind="policy", N=33, V=50021, pad=3, dtype=f32, clipped=True, entropy=0.01),
        # the example's draft model: two small tables, where latency counts
        dict(name="clip_draft_f32", kind="clip", shapes="tables", hidden=32, layers=0, vocab=2000, dtype=f32, out=f32, limit=5e-4),
        # a decoder stack in bf16 whose clipped gradients go to the optimizer in f32
        dict(name="clip_stack6x2048_bf16_f32", kind="clip", shapes="stack", hidden=2048, layers=6, vocab=32000, dtype=bf16, out=f32, limit=5e-4),
        # the norm that is logged: many tensors of odd sizes and both types, starting anywhere
        dict(name="norm_ragged_200", kind="norm", shapes="ragged", hidden=16384, layers=200, vocab=0, dtype="mixed", out="", limit=5e-4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["score", "score", "score_grad", "policy", "policy", "clip", "norm"])
    dtype = rng.choice(["bfloat16", "float32"])
    if kind in ("clip", "norm"):
        shapes = rng.choice(["tables", "stack", "ragged"])
        if shapes == "tables":
            case = dict(kind=kind, shapes=shapes, hidden=_log_int(rng, 1, 512), layers=0, vocab=_log_int(rng, 100, 262144))
        elif shapes == "stack":
            case = dict(kind=kind, shapes=shapes, hidden=_log_int(rng, 16, 2000), layers=_log_int(rng, 1, 6), vocab=_log_int(rng, 100, 32000))
        else:
            case = dict(kind=kind, shapes=shapes, hidden=_log_int(rng, 1, 300000), layers=_log_int(rng, 1, 60 if kind == "clip" else 400), vocab=0)
        if rng.random() < 0.3:
            dtype = "mixed"
        return {**case, "dtype": dtype, "out": rng.choice(["bfloat16", "float32"]) if kind == "clip" else "",
                "limit": rng.choice([5e-4, 5e-4, 5e-4, 1.0])}
    V = rng.choice([_log_int(rng, 1000, 262144), _log_int(rng, 1000, 262144), 32000, 151936])
    size = 2 if dtype == "bfloat16" else 4
    N = min(_log_int(rng, 1, 2048), max(1, 2048 * 151936 * 2 // (V * size)))
    case = dict(kind=kind, N=N, V=V, pad=rng.choice([0, 0, rng.randrange(1, 64)]), dtype=dtype)
    if kind == "policy":
        return {**case, "clipped": rng.random() < 0.7, "entropy": rng.choice([0.0, 0.01])}
    case["M"] = rng.choice([1, 1, rng.randrange(2, 9)])
    case["K"] = rng.choice([0, 1, 5, 20, rng.randrange(1, 65)]) if kind == "score" else 0
    case["masked"] = rng.random() < 0.25
    return case


# ----------------------------------------------------------------------------------------------
# Inputs: Zipf-ranked logit rows plus Gaussian noise, as the decode workloads have them; gradients whose scale differs
# from tensor to tensor.
# ----------------------------------------------------------------------------------------------


def _rows(gen, N, V, dtype, pad, masked):
    """[N, V] logits (a view of rows V + pad apart): a 12-logit Zipf profile, another shift of one random permutation
    for each row, plus noise. Masked rows keep between 64 and V tokens."""
    out = torch.empty((N, V + pad), dtype=getattr(torch, dtype), device="cuda")[:, :V]
    rank = torch.arange(1, V + 1, device="cuda", dtype=torch.float32)
    prof = rank.log() * (-12.0 / math.log(max(V, 2)))
    prof = prof[torch.randperm(V, generator=gen, device="cuda")]
    shift = torch.randint(0, V, (N, 1), generator=gen, device="cuda")
    for r in range(0, N, 256):
        k = min(256, N - r)
        x = prof[(torch.arange(V, device="cuda") + shift[r:r + k]) % V] + torch.randn((k, V), generator=gen, device="cuda")
        if masked:
            keep = (64.0 / V) ** torch.rand((k, 1), generator=gen, device="cuda")  # the share that is left
            key = torch.rand((k, V), generator=gen, device="cuda")
            limit = torch.maximum(key.topk(min(64, V), dim=1, largest=False).values[:, -1:], keep)
            x = torch.where(key <= limit, x, -math.inf)
        out[r:r + k] = x
    return out


def _sampled(gen, x, T):
    """One token of each row, drawn from its softmax."""
    parts = []
    for r in range(0, len(x), 256):
        noise = torch.empty(x[r:r + 256].shape, device="cuda").exponential_(generator=gen).log_()
        parts.append((x[r:r + 256].float() / T[r:r + 256, None] - noise).argmax(1))
    return torch.cat(parts).int()


def _sizes(case):
    """(elements, dtype, elements before the first) of each tensor."""
    h, n, vocab = case["hidden"], case["layers"], case["vocab"]
    if case["shapes"] == "tables":
        sizes = [vocab * h, h * vocab]
    elif case["shapes"] == "stack":
        sizes = [vocab * h] + n * (4 * [h * h] + 3 * [4 * h * h] + 2 * [h]) + [h, vocab * h]
    else:
        rng = random.Random(h * 1000 + n)
        sizes = [max(1, int(h * rng.lognormvariate(0.0, 1.0))) for _ in range(n)]
    ragged = case["shapes"] == "ragged"
    types = ["bfloat16", "float32"] if case["dtype"] == "mixed" else [case["dtype"]]
    return [(k, types[i % len(types)], i % 7 if ragged else 0) for i, k in enumerate(sizes)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    uniform = lambda *shape: torch.rand(shape, generator=gen, device="cuda")
    s = {"case": case}
    if case["kind"] in ("clip", "norm"):
        s["grads"], s["out"] = [], []
        for i, (k, dtype, offset) in enumerate(_sizes(case)):
            buf = torch.empty(k + offset, dtype=getattr(torch, dtype), device="cuda")
            s["grads"].append(buf[offset:].normal_(0.0, 1e-3 * 4.0 ** (i % 5), generator=gen))
            if case["kind"] == "clip":
                s["out"].append(torch.empty(k, dtype=getattr(torch, case["out"]), device="cuda"))
        count = sum(t.numel() for t in s["grads"])
        s["max_norm"] = case["limit"] * math.sqrt(count)  # 5e-4: every tensor's mean square is above it; 1: none is
        return s
    N, V = case["N"], case["V"]
    s["logits"] = _rows(gen, N, V, case["dtype"], case["pad"], case.get("masked", False))
    s["T"] = 0.7 + 0.6 * uniform(N)
    tokens = _sampled(gen, s["logits"], s["T"])
    if case["kind"] == "policy":
        x = s["logits"].gather(1, tokens.long()[:, None])[:, 0].double() / s["T"].double()
        lse = torch.cat([torch.logsumexp(s["logits"][r:r + 256].double() / s["T"][r:r + 256, None].double(), 1) for r in range(0, N, 256)])
        # the sampling policy a few updates back; no ratio within a thousandth of a border, where its side is a matter of rounding
        shift = 0.2 * torch.randn(N, generator=gen, device="cuda").double()
        for border in (math.log(1 - 0.2), math.log(1 + 0.28)):
            near = (shift - border).abs() < 1e-3
            shift = torch.where(near, shift + 2e-3, shift)
        s["old"] = (x - lse - shift).float() if case["clipped"] else None
        s["advantages"] = torch.randn(N, generator=gen, device="cuda") if case["clipped"] else uniform(N)
        s["grad"] = torch.full((N,), 1.0 / N, device="cuda")
        s["tokens"] = torch.where(uniform(N) < 0.05, -1, tokens) if N > 1 else tokens  # rows of padding
        return s
    if case["M"] > 1:  # the sampled token, others that the row gives a chance, and places left open
        more = torch.cat([(s["logits"][r:r + 256] > -math.inf).float().multinomial(case["M"] - 1, generator=gen)
                          for r in range(0, N, 256)]).int()
        tokens = torch.cat([tokens[:, None], torch.where(uniform(N, case["M"] - 1) < 0.2, -1, more)], 1).contiguous()
    s["tokens"] = tokens
    if case["kind"] == "score_grad":
        s["grads"] = [torch.randn(tokens.shape, generator=gen, device="cuda") / N, torch.randn(N, generator=gen, device="cuda") / N]
    return s


# ----------------------------------------------------------------------------------------------
# One pass.
# ----------------------------------------------------------------------------------------------


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import top_support_capture_gb300 as sfc

    c = s["case"]
    kind = c["kind"]
    if kind == "score":
        o = sfc.token_logprobs(s["logits"], s["T"], s["tokens"], top=c["K"])
        out = {"logprobs": o.logprobs, "entropy": o.entropy, "status": o.row_status}
        if c["K"]:
            out.update(top_ids=o.top_ids, top_logprobs=o.top_logprobs)
        return out
    if kind == "score_grad":
        x = s["logits"].detach().requires_grad_()
        o = sfc.token_logprobs(x, s["T"], s["tokens"])
        (grad,) = torch.autograd.grad([o.logprobs, o.entropy], x, s["grads"])
        return {"logprobs": o.logprobs.detach(), "entropy": o.entropy.detach(), "grad": grad, "status": o.row_status}
    if kind == "policy":
        o = sfc.policy_loss_and_grad(s["logits"], s["T"], s["tokens"], s["advantages"], s["grad"], old_logprobs=s["old"],
                                     clip_low=0.2, clip_high=0.28, entropy_weight=c["entropy"])
        return {"loss": o.loss, "logprobs": o.logprobs, "entropy": o.entropy, "grad": o.grad_logits, "status": o.row_status}
    if kind == "norm":
        return {"norm": sfc.grad_norm(s["grads"])}
    return {"norm": sfc.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"]), "clipped": s["out"]}


def _plain(s):
    kind = s["case"]["kind"]
    if kind in ("clip", "norm"):
        return _clip(s)
    return _policy(s) if kind == "policy" else _score(s)


def _softmax(x, T):
    """z - max z, its exponentials, their sum [N, 1], the entropies [N, 1] and z's logarithmic normaliser (64 bits)."""
    z = x.float() / T[:, None]
    z = z - z.max(1, keepdim=True).values
    e = z.exp()
    total = e.sum(1, keepdim=True)
    # -inf where a token is masked: its term is 0
    weighted = (e * z.clamp_min(-1e4)).sum(1, keepdim=True)
    ln = total.double().log()
    return z, e, total, ln - weighted.double() / total.double(), ln


def _top(x, K):
    """The K largest logits of each row, ties by the lowest id: (ids, logits)."""
    ids, values = [], []
    for r in range(0, len(x), 256):
        f = x[r:r + 256].float() + 0.0  # -0 to +0
        bits = f.view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2 ** 32 + (2 ** 31 - 1 - torch.arange(x.shape[1], device="cuda"))
        at = key.topk(K, dim=1).indices
        ids.append(at.int())
        values.append(f.gather(1, at))
    return torch.cat(ids), torch.cat(values)


def _score(s):
    c, T = s["case"], s["T"]
    tokens = s["tokens"].long().view(len(T), -1)
    there = tokens >= 0
    z, e, total, H, ln = _softmax(s["logits"], T)
    lp = torch.where(there, z.gather(1, tokens.clamp_min(0)).double() - ln, 0.0)
    out = {"logprobs": lp.float().view(s["tokens"].shape), "entropy": H[:, 0].float(),
           "status": torch.zeros(len(T), dtype=torch.int32, device="cuda")}
    if c["kind"] == "score_grad":
        g, h = torch.where(there, s["grads"][0].view(tokens.shape), 0.0), s["grads"][1][:, None]
        p = e / total
        grad = -p * (g.sum(1, keepdim=True) + h * (z.clamp_min(-1e4) - ln.float() + H.float()))
        grad.scatter_add_(1, tokens.clamp_min(0), g)
        out["grad"] = (grad / T[:, None]).to(s["logits"].dtype)
    elif c["K"]:
        out["top_ids"], x = _top(s["logits"], c["K"])
        at = z.gather(1, out["top_ids"].long())
        out["top_logprobs"] = (at.double() - ln).float()
    return out


def _policy(s):
    T, A = s["T"], s["advantages"]
    there, t = s["tokens"] >= 0, s["tokens"].clamp_min(0).long()[:, None]
    z, e, total, H, ln = _softmax(s["logits"], T)
    lp = (z.gather(1, t).double() - ln)[:, 0]
    if s["old"] is None:
        loss, g = -A * lp, -A.double()
    else:
        ratio = (lp - s["old"].double()).exp()
        loss = -torch.minimum(ratio * A, ratio.clamp(0.8, 1.28) * A)
        active = torch.where(A >= 0, ratio <= 1.28, ratio >= 0.8)
        g = torch.where(active, -ratio * A, 0.0)
    w = s["case"]["entropy"]
    loss = loss - w * H[:, 0]
    up = torch.where(there, s["grad"], 0.0)[:, None] / T[:, None]
    g = g.float()[:, None] * up
    p = e / total
    grad = p * (w * up * (z.clamp_min(-1e4) - ln.float() + H.float()) - g)
    grad.scatter_add_(1, t, g)
    zero = lambda v: torch.where(there, v, 0.0).float()
    return {"loss": zero(loss), "logprobs": zero(lp), "entropy": zero(H[:, 0]), "grad": grad.to(s["logits"].dtype),
            "status": torch.zeros(len(T), dtype=torch.int32, device="cuda")}


def _clip(s):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = total.sqrt()
    out = {"norm": norm.float()}
    if s["case"]["kind"] == "clip":
        scale = (s["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float()
        out["clipped"] = [(t.float() * scale).to(o.dtype) for t, o in zip(s["grads"], s["out"])]
    return out


# ----------------------------------------------------------------------------------------------
# The work that a pass cannot do without, and the outputs in 64 bits.
# ----------------------------------------------------------------------------------------------


def work(case):
    kind = case["kind"]
    width = {"bfloat16": 2, "float32": 4}
    if kind in ("clip", "norm"):
        sizes = _sizes(case)
        read = sum(k * width[dtype] for k, dtype, _ in sizes)
        count = sum(k for k, _, _ in sizes)
        if kind == "norm":
            return {"bytes": read + 4, "flops": 2 * count}
        return {"bytes": read + count * width[case["out"]] + 4, "flops": 3 * count}
    N, V, size = case["N"], case["V"], width[case["dtype"]]
    if kind == "score":
        return {"bytes": N * V * size + N * (12 + 8 * case["M"] + 8 * case["K"]), "flops": 6 * N * V}
    if kind == "score_grad":
        return {"bytes": 2 * N * V * size + N * (16 + 12 * case["M"]), "flops": 12 * N * V}
    return {"bytes": 2 * N * V * size + N * 36, "flops": 12 * N * V}


def _exact_row(x, T):
    """Log-probabilities of one row in 64 bits, and its entropy."""
    lp = torch.log_softmax(x.double() / T.double(), 0)
    p = torch.exp(lp)
    return lp, -torch.where(p > 0, p * lp, 0.0).sum()


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("clip", "norm"):
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]))
        out = {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda")}
        if case["kind"] == "clip":
            out["clipped"] = [t.double() * min(1.0, s["max_norm"] / (norm + 1e-6)) for t in s["grads"]]
        return out
    N, V = case["N"], case["V"]
    f64 = dict(dtype=torch.float64, device="cuda")
    logprobs, entropy = torch.zeros(s["tokens"].shape, **f64), torch.zeros(N, **f64)
    status = torch.zeros(N, dtype=torch.int32, device="cuda")
    given = [row if isinstance(row, list) else [row] for row in s["tokens"].tolist()]
    grad = None if case["kind"] == "score" else torch.zeros((N, V), **f64)
    if case["kind"] == "policy":
        loss = torch.zeros(N, **f64)
        for r, (t,) in enumerate(given):
            if t < 0:
                continue
            lp, H = _exact_row(s["logits"][r], s["T"][r])
            A, w = float(s["advantages"][r]), case["entropy"]
            at = float(lp[t])
            if s["old"] is None:
                value, slope = A * at, A
            else:
                ratio = math.exp(at - float(s["old"][r]))
                bound = (1 + 0.28) * A if A >= 0 else (1 - 0.2) * A
                value = min(ratio * A, bound)
                slope = ratio * A if ratio * A <= bound else 0.0
            logprobs[r], entropy[r] = lp[t], H
            loss[r] = -value - w * H
            p = torch.exp(lp)
            row = slope * p + w * p * (lp + H)
            row[t] -= slope
            grad[r] = row * (s["grad"][r].double() / s["T"][r].double())
        return {"loss": loss, "logprobs": logprobs, "entropy": entropy, "grad": grad, "status": status}
    K = case["K"]
    top_ids, top_lps = torch.zeros((N, K), dtype=torch.int32, device="cuda"), torch.zeros((N, K), **f64)
    flat = logprobs.view(N, -1)
    for r, row in enumerate(given):
        lp, H = _exact_row(s["logits"][r], s["T"][r])
        entropy[r] = H
        for j, t in enumerate(row):
            if t >= 0:
                flat[r, j] = lp[t]
        if grad is not None:
            p = torch.exp(lp)
            g = s["grads"][0].view(N, -1)[r].double()
            for j, t in enumerate(row):
                if t >= 0:
                    grad[r] -= g[j] * p
                    grad[r, t] += g[j]
            grad[r] -= s["grads"][1][r].double() * torch.where(p > 0, p * (lp + H), 0.0)
            grad[r] /= s["T"][r].double()
        if K:
            order = torch.sort(s["logits"][r].float(), descending=True, stable=True).indices[:K]
            top_ids[r], top_lps[r] = order.int(), lp[order]
    out = {"logprobs": logprobs, "entropy": entropy, "status": status}
    if grad is not None:
        out["grad"] = grad
    if K:
        out.update(top_ids=top_ids, top_logprobs=top_lps)
    return out
