"""What is measured of the operators that consume captured supports and a target's logits: distillation
from a teacher's top logits (loss and gradient), the gradient of the support replay, and the verification of
drafted tokens (over full rows and over captured supports).

Each operator has its plain form here, in elementary torch operations, beside the call that a user makes.
"""
import math

import torch

own = False

# ----------------------------------------------------------------------------------------------
# Cases. Vocabularies (32000, 151936, 129280, 262144), row counts and packed widths are those of this
# repository's decode workloads; 50021 is its tests' odd vocabulary.
# ----------------------------------------------------------------------------------------------


def listed():
    bf16, f32 = "bfloat16", "float32"
    return [
        # a draft model's training micro-batch on captured supports of the half-batch workload
        dict(name="distill_step_64x32000_bf16", kind="distill_step", N=64, V=32000, pad=0, W=1024, dtype=bf16, normalise=False),
        # a full training batch of tokens: the largest
        dict(name="distill_step_2048x151936_bf16", kind="distill_step", N=2048, V=151936, pad=0, W=1024, dtype=bf16, normalise=False),
        # teacher's raw top logits, wide supports, through autograd (loss, then backward)
        dict(name="distill_autograd_256x129280_f32", kind="distill_autograd", N=256, V=129280, pad=0, W=8192, dtype=f32, normalise=True),
        # evaluation of a few held-out tokens: the loss alone, where latency counts
        dict(name="distill_loss_8x262144_bf16", kind="distill_loss", N=8, V=262144, pad=0, W=50, dtype=bf16, normalise=False),
        # the smallest policy-gradient step, on the smallest decode workload
        dict(name="replay_grad_4x1024_f32", kind="replay_grad", N=4, V=1024, pad=0, W=1024, dtype=f32, entries=False),
        # a reinforcement-learning batch over the bench workload's supports
        dict(name="replay_grad_512x151936_bf16", kind="replay_grad", N=512, V=151936, pad=0, W=1024, dtype=bf16, entries=False),
        # wide supports, with an upstream gradient for every member (an entropy or KL term over the support)
        dict(name="replay_grad_256x129280_f32_entries", kind="replay_grad", N=256, V=129280, pad=0, W=8192, dtype=f32, entries=True),
        # one user's decode: the smallest verification
        dict(name="verify_1x4x151936_bf16", kind="verify", B=1, D=4, V=151936, pad=0, dtype=bf16, drafts="logits", ragged=False, greedy=False),
        # a serving batch
        dict(name="verify_64x4x151936_bf16", kind="verify", B=64, D=4, V=151936, pad=0, dtype=bf16, drafts="logits", ragged=False, greedy=False),
        # drafts looked up in the prompt (no draft distribution), ragged counts, greedy rows among them, odd rows
        dict(name="verify_33x7x50021_f32_lookup", kind="verify", B=33, D=7, V=50021, pad=0, dtype=f32, drafts="lookup", ragged=True, greedy=True),
        # one user's decode under top-k / top-p: verification over captured supports
        dict(name="verify_supports_1x4_w1024", kind="verify_supports", B=1, D=4, V=151936, W=1024, Wd=1024, ragged=False),
        # a serving batch with wide supports
        dict(name="verify_supports_128x4_w8192", kind="verify_supports", B=128, D=4, V=129280, W=8192, Wd=1024, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["distill_step", "distill_autograd", "distill_loss", "replay_grad", "verify", "verify_supports"])
    dtype = rng.choice(["bfloat16", "float32"])
    V = rng.choice([_log_int(rng, 1000, 262144), _log_int(rng, 1000, 262144), 32000, 151936])
    pad = rng.choice([0, 0, rng.randrange(1, 64)])
    size = 2 if dtype == "bfloat16" else 4
    W = min(_log_int(rng, 1, 8192), V)
    if kind in ("distill_step", "distill_autograd", "distill_loss", "replay_grad"):
        N = min(_log_int(rng, 1, 2048), max(1, 2048 * 151936 * 2 // (V * size)))
        case = dict(kind=kind, N=N, V=V, pad=pad, W=W, dtype=dtype)
        if kind == "replay_grad":
            case["entries"] = rng.random() < 0.5
        else:
            case["normalise"] = rng.random() < 0.5
        return case
    B, D = _log_int(rng, 1, 128), rng.randrange(1, 9)
    if kind == "verify":
        B = max(1, min(B, 128 * 5 * 151936 * 2 // ((2 * D + 1) * V * size)))
        return dict(kind=kind, B=B, D=D, V=V, pad=pad, dtype=dtype, drafts=rng.choice(["logits", "logits", "lookup"]),
                    ragged=rng.random() < 0.5, greedy=rng.random() < 0.25)
    return dict(kind=kind, B=B, D=D, V=V, W=W, Wd=min(_log_int(rng, 1, 8192), V), ragged=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------
# Inputs: Zipf-ranked logit rows plus Gaussian noise, as the decode workloads have them.
# ----------------------------------------------------------------------------------------------


def _rows(gen, N, V, dtype, pad=0, other=None, sigma=1.0):
    """[N, V] logits (a view of rows V + pad apart): a 12-logit Zipf profile, another shift of one random
    permutation for each row, plus noise; or `other` plus noise."""
    buf = torch.empty((N, V + pad), dtype=getattr(torch, dtype), device="cuda")
    out = buf[:, :V]
    rank = torch.arange(1, V + 1, device="cuda", dtype=torch.float32)
    prof = rank.log() * (-12.0 / math.log(max(V, 2)))
    prof = prof[torch.randperm(V, generator=gen, device="cuda")]
    shift = torch.randint(0, V, (N, 1), generator=gen, device="cuda")
    for r in range(0, N, 256):
        k = min(256, N - r)
        base = prof[(torch.arange(V, device="cuda") + shift[r:r + k]) % V] if other is None else other[r:r + k].float()
        out[r:r + k] = base + sigma * torch.randn((k, V), generator=gen, device="cuda")
    return out


def _supports(gen, logits, T, W, lowest=0):
    """Packed supports of the rows: the top entries (ids, largest first), their logprobs renormalised over
    the support, their raw logits, and ragged lengths."""
    N, V = logits.shape
    k = min(W, V)
    parts = [torch.topk(logits[r:r + 256].float(), k, dim=1) for r in range(0, N, 256)]
    val, ids = torch.cat([p.values for p in parts]), torch.cat([p.indices for p in parts])
    n = torch.randint(1, k + 1, (N,), generator=gen, device="cuda")
    if lowest == 0:
        n = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.05, torch.zeros_like(n), n)
    there = torch.arange(k, device="cuda") < n[:, None]
    z = torch.where(there, val / T[:, None], -math.inf)
    lp = torch.where(there, z - z.logsumexp(1, keepdim=True), 0.0)
    full = lambda x, fill, dt: torch.nn.functional.pad(torch.where(there, x, fill), (0, W - k), value=fill).to(dt).contiguous()
    return full(ids, -1, torch.int32), full(lp, 0.0, torch.float32), full(val, 0.0, torch.float32), n.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, V = case["kind"], case["V"]
    uniform = lambda *shape: torch.rand(shape, generator=gen, device="cuda")
    s = {"case": case}
    if kind in ("distill_step", "distill_autograd", "distill_loss", "replay_grad"):
        N = case["N"]
        s["logits"] = _rows(gen, N, V, case["dtype"], case["pad"])
        s["T"] = 0.7 + 0.6 * uniform(N)
        teacher = _rows(gen, N, V, case["dtype"], 0, s["logits"])
        s["ids"], lp, val, s["lengths"] = _supports(gen, teacher, s["T"], case["W"], 1 if kind == "replay_grad" else 0)
        s["grad"] = torch.randn(N, generator=gen, device="cuda") / N
        if kind == "replay_grad":
            at = (uniform(N) * s["lengths"]).long()
            s["tokens"] = s["ids"].gather(1, at[:, None])[:, 0].contiguous()
            s["grad_entries"] = torch.randn(s["ids"].shape, generator=gen, device="cuda") / N if case["entries"] else None
        else:
            s["values"] = val if case["normalise"] else lp
        return s
    B, D = case["B"], case["D"]
    s["seed"], s["step"] = seed, 17
    s["uniforms"] = uniform(B, D)
    s["num_drafts"] = torch.randint(0, D + 1, (B,), generator=gen, device="cuda").to(torch.int32) if case["ragged"] else None
    if kind == "verify":
        rows = _rows(gen, B * (D + 1), V, case["dtype"], case["pad"])
        s["target"] = rows.unflatten(0, (B, D + 1))
        s["T"] = 0.7 + 0.6 * uniform(B)
        if case["greedy"]:
            s["T"][::4] = 0.0
        near = _rows(gen, B * D, V, case["dtype"], case["pad"], s["target"][:, :D].flatten(0, 1))
        T = torch.where(s["T"] > 0, s["T"], 1.0).repeat_interleave(D)
        s["tokens"] = torch.cat([(near[r:r + 256].float() / T[r:r + 256, None] - torch.empty((len(near[r:r + 256]), V), device="cuda")
                                  .exponential_(generator=gen).log_()).argmax(1) for r in range(0, B * D, 256)]).to(torch.int32).view(B, D)
        s["draft"] = near.unflatten(0, (B, D)) if case["drafts"] == "logits" else None
        return s
    target = _rows(gen, B * (D + 1), V, "bfloat16")
    ones = torch.ones(B * (D + 1), device="cuda")
    ids, lp, _, n = _supports(gen, target, ones, case["W"], 1)
    s["ids"], s["lps"], s["lengths"] = ids.view(B, D + 1, -1), lp.view(B, D + 1, -1), n.view(B, D + 1)
    near = _rows(gen, B * D, V, "bfloat16", 0, target.view(B, D + 1, V)[:, :D].flatten(0, 1))
    ids, lp, _, n = _supports(gen, near, ones[:B * D], case["Wd"], 1)
    race = torch.where(torch.arange(ids.shape[1], device="cuda") < n[:, None],
                       lp - torch.empty_like(lp).exponential_(generator=gen).log_(), -math.inf)
    s["tokens"] = ids.gather(1, race.argmax(1, keepdim=True)).view(B, D).contiguous()
    s["draft_ids"], s["draft_lps"], s["draft_lengths"] = ids.view(B, D, -1), lp.view(B, D, -1), n.view(B, D)
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
    if kind == "distill_step":
        o = sfc.distill_loss_and_grad(s["logits"], s["T"], s["ids"], s["values"], s["lengths"], s["grad"], normalise=c["normalise"])
        return {"loss": o.loss, "grad": o.grad_logits, "status": o.row_status}
    if kind == "distill_autograd":
        x = s["logits"].detach().requires_grad_()
        o = sfc.distill_loss(x, s["T"], s["ids"], s["values"], s["lengths"], normalise=c["normalise"])
        (grad,) = torch.autograd.grad(o.loss, x, s["grad"])
        return {"loss": o.loss.detach(), "grad": grad, "status": o.row_status}
    if kind == "distill_loss":
        o = sfc.distill_loss(s["logits"], s["T"], s["ids"], s["values"], s["lengths"], normalise=c["normalise"])
        return {"loss": o.loss, "status": o.row_status}
    if kind == "replay_grad":
        return {"grad": sfc.replay_logprob_backward(s["logits"], s["T"], s["ids"], s["lengths"], s["tokens"], s["grad"],
                                                    grad_support_logprobs=s["grad_entries"])}
    if kind == "verify":
        o = sfc.verify_drafts(s["target"], s["draft"], s["tokens"], s["uniforms"], s["T"], s["seed"], s["step"],
                              num_drafts=s["num_drafts"], greedy_t0=c["greedy"])
    else:
        o = sfc.verify_supports(s["ids"], s["lps"], s["lengths"], s["draft_ids"], s["draft_lps"], s["draft_lengths"], s["tokens"],
                                s["uniforms"], s["seed"], s["step"], num_drafts=s["num_drafts"])
    return {"accepted": o.accepted, "tokens": o.tokens, "logprobs": o.token_logprobs, "status": o.row_status}


def _plain(s):
    kind = s["case"]["kind"]
    if kind.startswith("distill"):
        return _distill(s, kind != "distill_loss")
    if kind == "replay_grad":
        return _replay_grad(s)
    return _verify(s) if kind == "verify" else _verify_supports(s)


def _distill(s, backward):
    x, T = s["logits"].float(), s["T"][:, None]
    there = torch.arange(s["ids"].shape[1], device=x.device) < s["lengths"][:, None]
    ids = torch.where(there, s["ids"], 0).long()
    z = x / T
    m = z.max(1, keepdim=True).values
    e = (z - m).exp()
    total = e.sum(1, keepdim=True)
    y = s["values"]
    if s["case"]["normalise"]:
        y = torch.where(there, y / T, -math.inf)
        top = torch.where(s["lengths"][:, None] > 0, y.max(1, keepdim=True).values, 0.0)
        y = y - top
        y = y - torch.where(there, y, -math.inf).exp().sum(1, keepdim=True).clamp_min(1e-30).log()
    t = torch.where(there, y.exp(), 0.0)
    # a difference of near values: the sum is held in 64 bits
    lp = (z.gather(1, ids).double() - m.double()) - total.double().log()
    loss = torch.where(there, t.double() * (torch.where(there, y, 0.0).double() - lp), 0.0).sum(1).float()
    status = torch.zeros(len(x), dtype=torch.int32, device=x.device)
    if not backward:
        return {"loss": loss, "status": status}
    g = s["grad"][:, None] / T
    grad = e.mul_(g * t.sum(1, keepdim=True) / total)
    grad.scatter_add_(1, ids, -t * g)
    return {"loss": loss, "grad": grad.to(s["logits"].dtype), "status": status}


def _replay_grad(s):
    there = torch.arange(s["ids"].shape[1], device="cuda") < s["lengths"][:, None]
    ids, T = torch.where(there, s["ids"], 0).long(), s["T"][:, None]
    z = torch.where(there, s["logits"].gather(1, ids).float() / T, -math.inf)
    pi = (z - z.max(1, keepdim=True).values).exp()
    pi = pi / pi.sum(1, keepdim=True)
    up = torch.where(there & (s["ids"] == s["tokens"][:, None]), s["grad"][:, None], 0.0)
    if s["grad_entries"] is not None:
        up = up + torch.where(there, s["grad_entries"], 0.0)
    g = torch.where(there, (up - pi * up.sum(1, keepdim=True)) / T, 0.0)
    out = torch.zeros(s["logits"].shape, dtype=torch.float32, device="cuda").scatter_add_(1, ids, g)
    return {"grad": out.to(s["logits"].dtype)}


def _mulhilo(a, b):
    """High and low words of the product of two 32-bit numbers held in 64 bits (the product wraps there)."""
    p = a * b
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _waits(rows, ids, seed, step):
    """-ln u for every (row, id): u = (2 (w >> 9) + 1) 2^-24, w = word id % 4 of Philox4x32-10 at the counter
    (2^31 + id / 4, row, step lo, step hi) under the key (seed lo, seed hi)."""
    c0, c1 = (ids >> 2) | (1 << 31), rows.expand_as(ids)
    c2, c3 = torch.full_like(ids, step & 0xFFFFFFFF), torch.full_like(ids, step >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        (h0, l0), (h1, l1) = _mulhilo(c0, 0xD2511F53), _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    word = ids & 3
    w = torch.where(word == 0, c0, torch.where(word == 1, c1, torch.where(word == 2, c2, c3)))
    return -((2 * (w >> 9) + 1).double() * 2.0 ** -24).log()


def _emit(s, accept, tokens, drawn, lp_drafts, lp_drawn):
    """Outputs from the per-draft decisions and the token drawn at the first refusal."""
    B, D = tokens.shape
    accepted = accept.long().cumprod(1).sum(1)
    at = torch.arange(D + 1, device="cuda")
    pad = torch.nn.functional.pad
    put = lambda drafts, last, rest: torch.where(at < accepted[:, None], pad(drafts, (0, 1)), torch.where(at == accepted[:, None], last[:, None], rest))
    return {"accepted": accepted.int(), "tokens": put(tokens, drawn, -1).int(), "logprobs": put(lp_drafts, lp_drawn, 0.0).float(),
            "status": torch.zeros(B, dtype=torch.int32, device="cuda")}


def _counts(s, B, D):
    n = s["num_drafts"].long() if s["num_drafts"] is not None else torch.full((B,), D, device="cuda")
    return n, torch.arange(D, device="cuda") < n[:, None]


def _log_softmax(x, T):
    """Log-probabilities of [..., V] logits at T [B], in 64 bits (they are compared with numbers next to them);
    a row of T = 0 has all its mass at its first largest entry."""
    T = T.double().view(-1, *[1] * (x.dim() - 1))
    z = x.double() / torch.where(T > 0, T, 1.0)
    z = z - z.max(-1, keepdim=True).values
    lp = z - z.exp().sum(-1, keepdim=True).log()
    only = torch.arange(x.shape[-1], device="cuda") == x.float().argmax(-1, keepdim=True)
    return torch.where(T > 0, lp, torch.where(only, 0.0, -math.inf))


def _verify(s):
    B, D = s["tokens"].shape
    n, there = _counts(s, B, D)
    token = s["tokens"].long()[:, :, None]
    lp = _log_softmax(s["target"], s["T"])
    lq = _log_softmax(s["draft"], s["T"]) if s["draft"] is not None else None
    lp_drafts = lp[:, :D].gather(2, token)[:, :, 0]
    q = lq.gather(2, token)[:, :, 0].exp() if lq is not None else 1.0
    accept = there & (s["uniforms"].double() * q < lp_drafts.exp())
    a = accept.long().cumprod(1).sum(1)
    b = torch.arange(B, device="cuda")
    p, refused, ids = lp[b, a].exp(), a < n, torch.arange(lp.shape[2], device="cuda")
    last = a.clamp_max(D - 1)
    q = lq[b, last].exp() if lq is not None else (ids == token[b, last]).double()
    w = torch.where(refused[:, None], (p - q).clamp_min(0), p)
    w = torch.where(w.max(1, keepdim=True).values > 0, w, p)
    drawn = (w / _waits(b[:, None], ids.expand_as(w).contiguous(), s["seed"], s["step"])).argmax(1)
    return _emit(s, accept, s["tokens"].long(), drawn, lp_drafts, lp[b, a].gather(1, drawn[:, None])[:, 0])


def _spread(ids, lps, lengths, V):
    """[..., V] log-probabilities of packed supports, -inf outside them."""
    there = torch.arange(ids.shape[-1], device="cuda") < lengths[..., None]
    full = torch.full((*ids.shape[:-1], V + 1), -math.inf, dtype=torch.float32, device="cuda")
    return full.scatter_(-1, torch.where(there, ids, V).long(), torch.where(there, lps, -math.inf))[..., :V]


def _verify_supports(s):
    B, D = s["tokens"].shape
    V = s["case"]["V"]
    n, there = _counts(s, B, D)
    token = s["tokens"].long()
    find = lambda ids, lps, lengths: torch.where((ids == s["tokens"][:, :, None]) & (torch.arange(ids.shape[2], device="cuda") < lengths[:, :, None]),
                                                 lps, -math.inf).max(2).values
    lp_drafts = find(s["ids"][:, :D], s["lps"][:, :D], s["lengths"][:, :D])
    q = find(s["draft_ids"], s["draft_lps"], s["draft_lengths"]).double().exp()
    accept = there & (s["uniforms"].double() * q < lp_drafts.double().exp())
    a = accept.long().cumprod(1).sum(1)
    b, last = torch.arange(B, device="cuda"), a.clamp_max(D - 1)
    lp = _spread(s["ids"][b, a], s["lps"][b, a], s["lengths"][b, a], V)
    lq = _spread(s["draft_ids"][b, last], s["draft_lps"][b, last], s["draft_lengths"][b, last], V)
    p = lp.double().exp()
    w = torch.where((a < n)[:, None], (p - lq.double().exp()).clamp_min(0), p)
    w = torch.where(w.max(1, keepdim=True).values > 0, w, p)
    ids = torch.arange(V, device="cuda").expand_as(w).contiguous()
    drawn = (w / _waits(b[:, None], ids, s["seed"], s["step"])).argmax(1)
    return _emit(s, accept, token, drawn, lp_drafts, lp.gather(1, drawn[:, None])[:, 0])


# ----------------------------------------------------------------------------------------------
# The work that a pass cannot do without, and the outputs in 64 bits.
# ----------------------------------------------------------------------------------------------


def work(case):
    kind, V = case["kind"], case["V"]
    size = 2 if case.get("dtype") == "bfloat16" else 4
    if kind in ("distill_step", "distill_autograd", "distill_loss", "replay_grad"):
        N, n = case["N"], case["N"] * case["W"] // 2  # lengths are ragged: half of the width on average
        if kind == "replay_grad":  # ids and logits of the supports in, the gradient's rows out
            return {"bytes": N * V * size + n * (4 + size + (4 if case["entries"] else 0)) + 16 * N, "flops": 8 * n}
        if kind == "distill_loss":
            return {"bytes": N * V * size + n * 8 + 16 * N, "flops": 4 * N * V}
        return {"bytes": 2 * N * V * size + n * 8 + 20 * N, "flops": 8 * N * V}
    B, D = case["B"], case["D"]
    if kind == "verify":
        rows = B * (D + 1) + (B * D if case["drafts"] == "logits" else 0)
        return {"bytes": rows * V * size + B * (D + 1) * 16, "flops": 4 * rows * V + 20 * B * V}
    n = B * (D + 1) * case["W"] // 2 + B * D * case["Wd"] // 2
    return {"bytes": n * 8 + B * (D + 1) * 16, "flops": 4 * n}


def _exact_stats(x, T):
    z = x.to(torch.float64).div(T)
    return z, torch.logsumexp(z, dim=-1)


def exact(case, seed):
    kind = case["kind"]
    s = prepare(case, seed)
    if kind == "verify":
        return _exact_verify(s)
    if kind == "verify_supports":
        return _exact_verify_supports(s)
    N, V = case["N"], case["V"]
    lens = s["lengths"].tolist()
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    grad = torch.zeros((N, V), dtype=torch.float64, device="cuda") if kind != "distill_loss" else None
    for r, n in enumerate(lens):  # row by row, over the row's own entries
        if n == 0:
            continue
        T, ids = s["T"][r].double(), s["ids"][r, :n].long()
        if kind == "replay_grad":
            z, lse = _exact_stats(s["logits"][r, ids], T)
            up = torch.zeros(n, dtype=torch.float64, device="cuda")
            if s["grad_entries"] is not None:
                up += s["grad_entries"][r, :n]
            up += (ids == s["tokens"][r]) * s["grad"][r].double()
            grad[r, ids] = (up - torch.exp(z - lse) * up.sum()) / T
            continue
        z, lse = _exact_stats(s["logits"][r], T)
        y = s["values"][r, :n].double()
        ln_t = torch.log_softmax(y / T, dim=0) if case["normalise"] else y
        t = torch.exp(ln_t)
        loss[r] = torch.dot(t, ln_t - (z[ids] - lse))
        if grad is not None:
            grad[r] = torch.exp(z - lse) * t.sum()
            grad[r, ids] -= t
            grad[r] *= s["grad"][r].double() / T
    if kind == "replay_grad":
        return {"grad": grad}
    status = torch.zeros(N, dtype=torch.int32, device="cuda")
    return {"loss": loss, "status": status} if grad is None else {"loss": loss, "grad": grad, "status": status}


def _exact_race(s, b, w, ids):
    """The id that wins the race of weights w."""
    e = _waits(torch.full((1,), b, dtype=torch.int64, device="cuda"), ids, s["seed"], s["step"])
    score = torch.log(w) - torch.log(e)
    best = score.max()
    return int(ids[score == best].min())


def _exact_walk(s, target, draft):
    """Request by request: target(b, j) and draft(b, j) give (ids, probabilities in 64 bits), draft None for
    a certain draft."""
    B, D = s["tokens"].shape
    accepted, tokens, logprobs = [], [], []
    counts = s["num_drafts"].tolist() if s["num_drafts"] is not None else [D] * B
    drafted, u = s["tokens"].tolist(), s["uniforms"].double().tolist()
    for b in range(B):
        out, lps = [], []
        while True:
            j = len(out)
            ids, p = target(b, j)
            w = p
            if j < counts[b]:
                d = drafted[b][j]
                hit = p[ids == d]
                pd = float(hit[0]) if len(hit) else 0.0
                q_of = draft(b, j)
                if q_of is None:
                    qd, q = 1.0, (ids == d).double()
                else:
                    hit = q_of[1][q_of[0] == d]
                    qd = float(hit[0]) if len(hit) else 0.0
                    q = torch.zeros(s["case"]["V"], dtype=torch.float64, device="cuda").index_copy_(0, q_of[0], q_of[1])[ids]
                if u[b][j] * qd < pd:
                    out.append(d)
                    lps.append(math.log(pd))
                    continue
                w = torch.clamp(p - q, min=0)
                if not bool((w > 0).any()):
                    w = p
            token = _exact_race(s, b, w, ids)
            accepted.append(j)
            out.append(token)
            lps.append(math.log(float(p[ids == token][0])))
            break
        tokens.append(out + [-1] * (D + 1 - len(out)))
        logprobs.append(lps + [0.0] * (D + 1 - len(lps)))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    return {"accepted": i32(accepted), "tokens": i32(tokens), "logprobs": torch.tensor(logprobs, dtype=torch.float64, device="cuda"),
            "status": torch.zeros(B, dtype=torch.int32, device="cuda")}


def _exact_verify(s):
    V = s["case"]["V"]
    ids = torch.arange(V, device="cuda")

    def dist(x, b):
        T = float(s["T"][b])
        if T == 0.0:
            p = torch.zeros(V, dtype=torch.float64, device="cuda")
            p[int((x == x.max()).nonzero()[0])] = 1.0
            return p
        return torch.softmax(x.double() / s["T"][b].double(), 0)

    return _exact_walk(s, lambda b, j: (ids, dist(s["target"][b, j], b)),
                       (lambda b, j: (ids, dist(s["draft"][b, j], b))) if s["draft"] is not None else (lambda b, j: None))


def _exact_verify_supports(s):
    def packed(i, l, n):
        return lambda b, j: (i[b, j, :int(n[b, j])].long(), torch.exp(l[b, j, :int(n[b, j])].double()))

    return _exact_walk(s, packed(s["ids"], s["lps"], s["lengths"]), packed(s["draft_ids"], s["draft_lps"], s["draft_lengths"]))
