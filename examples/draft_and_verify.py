"""A small draft model learns a target's captured supports and then drafts for it.

The target is a fixed table of next-token logits, the draft a low-rank model of it. One program runs what the library
has for such a pair:

  1. the target decodes with top-k / top-p and captures each position's support     sample_filter_capture
  2. the draft is trained on those supports                                         distill_loss_and_grad
  3. the draft is tuned on its own samples, over their supports                     replay_logprob (differentiable)
     with the target's log-probabilities as reward                                  token_logprobs
  4. the draft drafts, the target verifies                                          verify_supports, verify_drafts
  5. the draft is tuned over its whole vocabulary, a few updates per sample         policy_loss_and_grad, clip_grad_norm

and prints how many tokens each call of the target yields before and after. `python examples/draft_and_verify.py`
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import top_support_capture_gb300 as sfc

V, RANK, WIDTH, TOP_K, TOP_P, DRAFTS = 2000, 32, 256, 64, 0.95, 4


class Draft(torch.nn.Module):
    def __init__(self, seed=0):
        super().__init__()
        gen = torch.Generator("cpu").manual_seed(seed)
        self.rows = torch.nn.Parameter(0.1 * torch.randn(V, RANK, generator=gen))
        self.cols = torch.nn.Parameter(0.1 * torch.randn(RANK, V, generator=gen))

    def forward(self, token):
        return self.rows[token.long()] @ self.cols


def target_table(seed=1):
    gen = torch.Generator("cpu").manual_seed(seed)
    return 3.0 * (torch.randn(V, RANK // 2, generator=gen) @ torch.randn(RANK // 2, V, generator=gen)) / (RANK // 2) ** 0.5


def capture(logits, seed, step):
    """One decode step of every row with its support captured."""
    rows, full = logits.shape[0], lambda v, dt: torch.full((logits.shape[0],), v, dtype=dt, device=logits.device)
    return sfc.sample_filter_capture(logits, full(1.0, torch.float32), full(TOP_K, torch.int32), full(TOP_P, torch.float32),
                                     full(0.0, torch.float32), seed, step, full(1, torch.uint8), packed_width=WIDTH)


def distil(draft, table, steps=150, batch=512):
    opt = torch.optim.Adam(draft.parameters(), lr=0.02)
    ones = torch.ones(batch, device=table.device)
    losses = []
    for step in range(steps):
        context = torch.randint(0, V, (batch,), device=table.device)
        teacher = capture(table[context], 11, step)
        logits = draft(context)
        out = sfc.distill_loss_and_grad(logits.detach(), ones, teacher.support_ids, teacher.support_logprobs, teacher.lengths,
                                        ones / batch)
        opt.zero_grad()
        logits.backward(out.grad_logits)
        opt.step()
        losses.append(out.loss.mean())
    return torch.stack(losses)


def tune(draft, table, steps=20, batch=512):
    """Policy gradient on the draft's own samples: the reward of a token is the target's log-probability."""
    opt = torch.optim.Adam(draft.parameters(), lr=0.002)
    ones = torch.ones(batch, device=table.device)
    for step in range(steps):
        context = torch.randint(0, V, (batch,), device=table.device)
        with torch.no_grad():
            own = capture(draft(context), 13, step)
            reward = sfc.token_logprobs(table[context], ones, own.tokens).logprobs
        replay = sfc.replay_logprob(draft(context), ones, own.support_ids, own.lengths, own.tokens)
        loss = -((reward - reward.mean()) * replay.token_logprob).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()


def tune_clipped(draft, table, steps=10, epochs=3, batch=512):
    """Towards the target's distribution by unfiltered samples (the reward is how much likelier the target finds them): clipped
    policy updates and clipped gradients. Returns the gradients' norms."""
    opt = torch.optim.Adam(draft.parameters(), lr=0.0005)
    ones, norms = torch.ones(batch, device=table.device), []
    for step in range(steps):
        context = torch.randint(0, V, (batch,), device=table.device)
        with torch.no_grad():
            logits = draft(context)
            tokens = torch.multinomial(logits.softmax(1), 1)[:, 0].int()
            old = sfc.token_logprobs(logits, ones, tokens).logprobs
            reward = sfc.token_logprobs(table[context], ones, tokens).logprobs - old
            advantages = (reward - reward.mean()) / (reward.std() + 1e-6)
        for _ in range(epochs):
            logits = draft(context)
            out = sfc.policy_loss_and_grad(logits.detach(), ones, tokens, advantages, ones / batch, old_logprobs=old)
            opt.zero_grad()
            logits.backward(out.grad_logits)
            norms.append(sfc.clip_grad_norm([p.grad for p in draft.parameters()], 1.0))
            opt.step()
    return torch.stack(norms)


@torch.no_grad()
def speculate(draft, table, rounds=16, requests=64, filtered=True):
    """Rounds of drafting and verification; returns the mean number of tokens per call of the target."""
    dev = table.device
    last = torch.randint(0, V, (requests,), dtype=torch.int32, device=dev)
    ones, emitted = torch.ones(requests, device=dev), 0
    for r in range(rounds):
        drafts, token = [], last
        for j in range(DRAFTS):  # the draft decodes
            logits = draft(token)
            if filtered:
                step = capture(logits, 21, r * DRAFTS + j)
                token = step.tokens
            else:
                step = logits
                token = torch.multinomial(logits.softmax(1), 1)[:, 0].int()
            drafts.append((token, step))
        tokens = torch.stack([t for t, _ in drafts], 1)
        rows = table[torch.cat([last[:, None], tokens], 1).long()]  # the target's rows, all positions in one call
        u = torch.rand(requests, DRAFTS, device=dev)
        if filtered:
            t = capture(rows.flatten(0, 1), 22, r)
            split = lambda x, k: x.view(requests, k, *x.shape[1:])
            side = lambda name: torch.stack([getattr(s, name) for _, s in drafts], 1)
            out = sfc.verify_supports(split(t.support_ids, DRAFTS + 1), split(t.support_logprobs, DRAFTS + 1),
                                      split(t.lengths, DRAFTS + 1), side("support_ids"), side("support_logprobs"), side("lengths"),
                                      tokens, u, 23, r)
        else:
            out = sfc.verify_drafts(rows, torch.stack([s for _, s in drafts], 1), tokens, u, ones, 23, r)
        last = out.tokens.gather(1, out.accepted.long()[:, None])[:, 0].contiguous()
        emitted += out.accepted.sum() + requests
    return float(emitted) / (rounds * requests)


def main():
    torch.manual_seed(0)
    table, draft = target_table().cuda(), Draft().cuda()
    before = speculate(draft, table)
    losses = distil(draft, table)
    after = speculate(draft, table)
    tune(draft, table)
    tuned, dense = speculate(draft, table), speculate(draft, table, filtered=False)
    norms = tune_clipped(draft, table)
    clipped = speculate(draft, table, filtered=False)
    print(f"distillation loss {float(losses[0]):.3f} -> {float(losses[-1]):.3f}")
    print(f"tokens per call of the target: untrained {before:.2f}, distilled {after:.2f}, tuned {tuned:.2f}, unfiltered {dense:.2f}")
    print(f"clipped updates over the whole vocabulary: gradient norm {float(norms[0]):.3f} -> {float(norms[-1]):.3f}, unfiltered {clipped:.2f}")
    return losses, before, after, tuned, dense


if __name__ == "__main__":
    main()
