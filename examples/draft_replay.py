"""A drafter trained from prioritized replay: the operators of rl_infra_gb300.ops around a ReplayBuffer.

An actor drafts tokens with a small recurrent model (a gated linear recurrence), has them verified against a
target's probabilities and stores what it saw: the context, the target's top logits there, and as the
row's priority how likely the draft was to be refused.  A learner samples rows by priority, runs the
drafter over their contexts, takes the distillation loss against the stored top logits with the batch's
importance weights, and writes the row losses back as the next priorities.  Every step stays on the GPU.

  python examples/draft_replay.py [--rounds 150] [--seed 0]

The target is a fixed random table of next-token logits, so that the example needs no data; what is
printed is the share of drafted tokens that the target accepts, which rises as the drafter learns.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from rl_infra_gb300 import capi, ops  # noqa: E402

VOCAB, CHANNELS, CONTEXT, TOP, DRAFTS, ACTORS, BATCH = 509, 128, 8, 16, 4, 64, 256


class Drafter:
    """Embedding, gate and input projections, the recurrence, and the head."""

    def __init__(self, gen):
        new = lambda *s, scale: (torch.randn(*s, generator=gen, device="cuda") * scale).requires_grad_()
        self.embed = new(VOCAB, CHANNELS, scale=1.0)
        self.project = new(CHANNELS, 2 * CHANNELS, scale=CHANNELS ** -0.5)
        self.head = new(CHANNELS, VOCAB, scale=CHANNELS ** -0.5)
        self.params = [self.embed, self.project, self.head]

    def parts(self, tokens):
        """gate and input [..., CHANNELS]: the two halves of one projection, used as they lie"""
        both = self.embed[tokens] @ self.project
        return both[..., :CHANNELS], both[..., CHANNELS:]

    def logits(self, tokens):
        """Next-token logits after each context [B, CONTEXT]."""
        gate, value = self.parts(tokens)
        _, last = ops.gated_scan(gate, value, gate=ops.GATE_SIGMOID)
        return last @ self.head

    @torch.no_grad()
    def draft(self, tokens, gen):
        """DRAFTS tokens after each context, and the probabilities that they were drawn from."""
        gate, value = self.parts(tokens)
        state = ops.scan_forward(gate, value, gate=ops.GATE_SIGMOID)["last"]
        drawn, probs = [], []
        for i in range(DRAFTS):
            probs.append(torch.softmax(state @ self.head, -1))
            drawn.append(torch.multinomial(probs[-1], 1, generator=gen).squeeze(1))
            if i + 1 < DRAFTS:   # one step of the recurrence, the state updated in place
                gate, value = self.parts(drawn[-1])
                ops.scan_step(gate, value, state, gate=ops.GATE_SIGMOID, out={"state": state})
        return torch.stack(drawn, 1), torch.stack(probs, 1)


def rollout(drafter, target, contexts, buffer, gen):
    """One verified draft a sequence; its positions enter the buffer.  Returns the new contexts and the
    share of drafted tokens that were accepted."""
    n = contexts.shape[0]
    tokens, q = drafter.draft(contexts, gen)
    run = torch.cat([contexts, tokens], 1)                           # [n, CONTEXT + DRAFTS]
    before = run[:, CONTEXT - 1:]                                    # the token before each drafted position
    logits = target[before]                                          # [n, DRAFTS + 1, VOCAB]
    got = ops.verify_draft(torch.softmax(logits, -1), q, tokens, torch.rand(n, DRAFTS, generator=gen, device="cuda"),
                           torch.rand(n, generator=gen, device="cuda"))
    top, at = logits[:, :DRAFTS].topk(TOP, dim=-1)
    windows = run.unfold(1, CONTEXT, 1)[:, :DRAFTS]                  # the context of each drafted position
    rows = torch.cat([windows.float(), at.float(), top], -1).reshape(n * DRAFTS, -1).contiguous()
    k = rows.shape[0]
    zero = torch.zeros(k, device="cuda")
    buffer.add(rows, rows, tokens.reshape(-1).int(), zero, zero.to(torch.uint8), (1.0 - got["accept_p"]).reshape(-1))
    # the next context: what was emitted, up to and with the token drawn after the last accepted one
    ended = torch.cat([contexts, got["tokens"].clamp_min(0).long()], 1)
    end = CONTEXT + got["accepted"].long() + 1
    cols = end[:, None] - CONTEXT + torch.arange(CONTEXT, device="cuda")
    return ended.gather(1, cols), got["accepted"].float().mean() / DRAFTS


def learn(drafter, buffer, optimizer, beta):
    """One weighted step; the row losses become the rows' priorities."""
    batch = buffer.sample(BATCH, beta)
    rows = batch["states"]
    contexts = rows[:, :CONTEXT].long()
    at = rows[:, CONTEXT:CONTEXT + TOP].int()
    top = rows[:, CONTEXT + TOP:CONTEXT + 2 * TOP]                   # a strided view of the gathered rows
    logits = drafter.logits(contexts)
    got = ops.distill_step(logits.detach(), top, at, batch["w"] / BATCH)
    optimizer.zero_grad(set_to_none=True)
    logits.backward(got["grad"])
    optimizer.step()
    buffer.update_priorities(batch["idx"], got["loss"])
    return got["loss"].mean()


def main(rounds=150, seed=0, say=print):
    """Returns the accepted share over the first and over the last tenth of the rounds."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    target = 2.5 * torch.randn(VOCAB, VOCAB, generator=gen, device="cuda")
    drafter = Drafter(gen)
    optimizer = torch.optim.Adam(drafter.params, lr=4e-3)
    buffer = capi.ReplayBuffer(1 << 15, CONTEXT + 2 * TOP, alpha=0.6, eps=1e-3, seed=seed)
    contexts = torch.randint(0, VOCAB, (ACTORS, CONTEXT), generator=gen, device="cuda")
    accepted, losses = [], []
    for r in range(rounds):
        contexts, share = rollout(drafter, target, contexts, buffer, gen)
        accepted.append(share)
        for _ in range(4):
            losses.append(learn(drafter, buffer, optimizer, beta=0.5))
        if say and (r + 1) % max(rounds // 5, 1) == 0:
            say(f"round {r + 1}: accepted {torch.stack(accepted[-10:]).mean().item():.3f}, "
                f"loss {torch.stack(losses[-40:]).mean().item():.3f}")
    tenth = max(rounds // 10, 1)
    shares = torch.stack(accepted).cpu()
    flags = buffer.status_device()
    buffer.close()
    if flags:
        raise RuntimeError(f"device flags {flags}")
    return shares[:tenth].mean().item(), shares[-tenth:].mean().item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rounds", type=int, default=150)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    first, last = main(args.rounds, args.seed)
    print(f"accepted share: first rounds {first:.3f}, last rounds {last:.3f}")
