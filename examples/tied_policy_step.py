"""One policy update after another on a toy policy, through every call of the
library that a step with tied weights needs:

    rollout     grpo_verify_drafts: a stale copy of the policy drafts tokens,
                the policy verifies them; gives the completions and the
                log-probs of their tokens (old_logp)
    loss        grpo_mask, grpo_advantage, grpo_embed_fwd (hidden states),
                grpo_lmhead_loss_fwd / _bwd (loss and gradients through the
                LM head, here the embedding's own matrix)
    gradient    grpo_embed_bwd with accumulate: the embedding's gradient is
                added to the LM head's
    update      grpo_clip_grad_norm, then a plain gradient step

The policy is a bigram model: the next token's logits are SCALE * (w_x . w_y).
The reward of a completion is the share of its tokens below V / 4; the mean
reward rises from about 0.25 to 0.85 and more.

    python examples/tied_policy_step.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocab_wide_logprob_gb300 as grpo  # noqa: E402

V, D = 512, 128          # vocabulary, hidden size (the LM head wants a multiple of 128)
B, G, P, C = 8, 8, 4, 48  # prompts, completions per prompt, prompt and completion tokens
K = 4                    # tokens drafted at a time
EOS = V - 1
SCALE = 2.0
MAX_NORM, RATE = 0.0025, 2000.0


def logits_after(weight, tokens):
    """Next-token logits [..., V] of the policy with matrix ``weight``."""
    hidden = grpo.grpo_embed_fwd(tokens, weight, SCALE)
    return hidden.float() @ weight.float().t()


def exponential(shape, gen):
    return torch.empty(shape, device="cuda").exponential_(generator=gen).clamp_(min=1e-20)


def rollout(weight, draft_weight, prompts, gen):
    """C tokens for every row of ``prompts`` [N, P]: drafted by ``draft_weight``,
    verified against ``weight``.  Returns ``(ids [N, P+C], old_logp [N, C],
    accepted share)``."""
    N = prompts.shape[0]
    ids = torch.full((N, P + C), EOS, device="cuda")
    ids[:, :P] = prompts
    old = torch.zeros(N, C, device="cuda")
    have = torch.zeros(N, dtype=torch.int64, device="cuda")  # completion tokens so far
    last = prompts[:, -1].contiguous()
    drafted = accepted = 0
    slot = torch.arange(K + 1, device="cuda")
    while int(have.min()) < C:
        # draft K tokens one after the other, keeping the draft's logits
        x, y, cur = [], [], last
        for _ in range(K):
            y.append(logits_after(draft_weight, cur))
            cur = (torch.log_softmax(y[-1], -1) - exponential((N, V), gen).log()).argmax(-1)
            x.append(cur)
        x, y = torch.stack(x, 1), torch.stack(y, 1)
        z = logits_after(weight, torch.cat([last[:, None], x], 1).contiguous())
        out = grpo.grpo_verify_drafts(z, x, torch.rand(N, K, device="cuda", generator=gen),
                                      exponential((N, V), gen), y)
        # append the accepted tokens and the emitted one
        n = out["n_accepted"].long()
        at = have[:, None] + slot
        keep = (slot <= n[:, None]) & (at < C)
        row = torch.arange(N, device="cuda")[:, None].expand_as(at)
        ids[row[keep], P + at[keep]] = out["tokens"][keep]
        old[row[keep], at[keep]] = out["logp"][keep]
        last = out["tokens"].gather(1, n[:, None]).squeeze(1)
        have += n + 1
        drafted += K * N
        accepted += int(n.sum())
    return ids, old, accepted / drafted


def gradients(weight, ids, old, lens, adv):
    """Loss and its gradient with respect to the tied matrix, float32 [V, D]."""
    hidden = grpo.grpo_embed_fwd(ids, weight, SCALE)
    f = grpo.grpo_lmhead_loss_fwd(hidden, weight, P, ids, lens, adv, old)
    dhidden, dweight, _ = grpo.grpo_lmhead_loss_bwd(hidden, weight, P, ids, lens, f["lse"], f["w"])
    # (positions after the last scored one have no gradient: nothing is padded out)
    grpo.grpo_embed_bwd(ids, dhidden, V, SCALE, dweight=dweight, accumulate=True)
    return f["loss"], dweight


def main(steps=30, seed=0, report=print):
    """Runs ``steps`` updates; returns the mean rewards, step by step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    master = torch.randn(V, D, device="cuda", generator=gen) / D ** 0.5
    stale = master.bfloat16()
    rewards = []
    for step in range(steps):
        weight = master.bfloat16()
        prompts = torch.randint(0, V - 1, (B, P), device="cuda", generator=gen)
        ids, old, share = rollout(weight, stale, prompts.repeat_interleave(G, 0), gen)
        _, lens = grpo.grpo_mask(ids, P, C, EOS)
        inside = torch.arange(C, device="cuda") < lens[:, None]
        reward = ((ids[:, P:] < V // 4) & inside).float().sum(1) / lens
        adv = grpo.grpo_advantage(reward, G)
        loss, grad = gradients(weight, ids, old, lens, adv)
        stats, _ = grpo.grpo_clip_grad_norm([grad], MAX_NORM)
        master.sub_(grad, alpha=RATE)
        stale = weight  # the next step's draft: one update behind
        rewards.append(float(reward.mean()))
        report(f"step {step:3d}  reward {rewards[-1]:.3f}  loss {float(loss):+.4f}  "
               f"gradient norm {float(stats[0]):.4f}  drafts accepted {share:.2f}")
    return rewards


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
