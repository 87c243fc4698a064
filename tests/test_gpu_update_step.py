"""One policy update through the operators as they are used together: rollout rows
scored with their alternatives, a loss with an entropy bonus over the log-probs,
its gradient through the token statistics, the LM head's product and the embedding,
the gradients' norm, and the AdamW step that clips on the way.  Against
torch's autograd in float64 and the formulas of the step."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
N, P, C, V, D = 6, 3, 10, 1003, 64
BETA1, BETA2, EPS, DECAY, LR, LIMIT, BONUS = 0.9, 0.99, 1e-8, 0.05, 1e-2, 0.02, 0.01


def inputs(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    ids = torch.randint(0, V, (N, P + C), generator=r, device="cuda")
    lens = torch.tensor([10, 0, 7, 1, 10, 4], dtype=torch.int32, device="cuda")
    adv = torch.randn(N, generator=r, device="cuda")
    embed = torch.randn(V, D, generator=r, device="cuda") * 0.3
    head = torch.randn(V, D, generator=r, device="cuda") * 0.3
    return ids, lens, adv, embed, head


def loss_of(logp, entropy, lens, adv):
    keep = torch.arange(C, device="cuda") < lens[:, None]
    each = -adv[:, None].to(logp.dtype) * logp - BONUS * entropy
    return torch.where(keep, each, torch.zeros_like(each)).sum() / (N * C)


def gradients64(ids, lens, adv, embed, head):
    embed, head = embed.double().requires_grad_(), head.double().requires_grad_()
    logits = embed[ids] @ head.t()
    lp = torch.log_softmax(logits[:, P - 1:-1], -1)
    logp = lp.gather(-1, ids[:, P:, None])[..., 0]
    loss = loss_of(logp, -(lp.exp() * lp).sum(-1), lens, adv)
    return loss.detach(), torch.autograd.grad(loss, (embed, head))


@pytest.mark.parametrize("bits", [32, 8])
def test_update(bits):
    import vocab_wide_logprob_gb300 as grpo
    from vocab_wide_logprob_gb300 import autograd
    ids, lens, adv, embed, head = inputs(1)
    params = [embed, head]
    state = grpo.grpo_adamw_state(params, bits)
    was = [p.clone().double() for p in params]
    moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in was]
    for step in range(1, 4):
        # the product with the LM head is the model's own; everything around it is the library's
        embed.requires_grad_()
        head.requires_grad_()
        hidden = autograd.grpo_embed(ids, embed)
        logits = hidden @ head.t()
        logp, entropy = autograd.grpo_logp_entropy(logits[:, P - 1:-1], ids[:, P:], lens)
        loss = loss_of(logp, entropy, lens, adv)
        grads = torch.autograd.grad(loss, (embed, head))
        embed.requires_grad_(False)
        head.requires_grad_(False)
        # (float32 products over D and V terms: 1e-5 of the largest entry is far above them)
        want_loss, want = gradients64(ids, lens, adv, embed, head)
        assert abs(float(loss.detach()) - float(want_loss)) <= 1e-5 * abs(float(want_loss))
        for g, w in zip(grads, want):
            assert (g.double() - w).abs().max() <= 1e-5 * w.abs().max()
        stats, ws = grpo.grpo_grad_norm(list(grads))
        assert grpo.grpo_check_error(ws) == 0
        grpo.grpo_adamw_step(params, list(grads), state, step, LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                             weight_decay=DECAY, norm=stats, max_norm=LIMIT)
        norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        coef = min(1.0, LIMIT / (norm + 1e-6))
        for k in range(2):
            m, v = moments[k]
            g = grads[k].double() * coef
            m.mul_(BETA1).add_(g, alpha=1 - BETA1)
            v.mul_(BETA2).add_(g * g, alpha=1 - BETA2)
            up = m / (1 - BETA1 ** step) / ((v / (1 - BETA2 ** step)).sqrt() + EPS)
            was[k] = was[k] - LR * (up + DECAY * was[k])
            if bits == 32:
                # each step's update is of the size of LR, and off by some 1e-6 of itself
                assert (params[k].double() - was[k]).abs().max() <= 3 * 1e-5 * LR
            else:
                # moments of earlier steps in e4m3: half a step of 2^-4 in each of m and the root
                # of what is left of them
                assert (params[k].double() - was[k]).abs().mean() <= 0.15 * LR * step
            was[k] = params[k].double()
            if bits == 8:  # (the next step begins with what is stored)
                n = params[k].numel()
                back = lambda c, j: (torch.nn.functional.pad(c.reshape(-1).view(torch.uint8), (0, -n % 256))
                                     .view(torch.float8_e4m3fn).double().view(-1, 256)
                                     * state["scales"][k][:, j:j + 1].double()).view(-1)[:n].view_as(params[k])
                moments[k] = (back(state["exp_avg"][k], 0), back(state["exp_avg_root"][k], 1) ** 2)


def test_scoring_of_a_rollout():
    """What verification emits is what the statistics score: the same log-probs at
    the sequences' own temperatures, the emitted tokens of greedy ones the first
    alternative."""
    import vocab_wide_logprob_gb300 as grpo
    r = torch.Generator(device="cuda")
    r.manual_seed(2)
    K = 3
    z = (torch.randn(8, K + 1, V, generator=r, device="cuda") * 2).to(BF16)
    T = torch.tensor([1.0, 0.0, 0.7, 2.0, 0.0, 1.3, 0.5, 1.0], device="cuda")
    x = z[:, :K].float().argmax(-1)
    u = torch.rand(8, K, generator=r, device="cuda")
    noise = torch.empty(8, V, device="cuda").exponential_(generator=r).clamp_(min=1e-9)
    out = grpo.grpo_verify_drafts(z, x, u, noise, temperature=T)
    stats = grpo.grpo_token_stats(z, out["tokens"].clamp(min=0), out["n_accepted"] + 1, T, top=4)
    # (both within some 1e-6 of the definition at these sizes)
    assert (stats["logp"] - out["logp"]).abs().max() <= 2e-5
    last = out["n_accepted"].long()
    row = torch.arange(8, device="cuda")
    greedy = T == 0
    assert torch.equal(stats["top_tokens"][row, last, 0][greedy], out["tokens"][row, last][greedy])


def test_the_update_in_a_graph():
    """Statistics, their gradient, norm and step captured once and replayed."""
    import vocab_wide_logprob_gb300 as grpo
    r = torch.Generator(device="cuda")
    r.manual_seed(3)
    z = torch.randn(4, 5, V, generator=r, device="cuda")
    y = torch.randint(0, V, (4, 5), generator=r, device="cuda")
    g = torch.randn(4, 5, generator=r, device="cuda")

    def update(param, state, step):
        out = grpo.grpo_token_stats(param, y, top=3)
        dz = grpo.grpo_token_stats_bwd(param, y, out["norm"], out["entropy"], g, g)
        stats, _ = grpo.grpo_grad_norm([dz])
        grpo.grpo_adamw_step([param], [dz], state, step, 1e-2, norm=stats, max_norm=0.5)
        return out["logp"], out["top_tokens"]

    eager, state = z.clone(), grpo.grpo_adamw_state([z])
    for t in (1, 2, 3):
        want = update(eager, state, torch.full((1,), t, dtype=torch.int64, device="cuda"))
    param, state = z.clone(), grpo.grpo_adamw_state([z])
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        got = update(param, state, step)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(param, eager)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_each_step_with_8_bit_states():
    """Every element of every step, from the states that it found: the update takes them as the
    numbers they are and uses its own moments unrounded, so that the bound is that of states in
    float32 (off by some 1e-6 of a step's size, and by half a step of float32 at 1)."""
    import vocab_wide_logprob_gb300 as grpo
    from vocab_wide_logprob_gb300 import autograd
    ids, lens, adv, embed, head = inputs(4)
    params = [embed, head]
    state = grpo.grpo_adamw_state(params, 8)

    def value(codes, k, j):
        n = codes.numel()
        each = state["scales"][k][:, j].double().repeat_interleave(256)[:n]
        return (codes.reshape(-1).float().double() * each).view(codes.shape)

    for step in range(1, 5):
        embed.requires_grad_()
        head.requires_grad_()
        logits = autograd.grpo_embed(ids, embed) @ head.t()
        logp, entropy = autograd.grpo_logp_entropy(logits[:, P - 1:-1], ids[:, P:], lens)
        grads = list(torch.autograd.grad(loss_of(logp, entropy, lens, adv), (embed, head)))
        embed.requires_grad_(False)
        head.requires_grad_(False)
        stats, _ = grpo.grpo_grad_norm(grads)
        coef = min(1.0, LIMIT / (float(stats[0]) + 1e-6))
        want = []
        for k, p in enumerate(params):
            g = grads[k].double() * coef
            m = BETA1 * value(state["exp_avg"][k], k, 0) + (1 - BETA1) * g
            v = BETA2 * value(state["exp_avg_root"][k], k, 1) ** 2 + (1 - BETA2) * g * g
            up = m / (1 - BETA1 ** step) / ((v / (1 - BETA2 ** step)).sqrt() + EPS)
            want.append(p.double() - LR * (up + DECAY * p.double()))
        grpo.grpo_adamw_step(params, grads, state, step, LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                             weight_decay=DECAY, norm=stats, max_norm=LIMIT)
        for p, w in zip(params, want):
            assert (p.double() - w).abs().max() <= 3e-5 * LR
