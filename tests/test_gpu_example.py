"""The example step: its gradient against torch's autograd, its rollout's
log-probs against the LM head's, and its learning."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location(
        "tied_policy_step", os.path.join(ROOT, "examples", "tied_policy_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_rollout_and_gradient(ex):
    g = ex.grpo
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    weight = (torch.randn(ex.V, ex.D, device="cuda", generator=gen) / ex.D ** 0.5).bfloat16()
    stale = (weight.float() + 0.02 * torch.randn(ex.V, ex.D, device="cuda", generator=gen)).bfloat16()
    prompts = torch.randint(0, ex.V - 1, (ex.B * ex.G, ex.P), device="cuda", generator=gen)
    ids, old, share = ex.rollout(weight, stale, prompts, gen)
    assert 0.3 < share < 1.0
    _, lens = g.grpo_mask(ids, ex.P, ex.C, ex.EOS)
    inside = torch.arange(ex.C, device="cuda") < lens[:, None]
    hidden = g.grpo_embed_fwd(ids, weight, ex.SCALE)
    logp, _, _ = g.grpo_lmhead_logprobs(hidden, weight, ex.P, ids, lens)
    assert (logp - old)[inside].abs().max() < 1e-4  # the same float32 products, other sums
    adv = torch.randn(ex.B * ex.G, device="cuda", generator=gen)
    loss, grad = ex.gradients(weight, ids, old, lens, adv)
    # the same through torch in float64 (the hidden states rounded as the lookup rounds them)
    w = weight.double().requires_grad_()
    h = w[ids] * ex.SCALE
    z = torch.log_softmax(h[:, ex.P - 1:-1] @ w.t(), -1)
    lp = z.gather(-1, ids[:, ex.P:].unsqueeze(-1)).squeeze(-1)
    r = (lp - old.double()).exp()
    a = adv.double()[:, None]
    ell = -torch.minimum(r * a, r.clamp(0.8, 1.2) * a)
    want = (ell * inside).sum() / inside.numel()
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 1e-5
    # dz is rounded to bfloat16 before the contractions: 2^-8 of each term
    err = (grad.double() - w.grad).norm() / w.grad.norm()
    assert err < 2.0 ** -8


def test_rewards_rise(ex):
    rewards = ex.main(steps=25, seed=1, report=lambda _: None)
    assert sum(rewards[-5:]) / 5 > sum(rewards[:5]) / 5 + 0.1
