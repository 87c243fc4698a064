"""Second derivatives through the library's backward passes are refused, not
left out; first-order gradients under create_graph=True are those without it."""
import pytest
import torch

from vocab_wide_logprob_gb300.autograd import grpo_embed, grpo_lmhead_loss, grpo_loss

pytestmark = pytest.mark.gpu


def inputs():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    N, P, C, V, d = 4, 3, 5, 1024, 128
    dev = dict(device="cuda", generator=gen)
    return dict(
        P=P, ids=torch.randint(0, V, (N, P + C), **dev),
        lens=torch.tensor([5, 2, 3, 1], dtype=torch.int32, device="cuda"),
        adv=torch.randn(N, **dev), logits=torch.randn(N, P + C, V, **dev),
        hidden=torch.randn(N, P + C, d, **dev).bfloat16(),
        weight=(torch.randn(V, d, **dev) * 0.1).bfloat16())


def losses():
    c = inputs()
    logits = c["logits"].requires_grad_()
    hidden, weight = c["hidden"].requires_grad_(), c["weight"].requires_grad_()
    table = torch.randn(1024, 64, device="cuda").requires_grad_()
    return {
        "loss": (lambda: grpo_loss(logits, c["P"], c["ids"], c["lens"], c["adv"]), [logits]),
        "lmhead": (lambda: grpo_lmhead_loss(hidden, weight, c["P"], c["ids"], c["lens"], c["adv"]),
                   [hidden, weight]),
        "embed": (lambda: grpo_embed(c["ids"], table).square().sum(), [table]),
    }


@pytest.mark.parametrize("name", ["loss", "lmhead", "embed"])
def test_second_derivatives_raise(name):
    f, leaves = losses()[name]
    want = torch.autograd.grad(f(), leaves)
    grads = torch.autograd.grad(f(), leaves, create_graph=True)
    for a, b in zip(grads, want):
        assert torch.equal(a.detach(), b) and a.dtype == b.dtype
    for k, leaf in enumerate(leaves):
        # beside another term, where a gradient without a graph would count as 0
        both = grads[k].float().sum() + leaf.float().pow(3).sum()
        with pytest.raises(RuntimeError, match="first-order"):
            torch.autograd.grad(both, leaf, retain_graph=True)


def test_a_gradient_that_depends_on_nothing_else():
    """The lookup is linear: with a constant upstream gradient its weight's is a
    constant too, and adds no second derivative."""
    table = torch.randn(50, 8, device="cuda").requires_grad_()
    ids = torch.tensor([1, 4, 4], device="cuda")
    up = torch.randn(3, 8, device="cuda")
    (dw,) = torch.autograd.grad(grpo_embed(ids, table), table, up, create_graph=True)
    (d2,) = torch.autograd.grad((dw * table).sum(), table)
    assert torch.equal(d2, dw.detach())
    # and one that is itself asked for a derivative
    up.requires_grad_()
    (dw,) = torch.autograd.grad(grpo_embed(ids, table), table, up, create_graph=True)
    with pytest.raises(RuntimeError, match="first-order"):
        torch.autograd.grad(dw.sum(), up)
