"""torch.autograd bindings of the loss: the forward is grpo_loss_fwd, the
backward grpo_loss_bwd (d loss / d logits, "loss.backward()" of "Making Dr
GRPO go brrr", salahadawi.com), both through the C ABI; torch only holds
the tensors.  GRPOLMHeadLoss does the same from hidden states and the LM head
(grpo_lmhead_loss_fwd / grpo_lmhead_loss_bwd).  GRPOEmbedding is the
embedding lookup (grpo_embed_fwd / grpo_embed_bwd), GRPOTokenStats the
log-probs and entropies of a caller's own loss (grpo_token_stats /
grpo_token_stats_bwd).

Of the losses, only the logits (or the hidden states and the LM head) receive a gradient.  The advantages, old and reference
log-probs are constants of the update step (the advantage comes from the
rewards, the old and reference log-probs from no-grad passes), so their
gradients are None.  The gradients are first-order: under create_graph=True they
can be used like any, but a second derivative through them raises.
"""
from __future__ import annotations

import torch

from . import _native as g


class _FirstOrder(torch.autograd.Function):
    """A gradient as it is, hung onto what it was computed from, so that a
    derivative of it is refused rather than left out."""

    @staticmethod
    def forward(ctx, grad, *of):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("this gradient has no derivative: the library's backward passes are "
                           "first-order")


def _first_order(grad, *of):
    """``grad`` of a backward pass that used the tensors ``of``.  (Gradients are
    enabled in a backward pass only under create_graph=True.)"""
    return _FirstOrder.apply(grad, *of) if torch.is_grad_enabled() else grad


class GRPOLoss(torch.autograd.Function):
    """loss = GRPOLoss.apply(logits, P, input_ids, lens, adv, old_logp,
    ref_logp, eps, beta, norm, agg): a 0-dim float32 tensor on the logits'
    device; ``loss.backward()`` writes d loss / d logits (same dtype and shape
    as the logits) scaled by the upstream gradient."""

    @staticmethod
    def forward(ctx, logits, P, input_ids, lens, adv, old_logp=None, ref_logp=None, eps=0.2,
                beta=0.0, norm=0.0, agg=None):
        out = g.grpo_loss_fwd(logits, P, input_ids, lens, adv, old_logp, ref_logp, eps, beta,
                              norm, agg=agg)
        ctx.save_for_backward(logits, input_ids, lens, out["lse"], out["w"])
        ctx.P = P
        return out["loss"].reshape(())

    @staticmethod
    def backward(ctx, grad_loss):
        logits, input_ids, lens, lse, w = ctx.saved_tensors
        gl = grad_loss.detach().reshape(1).to(torch.float32).contiguous()
        dlogits = g.grpo_loss_bwd(logits, ctx.P, input_ids, lens, lse, w, gl)
        return (_first_order(dlogits, logits, grad_loss),) + (None,) * 10


def grpo_loss(logits, P, input_ids, lens, adv, old_logp=None, ref_logp=None, eps=0.2, beta=0.0,
              norm=0.0, agg=None):
    """Functional form of :class:`GRPOLoss` (differentiable in ``logits``)."""
    return GRPOLoss.apply(logits, P, input_ids, lens, adv, old_logp, ref_logp, eps, beta, norm,
                          agg)


class GRPOEmbedding(torch.autograd.Function):
    """out = GRPOEmbedding.apply(ids, weight, scale, pad_id, out_dtype):
    grpo_embed_fwd, differentiable in ``weight`` [V, d]; the backward is
    grpo_embed_bwd (summed in float32, handed over in the weight's dtype).
    Tokens equal to ``pad_id`` give no gradient."""

    @staticmethod
    def forward(ctx, ids, weight, scale=1.0, pad_id=None, out_dtype=None):
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.V, ctx.scale, ctx.pad_id, ctx.wdtype = weight.shape[0], scale, pad_id, weight.dtype
        return g.grpo_embed_fwd(ids, weight, scale, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        # (the gradient of a broadcast or transposed use arrives with other strides)
        dw, _ = g.grpo_embed_bwd(ids, dout.contiguous(), ctx.V, ctx.scale, ctx.pad_id,
                                 out_dtype=ctx.wdtype)
        return None, _first_order(dw, dout), None, None, None


def grpo_embed(ids, weight, scale=1.0, pad_id=None, out_dtype=None):
    """Functional form of :class:`GRPOEmbedding` (differentiable in
    ``weight``)."""
    return GRPOEmbedding.apply(ids, weight, scale, pad_id, out_dtype)


class GRPOTokenStats(torch.autograd.Function):
    """logp, entropy = GRPOTokenStats.apply(logits, tokens, lens, temperature):
    grpo_token_stats of logits [N, R, V], both [N, R] float32 and differentiable
    in ``logits``; the backward is grpo_token_stats_bwd."""

    @staticmethod
    def forward(ctx, logits, tokens, lens=None, temperature=None):
        out = g.grpo_token_stats(logits, tokens, lens, temperature)
        ctx.save_for_backward(logits, tokens, out["norm"], out["entropy"], lens, temperature)
        ctx.set_materialize_grads(False)
        return out["logp"], out["entropy"]

    @staticmethod
    def backward(ctx, grad_logp, grad_entropy):
        if grad_logp is None and grad_entropy is None:
            return None, None, None, None
        logits, tokens, norm, entropy, lens, temperature = ctx.saved_tensors
        # (the gradient of a sum arrives expanded)
        gl, gh = (None if t is None else t.detach().float().contiguous()
                  for t in (grad_logp, grad_entropy))
        dz = g.grpo_token_stats_bwd(logits, tokens, norm, entropy, gl, gh, lens, temperature)
        of = [t for t in (logits, grad_logp, grad_entropy) if t is not None]
        return _first_order(dz, *of), None, None, None


def grpo_logp_entropy(logits, tokens, lens=None, temperature=None):
    """Functional form of :class:`GRPOTokenStats` (differentiable in
    ``logits``)."""
    return GRPOTokenStats.apply(logits, tokens, lens, temperature)


class GRPOLMHeadLoss(torch.autograd.Function):
    """loss = GRPOLMHeadLoss.apply(hidden, weight, P, input_ids, lens, adv,
    old_logp, ref_logp, eps, beta, norm, agg, rows_per_pass): the loss from
    hidden states [N, P+C, d] and the LM head [V, d] (both bfloat16), the
    projection fused on the tensor cores (grpo_lmhead_loss_fwd); the logits
    are never written.  ``loss.backward()`` writes d loss / d hidden and
    d loss / d weight (grpo_lmhead_loss_bwd, computed in float32 and handed
    to autograd, which stores them in the parameters' dtype), scaled by the
    upstream gradient.

    ``rows_per_pass``: rows per pass of the backward's workspace.  None (the
    default) takes the number of scored rows, read on the host from ``lens``
    (one synchronisation per backward), so that one pass covers them; 0 sizes
    it for every possible row (no synchronisation, N·C·V·2 bytes of logits
    gradient buffer)."""

    @staticmethod
    def forward(ctx, hidden, weight, P, input_ids, lens, adv, old_logp=None, ref_logp=None,
                eps=0.2, beta=0.0, norm=0.0, agg=None, rows_per_pass=None):
        out = g.grpo_lmhead_loss_fwd(hidden, weight, P, input_ids, lens, adv, old_logp, ref_logp,
                                     eps, beta, norm, agg=agg)
        ctx.save_for_backward(hidden, weight, input_ids, lens, out["lse"], out["w"])
        ctx.P = P
        ctx.rows_per_pass = rows_per_pass
        return out["loss"].reshape(())

    @staticmethod
    def backward(ctx, grad_loss):
        hidden, weight, input_ids, lens, lse, w = ctx.saved_tensors
        gl = grad_loss.detach().reshape(1).to(torch.float32).contiguous()
        rpp = ctx.rows_per_pass
        if rpp is None:
            rpp = max(1, int(lens.sum().item()))
        dh, dw, _ = g.grpo_lmhead_loss_bwd(hidden, weight, ctx.P, input_ids, lens, lse, w, gl,
                                           rows_per_pass=rpp)
        of = (hidden, weight, grad_loss)
        return (_first_order(dh, *of), _first_order(dw, *of)) + (None,) * 11


def grpo_lmhead_loss(hidden, weight, P, input_ids, lens, adv, old_logp=None, ref_logp=None,
                     eps=0.2, beta=0.0, norm=0.0, agg=None, rows_per_pass=None):
    """Functional form of :class:`GRPOLMHeadLoss` (differentiable in
    ``hidden`` and ``weight``)."""
    return GRPOLMHeadLoss.apply(hidden, weight, P, input_ids, lens, adv, old_logp, ref_logp, eps,
                                beta, norm, agg, rows_per_pass)
