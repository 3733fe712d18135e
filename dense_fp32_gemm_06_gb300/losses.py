"""Losses over rows of logits, each with its gradient by the logits in the
same call (argument marshalling only; include/adapters_gb300.h states the
operations, which rows count and the errors).

Logits are T x V, float32, bfloat16 or float16, with any row pitch; grad has
their type and receives the gradient of the rows' sum of losses.  It may be
the logits tensor itself, or None.  Means and masks go into ``weight``.
"""
from __future__ import annotations

from .adapters import run


def distill_topk(logits, teacher, index, loss, grad=None, *, weight=None, temperature=1.0, stream=None):
    """loss[t] = weight[t] tau^2 KL(q_t || softmax(logits[t] / tau)), q_t the
    softmax of the teacher's top logits ``teacher[t]`` (T x top, float32)
    over tau at the places ``index[t]`` (int32).  Places outside 0 .. V-1 and
    teacher logits of -inf are left out.  Returns loss."""
    run("distill_topk", logits, stream, logits, teacher, index, loss, grad, weight, temperature)
    return loss


def policy_loss(logits, labels, old_logp, advantage, loss, grad=None, *, ref=None, weight=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, logp=None, stream=None):
    """loss[t] = weight[t] (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
    + kl_coef (exp(ref - lp) - (ref - lp) - 1)) with lp the log-probability
    of labels[t] (int32), r = exp(lp - old_logp[t]) and A = advantage[t].
    ``logp`` receives lp.  A label outside 0 .. V-1 masks its row.  Returns
    loss."""
    run("policy_loss", logits, stream, logits, labels, old_logp, advantage, loss, grad, ref, weight, clip_low,
        clip_high, kl_coef, logp)
    return loss
