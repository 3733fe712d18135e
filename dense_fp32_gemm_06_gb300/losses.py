"""Losses over rows of logits, each with its gradient by the logits in the
same call (argument marshalling only; include/adapters_gb300.h states the
operations, which rows count and the errors).

Logits are T x V, float32, bfloat16 or float16, with any row pitch; grad has
their type and receives the gradient of the rows' sum of losses.  It may be
the logits tensor itself, or None.  Means and masks go into ``weight``.
"""
from __future__ import annotations

import torch

from . import _native
from .adapters import BF16, F16, F32, launch, matrix, refuse, vector

DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _rows(logits, loss, grad):
    """(device index, dtype code, T, V, pitch of the logits, pointer and pitch of the gradient, pointer of the loss)."""
    dev, dtype = logits.get_device(), logits.dtype
    if dtype not in DTYPES or dev < 0 or logits.dim() != 2:
        refuse("logits must be a 2-D float32, bfloat16 or float16 CUDA tensor")
    if loss is None:
        refuse("loss must be a float32 CUDA tensor of one value per row")
    T, V = logits.shape
    ldz = matrix(logits, "logits", dtype, T, V, dev)
    g, ldg = (grad.data_ptr(), matrix(grad, "grad", dtype, T, V, dev)) if grad is not None else (0, V or 1)
    return dev, DTYPES[dtype], T, V, ldz, g, ldg, vector(loss, "loss", torch.float32, (T,), dev)


def distill_topk(logits, teacher, index, loss, grad=None, *, weight=None, temperature=1.0, stream=None):
    """loss[t] = weight[t] tau^2 KL(q_t || softmax(logits[t] / tau)), q_t the
    softmax of the teacher's top logits ``teacher[t]`` (T x top, float32)
    over tau at the places ``index[t]`` (int32).  Places outside 0 .. V-1 and
    teacher logits of -inf are left out.  Returns loss."""
    dev, dtype, T, V, ldz, g, ldg, lp = _rows(logits, loss, grad)
    if teacher is None or index is None or teacher.dim() != 2:
        refuse("teacher and index must be T x top")
    top = teacher.shape[1]
    launch(_native.load().distill_topk, dev, stream, T, V, top, dtype, logits.data_ptr(), ldz,
           vector(teacher, "teacher", torch.float32, (T, top), dev), vector(index, "index", torch.int32, (T, top), dev),
           vector(weight, "weight", torch.float32, (T,), dev), temperature, lp, g, ldg)
    return loss


def policy_loss(logits, labels, old_logp, advantage, loss, grad=None, *, ref=None, weight=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, logp=None, stream=None):
    """loss[t] = weight[t] (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
    + kl_coef (exp(ref - lp) - (ref - lp) - 1)) with lp the log-probability
    of labels[t] (int32), r = exp(lp - old_logp[t]) and A = advantage[t].
    ``logp`` receives lp.  A label outside 0 .. V-1 masks its row.  Returns
    loss."""
    dev, dtype, T, V, ldz, g, ldg, lp = _rows(logits, loss, grad)
    if labels is None or old_logp is None or advantage is None:
        refuse("labels, old_logp and advantage are needed")
    if ref is None and kl_coef != 0.0:
        refuse("kl_coef needs ref")
    f32, rows = torch.float32, (T,)
    launch(_native.load().policy_loss, dev, stream, T, V, dtype, logits.data_ptr(), ldz,
           vector(labels, "labels", torch.int32, rows, dev), vector(old_logp, "old_logp", f32, rows, dev),
           vector(advantage, "advantage", f32, rows, dev), vector(ref, "ref", f32, rows, dev),
           vector(weight, "weight", f32, rows, dev), clip_low, clip_high, kl_coef, lp,
           vector(logp, "logp", f32, rows, dev), g, ldg)
    return loss
