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
from .adapters import BF16, F16, F32, matrix, need, on_device, vector

DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _rows(logits, loss, grad):
    need(logits.dim() == 2 and logits.dtype in DTYPES, "logits must be 2-D float32, bfloat16 or float16")
    device, dtype = logits.device, logits.dtype
    T, V = logits.shape
    ldz = matrix(logits, "logits", dtype, T, V, device)
    ldg = matrix(grad, "grad", dtype, T, V, device) if grad is not None else max(V, 1)
    need(loss is not None, "loss must be a float32 CUDA tensor of one value per row")
    return device, DTYPES[dtype], T, V, ldz, ldg, vector(loss, "loss", torch.float32, (T,), device)


def distill_topk(logits, teacher, index, loss, grad=None, *, weight=None, temperature=1.0, stream=None):
    """loss[t] = weight[t] tau^2 KL(q_t || softmax(logits[t] / tau)), q_t the
    softmax of the teacher's top logits ``teacher[t]`` (T x top, float32)
    over tau at the places ``index[t]`` (int32).  Places outside 0 .. V-1 and
    teacher logits of -inf are left out.  Returns loss."""
    device, dtype, T, V, ldz, ldg, lp = _rows(logits, loss, grad)
    need(teacher is not None and index is not None and teacher.dim() == 2, "teacher and index must be T x top")
    top = teacher.shape[1]
    tp, ip = vector(teacher, "teacher", torch.float32, (T, top), device), vector(index, "index", torch.int32, (T, top), device)
    wp = vector(weight, "weight", torch.float32, (T,), device)
    lib = _native.load()
    on_device(device, lambda st: lib.distill_topk(T, V, top, dtype, logits.data_ptr(), ldz, tp, ip, wp, float(temperature),
                                                  lp, grad.data_ptr() if grad is not None else 0, ldg, st), stream)
    return loss


def policy_loss(logits, labels, old_logp, advantage, loss, grad=None, *, ref=None, weight=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, logp=None, stream=None):
    """loss[t] = weight[t] (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
    + kl_coef (exp(ref - lp) - (ref - lp) - 1)) with lp the log-probability
    of labels[t] (int32), r = exp(lp - old_logp[t]) and A = advantage[t].
    ``logp`` receives lp.  A label outside 0 .. V-1 masks its row.  Returns
    loss."""
    device, dtype, T, V, ldz, ldg, lp = _rows(logits, loss, grad)
    need(labels is not None and old_logp is not None and advantage is not None, "labels, old_logp and advantage are needed")
    need(ref is not None or kl_coef == 0.0, "kl_coef needs ref")
    f32 = torch.float32
    yp = vector(labels, "labels", torch.int32, (T,), device)
    op, ap = vector(old_logp, "old_logp", f32, (T,), device), vector(advantage, "advantage", f32, (T,), device)
    rp, wp, gp = vector(ref, "ref", f32, (T,), device), vector(weight, "weight", f32, (T,), device), vector(logp, "logp", f32, (T,), device)
    lib = _native.load()
    on_device(device, lambda st: lib.policy_loss(T, V, dtype, logits.data_ptr(), ldz, yp, op, ap, rp, wp, float(clip_low),
                                                 float(clip_high), float(kl_coef), lp, gp,
                                                 grad.data_ptr() if grad is not None else 0, ldg, st), stream)
    return loss
