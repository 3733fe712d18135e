"""Fine-tunes low-rank adapters of a vocabulary projection and serves them together.

    python examples/adapters.py [--steps 80] [--vocab 4096] [--width 512]

Two adapters sit beside one frozen projection W (width x vocab).  Adapter 0
learns from a teacher's top logits (distillation), adapter 1 from rewards (the
clipped policy loss with a KL term against the frozen projection); both train
in the same batch, rows of either mixed, through lora_forward, the two losses
and lora_backward.  At the end a batch of single tokens of requests with
adapter 0, adapter 1 and none goes through one call, as a server would decode.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_gemm_06_gb300 as lib  # noqa: E402


def main(steps=80, vocab=4096, width=512, rank=16, rows=256, lr=1.0, quiet=False):
    """Returns (mean distillation loss at the start and the end, mean reward at the start and the end, served logits)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    bf16 = torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(bf16)

    W = normal(width, vocab, std=3.0 * width ** -0.5)                   # the frozen projection
    teacher_W = W.float() + torch.randn(width, 8, device="cuda", generator=g) @ torch.randn(8, vocab, device="cuda", generator=g) / width ** 0.5
    good = torch.randperm(vocab, device="cuda", generator=g)[: vocab // 8]  # what a reward is given for
    rewarded = torch.zeros(vocab, device="cuda")
    rewarded[good] = 1.0
    # FP32 copies of the adapters take the steps, bfloat16 ones the products
    A32 = torch.randn(2, rank, width, device="cuda", generator=g) * width ** -0.5
    B32 = torch.zeros(2, rank, vocab, device="cuda")
    scale = torch.full((2,), 2.0, device="cuda")
    ids = torch.arange(rows, device="cuda", dtype=torch.int32) % 2      # row t has adapter t % 2
    distil, policy = ids == 0, ids == 1
    weight_d, weight_p = distil.float() / distil.sum(), policy.float() / policy.sum()
    Y, dY = torch.empty(rows, vocab, device="cuda", dtype=bf16), torch.empty(rows, vocab, device="cuda", dtype=bf16)
    dY2 = torch.empty_like(dY)
    H = torch.empty(rows, rank, device="cuda")
    loss_d, loss_p, none = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.zeros(rows, device="cuda")
    old, ref = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dA, dB = torch.empty(2, rank, width, device="cuda", dtype=bf16), torch.empty(2, rank, vocab, device="cuda", dtype=bf16)
    base = torch.full((rows,), -1, device="cuda", dtype=torch.int32)    # no adapter: the frozen projection
    distils, rewards = [], []
    for step in range(steps):
        X = normal(rows, width)
        A, B = A32.to(bf16), B32.to(bf16)
        lib.lora_forward(X, W, A, B, ids, Y, scale, H=H)
        # the teacher's top logits, and a token for each row with its log-probability before the step and under the frozen W
        top = (X.float() @ teacher_W).topk(32, 1)
        labels = (Y.float() - torch.rand(rows, vocab, device="cuda", generator=g).clamp(1e-9, 1 - 1e-7).log().neg().log()).argmax(1).int()
        lib.policy_loss(Y, labels, none, none, loss_p, logp=old)
        lib.lora_forward(X, W, A, B, base, dY, scale)
        lib.policy_loss(dY, labels, none, none, loss_p, logp=ref)
        reward = rewarded[labels.long()]
        advantage = (reward - reward[policy].mean()) / (reward[policy].std() + 1e-6)
        # the losses with their gradients; rows of weight 0 get zeros
        lib.distill_topk(Y, top.values, top.indices.int(), loss_d, dY, weight=weight_d)
        lib.policy_loss(Y, labels, old, advantage, loss_p, dY2, ref=ref, weight=weight_p, kl_coef=0.02)
        dY.add_(dY2)
        lib.lora_backward(dY, X, W, A, B, ids, H, None, dA, dB, scale)
        A32.sub_(dA.float(), alpha=lr)
        B32.sub_(dB.float(), alpha=lr)
        distils.append(float(loss_d.sum()))
        rewards.append(float(reward[policy].mean()))
        if not quiet and step % 10 == 0:
            print(f"step {step:3d}  distillation {distils[-1]:.4f}  reward {rewards[-1]:.3f}")
    # a decoding step of six requests, one token each
    tokens = normal(6, width)
    served = torch.empty(6, vocab, device="cuda", dtype=bf16)
    lib.lora_forward(tokens, W, A32.to(bf16), B32.to(bf16), torch.tensor([0, 1, -1, 1, 0, -1], dtype=torch.int32, device="cuda"), served, scale)
    n = max(1, steps // 6)
    return (sum(distils[:n]) / n, sum(distils[-n:]) / n), (sum(rewards[:n]) / n, sum(rewards[-n:]) / n), (tokens, W, A32, B32, scale, served)


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("steps", 80), ("vocab", 4096), ("width", 512)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    d, r, _ = main(a.steps, a.vocab, a.width)
    print(f"distillation loss {d[0]:.4f} -> {d[1]:.4f}, reward {r[0]:.3f} -> {r[1]:.3f}")
