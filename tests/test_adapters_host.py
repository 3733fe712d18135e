"""The adapter and loss operators without a GPU: the header's functions are
the exported ones, every invalid argument is refused by its position before
any CUDA call, the binding refuses what is not a CUDA tensor, and the 64-bit
forms that the GPU tests compare with have the gradients that differences of
their values show."""
import ctypes
import os
import re

import pytest
import torch

import adapter_oracle as ao
import dense_fp32_gemm_06_gb300 as lib
from dense_fp32_gemm_06_gb300 import _native

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_and_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "adapters_gb300.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|const\s+char\s*\*)\s*(\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(_native.ADAPTER_EXPORTS)
    for checked in (False, True):
        so = _native.load(checked=checked)
        for name in names:
            assert hasattr(so, name), name


def test_status_strings():
    so = _native.load()
    for st in range(1, 23):
        assert so.adapters_status_string(st).decode().startswith(f"invalid argument {st}")
    assert b"unknown" not in so.adapters_status_string(100)
    assert so.adapters_status_string(12345) == b"unknown status"


P = 4096   # a pointer that is aligned and never read: every call below ends before any CUDA call
FORWARD = dict(t=4, k=6, n=5, l=2, r=3, dtype=0, X=P, ldx=6, op_w=0, W=P, ldw=5, A=P, B=P, ids=P, scale=P, Y=P, ldy=5, H=P, stream=0)
BACKWARD = dict(t=4, k=6, n=5, l=2, r=3, dtype=0, dY=P, lddy=5, X=P, ldx=6, op_w=0, W=P, ldw=5, A=P, B=P, ids=P, scale=P, H=P,
                dX=P, lddx=6, dA=P, dB=P, stream=0)
DISTILL = dict(t=4, v=9, top=3, dtype=0, logits=P, ldz=9, teacher=P, index=P, weight=P, temperature=2.0, loss=P, grad=P, ldg=9, stream=0)
POLICY = dict(t=4, v=9, dtype=0, logits=P, ldz=9, labels=P, old=P, adv=P, ref=P, weight=P, lo=0.2, hi=0.2, kl=0.1, loss=P, logp=P,
              grad=P, ldg=9, stream=0)


def call(name, base, over):
    return getattr(_native.load(), name)(*{**base, **over}.values())


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(k=-1), 2), (dict(n=-1), 3), (dict(l=-1), 4), (dict(r=-1), 5), (dict(r=257), 5), (dict(dtype=2), 6), (dict(dtype=-1), 6),
    (dict(X=0), 7), (dict(X=P + 2), 7), (dict(ldx=5), 8), (dict(op_w=2), 9), (dict(W=0), 10), (dict(W=P + 1), 10), (dict(ldw=4), 11),
    (dict(op_w=1, ldw=5), 11), (dict(A=0), 12), (dict(B=0), 13), (dict(B=P + 2), 13), (dict(ids=0), 14), (dict(ids=P + 2), 14),
    (dict(scale=P + 1), 15), (dict(Y=0), 16), (dict(ldy=4), 17), (dict(H=P + 2), 18), (dict(dtype=1, X=P + 1), 7),
])
def test_forward_refusals(over, status):
    assert call("lora_forward", FORWARD, over) == status


@pytest.mark.parametrize("over", [dict(t=0), dict(t=0, X=0, W=0, Y=0, ids=0), dict(n=0, H=0, Y=0, W=0, B=0)])
def test_forward_of_nothing(over):
    assert call("lora_forward", FORWARD, over) == 0


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(k=-1), 2), (dict(n=-1), 3), (dict(l=-1), 4), (dict(r=300), 5), (dict(dtype=7), 6), (dict(dY=0), 7), (dict(lddy=4), 8),
    (dict(X=0), 9), (dict(ldx=5), 10), (dict(op_w=-1), 11), (dict(W=0), 12), (dict(ldw=4), 13), (dict(A=0), 14), (dict(B=0), 15),
    (dict(ids=0), 16), (dict(scale=P + 2), 17), (dict(H=0), 18), (dict(dX=P + 2), 19), (dict(lddx=5), 20), (dict(dA=P + 2), 21), (dict(dB=P + 1), 22),
])
def test_backward_refusals(over, status):
    assert call("lora_backward", BACKWARD, over) == status


def test_backward_of_nothing():
    assert call("lora_backward", BACKWARD, dict(dX=0, dA=0, dB=0)) == 0
    assert call("lora_backward", BACKWARD, dict(t=0, dA=0, dB=0)) == 0


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(v=-1), 2), (dict(top=0), 3), (dict(top=1025), 3), (dict(dtype=3), 4), (dict(logits=0), 5), (dict(ldz=8), 6),
    (dict(teacher=0), 7), (dict(index=0), 8), (dict(index=P + 2), 8), (dict(weight=P + 2), 9), (dict(temperature=0.0), 10),
    (dict(temperature=-1.0), 10), (dict(temperature=float("nan")), 10), (dict(temperature=float("inf")), 10), (dict(loss=0), 11),
    (dict(grad=P + 2), 12), (dict(ldg=8), 13),
])
def test_distill_refusals(over, status):
    assert call("distill_topk", DISTILL, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(v=-1), 2), (dict(dtype=3), 3), (dict(logits=0), 4), (dict(ldz=8), 5), (dict(labels=0), 6), (dict(old=0), 7),
    (dict(adv=0), 8), (dict(ref=0), 9), (dict(weight=P + 2), 10), (dict(lo=-0.1), 11), (dict(hi=float("nan")), 12),
    (dict(kl=float("inf")), 13), (dict(loss=0), 14), (dict(logp=P + 2), 15), (dict(grad=P + 2), 16), (dict(ldg=8), 17),
])
def test_policy_refusals(over, status):
    assert call("policy_loss", POLICY, over) == status


def test_losses_of_no_rows():
    assert call("distill_topk", DISTILL, dict(t=0, logits=0, loss=0)) == 0
    assert call("policy_loss", POLICY, dict(t=0, logits=0, loss=0)) == 0


def test_binding_refuses_host_tensors():
    f = torch.zeros
    with pytest.raises(lib.SgemmError) as err:
        lib.lora_forward(f(4, 6), f(6, 5), f(2, 3, 6), f(2, 3, 5), f(4).int(), f(4, 5))
    assert err.value.status == -1 and "CUDA" in str(err.value)
    with pytest.raises(lib.SgemmError) as err:
        lib.lora_forward(f(4, 6), f(7, 5), f(2, 3, 6), f(2, 3, 5), f(4).int(), f(4, 5))
    assert "shape mismatch" in str(err.value)
    with pytest.raises(lib.SgemmError):
        lib.lora_forward(f(4, 6).half(), f(6, 5).half(), f(2, 3, 6), f(2, 3, 5), f(4).int(), f(4, 5))
    with pytest.raises(lib.SgemmError):
        lib.distill_topk(f(4, 9), f(4, 3), f(4, 3).int(), f(4))
    with pytest.raises(lib.SgemmError):
        lib.policy_loss(f(4, 9).double(), f(4).int(), f(4), f(4), f(4))


# ---------------------------------------------------------------- the 64-bit forms

def _g(seed):
    return torch.Generator().manual_seed(seed)


def test_lora_gradients_are_those_of_the_differences():
    g = _g(1)
    T, K, N, L, R = 5, 4, 3, 3, 2
    d = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    X, W, A, B, dY = d(T, K), d(K, N), d(L, R, K), d(L, R, N), d(T, N)
    ids, s = torch.tensor([0, 2, -1, 0, 2]), torch.tensor([0.5, 1.0, 2.0])
    Y, _, H, _ = ao.lora_forward(X, W, A, B, ids, s)
    grads = ao.lora_backward(dY, X, W, A, B, ids, H, s)
    for name, v in (("dX", X), ("dA", A), ("dB", B)):
        num = torch.zeros_like(v)
        for i in range(v.numel()):
            keep = float(v.reshape(-1)[i])
            side = []
            for e in (1e-6, -1e-6):
                v.reshape(-1)[i] = keep + e
                side.append(float((ao.lora_forward(X, W, A, B, ids, s)[0] * dY).sum()))
            v.reshape(-1)[i] = keep
            num.reshape(-1)[i] = (side[0] - side[1]) / 2e-6
        assert torch.allclose(grads[name][0], num, atol=1e-7), name


def test_loss_gradients_are_those_of_the_differences():
    g = _g(2)
    T, V, top = 6, 7, 3
    z = torch.randn(T, V, generator=g, dtype=torch.float64)
    z[1, 3] = -float("inf")
    t = torch.randn(T, top, generator=g)
    index = torch.tensor([[0, 1, 2], [4, 4, 6], [-1, 2, 3], [9, -1, 100], [5, 6, 0], [3, 2, 1]])
    w = torch.tensor([1.0, 0.5, 2.0, 1.0, 0.0, 1.0])
    y = torch.tensor([0, 2, 6, -1, 3, 7])
    old, adv, ref = torch.randn(T, generator=g) - 2, torch.randn(T, generator=g), torch.randn(T, generator=g) - 2
    forms = {"distill": lambda: (ao.distill(z, t, index, w, 1.5, torch.float32)[i] for i in (0, 2)),
             "policy": lambda: (ao.policy(z, y, old, adv, ref, w, 0.2, 0.3, 0.1, torch.float32)[i] for i in (0, 4))}
    for name, form in forms.items():
        loss, grad = form()
        num = torch.zeros_like(z)
        for i in range(z.numel()):
            keep = float(z.reshape(-1)[i])
            if keep == -float("inf"):
                continue
            side = []
            for e in (1e-6, -1e-6):
                z.reshape(-1)[i] = keep + e
                side.append(float(list(form())[0].sum()))
            z.reshape(-1)[i] = keep
            num.reshape(-1)[i] = (side[0] - side[1]) / 2e-6
        assert torch.allclose(grad, num, atol=1e-7), name
        assert loss[3] == 0 and not grad[3].any()
    assert list(forms["distill"]())[0][4] == 0
