"""The device's one-time set-up of the microscaled operators, each in a process
of its own: a first call inside a capture is refused, and the calls after it
work; first calls from several threads at once all have their results."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

START = """
import threading, torch
import dense_fp32_gemm_06_gb300 as lib
from dense_fp32_gemm_06_gb300 import microscale
T, K, N = 40, 64, 33
x, dy = torch.ones(T, K, device="cuda"), torch.ones(T, N, device="cuda")
c = torch.full((N, 32), 0x22, device="cuda", dtype=torch.uint8)              # ones
s = torch.full((N, 16), 127, device="cuda", dtype=torch.uint8)[:, :2]
y, dx = torch.zeros(T, N, device="cuda"), torch.zeros(T, K, device="cuda")
q = lib.mx_empty(T, K, 8)
calls = {"linear": lambda: lib.mx4_linear(x, c, s, y), "grad_input": lambda: lib.mx_grad_input(dy, c, s, dx), "quantize": lambda: lib.mx_quantize(x, *q)}
def right(name):
    torch.cuda.synchronize()
    assert microscale.device_status() == 0
    assert {"linear": lambda: (y == K).all(), "grad_input": lambda: (dx == N).all(), "quantize": lambda: (q[0] == 64).all() and (q[1] == 121).all()}[name]()
torch.cuda.synchronize()
"""


def child(code):
    r = subprocess.run([sys.executable, "-c", START + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.parametrize("name", ["linear", "grad_input", "quantize"])
def test_a_first_call_inside_a_capture_is_refused(name):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    child(f"""
graph, refused = torch.cuda.CUDAGraph(), False
try:
    with torch.cuda.graph(graph):
        try:
            calls["{name}"]()
        except lib.SgemmError as e:
            refused = e.status == 100
except RuntimeError:
    pass
assert refused
calls["{name}"]()
right("{name}")
graph = torch.cuda.CUDAGraph()
y.zero_(), dx.zero_(), q[0].zero_(), q[1].zero_()
with torch.cuda.graph(graph):
    calls["{name}"]()
graph.replay()
right("{name}")
""")


def test_first_calls_from_several_threads():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    child("""
errors, gate = [], threading.Barrier(6)
def work(name):
    try:
        gate.wait()
        calls[name]()
    except BaseException as e:
        errors.append(e)
threads = [threading.Thread(target=work, args=(n,)) for n in ("linear", "grad_input", "quantize") * 2]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
for n in calls:
    right(n)
""")
