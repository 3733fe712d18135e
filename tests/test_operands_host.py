"""The extension module that looks the adapter and loss calls' tensors over,
without a GPU: built once whatever the number of threads that come first, not
needed by the GEMM, and required operands that are missing are refused."""
import os
import threading

import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
from dense_fp32_gemm_06_gb300 import _native, adapters


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The module's place moved to an empty folder, nothing loaded."""
    monkeypatch.setattr(_native, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(_native, "_operands", None, raising=False)
    monkeypatch.setattr(adapters, "_operands", None)
    return tmp_path


def test_threads_that_come_first_together_build_once(elsewhere, monkeypatch):
    runs, real = [], _native.subprocess.run
    started = threading.Barrier(8)

    def counted(cmd, **kw):
        runs.append(cmd)
        return real(cmd, **kw)

    monkeypatch.setattr(_native.subprocess, "run", counted)
    errors, modules = [], []

    def first_call():
        started.wait()
        try:
            modules.append(adapters._load_operands())
        except BaseException as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=first_call) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and len(runs) == 1, (errors, len(runs))
    assert all(m is modules[0] for m in modules)
    assert [f for f in os.listdir(elsewhere) if ".tmp" in f] == []


def test_the_gemm_builds_without_pythons_headers(elsewhere, monkeypatch, capsys):
    monkeypatch.setattr(_native.sysconfig, "get_paths", lambda: {"include": str(elsewhere / "none")})
    monkeypatch.setattr(_native, "_stale", lambda target: False)   # the library itself is there
    assert _native.build_all() == [_native.lib_path(False), _native.lib_path(True)]
    assert "Python.h" in capsys.readouterr().out
    f = torch.zeros
    with pytest.raises(lib.SgemmError) as err:                     # the calls that need the module say so
        lib.policy_loss(f(4, 9), f(4).int(), f(4), f(4), f(4))
    assert "Python.h" in str(err.value)


def test_missing_operands_are_refused():
    f, i = torch.zeros, torch.zeros(4).int()
    calls = [lambda: lib.lora_forward(f(4, 6), f(6, 5), f(2, 3, 6), f(2, 3, 5), i, None),
             lambda: lib.lora_forward(None, f(6, 5), f(2, 3, 6), f(2, 3, 5), i, f(4, 5)),
             lambda: lib.lora_forward(f(4, 6), None, f(2, 3, 6), f(2, 3, 5), i, f(4, 5)),
             lambda: lib.lora_forward(f(4, 6), f(6, 5), None, f(2, 3, 5), i, f(4, 5)),
             lambda: lib.lora_backward(None, f(4, 6), f(6, 5), f(2, 3, 6), f(2, 3, 5), i, f(4, 3)),
             lambda: lib.lora_backward(f(4, 5), None, None, None, None, i, f(4, 3)),
             lambda: lib.distill_topk(None, f(4, 3), f(4, 3).int(), f(4)),
             lambda: lib.distill_topk(f(4, 9), None, f(4, 3).int(), f(4)),
             lambda: lib.policy_loss(None, i, f(4), f(4), f(4))]
    for n, call in enumerate(calls):
        with pytest.raises(lib.SgemmError) as err:
            call()
        assert err.value.status == -1, n
