"""The extension module that looks the adapter and loss calls' tensors over,
without a GPU: built once whatever the number of threads that come first."""
import os
import threading

import pytest

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
