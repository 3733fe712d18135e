"""Builds and loads the C-ABI CUDA library (in-tree, sm_103a only)."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import platform
import shutil
import subprocess
import sysconfig
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
CSRC = os.path.join(_PKG, "csrc")
INCLUDE = os.path.join(_ROOT, "include")
LIB_DIR = os.path.join(_PKG, "_lib")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]
# the C ABI and planning, and the kernel units (compiled in parallel)
SOURCES = ["sgemm_api.cu", "tc_wide.cu", "tc_narrow.cu", "tc_trans.cu", "tc_pair.cu", "ffma.cu",
           "adapters_api.cu", "lora_simt.cu", "lora_tc.cu", "lora_skinny.cu", "row_loss.cu",
           "microscale_api.cu", "mx_store.cu", "mx4_tc.cu", "mx_grad.cu", "mx_grad_4.cu", "mx_grad_8.cu"]

_lock = threading.Lock()
_libs = {}
_operands = None


class SgemmError(RuntimeError):
    """A non-zero status from the C ABI, or a missing library."""

    def __init__(self, status: int, message: str):
        super().__init__(f"sgemm status {status}: {message}")
        self.status = status


def lib_path(checked: bool = False) -> str:
    """The release library, or (checked=True) the one compiled with
    SGEMM_GB300_CHECKED: every kernel index tested before its access."""
    kind = "checked_" if checked else ""
    return os.path.join(LIB_DIR, f"libsgemm_gb300_{kind}{platform.machine()}.so")


def _deps():
    out = [os.path.join(INCLUDE, "sgemm_gb300.h"), os.path.join(INCLUDE, "adapters_gb300.h"), os.path.join(INCLUDE, "microscale_gb300.h")]
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, name))
    return out


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in _deps())


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise SgemmError(-1, "nvcc not found: cannot build the CUDA library")


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Compiles csrc/*.cu into one shared library for sm_103a; returns its
    path (the checked variant with checked=True)."""
    return build_all(force=force, verbose=verbose, variants=(checked,))[0]


def build_all(force: bool = False, verbose: bool = False, variants=(False, True)) -> list:
    """Compiles the release library and (variants containing True) the
    checked one, every object of every variant in parallel, then one link
    each.  Skips a variant whose library is newer than every source.  The
    argument module of the adapter and loss calls is built too, where
    Python's headers are; without them those calls alone are refused."""
    os.makedirs(LIB_DIR, exist_ok=True)
    if os.path.exists(_python_header()):
        build_operands(force=force)
    else:
        print(f"no {_python_header()}: the adapter, loss and microscaled calls from Python need it")
    cc = nvcc()
    jobs = []   # (target, objs, procs)
    for checked in variants:
        target = lib_path(checked)
        if not force and not _stale(target):
            jobs.append((target, None, []))
            continue
        obj_dir = os.path.join(LIB_DIR, f"obj_{'checked_' if checked else ''}{platform.machine()}")
        os.makedirs(obj_dir, exist_ok=True)
        objs, procs = [], []
        for src in SOURCES:
            obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
            objs.append(obj)
            cmd = [cc, *ARCH_FLAGS, *NVCC_FLAGS, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
            if checked:
                cmd.insert(1, "-DSGEMM_GB300_CHECKED")
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        jobs.append((target, objs, procs))
    out_paths = []
    for target, objs, procs in jobs:
        for cmd, p in procs:
            out, _ = p.communicate()
            if verbose or p.returncode:
                print(out.decode(errors="replace"))
            if p.returncode:
                raise SgemmError(-1, "nvcc failed: " + " ".join(cmd))
        if objs is not None:
            tmp = target + f".tmp{os.getpid()}"
            link = [cc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
            r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
            if r.returncode:
                print(r.stdout.decode(errors="replace"))
                raise SgemmError(-1, "nvcc link failed")
            os.replace(tmp, target)
        out_paths.append(target)
    return out_paths


def operands_path() -> str:
    """The extension module that looks the adapter, loss and microscaled calls' tensors over."""
    return os.path.join(LIB_DIR, "_operands" + sysconfig.get_config_var("EXT_SUFFIX"))


def _python_header() -> str:
    return os.path.join(sysconfig.get_paths()["include"], "Python.h")


def build_operands(force: bool = False) -> str:
    """Compiles csrc/operands.c for this interpreter (a second or so)."""
    src, target = os.path.join(CSRC, "operands.c"), operands_path()
    if force or not os.path.exists(target) or os.path.getmtime(src) > os.path.getmtime(target):
        if not os.path.exists(_python_header()):
            raise SgemmError(-1, f"the adapter, loss and microscaled calls from Python need {_python_header()}, which is not there")
        os.makedirs(LIB_DIR, exist_ok=True)
        tmp = target + f".tmp{os.getpid()}"
        cmd = ["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I", os.path.dirname(_python_header()), src, "-o", tmp]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode:
            print(r.stdout.decode(errors="replace"))
            raise SgemmError(-1, "gcc failed: " + " ".join(cmd))
        os.replace(tmp, target)
    return target


def load_operands(setup):
    """That module, built and passed to ``setup`` on first use, once whatever the number of threads."""
    global _operands
    with _lock:
        if _operands is None:
            path = build_operands()
            loader = importlib.machinery.ExtensionFileLoader("_operands", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_operands", path, loader=loader))
            loader.exec_module(module)
            setup(module)
            _operands = module
        return _operands


# Exported symbols, in the order the header declares them.
EXPORTS = ["sgemm", "sgemm_ex", "sgemm_op", "sgemm_strided_batched", "sgemm_tf32x3_split_a", "sgemm_tf32x3_split_b", "sgemm_tf32x3_split_gemm",
           "sgemm_tf32x3_noalloc", "reduce_sum_f32", "sgemm_status_string", "sgemm_last_cuda_error", "sgemm_plan_for", "sgemm_device_status",
           "sgemm_selftest_wait", "sgemm_bounds_line", "sgemm_selftest_bounds", "sgemm_version"]

# The same of adapters_gb300.h.
ADAPTER_EXPORTS = ["lora_forward", "lora_backward", "distill_topk", "policy_loss", "adapters_status_string",
                   "adapters_last_cuda_error", "adapters_plan_for", "adapters_device_status"]


# The same of microscale_gb300.h.
MX_EXPORTS = ["mx_quantize", "mx_dequantize", "mx4_linear", "mx4_matmul", "mx_grad_input", "mx_grad_weight", "mx_status_string",
              "mx_last_cuda_error", "mx_plan_for", "mx_device_status"]


class AdaptersPlan(ctypes.Structure):   # adapters_plan, and mx_plan
    _fields_ = [(name, ctypes.c_int) for name in ("rows", "split", "pair", "tiles")]


class Plan(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int) for name in (
        "path", "kernel", "bm", "bn", "bk", "rm", "rn", "threads", "stages", "grid", "tiles",
        "k_tiles", "smem_bytes", "b_vec", "c_vec", "group_m", "split_k", "op_a", "op_b", "a_vec",
        "a_in_kernel", "trans", "stream_k", "b_in_kernel", "pair", "persistent", "sk_parts")]


def _declare(lib):
    i, f, vp = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
    gemm = [i, i, i, f, vp, i, vp, i, f, vp, i, vp]
    lib.sgemm.argtypes = gemm
    lib.sgemm.restype = i
    lib.sgemm_ex.argtypes = gemm + [i]
    lib.sgemm_ex.restype = i
    lib.sgemm_op.argtypes = [i, i] + gemm + [i]
    lib.sgemm_op.restype = i
    ll = ctypes.c_longlong
    lib.sgemm_strided_batched.argtypes = [i, i, i, i, i, f, vp, i, ll, vp, i, ll, f, vp, i, ll, i, vp, i]
    lib.sgemm_strided_batched.restype = i
    lib.sgemm_tf32x3_split_a.argtypes = [i, i, vp, i, vp, vp, vp]
    lib.sgemm_tf32x3_split_a.restype = i
    lib.sgemm_tf32x3_split_b.argtypes = [i, i, vp, i, vp, vp, vp]
    lib.sgemm_tf32x3_split_b.restype = i
    lib.sgemm_tf32x3_split_gemm.argtypes = [i, i, i, f, vp, vp, vp, vp, f, vp, i, vp]
    lib.sgemm_tf32x3_split_gemm.restype = i
    lib.sgemm_tf32x3_noalloc.argtypes = gemm
    lib.sgemm_tf32x3_noalloc.restype = i
    lib.reduce_sum_f32.argtypes = [vp, ctypes.c_longlong, vp, vp]
    lib.reduce_sum_f32.restype = i
    lib.sgemm_status_string.argtypes = [i]
    lib.sgemm_status_string.restype = ctypes.c_char_p
    lib.sgemm_last_cuda_error.argtypes = []
    lib.sgemm_last_cuda_error.restype = i
    lib.sgemm_plan_for.argtypes = [i, i, i, f, vp, i, vp, i, f, vp, i, i, i, ctypes.POINTER(Plan)]
    lib.sgemm_plan_for.restype = i
    lib.sgemm_device_status.argtypes = [ctypes.POINTER(i), i]
    lib.sgemm_device_status.restype = i
    lib.sgemm_selftest_wait.argtypes = [ctypes.c_ulonglong, ctypes.POINTER(i)]
    lib.sgemm_selftest_wait.restype = i
    lib.sgemm_bounds_line.argtypes = [ctypes.POINTER(i), i]
    lib.sgemm_bounds_line.restype = i
    lib.sgemm_selftest_bounds.argtypes = [ctypes.POINTER(i)]
    lib.sgemm_selftest_bounds.restype = i
    lib.sgemm_version.argtypes = []
    lib.sgemm_version.restype = ctypes.c_char_p
    lib.lora_forward.argtypes = [i, i, i, i, i, i, vp, i, i, vp, i, vp, vp, vp, vp, vp, i, vp, vp]
    lib.lora_forward.restype = i
    lib.lora_backward.argtypes = [i, i, i, i, i, i, vp, i, vp, i, i, vp, i, vp, vp, vp, vp, vp, vp, i, vp, vp, vp]
    lib.lora_backward.restype = i
    lib.distill_topk.argtypes = [i, i, i, i, vp, i, vp, vp, vp, f, vp, vp, i, vp]
    lib.distill_topk.restype = i
    lib.policy_loss.argtypes = [i, i, i, vp, i, vp, vp, vp, vp, vp, f, f, f, vp, vp, vp, i, vp]
    lib.policy_loss.restype = i
    lib.adapters_status_string.argtypes = [i]
    lib.adapters_status_string.restype = ctypes.c_char_p
    lib.adapters_last_cuda_error.argtypes = []
    lib.adapters_last_cuda_error.restype = i
    lib.adapters_plan_for.argtypes = [i, i, i, ctypes.POINTER(AdaptersPlan)]
    lib.adapters_plan_for.restype = i
    lib.adapters_device_status.argtypes = [ctypes.POINTER(i), i]
    lib.adapters_device_status.restype = i
    lib.mx_quantize.argtypes = [i, i, i, i, vp, i, i, vp, i, vp, i, vp]
    lib.mx_dequantize.argtypes = [i, i, i, i, vp, i, vp, i, vp, i, vp]
    lib.mx4_linear.argtypes = [i, i, i, i, vp, i, vp, i, vp, i, vp, i, vp]
    lib.mx4_matmul.argtypes = [i, i, i, i, vp, i, vp, i, vp, i, vp, i, vp, i, vp]
    lib.mx_grad_input.argtypes = [i, i, i, i, vp, i, i, vp, i, vp, i, vp, i, vp]
    lib.mx_grad_weight.argtypes = [i, i, i, i, vp, i, i, vp, i, vp, i, i, vp, i, vp]
    for name in ("mx_quantize", "mx_dequantize", "mx4_linear", "mx4_matmul", "mx_grad_input", "mx_grad_weight"):
        getattr(lib, name).restype = i
    lib.mx_status_string.argtypes = [i]
    lib.mx_status_string.restype = ctypes.c_char_p
    lib.mx_last_cuda_error.argtypes = []
    lib.mx_last_cuda_error.restype = i
    lib.mx_plan_for.argtypes = [i, i, i, i, i, i, ctypes.POINTER(AdaptersPlan)]
    lib.mx_plan_for.restype = i
    lib.mx_device_status.argtypes = [ctypes.POINTER(i), i]
    lib.mx_device_status.restype = i
    lib.address = {name: ctypes.cast(getattr(lib, name), vp).value for name in ADAPTER_EXPORTS + MX_EXPORTS}
    return lib


def load(build_if_missing: bool = True, checked: bool = False):
    """The loaded library (ctypes.CDLL): the release one, or with
    checked=True the bounds-checking one.  Raises SgemmError when it is not
    built and cannot be built -- there is no fallback implementation."""
    lib = _libs.get(checked)
    if lib is not None:   # (every call of the operators passes here)
        return lib
    with _lock:
        if checked not in _libs:
            path = lib_path(checked)
            if build_if_missing:
                path = build(checked=checked)
            if not os.path.exists(path):
                raise SgemmError(-1, f"CUDA library not built ({path}); run __graft_entry__.build()")
            _libs[checked] = _declare(ctypes.CDLL(path))
        return _libs[checked]
