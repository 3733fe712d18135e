"""The bounds-checking library tests reads as well as writes: the functions of
the microscaled operators through which computed global addresses are read,
and the fused quantiser's stores into shared memory, have their tests."""
import os
import re

import pytest

from dense_fp32_gemm_06_gb300 import _native


def body(name, text):
    """From the function's (or lambda's) name to the brace that closes it."""
    at = re.search(name, text).end()
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("file,name,access", [
    ("mx_store.cuh", r"void load8\(", r"m\.has\(row \+ c(, 8| \+ i, 1)"),
    ("mx_store.cuh", r"void load_run\(", r"m\.has"),
    ("mx_store.cuh", r"auto fetch = ", r"m\.has\(x \+ i \* 256, 8"),
    ("mx_store.cuh", r"auto load = ", r"m\.has\(at"),
    ("mx_store.cuh", r"void __launch_bounds__\(STORE_THREADS\) dequantize_kernel\(", r"a\.lds .* a\.ldc"),
    ("mx_drain.cuh", r"float before\(", r"o\.ldy"),
    ("mx_drain.cuh", r"bool drain_deep\(", r"o\.ldy"),
    ("mx4_tc.cuh", r"auto fetch = ", r"x\.has"),
    ("mx4_tc.cuh", r"codes\[R\], bytes\[R\];.*?(?=for \(int i = 0; i < R; \+\+i\) \{   // \(rows)", r"r < XR && 2048 \+ word < UNIT"),
])
def test_reads_are_tested(file, name, access):
    with open(os.path.join(_native.CSRC, file)) as f:
        text = f.read()
    part = body("(?s)" + name, text)
    assert re.search(r"SG_IN\((.(?!\) \?|\)\)))*" + access, part), part


def test_the_decoders_reads_are_tested():
    with open(os.path.join(_native.CSRC, "mx_grad.cuh")) as f:
        part = re.search(r"const uint8_t \*raw = .*?load_transposed_bytes", f.read(), re.S).group()
    assert part.count("SG_IN(") == 2   # the scales, the codes


def test_values_are_read_nowhere_else():
    """Real matrices are addressed through Source alone."""
    for file in ("mx_store.cuh", "mx_grad.cuh", "mx4_tc.cuh"):
        with open(os.path.join(_native.CSRC, file)) as f:
            text = f.read()
        for cast in re.finditer(r"static_cast<const T \*>\(a\.(x|real)\)", text):
            line = text[text.rfind("\n", 0, cast.start()) + 1:text.index("\n", cast.end())]
            assert "Source" in line or line.strip().startswith("return {"), line
