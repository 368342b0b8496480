"""Kernels launched with programmatic stream serialisation run beside the end of
their predecessor: what their sources must (not) contain, read without a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_dense_matrix_spmm_gb300", "csrc")
UNITS = ["route.cu", "embed.cu", "experts.cu"]
HEADERS = ["rowvec.cuh", "sm103_more.cuh"]


def _code(name):
    """The file without comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _block(code, at):
    """The braces that open at or after `at`, and what they hold."""
    start = code.index("{", at)
    depth = 0
    for i in range(start, len(code)):
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth == 0:
            return code[start:i + 1]
    raise AssertionError("unbalanced braces")


def test_units_are_the_chained_ones():
    found = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "launch_chained" in _code(f)]
    assert found == sorted(UNITS)


@pytest.mark.parametrize("name", UNITS + HEADERS)
def test_no_load_may_pass_the_dependency_wait(name):
    """Non-coherent loads (ld.global.nc, __ldg, restrict-qualified read-only pointers) of what the
    predecessor may still be writing are undefined and may be moved over the wait, and nothing says
    that the cache-hint intrinsics stay behind it.  Ordinary loads and volatile PTX do."""
    code = _code(name)
    assert not re.findall(r"__ld(?:g|ca|cg|cs|lu|cv)\b", code)
    assert not re.findall(r"\bld\.global[\w.]*\.nc\b", code)
    assert not re.findall(r"__restrict__|\brestrict\b", code)
    for m in re.finditer(r"\basm\b[^;]*?\bld\.global", code):
        assert re.match(r"asm\s+volatile", m.group(0)), m.group(0)


@pytest.mark.parametrize("name", UNITS)
def test_every_kernel_waits_for_its_predecessor(name):
    code = _code(name)
    kernels = [m.start() for m in re.finditer(r"__global__", code)]
    assert kernels
    for at in kernels:
        assert "grid_dep_wait()" in _block(code, code.index(")", code.index("const", at)))
