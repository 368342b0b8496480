"""The units that launch chained kernels through launch_rows: what their sources must (not) contain, read without a
GPU (the other chained units have the same checks in test_chained_kernels.py)."""
import os
import re

import pytest

from tests.test_chained_kernels import CSRC, _block, _code

UNITS = ["gated.cu", "rows8.cu", "topk.cu"]
HEADERS = ["gated.cuh"]


def test_units_are_the_chained_ones():
    found = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and f not in ("route.cu", "embed.cu", "experts.cu")
             and re.search(r"launch_rows\(|SPMM_ROWS_TYPED|launch_chained", _code(f))]
    assert found == UNITS


@pytest.mark.parametrize("name", UNITS + HEADERS)
def test_no_load_may_pass_the_dependency_wait(name):
    code = _code(name)
    assert not re.findall(r"__ld(?:g|ca|cg|cs|lu|cv)\b", code)
    assert not re.findall(r"\bld\.global[\w.]*\.nc\b", code)
    assert not re.findall(r"__restrict__|\brestrict\b", code)


@pytest.mark.parametrize("name", UNITS)
def test_every_kernel_waits_for_its_predecessor(name):
    code = _code(name)
    kernels = [m.start() for m in re.finditer(r"__global__", code)]
    assert kernels
    for at in kernels:
        assert "grid_dep_wait()" in _block(code, code.index(")", code.index("const", at)))


def test_gated_epilogue_reads_tmem_together():
    """TMEM loads and transposing stores need whole warps, which come from spinning waits and one thread's stores."""
    from tests.test_warp_convergence import _NEEDS, _body, _unsafe
    code = _code("experts.cu")
    for head in (r"void store_gated\(", r"void fold_halves\(", r"void store_part\("):
        body = _body(code, head)
        loop = body[body.index("for (int c = c0"):]
        assert re.search(_NEEDS, loop) and _unsafe(loop + loop, True) is None, head
    assert re.search(r"__syncwarp\(\);\s*tmem_st_wait\(\)", _body(code, r"void fold_halves\("))
