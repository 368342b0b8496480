"""Instructions marked .aligned need all threads of a warp at once: the sources must
bring a warp together (__syncwarp) between a branch or a spinning wait and such an
instruction, read without a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_dense_matrix_spmm_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _body(code, head):
    """The body of the function whose text matches `head`."""
    start = code.index("{", re.search(head, code).end())
    depth = 0
    for i in range(start, len(code)):
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth == 0:
            return code[start:i + 1]
    raise AssertionError("unbalanced braces")


def test_cluster_barrier_brings_its_warps_together():
    """Callers reach the cluster barrier out of branches (a warp's digits past the last one, dropped lanes)."""
    body = _body(_code("sm103_more.cuh"), r"void cluster_sync_all\(\)")
    assert ".aligned" in body
    assert body.index("__syncwarp()") < body.index("asm")
