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


# What may leave a warp's threads apart, what brings them together, what needs them together.
_APART = r"if \(lane|mbar_wait\w*\(|mbar_try_wait\("
_TOGETHER = r"__syncwarp\(\)|__syncthreads\(\)|__shfl\w*_sync\(|__ballot_sync\(|__all_sync\(|cluster_sync_all\(\)|sync_all<"
_NEEDS = r"tmem_ld\w*\(|stmatrix_\w+\("


def _unsafe(body, apart):
    """The first collective call that a warp may reach apart, walking the text in order."""
    for m in re.finditer(f"(?P<apart>{_APART})|(?P<together>{_TOGETHER})|(?P<needs>{_NEEDS})", body):
        if m.group("together"):
            apart = False
        elif m.group("apart"):
            apart = True
        elif apart:
            return m.group(0)
    return None


def test_the_walk_itself():
    assert _unsafe("mbar_wait(x); tmem_ld16(t);", False) == "tmem_ld16("
    assert _unsafe("mbar_wait(x); __syncwarp(); tmem_ld16(t);", False) is None
    assert _unsafe("tmem_ld16(t); if (lane == 0) {}", False) is None


def test_experts_read_tmem_together():
    """The epilogue's loops are entered from a wait that each thread spins in, and go round after one thread's store."""
    code = _code("experts.cu")
    for head in (r"void store_rows\(", r"void store_dw\("):
        body = _body(code, head)
        loop = body[body.index("for (int c = c0"):]
        assert re.search(_NEEDS, loop)
        assert _unsafe(loop + loop, True) is None, head
