"""Arrivals on a barrier of the other CTA of a pair, read from the sources without a GPU.  A release and an acquire order
memory only if each one's scope holds the other's thread; the waiting thread is in another CTA, so the scope is the
cluster's.  What hands over cleared shared memory has to be such a release."""
import re

from tests.test_warp_convergence import _body, _code


def _arrivals(code):
    """The remote arrivals in `code` as (semantics, scope)."""
    found = re.findall(r"mbarrier\.arrive((?:\.\w+)*?)\.shared::cluster\.b64", code)
    assert found
    return [tuple(f.split(".")[1:]) for f in found]


def test_their_scope_holds_the_waiting_thread():
    for arrival in _arrivals(_code("sm103_more.cuh")):
        assert arrival in (("release", "cluster"), ("relaxed", "cluster"))
    assert ".acquire.cluster." in _body(_code("sm103_more.cuh"), r"bool mbar_wait_cluster\(")


def test_cleared_tails_are_released():
    """Rank 1 clears its rows with ordinary stores, which rank 0's MMA then reads."""
    code = _code("experts.cu")
    (handed,) = re.findall(r"(mbar_\w+)\(map_shared\(zeroed_bar\(last\), 0\)\)", code)
    assert _arrivals(_body(_code("sm103_more.cuh"), rf"void {handed}\(")) == [("release", "cluster")]
    assert "fence_proxy_async_smem()" in _body(code, r"void clear_tail\(")
    assert re.search(r"mbar_wait_cluster\(zeroed_bar\(s\)", code)


def test_accumulators_are_handed_back_between_fences():
    """A relaxed arrival orders no memory: the accumulator has been read (wait::ld in every epilogue) and fenced before it."""
    code = _code("experts.cu")
    back = code[code.index("auto give_back = "):]
    assert back.index("tc_fence_before()") < back.index("mbar_hand_back_remote(")
    for head in (r"void store_rows\(", r"void store_gated\(", r"void store_dw\(", r"void store_part\(", r"void fold_halves\("):
        assert "tmem_ld_wait()" in _body(code, head), head
    waits = [m.end() for m in re.finditer(r"mbar_wait_cluster\(acce_bar", code)]
    assert len(waits) == 2
    for at in waits:
        assert "tc_fence_after()" in code[at:at + 600]
