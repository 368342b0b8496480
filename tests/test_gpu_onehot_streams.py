"""The one-hot operators on a stream of their own while the current one is busy, and
captured in a graph that is replayed on new inputs."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import matrix

pytestmark = pytest.mark.gpu

T, K_CHOICES, E, H, N, V = 96, 3, 12, 264, 136, 700


def _inputs(torch, seed):
    rng = np.random.default_rng(seed)
    ids = np.where(rng.random((T, K_CHOICES)) < 0.1, -1, rng.integers(0, E, (T, K_CHOICES)))
    tokens = np.where(rng.random(T) < 0.1, -1, rng.integers(0, V, T))
    return dict(ids=torch.from_numpy(ids).cuda(), tokens=torch.from_numpy(tokens).cuda(),
                w=torch.rand((T, K_CHOICES), generator=torch.Generator().manual_seed(seed)).cuda(),
                table=matrix((V, H), "bf16", seed + 1), dy=matrix((T, N), "bf16", seed + 2),
                W=matrix((E, N, H), "bf16", seed + 3, H ** -0.5))


def _run(spmm, s, stream=None):
    """Every operator once: embedding, route, dispatch, experts, combine, and their gradients."""
    x = spmm.spmm_embed(s["table"], s["tokens"], 2.0, stream=stream)
    R = spmm.spmm_build_route(s["ids"], E, stream=stream)
    xs = spmm.spmm_dispatch(R, x, stream=stream)
    ys = spmm.spmm_experts(R, xs, s["W"], stream=stream)
    y = spmm.spmm_combine(R, ys, s["w"], stream=stream)
    dys, dw = spmm.spmm_combine_grad(R, s["dy"], ys, s["w"], stream=stream)
    dxs, dW = spmm.spmm_experts_grad(R, dys, xs, s["W"], stream=stream)
    dx = spmm.spmm_dispatch_grad(R, dxs, stream=stream)
    RV = spmm.spmm_build_route(s["tokens"], V, stream=stream)
    dtable = spmm.spmm_embed_grad(RV, dx, 2.0, stream=stream)
    return [x, R.order, R.pos, R.offsets, xs, ys, y, dys, dw, dxs, dW, dx, RV.order, RV.keys, RV.offsets, dtable]


def _same(torch, a, b):
    assert len(a) == len(b)
    for i, (p, q) in enumerate(zip(a, b)):
        assert torch.equal(p, q), i


def test_a_stream_of_its_own_does_not_wait_for_the_current_one():
    """Work of about half a second is queued on the current stream.  The operators finish on theirs before it
    does, which they could not if one of them had gone to the current stream."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    s = _inputs(torch, 3)
    want = _run(spmm, s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _run(spmm, s, side)  # kernels loaded, memory of the side stream at hand
    a, b = (torch.empty(1 << 30, dtype=torch.uint8, device="cuda") for _ in range(2))
    b.copy_(a)
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    for _ in range(800):  # 0.3 ms or more each
        b.copy_(a)
    done.record()
    got = _run(spmm, s, side)
    side.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    _same(torch, got, want)
    assert spmm.last_device_error() == 0


def test_inputs_made_late_on_the_side_stream():
    """The inputs reach their buffers on the side stream after a long wait there: an operator on another stream
    would read what they held before."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    old, new = _inputs(torch, 4), _inputs(torch, 5)
    want = _run(spmm, new)
    side = torch.cuda.Stream()
    a, b = (torch.empty(1 << 30, dtype=torch.uint8, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):
            b.copy_(a)
        for name, t in old.items():
            t.copy_(new[name])
    got = _run(spmm, old, side)
    side.synchronize()
    _same(torch, got, want)


def test_captured_in_a_graph():
    """Captured once, replayed on other ids, weights and rows: the bits of the same calls outside a graph."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    s = _inputs(torch, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(spmm, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _run(spmm, s)
    for seed in (6, 7, 8):
        new = _inputs(torch, seed)
        for name, t in s.items():
            t.copy_(new[name])
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _same(torch, outs, _run(spmm, new))
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("tokens,keys", [(700, 40), (2100, 5000), (20000, 300)])
def test_larger_routes_in_a_graph(tokens, keys):
    """The sort's other forms (one tile, a cluster, several launches) and the table gradient's join in a graph."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = torch.empty(tokens, dtype=torch.int64, device="cuda")
    dy = matrix((tokens, 72), "bf16", 1)

    def fill(seed):
        rng = np.random.default_rng(seed)
        ids.copy_(torch.from_numpy(np.where(rng.random(tokens) < 0.3, keys // 2, rng.integers(-1, keys, tokens))))

    def run():
        R = spmm.spmm_build_route(ids, keys)
        return [R.order, R.pos, R.offsets, R.keys, spmm.spmm_embed_grad(R, dy)]

    fill(1)
    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = run()
    for seed in (2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        _same(torch, outs, run())
