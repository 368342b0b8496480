"""The gated experts' operators on a stream of their own while the current one is busy, captured in a graph that is
replayed on new inputs, in two graphs at once, and past 32-bit offsets."""
import numpy as np
import pytest

from tests.gated_util import act, act_slope
from tests.gpu_util import need_gpu
from tests.onehot_util import f64, matrix

pytestmark = pytest.mark.gpu

T, K_CHOICES, E, H, N = 96, 3, 12, 264, 144


def _inputs(torch, seed, T=T):
    x = matrix((T, E), "f32", seed, 2.0)
    x[T // 2] = -float("inf")
    return dict(logits=x, x=matrix((T, H), "bf16", seed + 1), W=matrix((E, 2 * N, H), "bf16", seed + 2, H ** -0.5),
                dh=matrix((T * K_CHOICES, N), "bf16", seed + 3), dw=matrix((T, K_CHOICES), "f32", seed + 4))


def _run(spmm, s, stream=None):
    """Every operator once, as a layer uses them; results that are tensors."""
    ids, w = spmm.spmm_topk(s["logits"], K_CHOICES, stream=stream)
    R = spmm.spmm_build_route(ids, E, stream=stream)
    xs = spmm.spmm_dispatch(R, s["x"], stream=stream)
    P = spmm.spmm_pack_rows(xs, stream=stream)
    h, gu = spmm.spmm_experts_gated(R, xs, s["W"], act="silu", save="rows", stream=stream)
    _, G = spmm.spmm_experts_gated(R, xs, s["W"], act="silu", save="packed", stream=stream)
    served = spmm.spmm_experts_gated(R, xs, s["W"], act="silu", stream=stream)
    dgu, h2 = spmm.spmm_gated_grad(R, s["dh"], gu, with_h=True, stream=stream)
    grads = spmm.spmm_experts_gated_grad(R, s["dh"], P, s["W"], G, stream=stream)
    back = spmm.spmm_unpack_rows(P, stream=stream)
    dl = spmm.spmm_topk_grad(s["logits"], ids, w, s["dw"], stream=stream)
    return [ids, w, R.pos, xs, P.q, P.scale, h, gu, G.q, G.scale, served, dgu, h2, *grads, back, dl]


def _same(torch, a, b):
    assert len(a) == len(b)
    for i, (p, q) in enumerate(zip(a, b)):
        assert torch.equal(p, q), i


@pytest.mark.parametrize("tokens", [T, 4])
def test_a_stream_of_its_own_does_not_wait_for_the_current_one(tokens):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    s = _inputs(torch, 3, tokens)
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


@pytest.mark.parametrize("tokens", [T, 5, 1])
def test_captured_in_a_graph(tokens):
    """Captured once, replayed on other logits, weights and rows: the bits of the same calls outside a graph."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    s = _inputs(torch, 6, tokens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(spmm, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _run(spmm, s)
    for seed in (6, 7, 8):
        new = _inputs(torch, seed, tokens)
        for name, t in s.items():
            t.copy_(new[name])
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _same(torch, outs, _run(spmm, new))
    assert spmm.last_device_error() == 0


def test_two_graphs_on_two_streams():
    """Two captured passes replayed at the same time share nothing."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    both = []
    for seed in (1, 2):
        s = _inputs(torch, 10 * seed, 700 * seed)
        want = _run(spmm, s)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs = _run(spmm, s)
        both.append((s, want, graph, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, _, graph, _, stream in both:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, want, _, outs, _ in both:
        _same(torch, outs, want)
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("save", ["rows", "packed"])
def test_offsets_past_32_bits(save):
    """[g u] of more than 2^31 values (of more than 2^32 bytes): rows at the end, dropped ones among them."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    n, N, K = (1 << 20) + (1 << 17) + 77, 1024, 8
    if save == "packed":
        n *= 2
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    ids[-100:] = -1
    R = spmm.spmm_build_route(ids, 1)
    xs = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    xs[-400:] = matrix((400, K), "bf16", 1)
    W = matrix((1, 2 * N, K), "bf16", 2)
    h, gu = spmm.spmm_experts_gated(R, xs, W, save=save)
    tail = slice(n - 400, n - 100)  # kept rows: the sort is stable
    if save == "rows":
        ref = (f64(xs[tail]) @ f64(W[0]).T)
        assert np.abs(f64(gu[tail]) - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
        assert not gu[-100:].any()
        V = f64(gu[tail])
    else:
        assert not gu.q[-100:].any() and (gu.scale[-100:] == 1).all()
        V = f64(spmm.spmm_unpack_rows(spmm.Rows8(300, 2 * N, gu.dtype, gu.q[tail], gu.scale[tail])))
        ref = f64(xs[tail]) @ f64(W[0]).T
        assert np.abs(V - ref).max() <= np.abs(ref).max() / 100
    del h
    dh = torch.ones(n, N, dtype=torch.bfloat16, device="cuda")
    dgu = spmm.spmm_gated_grad(R, dh, gu)
    g, u = V[:, :N], V[:, N:]
    got = f64(dgu[tail])
    # one rounding of bf16, and of differences
    assert np.allclose(got[:, :N], u * act_slope(g, "silu"), rtol=2.0 ** -7, atol=1e-6)
    assert np.allclose(got[:, N:], act(g, "silu"), rtol=2.0 ** -7, atol=1e-6)
    assert not dgu[-100:].any()
    assert spmm.last_device_error() == 0


def test_router_past_32_bits():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rows, experts = (1 << 23) + 5, 264
    x = torch.zeros(rows, experts, dtype=torch.bfloat16, device="cuda")
    x[-9:] = matrix((9, experts), "bf16", 1)
    ids, w = spmm.spmm_topk(x, 2)
    last = spmm.spmm_topk(x[-9:].clone(), 2)
    assert torch.equal(ids[-9:], last[0]) and torch.equal(w[-9:], last[1])
    assert (ids[:-9] == torch.tensor([0, 1], device="cuda")).all() and (w[:-9] == 0.5).all()
    d = spmm.spmm_topk_grad(x, ids, w, torch.ones_like(w) * torch.tensor([1.0, 0.0], device="cuda"))
    assert (d[:-9, 0] == 0.25).all() and (d[:-9, 1] == -0.25).all() and not d[:-9, 2:].any()
