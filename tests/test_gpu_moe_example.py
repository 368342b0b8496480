"""The example layer: its forward pass and gradients against the same layer in 64
bits (autograd), and a training run whose loss falls."""
import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _example():
    from examples import moe_layer
    return moe_layer


# Eight stored intermediates (x, h, a, ys, the sum, dys, da / dh, dxs) are rounded to bf16
# with a relative error of 2^-8 each, and each passes on through products whose terms
# carry it independently: in norm at most 8 roundings of 2^-8.
TOL = 8 * 2.0 ** -8


def test_layer_against_64_bits():
    torch = need_gpu()
    m = _example()
    V, E, H, F, top, T = 50, 6, 64, 96, 2, 41
    layer = m.Layer.random(V, E, H, F, top, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    tokens[5] = tokens[6] = -1
    y, saved = m.forward(layer, tokens)
    dy = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    got = m.backward(layer, saved, dy)

    p = [t.detach().double().cpu().requires_grad_() for t in (layer.table, layer.router, layer.W1, layer.W2)]
    table, router, W1, W2 = p
    ids, chosen = tokens.cpu(), saved[4].cpu()
    x = torch.where(ids[:, None] >= 0, table[ids.clamp(min=0)], 0.0)
    w = torch.softmax((x @ router.t()).gather(1, chosen), dim=1)
    out = x
    for j in range(top):
        e = chosen[:, j]
        h = torch.einsum("tfh,th->tf", W1[e], x)
        out = out + w[:, j, None] * torch.einsum("thf,tf->th", W2[e], torch.nn.functional.silu(h))
    (out * dy.double().cpu()).sum().backward()
    for name, a, b in [("y", y, out.detach())] + [(n, a, t.grad) for n, a, t in
                                                  zip(("dtable", "drouter", "dW1", "dW2"), got, p)]:
        a = a.double().cpu()
        assert torch.linalg.vector_norm(a - b) <= TOL * torch.linalg.vector_norm(b), name
    assert not got[0].cpu()[torch.tensor([v for v in range(V) if v not in ids.tolist()])].any()


def test_example_trains():
    need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    losses = _example().main(["--tokens", "512", "--experts", "8", "--width", "256", "--hidden", "192", "--vocab", "500",
                              "--steps", "4"])
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert spmm.last_device_error() == 0
