"""Plain 64-bit definitions and error bounds for the one-hot operators' tests.

Bounds, derived from the arithmetic the header promises (fp32 sums, one rounding
to the output type): a sum of n products with terms of total magnitude S has an
fp32 error of at most (n + 2) 2^-23 S (2^-23 per step also covers truncating
adders), and rounding to the output type adds at most half a unit in the last
place, 2^-p of the value for a significand of p bits (bf16 8, fp16 11, fp32 24),
or half the smallest subnormal.
"""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
_TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


def bound(ref, magnitude, n, dtype):
    acc = (n + 2) * 2.0 ** -23 * magnitude
    return acc + _UNIT[dtype] * (np.abs(ref) + acc) + _TINY[dtype]


def check(got, ref, magnitude, n, dtype, what):
    g = got.detach().cpu().to(torch.float64).numpy()
    assert g.shape == ref.shape, what
    bad = ~(np.abs(g - ref) <= bound(ref, magnitude, n, dtype))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: "
                             f"{g[i]} against {ref[i]}, bound {np.broadcast_to(bound(ref, magnitude, n, dtype), g.shape)[i]}")


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def route(ids, n_keys):
    """order, pos, offsets of a T x k array of ids from the definition."""
    flat = np.asarray(ids).reshape(-1)
    key = np.where((flat < 0) | (flat >= n_keys), n_keys, flat).astype(np.int64)
    order = np.argsort(key, kind="stable")
    pos = np.full(flat.size, -1, np.int64)
    kept = int((key < n_keys).sum())
    pos[order[:kept]] = np.arange(kept)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=n_keys + 1)[:n_keys])])
    return order, pos.reshape(np.asarray(ids).shape), offsets


def matrix(shape, dtype, seed, scale=1.0, pitch=None):
    """A device matrix of normal values; with a pitch, a view of wider rows."""
    g = torch.Generator().manual_seed(seed)
    full = torch.randn((*shape[:-1], pitch or shape[-1]), generator=g) * scale
    return full.to(DT[dtype]).cuda()[..., :shape[-1]]
