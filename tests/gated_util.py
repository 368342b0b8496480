"""Plain 64-bit definitions and error bounds for the gated experts' tests.

Bounds, derived from the arithmetic the header promises.  A sum of n products whose
terms have the total magnitude S is off by at most (n + 2) 2^-23 S.  The activations and
their derivatives are made of expf and erfcf (a few units in the last place, each
2^-23 of the value), of arguments that are themselves rounded (an error of a 2^-24 in an
exponent a is one of a 2^-24 of the result; here a is at most g^2 / 2 or, in the tanh form,
1.6 |g| + 0.08 |g|^3) and of a few products: ACT(g) 2^-22 bounds the error of act relative to itself and that of
act' absolutely, with ACT(g) = 16 + 4 |g| + 4 g^2 + |g|^3.  Rounding to the rows' type adds half a unit
in the last place.
"""
import numpy as np

from tests.onehot_util import bound

ACTS = ["silu", "gelu", "gelu_tanh"]
GROUP = 16


def act(x, name):
    """act(x) in 64 bits."""
    import torch
    t = torch.from_numpy(np.asarray(x, np.float64))
    if name == "silu":
        return (t * torch.sigmoid(t)).numpy()
    if name == "gelu":
        return (t * 0.5 * torch.erfc(-t / 2 ** 0.5)).numpy()
    return (t * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (t + 0.044715 * t ** 3))).numpy()


def act_slope(x, name):
    """act'(x) by central differences of act in 64 bits (off by 1e-9 or less for |x| < 30: the third derivative
    times h^2 / 6 and 2^-52 |x| / h)."""
    h = 1e-5
    x = np.asarray(x, np.float64)
    return (act(x + h, name) - act(x - h, name)) / (2 * h)


def act_error(g):
    g = np.abs(g)
    return (16 + 4 * g + 4 * g * g + g ** 3) * 2.0 ** -22


def near(got, ref, error, dtype, what):
    """got within error of ref before its rounding to dtype."""
    g = got.detach().cpu().double().numpy()
    assert g.shape == ref.shape, what
    lim = error + bound(np.abs(ref) + error, 0.0, 0, dtype)
    bad = ~(np.abs(g - ref) <= lim)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: {g[i]} against "
                             f"{ref[i]}, bound {lim[i]}")


def packed(x):
    """(q, scale byte) of rows x (64 bits) from the definition: the smallest exponent found by trying them upwards."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    q, scale = np.zeros((rows, cols), np.int64), np.zeros((rows, groups), np.int64)
    for r in range(rows):
        for j in range(groups):
            v = x[r, j * GROUP:(j + 1) * GROUP]
            if not np.isfinite(v).all():
                scale[r, j] = 255
                continue
            # exponents below this one have |v| 2^-e of 255 or more
            e = int(np.floor(np.log2(np.abs(v).max()))) - 8 if v.any() else -126
            e = max(e, -126)
            while e < 121 and np.abs(np.rint(v * 2.0 ** -e)).max() > 127:
                e += 1
            q[r, j * GROUP:(j + 1) * GROUP] = np.clip(np.rint(v * 2.0 ** -e), -127, 127)
            scale[r, j] = e + 127
    return q, scale


def held(q, scale):
    """The values of packed rows in 64 bits."""
    s = np.repeat(np.asarray(scale), GROUP, axis=1)[:, :q.shape[1]].astype(np.float64)
    return np.where(s == 255, np.nan, q * 2.0 ** (s - 127))
