"""Plain 64-bit definitions of the operators around a memory layer, and the
arithmetic their tests' tolerances are made of.

U32 is half a step of fp32 relative to the value; ``half_step`` that of a
storage type.  A sum of n fp32 terms in any order is off by at most about
n * U32 times the sum of the terms' magnitudes.
"""

import torch

U32 = 2.0 ** -24
GROUP = 128
Q8_MAX = {"e4m3": 448.0, "int8": 127.0}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def q8_groups(d):
    return (d + GROUP - 1) // GROUP


def group_amax(v):
    """[T, d] fp64 -> largest magnitude of each 128-column group."""
    return torch.stack([c.abs().amax(1) for c in v.split(GROUP, dim=1)], 1)


def expand_scales(scales, d):
    return scales.double().repeat_interleave(GROUP, 1)[:, :d]


def scale_of(amax, fmt):
    """Smallest 2^k >= 2^-100 with amax <= 2^k * max, by search."""
    s = torch.full_like(amax, 2.0 ** -100)
    while True:
        grow = amax > s * Q8_MAX[fmt]
        if not grow.any():
            return s
        s = torch.where(grow, s * 2, s)


def q8_values(q, scales):
    return q.float().double() * expand_scales(scales, q.shape[1])


def q8_half_step(v, scales, fmt):
    """Half a step of the 8-bit format at each value."""
    s = expand_scales(scales, v.shape[1])
    if fmt == "int8":
        return s / 2
    return torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10)


def embed(table, ids, scale, pad_id=None):
    out = table.double()[ids.long()] * scale
    if pad_id is not None:
        out[ids == pad_id] = 0
    return out


def embed_grad(dout, ids, n_rows, scale, pad_id=None):
    """(gradient, sum of magnitudes, terms per row), one token at a time."""
    d = dout.shape[-1]
    g = torch.zeros(n_rows, d, dtype=torch.float64)
    mag = torch.zeros(n_rows, d, dtype=torch.float64)
    n = torch.zeros(n_rows, 1, dtype=torch.float64)
    for t, r in enumerate(ids.reshape(-1).tolist()):
        if r == pad_id or not 0 <= r < n_rows:
            continue
        row = dout.reshape(-1, d)[t].double() * scale
        g[r] += row
        mag[r] += row.abs()
        n[r] += 1
    return g, mag, n


def norm(h, weight, eps):
    """(y, rstd) of the root-mean-square norm, fp64."""
    h = h.double()
    rstd = (h.square().mean(1) + eps) ** -0.5
    y = h * rstd[:, None]
    return (y if weight is None else y * weight.double()), rstd
