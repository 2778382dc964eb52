"""Norm and rotation of query and key rows in plain numpy. Test infrastructure;
shares no code with the CUDA path."""
import numpy as np


def table(inv_freq, n_positions):
    """[n_positions, 2, pairs] float64: cosines and sines."""
    angle = np.arange(n_positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    return np.stack([np.cos(angle), np.sin(angle)], 1)


def turn_of(tab, pos, axes=None):
    """Cosines and sines [..., pairs] of positions pos [...] (with axes: [axes, ...]);
    positions outside the table turn nothing."""
    pos = np.asarray(pos)
    n = tab.shape[2]
    out = np.empty((2,) + (pos.shape if axes is None else pos.shape[1:]) + (n,), tab.dtype)
    for i in range(n):
        p = pos if axes is None else pos[axes[i]]
        ok = (p >= 0) & (p < len(tab))
        row = tab[np.where(ok, p, 0), :, i]
        out[0, ..., i] = np.where(ok, row[..., 0], 1.0)
        out[1, ..., i] = np.where(ok, row[..., 1], 0.0)
    return out[0], out[1]


def pair_places(pairs, interleaved):
    i = np.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def turned(x, cos, sin, interleaved):
    """Rows x [..., d], each with its own cosines and sines [..., pairs], in x's type (every
    product and sum rounded to it) -> (rows, |a c| + |b s| of each element)."""
    a, b = pair_places(cos.shape[-1], interleaved)
    out, mag = x.copy(), np.abs(x)
    ac, bs, bc, as_ = x[..., a] * cos, x[..., b] * sin, x[..., b] * cos, x[..., a] * sin
    out[..., a], out[..., b] = ac - bs, bc + as_
    mag[..., a], mag[..., b] = np.abs(ac) + np.abs(bs), np.abs(bc) + np.abs(as_)
    return out, mag


def normalised(x, weight, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
