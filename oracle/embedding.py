"""fp64 CPU oracle of the scaled token embedding lookup and its gradient.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path.

    out[t] = scale * E[id_t]
    dE[v]  = scale * sum over t with id_t = v, v != padding_idx, of dOut[t]

A token whose id lies outside [0, V) gives a row of NaN and no gradient.
"""
from __future__ import annotations

import numpy as np


def forward(ids: np.ndarray, E: np.ndarray, scale: float = 1.0) -> np.ndarray:
    ok = (ids >= 0) & (ids < E.shape[0])
    out = np.full((len(ids), E.shape[1]), np.nan)
    out[ok] = scale * E[ids[ok]].astype(np.float64)
    return out


def backward(dOut: np.ndarray, ids: np.ndarray, V: int, scale: float = 1.0, padding_idx=None):
    """(dE, the sums of magnitudes that bound its rounding errors, tokens of each row)."""
    ok = (ids >= 0) & (ids < V)
    if padding_idx is not None:
        ok &= ids != padding_idx
    dE = np.zeros((V, dOut.shape[1]))
    mag = np.zeros_like(dE)
    x = dOut[ok].astype(np.float64)
    np.add.at(dE, ids[ok], x)
    np.add.at(mag, ids[ok], np.abs(x))
    return scale * dE, abs(scale) * mag, np.bincount(ids[ok], minlength=V)
