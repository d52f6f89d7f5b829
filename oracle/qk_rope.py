"""fp64 CPU oracle of the norm of queries and keys for each head with the
position rotation, forward and backward.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path.

    n = x * rstd * gain,  rstd = 1/sqrt(mean(x^2) + eps)   (n = x without a gain)
    pairs (a, b) of the first rot elements: a' = a cos - b sin, b' = b cos + a sin

The rotation is a complex product here: a + ib times cos + i sin.
"""
from __future__ import annotations

import numpy as np


def _turn(x, cos, sin, interleaved, back=False):
    """x [..., D] turned by angles cos, sin [..., rot/2] (backwards: by their negatives)."""
    half = cos.shape[-1]
    w = cos - 1j * sin if back else cos + 1j * sin
    y = np.array(x, dtype=np.float64)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z = (y[..., a] + 1j * y[..., b]) * w
    y[..., a], y[..., b] = z.real, z.imag
    return y


def forward(x, gain, eps, cos, sin, interleaved=False):
    """x [T, H, D], cos and sin [T, rot/2] of each token's position; gain [D] or None."""
    n = np.array(x, dtype=np.float64)
    if gain is not None:
        n = n / np.sqrt(np.mean(n * n, axis=-1, keepdims=True) + eps) * gain
    return _turn(n, cos[:, None, :], sin[:, None, :], interleaved)


def backward(x, gain, eps, cos, sin, dy, interleaved=False):
    """(dx [T, H, D], dgain [D] or None)."""
    dn = _turn(dy, cos[:, None, :], sin[:, None, :], interleaved, back=True)
    if gain is None:
        return dn, None
    rstd = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    xh = x * rstd
    dgain = np.sum(dn * xh, axis=(0, 1))
    dn = dn * gain
    return rstd * (dn - xh * np.mean(dn * xh, axis=-1, keepdims=True)), dgain
