"""fp64 CPU oracle of distillation from a teacher's top logits.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path.

    t = s z (cap tanh(t / cap) with softcapping),  q = softmax(t / T) over V,
    p = softmax(a / T) over the entries with an id >= 0
    loss = T^2 sum p_i (log p_i - log q_ci)
    dz_j = dloss T (q_j - sum of p_i with c_i = j) dt/dz

Rows labelled ignore_index and rows without a live entry (no id, or every
value -inf) have loss and gradient 0.
"""
from __future__ import annotations

import numpy as np


def run(z, values, ids, dloss, labels=None, T=1.0, s=1.0, cap=0.0, ignore_index=-100):
    """(loss [N], dz [N, V], q [N, V], p summed by id [N, V])."""
    N, V = z.shape
    with np.errstate(all="ignore"):
        t = s * z
        slope = np.full_like(t, s)
        if cap > 0:
            slope = s / np.cosh(t / cap) ** 2
            t = cap * np.tanh(t / cap)
        x = t / T
        x = x - x.max(axis=1, keepdims=True)
        logq = x - np.log(np.exp(x).sum(axis=1, keepdims=True))
    loss, P = np.zeros(N), np.zeros((N, V))
    live = np.zeros(N, dtype=bool)
    for r in range(N):
        if labels is not None and labels[r] == ignore_index:
            continue
        has = ids[r] >= 0
        a, c = values[r][has], ids[r][has]
        if not len(a) or np.all(a == -np.inf):
            continue
        live[r] = True
        a = (a - a.max()) / T
        p = np.exp(a) / np.exp(a).sum()
        np.add.at(P[r], c, p)
        some = p > 0
        loss[r] = T * T * np.sum(p[some] * (np.log(p[some]) - logq[r][c[some]]))
    q = np.exp(logq)
    with np.errstate(all="ignore"):
        dz = (q - P) * slope * (T * np.asarray(dloss, dtype=np.float64))[:, None]
    dz[~live] = 0.0
    return loss, dz, q, P
