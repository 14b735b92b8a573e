"""CPU oracle of cache eviction by accumulated attention weight (include/kv4.h)."""
from __future__ import annotations

import numpy as np


def weights(q, K, lse, G: int):
    """Weight of each position summed over a kv head's G query heads: [Hkv, L] float64.
    q [Hq, D]; K [L, Hkv, D]; lse [Hq]."""
    L, H, D = K.shape
    w = np.zeros((H, L))
    for j in range(H * G):
        w[j // G] += np.exp(K[:, j // G] @ q[j].astype(np.float64) / np.sqrt(D) - float(lse[j]))
    return w


def select(acc, S: int, R: int, budget: int):
    """Kept positions of one (sequence, kv head) with totals acc [L], ascending."""
    L = len(acc)
    if L <= budget:
        return list(range(L))
    need = budget - S - R

    def order(p):  # largest total first, NaN last, equal totals from the lowest position on
        return (1, 0.0, p) if np.isnan(acc[p]) else (0, -float(acc[p]), p)

    best = sorted(range(S, L - R), key=order)[:need]
    return sorted(list(range(S)) + best + list(range(L - R, L)))
