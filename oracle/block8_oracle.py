"""CPU oracle of the 8-bit block-scaled cache (include/kv4.h): plain numpy in float64, one
block and one sequence at a time. Codes are kept as the numbers they stand for."""
from __future__ import annotations

import numpy as np

PAGE, D = 16, 128
TOP = {"int8": 127.0, "e4m3": 448.0}


def up16(x: float) -> float:
    """x >= 0 to the next fp16 at or above it, at most 65504."""
    x = min(float(x), 65504.0)
    h = np.float16(x)
    return float(h if float(h) >= x else np.nextafter(h, np.float16(np.inf)))


def nearest(y: np.ndarray, fmt: str) -> np.ndarray:
    """The nearest code of each quotient, ties to even, clamped."""
    top = TOP[fmt]
    if fmt == "int8":
        return np.clip(np.rint(y), -top, top)
    a = np.abs(y)
    # e4m3: 3 mantissa bits; below 2^-6 the step stays 2^-9
    _, e = np.frexp(np.maximum(a, 2.0 ** -6))
    step = 2.0 ** (e - 1.0 - 3.0)
    return np.sign(y) * np.minimum(np.rint(a / step) * step, top)


class Block:
    """One (page, kv head) block of K or V."""

    def __init__(self, fmt: str):
        self.fmt = fmt
        self.codes = np.zeros((PAGE, D))
        self.scale = 0.0

    def append(self, slot: int, rows: np.ndarray) -> None:
        """One call's rows into slots slot .. slot + len(rows) - 1."""
        rows = rows.astype(np.float64)
        # the quotient is the fp32 one: an fp16 at or above the exact quotient is at or above it
        want = up16(np.float32(np.abs(rows).max()) / np.float32(TOP[self.fmt]))
        new = want if slot == 0 else max(self.scale, want)
        if slot and new > self.scale:
            self.codes[:slot] = nearest(self.codes[:slot] * self.scale / new, self.fmt)
        self.scale = new
        self.codes[slot:slot + len(rows)] = nearest(rows / new, self.fmt) if new else 0.0


def attention(q, K, V, G: int):
    """Causal attention of the last n positions of L: q [n, Hq, D]; K, V [L, Hkv, D] float64.
    Returns O [n, Hq, D], lse [n, Hq], and two magnitudes for error bounds: A = sum p |v|
    like O and the largest sum |q_d k_d| / sqrt(D) of a visible key like lse."""
    n, Hq, _ = q.shape
    L = K.shape[0]
    O, A = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, mag = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        seen = L - n + i + 1
        if seen <= 0:
            continue
        for j in range(Hq):
            k, v = K[:seen, j // G], V[:seen, j // G]
            s = k @ q[i, j].astype(np.float64) / np.sqrt(D)
            m = s.max()
            p = np.exp(s - m)
            z = p.sum()
            O[i, j] = p @ v / z
            A[i, j] = p @ np.abs(v) / z
            lse[i, j] = m + np.log(z)
            mag[i, j] = (np.abs(k) @ np.abs(q[i, j].astype(np.float64))).max() / np.sqrt(D)
    return O, lse, A, mag
