"""Plain fp64 definition of the 4-bit paged cache (TEST INFRASTRUCTURE, see core.py). The pages core.py cites have
no counterpart of it; the definition is the library's own:

* A head vector x (one token, one head) is stored in blocks of 32 columns, each with one power of two: a = max |x|,
  E = floor(log2 a) - 2, one more when a > 7 * 2^E, at most 125; the value is the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4,
  6} * 2^E, ties to the step of even index. Zeros when a < 2^-77; the whole vector is NaN when x holds an infinity or
  NaN.
* What a layer stores of a token, and the attention over it, are those of the 8-bit cache (kv8.py).
"""
from __future__ import annotations

import numpy as np

STEPS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def exponents(x: np.ndarray) -> np.ndarray:
    """E of every block of x [..., n]: [..., n / 32] (any value for a block of zeros)."""
    a = np.abs(np.asarray(x, np.float64)).reshape(*x.shape[:-1], -1, 32).max(axis=-1)
    e = np.frexp(np.where(a == 0, 1.0, a))[1] - 3.0
    return np.minimum(e + (a > 7.0 * np.exp2(e)), 125.0)


def stored(x: np.ndarray) -> np.ndarray:
    """The values that the 4-bit form of the vectors x [..., n] stands for."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(axis=-1, keepdims=True)
    y = np.where(fine, x, 0.0)
    unit = np.exp2(np.repeat(exponents(y), 32, axis=-1))
    m = np.abs(y) / unit
    below = np.abs(m[..., None] - STEPS)
    best = below.min(axis=-1, keepdims=True)
    ties = below == best                                           # one step, or two neighbours
    even = ties & (np.arange(8) % 2 == 0)
    index = np.where(ties.sum(-1) == 2, even.argmax(-1), ties.argmax(-1))
    small = np.repeat(np.abs(y).reshape(*y.shape[:-1], -1, 32).max(axis=-1) < 2.0 ** -77, 32, axis=-1)
    return np.where(fine, np.where(small, 0.0, STEPS[index] * unit * np.sign(y)), np.nan)
