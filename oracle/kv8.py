"""Plain fp64 definition of the 8-bit paged cache and of the page eviction (TEST INFRASTRUCTURE, see
core.py). The pages core.py cites have no counterpart of either; the definition is the library's own:

* A head vector x (one token, one head) is stored with one power-of-two step: a = max |x|,
  E = floor(log2 a) - 6, code = clamp(round_half_even(x / 2^E), -127, 127), value = code * 2^E; all
  zeros when a < 2^-119; NaN when x holds an infinity or NaN.
* A sliding layer stores K' = RoPE(norm(k)) and V = norm(v); a global layer stores S = norm(s) and the
  128 turned columns of RoPE(w_k norm(s)); scores read K from the turned columns and from S elsewhere.
* Page weights: the softmax weight of a page's 16 keys, summed over the query heads.
* Eviction: of n held pages, n - keep leave, the lightest of those that are neither among the first
  `first` nor among the last `last`; of equal weights the lower index leaves first.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from .core import Layer, Norms, normed_kv, rope, rope_rotated_pairs


def exponent(x: np.ndarray) -> np.ndarray:
    """floor(log2 max|x|) over the last axis (exact; -inf for zeros)."""
    a = np.abs(np.asarray(x, np.float64)).max(axis=-1)
    m, e = np.frexp(a)
    return np.where(a == 0, -np.inf, e - 1.0)


def stored(x: np.ndarray) -> np.ndarray:
    """The values that the 8-bit form of the vectors x [..., n] stands for."""
    x = np.asarray(x, np.float64)
    e = exponent(np.where(np.isfinite(x), x, 0.0))[..., None]
    step = np.exp2(np.where(np.isfinite(e), e, 0.0) - 6)
    y = np.where(e < -119, 0.0, np.clip(np.rint(np.where(np.isfinite(x), x, 0.0) / step), -127, 127) * step)
    return np.where(np.isfinite(x).all(axis=-1, keepdims=True), y, np.nan)


def turned_columns(layer: Layer) -> np.ndarray:
    r, h = rope_rotated_pairs(layer.head_dim, layer.rope_partial), layer.head_dim // 2
    return np.concatenate([np.arange(r), np.arange(h, h + r)])


def parts(layer: Layer, k: np.ndarray, v: Optional[np.ndarray], pos, norms: Optional[Norms] = None):
    """The two tensors a layer stores of its rows [n, H, D] at positions pos [n], before the 8-bit cast."""
    src, val = normed_kv(layer, norms, k, v)
    key = rope(src, np.asarray(pos)[:, None], layer.rope_theta, layer.rope_partial)
    if layer.kv_shared:
        return val, key[..., turned_columns(layer)]
    return key, val


def keys_values(layer: Layer, one: np.ndarray, two: np.ndarray):
    """K and V [n, H, D] from the two stored tensors."""
    if not layer.kv_shared:
        return one, two
    k = np.array(one, np.float64)
    k[..., turned_columns(layer)] = two
    return k, one


def decode(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, first: int = 0):
    """One query row q [Hq, D] over keys first .. n-1 of k, v [n, H, D]: output [Hq, D], the weights
    p [Hq, n], sum_j p_j |v_j| (the scale of the relative rounding errors of P.V) and n max_j p_j max|v_j|
    (that of the absolute ones)."""
    hq, n = q.shape[0], k.shape[0]
    group = hq // k.shape[1]
    out, mag, peak, p = np.zeros(q.shape), np.zeros(q.shape), np.zeros((hq, 1)), np.zeros((hq, n))
    for h in range(hq):
        s = (k[first:, h // group] @ q[h]) * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        p[h, first:] = w
        out[h] = w @ v[first:, h // group]
        mag[h] = w @ np.abs(v[first:, h // group])
        peak[h] = (n - first) * (w * np.abs(v[first:, h // group]).max(axis=-1)).max()
    return out, p, mag, peak


def page_sums(p: np.ndarray) -> np.ndarray:
    """[Hq, n] weights -> [pages] sums over heads and keys."""
    w = p.sum(axis=0)
    return np.array([w[i:i + 16].sum() for i in range(0, len(w), 16)])


def evict(seq_len: int, table: Sequence[int], weights: Sequence[float], keep: int, first: int, last: int):
    """(new length, kept pages, their weights, evicted pages) of one sequence."""
    n = (seq_len + 15) // 16
    order = sorted(range(first, n - last),
                   key=lambda i: (math.inf if math.isnan(weights[i]) else weights[i], math.isnan(weights[i]), i))
    out = set(order[:max(0, n - keep)])
    kept = [i for i in range(n) if i not in out]
    return (seq_len - 16 * len(out), [table[i] for i in kept], [weights[i] for i in kept],
            [table[i] for i in sorted(out)])
