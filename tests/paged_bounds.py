"""Bounds of paged attention that do not grow with the number of keys."""
import math

import numpy as np


def attention_rows(q, k, v, past):
    """Rows of one head in 64 bits and the bound that each element is held to: q [n][d], k and v
    [len][d] (what the cache holds), row t at position past + t.

    The bound counts, for o = sum p v with weights p (sum 1):
    * the output's rounding, 2^-11 |o| (and half the fp16 subnormal step);
    * the weights' rounding to fp16, 2^-11 sum p |v|, and for those below fp16's normal range 2^-32 of
      the exponent base's unit, which is at most twice the row's largest weight; once more for a
      weight that is scaled after it is stored: 2^-30 max p * max|v| for each key;
    * a score's error e, (d + 4) 2^-23 sum |q k| / sqrt d for its products and sums and 2^-22 of that
      for the exponent's argument, and exp2's 2^-21: a factor within 1 +- 2 e of each
      weight, and the same again through the weights' sum;
    * the sums over the keys, whatever their number: 2^-13 sum p |v| for the products, folded
      into rounded sums before 1024 truncations of 2^-23 each have come together (and at most 2048
      roundings of 2^-24 behind that), and 2^-13 for the weights' sum.
    """
    n, d = q.shape
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    s = q @ k.T / math.sqrt(d)
    sa = (np.abs(q) @ np.abs(k).T / math.sqrt(d)).max(1)
    mask = np.arange(len(k))[None] > (past + np.arange(n))[:, None]
    s[mask] = -np.inf
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    o, a = p @ v, p @ np.abs(v)
    e = (d + 4) * 2.0 ** -23 * sa + 2.0 ** -22 * sa + 2.0 ** -21
    lost = 2.0 ** -30 * p.max(1) * (~mask).sum(1) * np.abs(v).max()
    rel = 2.0 ** -11 + 4 * e + 2.0 ** -12
    return o, 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + rel[:, None] * a + lost[:, None]
