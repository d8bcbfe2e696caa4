"""CPU float64 oracle for the per-head norm and rotation of queries and keys -- TEST INFRASTRUCTURE ONLY.

    y = x / sqrt(mean(x^2) + eps) * weight
    out = the pairs of the first rotary_dim dims turned by the angle whose cosine and sine the
          table holds for the row's position; pairs (i, i + rotary_dim / 2) or (2 i, 2 i + 1)

``norm_rope`` returns the result and, per element, the sum of the sizes of its two addends (what
rounding errors of the factors are measured against).
"""

from __future__ import annotations

import numpy as np


def norm_rope(x, weight, cos_sin, positions, eps, interleaved):
    """x [T, heads, D] float64; weight [D] or None; cos_sin [P, R] or None; positions [T]."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(axis=2, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    size = np.abs(y)
    if cos_sin is None or cos_sin.shape[1] == 0:
        return y, size
    P, R = cos_sin.shape
    out, add = y.copy(), size.copy()
    for t in range(y.shape[0]):
        p = int(positions[t])
        row = np.asarray(cos_sin[p], dtype=np.float64) if 0 <= p < P else np.zeros(R)
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            c, s = row[i], row[R // 2 + i]
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            add[t, :, a] = add[t, :, b] = size[t, :, a] + size[t, :, b]
    return out, add
