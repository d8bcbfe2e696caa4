"""CPU float64 oracle for attention with a sliding window and first tokens that stay visible
-- TEST INFRASTRUCTURE ONLY.

A query at position p sees the keys t <= p with t > p - window or t < sinks, softmax over those and
nothing else: a row's other keys and values are not touched, so they may hold anything and their
pages need not exist.
"""

from __future__ import annotations

import numpy as np

from .attention import NEG_INF, _arr, _f64, _ints


def window_tokens(p: int, window: int, sinks: int) -> np.ndarray:
    """The keys that a query at position p sees, in order."""
    lo = max(0, p - window + 1)
    return np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, p + 1)])


def paged_window(q, cu_q_lens, k_cache, v_cache, block_table, seq_lens, scale, window, sinks):
    """Query rows cu_q_lens[s] .. of q [T, H, D] are the last tokens of sequence s.  Returns
    (out [T, H, D], lse [T, H], size [T, H, D]): size is the sum of weight * |v|."""
    q, k_cache, v_cache = _f64(q), _arr(k_cache), _arr(v_cache)
    T, H, D = q.shape
    bs, G = k_cache.shape[1:3]
    r = H // G
    out, size = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse = np.full((T, H), NEG_INF)
    cu, lens, table = _ints(cu_q_lens), _ints(seq_lens), _ints(block_table)
    for s in range(len(lens)):
        n = int(cu[s + 1] - cu[s])
        for i in range(n):
            t = window_tokens(int(lens[s]) - n + i, window, sinks)
            page = table[s, t // bs].astype(np.int64)
            assert (page >= 0).all() and (page < k_cache.shape[0]).all()
            k, v = _f64(k_cache[page, t % bs]), _f64(v_cache[page, t % bs])
            row = int(cu[s]) + i
            for h in range(H):
                z = float(scale) * (k[:, h // r] @ q[row, h])
                e = np.exp(z - z.max())
                lse[row, h] = z.max() + np.log(e.sum())
                w = e / e.sum()
                out[row, h] = w @ v[:, h // r]
                size[row, h] = w @ np.abs(v[:, h // r])
    return out, lse, size


def paged_window_decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, sinks):
    """One query per sequence (its last token); a sequence without tokens: zeros and lse -inf."""
    lens = _ints(seq_lens)
    live = np.flatnonzero(lens > 0)
    S, H, D = q.shape
    out, size, lse = np.zeros((S, H, D)), np.zeros((S, H, D)), np.full((S, H), NEG_INF)
    out[live], lse[live], size[live] = paged_window(q[live], np.arange(len(live) + 1), k_cache, v_cache,
                                                    _ints(block_table)[live], lens[live], scale, window, sinks)
    return out, lse, size
