"""CPU oracle for the 8-bit paged cache -- TEST INFRASTRUCTURE ONLY.

It shares no code with the CUDA library.  The definition, written out page by
page in float64:

* a code is sign, four exponent bits (bias 7), three mantissa bits; exponent 0 is
  subnormal, code 0x7f / 0xff is NaN, there is no infinity, the largest value 448;
* an element is ``value(code) * 2 ** (byte - 127)``, one byte per page and KV head;
* a write takes, for each page its new rows fall into and each head, the smallest
  exponent ``e >= -126`` with ``max |x| <= 448 * 2 ** e`` over the page's new finite
  values; a page that holds earlier tokens of its sequence keeps the larger of ``e``
  and its exponent, and its earlier codes are rounded again if it grows;
* rounding is to nearest, ties to the even code; NaN and infinities become NaN.

Codes and bytes are NumPy uint8 arrays; results are modified copies.
"""

from __future__ import annotations

import math

import numpy as np
import torch


def _values() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            x = math.nan
        v[c] = -x if c & 128 else x
    return v


E4M3_VALUES = _values()
_POSITIVE = E4M3_VALUES[:127]  # increasing: 0 .. 448


def encode_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest code of each float64 value (ties to the even code, past 448: 448); NaN and infinities: 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    below, above = a - _POSITIVE[lo], _POSITIVE[hi] - a
    take_hi = (above < below) | ((above == below) & (hi % 2 == 0))
    code = np.where(take_hi, hi, lo)
    code = np.where(a == 0, 0, code).astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def scale_byte(amax: float) -> int:
    """The byte of the smallest 2 ** e with amax <= 448 * 2 ** e, e >= -126."""
    e = -126
    if amax > 0:
        e = max(-126, math.frexp(amax)[1] - 10)
        while amax > 448.0 * 2.0 ** e:
            e += 1
    return e + 127


def dequantize(codes: np.ndarray, bytes_: np.ndarray) -> np.ndarray:
    """float64 elements of a cache [nb, bs, G, D] with scale bytes [nb, G]."""
    return E4M3_VALUES[codes] * (2.0 ** (bytes_.astype(np.float64) - 127))[:, None, :, None]


def quantize_pages(x: np.ndarray):
    """A pool [nb, bs, G, D] quantised page by page; returns (codes, bytes)."""
    nb, bs, G, D = x.shape
    bytes_ = np.array([[scale_byte(float(np.abs(x[b, :, g]).max())) for g in range(G)] for b in range(nb)], np.uint8)
    return encode_e4m3(x * (2.0 ** (127 - bytes_.astype(np.float64)))[:, None, :, None]), bytes_


def write_cache(rows, codes: np.ndarray, bytes_: np.ndarray, cu_q_lens, block_table, seq_lens):
    """New rows [T, G, D] of one of the caches into its pages; returns (codes, bytes)."""
    x = rows.detach().cpu().to(torch.float64).numpy() if isinstance(rows, torch.Tensor) else np.asarray(rows)
    codes, bytes_ = codes.copy(), bytes_.copy()
    bs, G = codes.shape[1:3]
    for s, L in enumerate(np.asarray(seq_lens)):
        r0, r1 = int(cu_q_lens[s]), int(cu_q_lens[s + 1])
        first, L = int(L) - (r1 - r0), int(L)
        for page in range(first // bs, -(-L // bs) if r1 > r0 else 0):
            b = int(block_table[s][page])
            lo, hi = max(first, page * bs), min(L, page * bs + bs)
            new = x[r0 + lo - first:r0 + hi - first]
            kept = lo - page * bs
            for g in range(G):
                fin = np.abs(new[:, g][np.isfinite(new[:, g])])
                byte = scale_byte(float(fin.max()) if fin.size else 0.0)
                if kept:
                    old = min(int(bytes_[b, g]), 254)
                    if byte > old:
                        v = E4M3_VALUES[codes[b, :kept, g]] * 2.0 ** (old - byte)
                        codes[b, :kept, g] = encode_e4m3(v)
                    byte = max(byte, old)
                bytes_[b, g] = byte
                with np.errstate(over="ignore"):
                    codes[b, kept:kept + hi - lo, g] = encode_e4m3(new[:, g] * 2.0 ** (127 - byte))
    return codes, bytes_
