"""The 8-bit cache's attention where the pages' V scales differ widely or lie near the ends of
fp32's range: contributions of small pages beside large ones, and results near 2^126 or 2^-113.

The bound of an output column is that of a softmax whose weights are rounded, whatever the pages'
scales: (2 ds + step + 2^-16) sum_t w_t |v_t| + sum_t min(w_t, floor * max w) |v_t|, and the final
rounding (a weight below the floor is rounded to zero or to twice itself at most).  ds bounds a score's error (fp32 sums of exact products, at most 2^-18 of
|scale| sum |q k|, and 2^-20; chunks take the query as two e4m3 parts, 2^-17 of its largest
element more); `step` is a weight's relative rounding and `floor` its absolute one, against the
largest weight:

* decode, bf16 queries: fp16 weights, 2^-11.  They are subnormal below 2^-14, off by up to 2^-25
  there, where the largest weight is 2^14: 2^-39.  A weight may carry its page's V exponent while
  that is at most 2^12 below the largest one: 2^-27.
* decode, fp32 queries: two fp16 parts, 2^-21; the second, times 2^11, is off by up to 2^-25:
  2^-25 - 11 - 14 = 2^-50.
* chunks: bf16 weights, 2^-8 (their range is fp32's: no floor).
"""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from test_gpu_cache_fp8 import BF16, DEV, F32, Cache, check, check_lse, gpu, i32

pytestmark = pytest.mark.gpu

STEP = {BF16: 2.0 ** -11, F32: 2.0 ** -21, "chunk": 2.0 ** -8}
FLOOR = {BF16: 2.0 ** -27, F32: 2.0 ** -50, "chunk": 0.0}


def exact(cache, q, rows, scale, kind):
    """q [R, H, D] float64, rows[i] = (sequence, visible tokens): out, its bound, lse and its bound."""
    R, H, D = q.shape
    r = H // cache.G
    out, tol = np.zeros((R, H, D)), np.zeros((R, H, D))
    lse, ltol = np.full((R, H), -np.inf), np.zeros((R, H))
    for i, (s, n) in enumerate(rows):
        if n == 0:
            continue
        k, v = cache.rows(s, n, "k"), cache.rows(s, n, "v")
        for h in range(H):
            g = h // r
            z = scale * (k[:, g] @ q[i, h])
            m = z.max()
            e = np.exp(z - m)
            w = e / e.sum()
            a = np.abs(v[:, g])
            ds = 2.0 ** -18 * abs(scale) * (np.abs(k[:, g]) @ np.abs(q[i, h])).max() + 2.0 ** -20
            if kind == "chunk":
                ds += 2.0 ** -17 * abs(scale) * np.abs(q[i, h]).max() * np.abs(k[:, g]).sum(axis=1).max()
            out[i, h] = w @ v[:, g]
            lse[i, h] = m + np.log(e.sum())
            tol[i, h] = (2 * ds + STEP[kind] + 2.0 ** -16) * (w @ a) + np.minimum(w, FLOOR[kind] * w.max()) @ a
            ltol[i, h] = ds + 2.0 ** -21 * abs(lse[i, h])
    return out, tol, lse, ltol


def lifted(rng, lens, G, D, bs, gap, where):
    """Ordinary pages but one per sequence (the first, a middle or the last one), where one token has V
    2^gap times as large, a score about e^-60 of the others' for queries whose first element is 8, and
    leaves the page's other tokens codes of zero."""
    c = Cache(rng, lens, G, D, bs, spread=0.0, poisoned=False)
    for s, n in enumerate(lens):
        pages = -(-n // bs)
        page = c.table[s, {"first": 0, "middle": pages // 2, "last": pages - 1}[where]]
        x = rng.standard_normal((2, 1, bs, G, D))
        x[0, 0, 0, :, 0] = -60 / (8 * D ** -0.5)
        x[1, 0, 0] *= 2.0 ** gap
        for codes, byte, y in ((c.k, c.ks, x[0]), (c.v, c.vs, x[1])):
            a, b = oracle.quantize_pages(y)
            codes[page], byte[page] = a[0], b[0]
    c.k[..., 0][np.abs(oracle.E4M3_VALUES[c.k[..., 0]]) < 200] = 0  # (no other score moves with that element)
    c.put()
    return c


def queries(rng, rows, H, D):
    q = torch.from_numpy(rng.standard_normal((rows, H, D)))
    q[:, :, 0] = 8.0
    return q


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("gap", [8, 14, 20, 34, 40, 60])
def test_decode_small_pages_beside_a_large_one(gap, where, dtype):
    """Unsplit, joined and merged calls: what the ordinary pages add to a column stays."""
    rng = np.random.default_rng(gap)
    for D, bs, G, lens, partitions in ((128, 16, 2, [400, 33, 200], (0, 48, 64)), (64, 32, 1, [500], (0, 32, 128)),
                                       (128, 64, 1, [130, 700], (0, 64))):
        c = lifted(rng, lens, G, D, bs, gap, where)
        q = queries(rng, len(lens), 4 * G, D).to(dtype)
        ref, tol, rl, lt = exact(c, q.double().numpy(), list(enumerate(lens)), D ** -0.5, dtype)
        for partition in partitions:
            out, lse = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, c.sl, D ** -0.5, partition_size=partition,
                                                      want_lse=True)
            check(out, ref, tol, dtype, f"out, head_dim {D}, partitions of {partition}")
            check_lse(lse, rl, lt)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,S", [(128, 40), (64, 40)])
def test_decode_small_pages_beside_a_large_one_more_items_than_sms(D, S, dtype):
    rng = np.random.default_rng(D)
    lens = [int(n) for n in rng.integers(20, 150, S)]
    c = lifted(rng, lens, 4, D, 16, 40, "middle")
    q = queries(rng, S, 8, D).to(dtype)
    ref, tol, rl, lt = exact(c, q.double().numpy(), list(enumerate(lens)), D ** -0.5, dtype)
    for partition in (0, 16):
        out, lse = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, c.sl, D ** -0.5, partition_size=partition,
                                                  want_lse=True)
        check(out, ref, tol, dtype, f"out, partitions of {partition}")
        check_lse(lse, rl, lt)


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("gap", [14, 40, 60])
def test_small_pages_beside_a_large_one_in_a_mixed_batch(gap, where):
    """The single-token rows of a chunked call, and its chunks."""
    rng = np.random.default_rng(gap + 1)
    D = 128
    spans = [(400, 1), (150, 40), (90, 1), (300, 3)]
    c = lifted(rng, [n for n, _ in spans], 1, D, 16, gap, where)
    cu = np.concatenate([[0], np.cumsum([q for _, q in spans])])
    q = queries(rng, int(cu[-1]), 4, D).to(BF16)
    out, lse = pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32(cu), *c.dev, c.bt, c.sl, D ** -0.5, want_lse=True)
    for s, (n, m) in enumerate(spans):
        rows = [(s, n - m + i + 1) for i in range(m)]
        at = slice(int(cu[s]), int(cu[s + 1]))
        ref, tol, rl, lt = exact(c, q[at].double().numpy(), rows, D ** -0.5, BF16 if m == 1 else "chunk")
        check(out[at], ref, tol, BF16, f"sequence {s}")
        check_lse(lse[at], rl, lt)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [2.0 ** 119, 2.0 ** 100, 2.0 ** -100, 2.0 ** -113])
def test_decode_values_near_the_ends_of_the_range(size, dtype):
    """V of one size throughout: no sum on the way overflows, and no factor is flushed to zero
    (results of 2^-113 are still normal numbers of both types)."""
    rng = np.random.default_rng(3)
    lens, D = [100, 300, 1], 128
    c = Cache(rng, lens, 1, D, 16, spread=0.0, poisoned=False)
    c.v, c.vs = oracle.quantize_pages(rng.standard_normal((c.nb, 16, 1, D)) * size)
    c.put()
    q = torch.from_numpy(rng.standard_normal((3, 4, D))).to(dtype)
    ref, tol, rl, lt = exact(c, q.double().numpy(), list(enumerate(lens)), 0.1, dtype)
    for partition in (0, 16, 64):
        out, lse = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, c.sl, 0.1, partition_size=partition,
                                                  want_lse=True)
        check(out, ref, tol, dtype, f"out, partitions of {partition}")
        check_lse(lse, rl, lt)
        # (an output of nothing but zeros would pass the comparison's absolute part at 2^-113)
        assert np.abs(out.double().cpu().numpy()).max() >= 0.5 * np.abs(ref).max()
    if dtype == BF16:  # single-token rows of a chunked call
        out, lse = pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32([0, 1, 2, 3]), *c.dev, c.bt, c.sl, 0.1, want_lse=True)
        check(out, ref, tol, dtype, "single-token rows")
        assert np.abs(out.double().cpu().numpy()).max() >= 0.5 * np.abs(ref).max()
