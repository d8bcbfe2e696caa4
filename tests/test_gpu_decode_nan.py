"""NaN among what a decode's query sees reaches its output and its log-sum-exp, whichever kernel runs the call,
and no other row: a NaN query, one NaN key, a page of NaN keys, the keys of a whole length, a NaN value.

The reference is the float64 oracle, where a NaN score makes the row's maximum, sum and weights NaN.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from test_gpu_window import BF16, DEV, F32, Batch, i32

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(autouse=True)
def _clear_status():
    pa.metis_read_status(clear=True)
    yield


def same_nan(out, lse, want):
    o, l = want[:2]
    assert np.array_equal(np.isnan(out.double().cpu().numpy()), np.isnan(o)), "output"
    assert np.array_equal(np.isnan(lse.double().cpu().numpy()), np.isnan(l)), "lse"


def plant(b, what, s):
    """Into what the query of sequence s sees, of KV head 0 (a value: in column 3)."""
    seen = oracle.window_tokens(int(b.lens[s]) - 1, b.window, b.sinks)
    bs = b.k.shape[1]
    if what == "query":
        b.q[s, 0, 5] = NAN
    elif what == "key":
        b.k[b.slot(s, int(seen[len(seen) // 2]))][0] = NAN
    elif what == "first key":
        b.k[b.slot(s, int(seen[0]))][0] = NAN
    elif what == "last key":
        b.k[b.slot(s, int(seen[-1]))][0] = NAN
    elif what == "page":
        for t in seen[seen // bs == seen[-1] // bs]:
            b.k[b.slot(s, int(t))][0] = NAN
    elif what == "all keys":
        for t in seen:
            b.k[b.slot(s, int(t))][0] = NAN
    else:
        b.v[b.slot(s, int(seen[-1]))][0, 3] = NAN


WHAT = ["query", "key", "first key", "last key", "page", "all keys", "value"]


@pytest.mark.parametrize("S,H,G,D,bs,window,sinks,dtype", [
    (1, 32, 8, 128, 16, 700, 4, BF16),   # few items: each shared by eight CTAs
    (3, 8, 8, 64, 64, 1500, 130, BF16),
    (40, 16, 8, 64, 16, 90, 33, BF16),   # a CTA an item
    (700, 16, 4, 128, 16, 40, 2, BF16),  # a warp walks items
    (6, 4, 1, 64, 16, 5, 0, F32),        # a token for each warp
    (6, 7, 1, 128, 64, 100, 17, F32),
])
def test_windowed_decode(S, H, G, D, bs, window, sinks, dtype):
    lens = np.random.default_rng(S).integers(window + sinks + 20, window + sinks + 900, S)
    b = Batch(S, [(int(n), 1) for n in lens], H, G, D, bs, window, sinks, dtype, True)
    clean = b.q.clone(), b.k.clone(), b.v.clone()
    for i, what in enumerate(WHAT):
        b.q, b.k, b.v = (x.clone() for x in clean)
        plant(b, what, i * 5 % S)
        same_nan(*b.run(), b.want())


@pytest.mark.parametrize("partition", [0, 64, 512])
@pytest.mark.parametrize("H,G,D,dtype", [(8, 2, 128, BF16), (4, 1, 64, BF16), (7, 1, 64, F32)])
def test_decode_of_all_tokens(partition, H, G, D, dtype):
    seqs = [(n, 1) for n in (900, 30, 5, 1300, 64, 129, 700)]
    b = Batch(9, seqs, H, G, D, 16, 10 ** 6, 0, dtype, True)
    clean = b.q.clone(), b.k.clone(), b.v.clone()
    for i, what in enumerate(WHAT):
        b.q, b.k, b.v = (x.clone() for x in clean)
        plant(b, what, i)
        out, lse = pa.metis_paged_attn_decode(b.q.to(DEV), b.k.to(DEV), b.v.to(DEV), i32(b.table), i32(b.lens), b.scale,
                                              partition_size=partition, max_seq_len=1300, want_lse=True)
        same_nan(out, lse, b.want())


@pytest.mark.parametrize("window,sinks", [(60, 3), (10 ** 6, 0)])
def test_decodes_beside_chunks(window, sinks):
    seqs = [(n, 1) for n in (900, 30, 5, 1300, 64, 129, 700)] + [(300, 100)]
    b = Batch(10, seqs, 8, 2, 128, 16, window, sinks)
    clean = b.q.clone(), b.k.clone(), b.v.clone()
    for i, what in enumerate(WHAT):
        b.q, b.k, b.v = (x.clone() for x in clean)
        plant(b, what, i)
        want = b.want()
        same_nan(*b.run(), want)
        if window == 10 ** 6:
            same_nan(*pa.metis_paged_attn_prefill_chunk(b.q.to(DEV), i32(b.cu), b.k.to(DEV), b.v.to(DEV), i32(b.table),
                                                        i32(b.lens), b.scale, max_seq_len=1300, want_lse=True), want)


def test_decode_over_shared_prefixes():
    from test_gpu_shared_prefix import Batch as Shared
    b = Shared(3, [(300, [310, 300, 390, 301]), (16, [16, 40])], 8, 2, 128, 16, after=[50])
    clean = b.q.clone(), b.k.clone(), b.v.clone()
    slot = lambda s, t: (int(b.table[s, t // 16]), t % 16)
    for s, t in ((0, 305), (2, 320), (0, 7), (1, 299), (4, 15), (6, 49)):
        for keys in (True, False):
            b.q, b.k, b.v = (x.clone() for x in clean)
            g = int(np.searchsorted(b.cu, s, side="right")) - 1
            shared = g < len(b.shared) and t < b.shared[g]  # the members' copies are alike
            for m in range(b.cu[g], b.cu[g + 1]) if shared else [s]:
                (b.k if keys else b.v)[slot(m, t)][1, 3] = NAN
            same_nan(*b.run(), b.want())
    for s in range(7):
        b.q, b.k, b.v = (x.clone() for x in clean)
        b.q[s, 2, 9] = NAN
        same_nan(*b.run(), b.want())
