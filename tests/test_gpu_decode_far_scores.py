"""A key whose score lies below fp32's range weighs nothing, wherever it stands: alone among the tokens that a
warp or a unit of 16 holds, first in the sequence, or all of a shared prefix.

Queries are positive and such a key's elements the type's lowest value, so that every product is negative and the
sum passes -infinity; the oracle's float64 has it as a finite score and a weight of zero.
"""
import numpy as np
import pytest
import torch

import paged_attention_kv_decode_gb300 as pa
from test_gpu_window import BF16, DEV, F32, Batch, compare, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    pa.metis_read_status(clear=True)
    yield


def lower(b, tokens):
    """Keys of every sequence's `tokens` (those it has, the last one aside)."""
    b.q = b.q.abs() + 0.25
    for s, n in enumerate(b.lens):
        for t in tokens:
            if t < n - 1:
                b.k[b.slot(s, t)] = torch.finfo(b.k.dtype).min
    return b


@pytest.mark.parametrize("S,H,G,D,bs,window,sinks,dtype", [
    (1, 32, 8, 128, 16, 700, 1, BF16),   # few items: each shared by eight CTAs
    (40, 16, 8, 64, 16, 90, 1, BF16),    # a CTA an item
    (700, 16, 4, 128, 16, 40, 1, BF16),  # a warp walks items
    (6, 7, 1, 128, 64, 30, 1, F32),
])
def test_windowed_decode(S, H, G, D, bs, window, sinks, dtype):
    lens = np.random.default_rng(S).integers(window + sinks + 20, window + sinks + 900, S)
    lower(Batch(S, [(int(n), 1) for n in lens], H, G, D, bs, window, sinks, dtype, True), [0]).check()


@pytest.mark.parametrize("partition", [0, 16, 512])
@pytest.mark.parametrize("H,G,D,dtype", [(8, 2, 128, BF16), (7, 1, 64, F32)])
def test_decode_of_all_tokens(partition, H, G, D, dtype):
    b = lower(Batch(9, [(n, 1) for n in (900, 30, 2, 1300, 64, 129)], H, G, D, 16, 10 ** 6, 0, dtype, True),
              list(range(16)) + list(range(64, 80)))
    out, lse = pa.metis_paged_attn_decode(b.q.to(DEV), b.k.to(DEV), b.v.to(DEV), i32(b.table), i32(b.lens), b.scale,
                                          partition_size=partition, max_seq_len=1300, want_lse=True)
    compare(out, lse, b.want(), dtype)


def test_decodes_beside_chunks():
    lower(Batch(10, [(n, 1) for n in (900, 30, 1300, 64)] + [(300, 100)], 8, 2, 128, 16, 60, 1), [0]).check()


def test_decode_over_shared_prefixes():
    """A prefix of one token, and own tokens whose first unit is such."""
    from test_gpu_shared_prefix import Batch as Shared
    b = Shared(3, [(1, [40, 2, 300]), (32, [60, 52, 80])], 8, 2, 128, 16)
    b.q = b.q.abs() + 0.25
    low = torch.finfo(BF16).min
    for s in range(3):
        b.k[int(b.table[s, 0]), 0] = low
    for s in range(3, 6):
        for t in range(32, 48):
            b.k[int(b.table[s, t // 16]), t % 16] = low
    b.check()
