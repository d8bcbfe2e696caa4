"""Windows and first tokens beyond every length, up to the largest numbers a call can be given: every query sees all
that is before it, as without a window."""
import numpy as np
import pytest
import torch

import paged_attention_kv_decode_gb300 as pa
from test_gpu_window import CHUNKS, DEV, Batch, i32

pytestmark = pytest.mark.gpu
INT_MAX = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def _clear_status():
    pa.metis_read_status(clear=True)
    yield


@pytest.mark.parametrize("window,sinks", [(INT_MAX, 0), (INT_MAX, 4), (INT_MAX, 300), (INT_MAX - 100, 0), (INT_MAX - 800, 1)])
@pytest.mark.parametrize("H,G,D,bs,which", [(8, 2, 128, 16, 0), (4, 4, 64, 32, 0), (4, 4, 128, 16, 1), (8, 1, 64, 16, 1),
                                            (4, 1, 128, 64, 1)])
def test_chunks(window, sinks, H, G, D, bs, which):
    b = Batch(window % 91 + sinks + H, CHUNKS[which], H, G, D, bs, 10 ** 6, 0)
    cache = b.k.to(DEV), b.v.to(DEV), i32(b.table), i32(b.lens)
    want, wl = pa.metis_paged_attn_prefill_chunk(b.q.to(DEV), i32(b.cu), *cache, b.scale, max_seq_len=1000, want_lse=True)
    b.window, b.sinks = window, sinks
    out, lse = b.run(max_seq_len=1000)
    assert torch.equal(out, want) and torch.equal(lse, wl) and pa.metis_read_status() == 0


@pytest.mark.parametrize("window,sinks", [(2 ** 32 + 5, 0), (2 ** 40, 4), (5, 2 ** 32 + 3), (2 ** 31, 2 ** 63)])
@pytest.mark.parametrize("decode", [False, True])
def test_numbers_past_int32_are_beyond_every_length(window, sinks, decode):
    seqs = [(n, min(n, 1 if decode else q)) for n, q in CHUNKS[0]]
    b = Batch(3, seqs, 8, 2, 128, 16, 10 ** 6, 0, decode=decode)
    want, wl = b.run()
    b.window, b.sinks = window, sinks
    out, lse = b.run()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    for window, sinks in ((-2 ** 32 + 5, 0), (5, -2 ** 32 + 3)):  # (their low 32 bits are positive)
        b.window, b.sinks = window, sinks
        with pytest.raises(pa.MetisError):
            b.run()
