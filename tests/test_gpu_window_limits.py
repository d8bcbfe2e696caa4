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
