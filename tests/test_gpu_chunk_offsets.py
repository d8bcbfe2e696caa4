"""Offsets and lengths of chunked calls (bf16 and 8-bit cache) that do not fit together: reported, and
the other sequences' rows as without them."""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from test_gpu_cache_fp8 import BF16, DEV, Cache, gpu, i32

pytestmark = pytest.mark.gpu


class Batch:
    def __init__(self, fp8, D=128, bs=16):
        rng = np.random.default_rng(4)
        self.lens, self.rows = [90, 40, 33, 70], 64
        self.c = Cache(rng, self.lens, 2, D, bs, spread=0.0, poisoned=False)
        self.q = gpu(torch.from_numpy(rng.standard_normal((self.rows, 8, D))).to(BF16))
        if fp8:
            self.fn, self.cache = pa.metis_paged_attn_prefill_chunk_fp8, self.c.dev
        else:
            self.fn = pa.metis_paged_attn_prefill_chunk
            self.cache = [gpu(torch.from_numpy(oracle.dequantize(a, b)).to(BF16))
                          for a, b in ((self.c.k, self.c.ks), (self.c.v, self.c.vs))]

    def run(self, cu, lens=None, max_seq_len=96):
        """The outputs (7.0 where nothing was written), their lse and the status bits.  The outputs are
        the middle of larger tensors whose other rows must stay."""
        n = self.rows
        out = torch.full((3 * n, 8, self.q.shape[2]), 7.0, dtype=BF16, device=DEV)
        lse = torch.full((3 * n, 8), 7.0, device=DEV)
        pa.metis_read_status(clear=True)
        self.fn(self.q, i32(cu), *self.cache, self.c.bt, i32(self.lens if lens is None else lens), 0.1,
                out=out[n:2 * n], lse_out=lse[n:2 * n], max_seq_len=max_seq_len)
        status = pa.metis_read_status(clear=True)
        for t in (out, lse):
            assert (t[:n] == 7.0).all() and (t[2 * n:] == 7.0).all()
        return out[n:2 * n], lse[n:2 * n], status


@pytest.fixture(params=[True, False], ids=["fp8", "bf16"])
def batch(request):
    return Batch(request.param)


def same(a, b, rows):
    return torch.equal(a[0][rows].view(torch.int16), b[0][rows].view(torch.int16)) and torch.equal(a[1][rows], b[1][rows])


def untouched(a, rows):
    return bool((a[0][rows] == 7.0).all() and (a[1][rows] == 7.0).all())


def test_query_counts_that_do_not_fit_are_reported(batch):
    good = batch.run([0, 20, 21, 24, 64])
    assert good[2] == 0
    # a count below zero: that sequence has no rows
    got = batch.run([0, 20, 21, 24, 10])
    assert got[2] == pa.STATUS_BAD_Q_LEN
    assert same(got, good, slice(0, 24)) and untouched(got, slice(24, 64))
    # more queries than cached tokens: clamped, also where nothing is cached
    got = batch.run([0, 20, 21, 24, 64], [90, 40, 0, 70])
    assert got[2] == pa.STATUS_BAD_Q_LEN
    assert same(got, good, slice(0, 21)) and same(got, good, slice(24, 64)) and untouched(got, slice(21, 24))
    got = batch.run([0, 20, 21, 24, 64], [90, 40, 2, 70])
    assert got[2] == pa.STATUS_BAD_Q_LEN and same(got, good, slice(0, 21)) and same(got, good, slice(24, 64))
    # a length past the bound counts only where there are queries
    assert batch.run([0, 20, 21, 21, 61], [90, 40, 500, 70])[2] == 0
    assert batch.run([0, 20, 21, 24, 64], [90, 40, 500, 70])[2] & pa.STATUS_SEQ_TOO_LONG


@pytest.mark.parametrize("cu,out_of_it", [
    ([0, 20, 21, 24, 65], [3]),                    # a chunk past the last row
    ([0, 20, 21, 24, (1 << 31) - 1], [3]),
    ([0, 20, 21, 30, 1 << 20], [3]),
    ([64, 65, 65, 65, 65], [0, 1, 2, 3]),          # a single row past it
    ([(1 << 31) - 1, -(1 << 31), 1, 4, 44], [0, 1]),
    ([-1, 0, 1, 4, 44], [0]),                      # a single row in front of the first
    ([-30, 20, 21, 24, 64], [0]),
    ([-(1 << 31), 20, 21, 24, 64], [0]),
    ([0, 20, 1 << 30, 24, 64], [1, 2]),
])
def test_rows_outside_the_batch_are_left_out(batch, cu, out_of_it):
    got = batch.run(cu)
    assert got[2] == pa.STATUS_BAD_OFFSETS
    # the other sequences, each alone in a call of its own
    written = np.zeros(batch.rows, bool)
    for s in range(4):
        if s in out_of_it:
            continue
        alone = [cu[s]] * (s + 1) + [cu[s + 1]] * (4 - s)
        ref = batch.run(alone)
        assert ref[2] == 0
        rows = slice(cu[s], cu[s + 1])
        written[rows] = True
        assert np.abs((got[0][rows].float() - ref[0][rows].float()).cpu().numpy()).max(initial=0.0) <= 0.05
        assert np.abs((got[1][rows] - ref[1][rows]).cpu().numpy()).max(initial=0.0) <= 1e-3
    assert untouched(got, torch.from_numpy(np.flatnonzero(~written)).to(DEV))


def test_rows_behind_the_last_sequence_stay(batch):
    got = batch.run([0, 20, 21, 24, 50])
    assert got[2] == 0 and untouched(got, slice(50, 64)) and not untouched(got, slice(49, 50))
