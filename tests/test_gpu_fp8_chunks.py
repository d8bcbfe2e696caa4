"""Chunked prefill over the 8-bit cache: softmax scales of either sign and zero, query rows of any
size, and the split over keys held to each row's own bound."""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from test_gpu_cache_fp8 import BF16, CHUNK_STEP, DEV, Cache, attention, check, check_lse, gpu, i32
from test_gpu_fp8_value_ranges import exact

pytestmark = pytest.mark.gpu


def run(c, q, q_lens, scale, **kw):
    cu = i32(np.concatenate([[0], np.cumsum(q_lens)]))
    return pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), cu, *c.dev, c.bt, c.sl, scale, want_lse=True, **kw)


def rows_of(lens, q_lens):
    return [(s, n - m + i + 1) for s, (n, m) in enumerate(zip(lens, q_lens)) for i in range(m)]


@pytest.mark.parametrize("r,D,bs", [(4, 128, 16), (8, 64, 64), (16, 128, 32)])
@pytest.mark.parametrize("scale", [0.0, -0.05, -0.3, 0.7])
def test_chunk_softmax_scales(scale, r, D, bs):
    """Masked, whole and split tiles; a prefix long enough to be split over its keys."""
    rng = np.random.default_rng(r + D)
    lens, q_lens = [200, 70, 2100, 33], [150, 70, 40, 5]
    c = Cache(rng, lens, 1, D, bs, spread=0.5)
    q = torch.from_numpy(rng.standard_normal((sum(q_lens), r, D))).to(BF16)
    out, lse = run(c, q, q_lens, scale)
    ref, tol, rl, lt = attention(c, q.double().numpy(), rows_of(lens, q_lens), scale, CHUNK_STEP, parts=True)
    check(out, ref, tol, BF16, "out")
    check_lse(lse, rl, lt)


@pytest.mark.parametrize("size,scale", [(1e30, 1e-31), (1e-30, 1e29), (0.0, 1.0), (1.0, 0.01), (1e30, 0.0), (1e30, -1e-31)])
def test_chunk_query_rows_of_any_size(size, scale):
    """The power of two that brings a row into e4m3's range is undone; a scale of zero weighs every
    visible token alike, whatever the scores."""
    rng = np.random.default_rng(6)
    lens, q_lens = [180, 40], [130, 40]
    c = Cache(rng, lens, 2, 128, 16, spread=0.0)
    q = rng.standard_normal((170, 8, 128)) * size
    q[100, 2, 5] = 4096.0 * size  # one large element beside small ones
    q[7] = 0.0
    q = torch.from_numpy(q).to(BF16)
    out, lse = run(c, q, q_lens, scale)
    ref, tol, rl, lt = attention(c, q.double().numpy(), rows_of(lens, q_lens), scale, CHUNK_STEP, parts=True)
    check(out, ref, tol, BF16, "out")
    check_lse(lse, rl, lt)


def test_chunk_split_and_whole_within_each_rows_own_bound():
    """The same call with and without the memory for parts, every element against its own bound."""
    rng = np.random.default_rng(31)
    lens, q_lens = [2900, 64, 1500], [100, 1, 300]
    c = Cache(rng, lens, 2, 128, 16)
    q = torch.from_numpy(rng.standard_normal((401, 8, 128))).to(BF16)
    at = np.sort(np.concatenate([rng.choice(401, 40, replace=False), [100]]))
    rows = rows_of(lens, q_lens)
    ref, tol, rl, lt = attention(c, q[torch.from_numpy(at)].double().numpy(), [rows[i] for i in at], 0.088, CHUNK_STEP,
                                 parts=True)
    dev_at = torch.from_numpy(at).to(DEV)
    for n in (pa.metis_prefill_workspace_bytes(3, 401, 8, 2),
              pa.metis_prefill_fp8_workspace_bytes(3, 401, 8, 2, 128, 2900)):
        out, lse = run(c, q, q_lens, 0.088, max_seq_len=2900,
                       workspace=torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV))
        check(out[dev_at], ref, tol, BF16, "out")
        check_lse(lse[dev_at], rl, lt)


@pytest.mark.parametrize("r,D,bs", [(4, 128, 16), (1, 64, 32), (8, 64, 64)])
def test_chunk_lowest_value_of_an_unseen_token_stays_out(r, D, bs):
    """V rows hold the type's lowest and largest value (2^128 once rounded to a code): rows of the same
    chunk that do not see them are what they are without them."""
    rng = np.random.default_rng(r + D)
    lens, q_lens = [200, 150], [170, 150]
    c = Cache(rng, lens, 1, D, bs, spread=0.0, poisoned=False)
    rows = [torch.from_numpy(rng.standard_normal((350, 1, D))).to(BF16) for _ in range(2)]
    extreme = ((0, 150, 5, torch.finfo(BF16).min), (0, 151, 9, torch.finfo(BF16).max), (1, 20, 7, torch.finfo(BF16).min),
               (1, 149, 0, torch.finfo(BF16).max))
    for s, t, d, x in extreme:
        rows[1][200 * s + t, 0, d] = x
    pa.metis_reshape_and_cache_fp8(gpu(rows[0]), gpu(rows[1]), *c.dev, i32([0, 200, 350]), c.bt, c.sl)
    c.k, c.ks = oracle.write_cache(rows[0], c.k, c.ks, [0, 200, 350], c.table, lens)
    c.v, c.vs = oracle.write_cache(rows[1], c.v, c.vs, [0, 200, 350], c.table, lens)
    q = torch.from_numpy(rng.standard_normal((320, r, D))).to(BF16)
    out, lse = run(c, q, q_lens, D ** -0.5)
    visible = rows_of(lens, q_lens)
    ref, tol, rl, lt = exact(c, q.double().numpy(), visible, D ** -0.5, "chunk")
    check_lse(lse, rl, lt)
    sees = np.zeros((320, D), bool)
    for s, t, d, _ in extreme:
        sees[[i for i, (seq, n) in enumerate(visible) if seq == s and n > t], d] = True
    sees = np.broadcast_to(sees[:, None], ref.shape)
    got = out.double().cpu().numpy()
    assert not np.isnan(got).any()
    check(torch.from_numpy(np.where(sees, 0.0, got)), np.where(sees, 0.0, ref), tol, BF16, "columns that see none")
    assert sees.any() and (np.abs(ref[sees]) > 1e30).all() and (np.sign(got[sees]) == np.sign(ref[sees])).all()
