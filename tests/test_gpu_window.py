"""Windowed decode and chunked prefill against the float64 oracle.

Pages without a token that a query sees do not exist (table entries -1 or ids far outside the pool), and
other tokens' slots hold NaN, so a read of either shows.  Tolerance of bf16 outputs per element: the weights
are rounded to bf16 in front of the product with V (eps / 2 = 2^-8 of the sum of weight * |v|), the output once
more (2^-8 of its value), and scores, exponentials and sums in fp32 come to less than 2^-14 of that sum.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from helpers import BF16_LSE_ATOL, F32_ATOL

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clear_status():
    pa.metis_read_status(clear=True)
    yield


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Batch:
    """seqs: (tokens with the queried ones, queried tokens).  Decodes: a query row for every sequence."""

    def __init__(self, seed, seqs, H, G, D, bs, window, sinks, dtype=BF16, decode=False, absent=-1):
        rng = np.random.default_rng(seed)
        self.seqs, self.window, self.sinks, self.dtype, self.decode = seqs, window, sinks, dtype, decode
        self.scale = D ** -0.5
        width = max(1, max(-(-n // bs) for n, _ in seqs)) + 1
        seen = np.zeros((len(seqs), width * bs), dtype=bool)
        for s, (n, q) in enumerate(seqs):
            for p in range(n - q, n):
                seen[s, oracle.window_tokens(p, window, sinks)] = True
        held = seen.reshape(len(seqs), width, bs).any(2)
        nb = int(held.sum()) + 2
        self.table = np.full((len(seqs), width), absent)
        self.table[held] = rng.permutation(nb)[: held.sum()]
        k, v = (torch.from_numpy(rng.standard_normal((nb, bs, G, D))).to(dtype) for _ in range(2))
        free = np.ones((nb, bs), dtype=bool)
        free[self.table[held]] = ~seen.reshape(len(seqs), width, bs)[held]
        k[torch.from_numpy(free)] = float("nan")
        v[torch.from_numpy(free)] = float("nan")
        self.k, self.v = k, v
        self.lens = np.array([n for n, _ in seqs])
        self.cu = np.concatenate([[0], np.cumsum([q for _, q in seqs])])
        rows = len(seqs) if decode else int(self.cu[-1])
        self.q = torch.from_numpy(rng.standard_normal((rows, H, D))).to(dtype)

    def slot(self, s, t):
        bs = self.k.shape[1]
        return int(self.table[s, t // bs]), t % bs

    def want(self):
        args = self.k, self.v, self.table, self.lens, self.scale, self.window, self.sinks
        if self.decode:
            return oracle.paged_window_decode(self.q, *args)
        return oracle.paged_window(self.q, self.cu, *args)

    def run(self, **kw):
        cache = self.k.to(DEV), self.v.to(DEV), i32(self.table), i32(self.lens)
        kw.setdefault("max_seq_len", max(1, int(self.lens.max())))
        if self.decode:
            return pa.metis_paged_attn_decode_window(self.q.to(DEV), *cache, self.scale, self.window, self.sinks,
                                                     want_lse=True, **kw)
        return pa.metis_paged_attn_prefill_chunk_window(self.q.to(DEV), i32(self.cu), *cache, self.scale, self.window,
                                                        self.sinks, want_lse=True, **kw)

    def check(self, status=0, **kw):
        out, lse = self.run(**kw)
        torch.cuda.synchronize()
        assert pa.metis_read_status() == status
        compare(out, lse, self.want(), self.dtype)


def compare(out, lse, want, dtype):
    o, l, size = want
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    fine = np.isfinite(o)
    assert np.array_equal(np.isfinite(got), fine), np.argwhere(np.isfinite(got) != fine)[:5]
    tol = np.full(o.shape, F32_ATOL) if dtype == F32 else (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * np.abs(o)
    d = np.abs(np.where(fine, got - np.where(fine, o, 0), 0))
    bad = d > np.where(fine, tol, 1)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], d[bad][0], tol[bad][0])
    assert np.array_equal(np.isneginf(gl), np.isneginf(l))
    live = ~np.isneginf(l)
    assert np.abs(gl[live] - l[live]).max(initial=0) <= (F32_ATOL if dtype == F32 else BF16_LSE_ATOL)


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 127, 128, 129, 300, 0]


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (15, 0), (16, 16), (17, 3), (33, 100), (64, 4), (100, 17),
                                          (128, 0), (1000, 1000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("H,G,D,bs,dtype", [(8, 2, 128, 16, BF16), (6, 2, 64, 32, BF16), (4, 1, 64, 16, F32),
                                            (7, 1, 128, 64, F32)])
def test_decode_parity(window, sinks, H, G, D, bs, dtype):
    Batch(window % 97 + sinks % 89, [(n, min(n, 1)) for n in LENS], H, G, D, bs, window, sinks, dtype, True).check()


@pytest.mark.parametrize("S,H,G,D,bs,window,sinks", [
    (1, 32, 8, 128, 16, 700, 4),     # few items: each shared by eight CTAs
    (3, 8, 8, 64, 64, 1500, 130),
    (5, 28, 4, 128, 32, 513, 1),
    (40, 16, 8, 64, 16, 90, 33),     # one CTA an item
    (130, 8, 4, 128, 16, 40, 2),     # more than the ranked ones
    (700, 16, 4, 128, 16, 40, 2),    # a warp walks items: short windows,
    (700, 4, 4, 64, 32, 70, 20),
    (2500, 7, 1, 128, 16, 33, 0),
])
def test_decode_batches(S, H, G, D, bs, window, sinks):
    rng = np.random.default_rng(S)
    lens = rng.integers(1, 2000, S)
    lens[0] = 1999
    lens[rng.integers(1, S, S // 50)] = 0
    Batch(S, [(int(n), min(int(n), 1)) for n in lens], H, G, D, bs, window, sinks, decode=True, absent=10 ** 6).check()


def test_decode_of_long_sequences_reads_only_the_window():
    """A million cached tokens per sequence, of which 600 pages exist."""
    Batch(8, [(1 << 20, 1), ((1 << 20) - 5, 1)], 8, 2, 128, 16, 9000, 100, decode=True, absent=-7).check()


CHUNKS = [
    [(40, 40), (200, 1), (333, 100), (0, 0), (1, 1), (130, 130)],
    [(700, 5), (129, 128), (512, 64), (65, 65), (1000, 1)],
]


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 2), (33, 0), (64, 5), (100, 130), (128, 0), (129, 1), (300, 16),
                                          (5000, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("H,G,D,bs,which", [(8, 2, 128, 16, 0), (4, 4, 64, 32, 0), (16, 1, 128, 64, 1), (8, 1, 64, 16, 1),
                                            (4, 2, 128, 32, 1)])
def test_prefill_parity(window, sinks, H, G, D, bs, which):
    Batch(window % 91 + sinks % 83 + H, CHUNKS[which], H, G, D, bs, window, sinks).check()


@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (2, 2, 64)])
def test_prefill_of_many_units(H, G, D):
    """Several units per SM, first tokens and window tiles far apart, decodes beside."""
    rng = np.random.default_rng(H)
    seqs = [(int(rng.integers(400, 900)), int(rng.integers(1, 300))) for _ in range(20)]
    seqs += [(int(rng.integers(1, 3000)), 1) for _ in range(12)]
    Batch(77, seqs, H, G, D, 16, 150, 9, absent=2 ** 31 - 1).check()


def test_long_prefix():
    Batch(5, [(20000, 150), (9000, 70)], 8, 2, 128, 16, 2000, 200).check()


@pytest.mark.parametrize("H,G,D,window,sinks", [(8, 2, 128, 50, 3), (4, 4, 64, 20, 0), (2, 2, 128, 200, 300),
                                                (16, 1, 64, 300, 0), (4, 1, 128, 1, 1)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_values_of_unseen_tokens_do_not_reach_a_row(H, G, D, window, sinks, value):
    """V elements of tokens inside the chunk and the window: the rows that see them have them in their column
    (weights that round to nothing aside), the others do not."""
    b = Batch(int(window + D), [(400, 300), (90, 90), (250, 40)], H, G, D, 16, window, sinks)
    rng = np.random.default_rng(3)
    for s, (n, q) in enumerate(b.seqs):
        for t in rng.integers(max(0, n - q - window + 1), n, 12):
            page, off = b.slot(s, int(t))
            b.v[page, off, rng.integers(G), rng.integers(D)] = value
    b.v[b.slot(1, 89)] = value  # the last token's whole row
    b.check()


def test_keys_of_unseen_tokens_do_not_reach_a_row():
    b = Batch(4, [(400, 300)], 8, 2, 128, 16, 60, 2)
    b.k[b.slot(0, 250)] = float("nan")
    out, lse = b.run()
    rows = np.arange(100, 400)
    sees = (rows >= 250) & (rows < 310)
    got = torch.isfinite(out).all(2).all(1).cpu().numpy()
    assert np.array_equal(got, ~sees) and np.array_equal(torch.isfinite(lse).all(1).cpu().numpy(), ~sees)


def test_units_whose_queries_all_see_every_key():
    """The last query of 65 that end at a tile's last key: a unit without a tile to look at, behind units
    of the same SM in which infinities and NaN were noted."""
    b = Batch(21, [(128, 65)] * 160 + [(256, 65)] * 8, 8, 2, 128, 16, 10 ** 6, 0)
    rng = np.random.default_rng(4)
    for s, (n, q) in enumerate(b.seqs):
        if s % 4:
            page, off = b.slot(s, int(rng.integers(n - q + 1, n)))
            b.v[page, off, rng.integers(2), rng.integers(128)] = (float("nan"), float("inf"))[s % 2]
    b.check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-20, 4.0])
def test_scales(scale):
    for decode in (True, False):
        b = Batch(6, [(300, 1 if decode else 120), (40, 1 if decode else 40)], 8, 2, 128, 16, 100, 4, decode=decode)
        b.scale = scale
        b.check()


def test_a_window_over_everything_is_the_plain_call():
    rng = np.random.default_rng(9)
    seqs = [(int(n), int(min(n, m))) for n, m in zip(rng.integers(1, 900, 12), rng.integers(1, 200, 12))]
    b = Batch(9, seqs, 8, 2, 128, 16, 10 ** 9, 0)
    cache = b.k.to(DEV), b.v.to(DEV), i32(b.table), i32(b.lens)
    plain, pl = pa.metis_paged_attn_prefill_chunk(b.q.to(DEV), i32(b.cu), *cache, b.scale, max_seq_len=900, want_lse=True)
    out, lse = b.run()
    assert torch.equal(out, plain) and torch.equal(lse, pl)


def test_rows_of_no_sequence_are_left_and_bad_contents_flagged():
    b = Batch(10, [(100, 50), (60, 1), (80, 30)], 8, 2, 64, 16, 40, 2)
    out = torch.full((b.q.shape[0], 8, 64), 7.0, dtype=BF16, device=DEV)
    cu = b.cu.copy()
    cu[2:] -= 1  # the second sequence has no row, the last row belongs to none
    cache = b.k.to(DEV), b.v.to(DEV), i32(b.table), i32(b.lens)
    pa.metis_paged_attn_prefill_chunk_window(b.q.to(DEV), i32(cu), *cache, b.scale, 40, 2, max_seq_len=100, out=out)
    assert (out[-1] == 7).all() and not (out[:-1] == 7).all(2).any() and pa.metis_read_status() == 0
    table = b.table.copy()
    table[0, 5] = 10 ** 6
    pa.metis_paged_attn_prefill_chunk_window(b.q.to(DEV), i32(b.cu), *cache[:2], i32(table), cache[3], b.scale, 40, 2,
                                             max_seq_len=100)
    assert pa.metis_read_status() == pa.STATUS_BAD_BLOCK_ID
    q = b.q[:3].to(DEV)
    pa.metis_paged_attn_decode_window(q, *cache[:2], i32(table), cache[3], b.scale, 40, 2, max_seq_len=100)
    assert pa.metis_read_status() == pa.STATUS_BAD_BLOCK_ID
    pa.metis_paged_attn_decode_window(q, *cache, b.scale, 40, 2, max_seq_len=90)
    assert pa.metis_read_status() == pa.STATUS_SEQ_TOO_LONG
    pa.metis_paged_attn_prefill_chunk_window(b.q.to(DEV), i32(b.cu + 1000), *cache, b.scale, 40, 2, max_seq_len=100)
    assert pa.metis_read_status() == pa.STATUS_BAD_OFFSETS


def test_captured_and_replayed_twice_at_once():
    """Two captured calls of one kind share no memory but their inputs; lengths change between replays."""
    rng = np.random.default_rng(11)
    seqs = [(int(n), 1) for n in rng.integers(300, 600, 6)]
    d = Batch(11, seqs, 8, 2, 128, 16, 10 ** 6, 0, decode=True)  # every page is there
    c = Batch(12, [(n, 100) for n, _ in seqs], 8, 2, 128, 16, 10 ** 6, 0)
    graphs, streams, runs = [], [torch.cuda.Stream() for _ in range(4)], []
    for b in (d, c):
        q, k, v, table, lens, cu = b.q.to(DEV), b.k.to(DEV), b.v.to(DEV), i32(b.table), i32(b.lens), i32(b.cu)
        for window, sinks in ((70, 3), (250, 0)):
            out = torch.empty_like(q)
            ws = torch.empty(max(256, pa.metis_prefill_workspace_bytes(6, q.shape[0], 8, 2)), dtype=torch.uint8, device=DEV)

            def call(q=q, k=k, v=v, table=table, lens=lens, cu=cu, out=out, ws=ws, b=b, window=window, sinks=sinks):
                if b.decode:
                    pa.metis_paged_attn_decode_window(q, k, v, table, lens, b.scale, window, sinks, out=out, max_seq_len=600)
                else:
                    pa.metis_paged_attn_prefill_chunk_window(q, cu, k, v, table, lens, b.scale, window, sinks, out=out,
                                                             max_seq_len=600, workspace=ws)
            runs.append((call, out, lens))
    torch.cuda.synchronize()
    for (call, _, _), st in zip(runs, streams):
        with torch.cuda.stream(st):
            call()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        graphs.append(g)
    for step in range(3):
        for _, _, lens in runs[::2]:
            lens.sub_(17)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        got = [out.clone() for _, out, _ in runs]
        for (call, out, _), seen in zip(runs, got):
            call()
            assert torch.equal(out, seen)
    assert pa.metis_read_status() == 0


def test_refusals():
    b = Batch(13, [(40, 1)], 8, 2, 64, 16, 10, 0, decode=True)
    q, cache = b.q.to(DEV), (b.k.to(DEV), b.v.to(DEV), i32(b.table), i32(b.lens))
    for window, sinks in ((0, 0), (-1, 0), (5, -1)):
        with pytest.raises(pa.MetisError):
            pa.metis_paged_attn_decode_window(q, *cache, 0.1, window, sinks, max_seq_len=40)
        with pytest.raises(pa.MetisError):
            pa.metis_paged_attn_prefill_chunk_window(q, i32([0, 1]), *cache, 0.1, window, sinks, max_seq_len=40)
    with pytest.raises(TypeError):
        pa.metis_paged_attn_decode_window(q.float(), *cache, 0.1, 4, max_seq_len=40)
    with pytest.raises(ValueError):
        pa.metis_paged_attn_decode_window(q, cache[0], cache[1], cache[2], i32([40, 1]), 0.1, 4, max_seq_len=40)
    with pytest.raises(pa.MetisError):
        pa.metis_paged_attn_prefill_chunk_window(q.float(), i32([0, 1]), cache[0].float(), cache[1].float(), *cache[2:], 0.1,
                                                 4, max_seq_len=40)
    empty, _ = pa.metis_paged_attn_decode_window(q[:0], *cache[:2], cache[2][:0], cache[3][:0], 0.1, 4, max_seq_len=1)
    assert empty.shape == (0, 8, 64)
