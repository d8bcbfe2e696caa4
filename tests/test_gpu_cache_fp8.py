"""GPU parity of the 8-bit cache's operators: the quantising write and the read-back bit for
bit, decode and chunked prefill against softmax attention in float64 over the same codes.

Tolerances of the attention outputs (derived, not tuned).  With w the exact softmax
weights of a row and A = sum_t w_t |v_t| per output column:

* scores are fp32 sums of exact products.  A sum of D products, added 16 or 32 at a time in
  the tensor core with at most one unit of 2^-23 of the partial sums lost per addition,
  is off by at most 24 * 2^-23 < 2^-18 of sum |q k|; the multiplication by the scales, the
  subtraction of the maximum and ex2.approx add less than 2^-21 (1 + sum |q k| scale).
  Prefill chunks take the query as two e4m3 parts at one power of two, the row's largest
  element in [2^7, 2^8): an element is off by at most half of e4m3's smallest step, 2^-10,
  that is 2^-17 of the largest.  So ds = 2^-18 T + 2^-20 (+ 2^-17 U for prefill) bounds the
  error of a score, T = |scale| max_t sum_d |q_d k_td|, U = |scale| max_d |q_d| max_t sum_d |k_td|,
  and a weight is off by a factor within 1 +- 2 ds (numerator and denominator): 2 ds A.
* each weight is rounded once for the P V product: bf16 2^-8 (half a step, relative; chunks),
  fp16 2^-11 (decode, bf16 queries), two fp16 parts 2^-21 (fp32): that times A.  fp16 weights
  are also off by up to 2^-25 where the largest w 2^vb (vb: V's page exponent) of the
  tokens is 2^14 or more: at most B = 2^-39 max(w 2^vb) sum_t |code_t|.
* the accumulation of P V and the merges: less than 2^-16 A for the lengths here.
* the result is rounded once: 2^-8 |o| for bf16.

lse: ds plus 2^-21 |lse| for log2 and the final product.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def deal(rng, lens, bs, extra=3):
    """A block table over a pool with `extra` pages that no sequence owns."""
    pages = [-(-int(n) // bs) for n in lens]
    nb = sum(pages) + extra
    perm = rng.permutation(nb)
    table = np.full((len(lens), max(1, max(pages))), -1, np.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    return table, nb


def pool(rng, nb, bs, G, D, spread=2.0):
    """Codes and bytes of a pool whose pages and heads differ in size by up to 2^(2 spread)."""
    x = rng.standard_normal((nb, bs, G, D)) * 2.0 ** rng.uniform(-spread, spread, (nb, 1, G, 1))
    return oracle.quantize_pages(x)


def poison(codes, bytes_, table, lens, bs):
    """NaN codes in every slot no token owns, NaN scales in the pages no sequence owns."""
    codes, bytes_ = codes.copy(), bytes_.copy()
    free = np.ones(codes.shape[:2], bool)
    for s, n in enumerate(lens):
        t = np.arange(int(n))
        free[table[s, t // bs], t % bs] = False
    codes[free] = 0x7F
    bytes_[free.all(axis=1)] = 255
    return codes, bytes_


def gpu(x, dtype=None):
    t = x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))
    return t.to(DEV) if dtype is None else t.to(DEV, dtype)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Cache:
    """A K and a V pool on the GPU with the oracle's view of both."""

    def __init__(self, rng, lens, G, D, bs, spread=2.0, poisoned=True, extra=3):
        self.bs, self.G, self.D, self.lens = bs, G, D, list(lens)
        self.table, self.nb = deal(rng, lens, bs, extra)
        self.k, self.ks = pool(rng, self.nb, bs, G, D, spread)
        self.v, self.vs = pool(rng, self.nb, bs, G, D, spread)
        if poisoned:
            self.k, self.ks = poison(self.k, self.ks, self.table, lens, bs)
            self.v, self.vs = poison(self.v, self.vs, self.table, lens, bs)
        self.put()

    def put(self):
        self.dev = [gpu(self.k).view(torch.float8_e4m3fn), gpu(self.v).view(torch.float8_e4m3fn), gpu(self.ks),
                    gpu(self.vs)]
        self.bt = i32(self.table)
        self.sl = i32(self.lens)

    def rows(self, s, n, which):
        """The first n tokens of sequence s as float64 [n, G, D]."""
        codes, b = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        t = np.arange(n)
        page = self.table[s, t // self.bs]
        return oracle.E4M3_VALUES[codes[page, t % self.bs]] * (2.0 ** (b[page].astype(np.float64) - 127))[:, :, None]


STEP = {BF16: 2.0 ** -11, F32: 2.0 ** -21}  # decode's rounding of a weight
CHUNK_STEP = 2.0 ** -8                      # prefill's


def attention(cache, q, rows, scale, p_step, parts=False):
    """q [R, H, D] float64; rows[i] = (sequence, visible tokens).  Returns out, its bound
    without the final rounding, lse and its bound.  parts: queries as two e4m3 parts."""
    R, H, D = q.shape
    r = H // cache.G
    out, tol = np.zeros((R, H, D)), np.zeros((R, H, D))
    lse, ltol = np.full((R, H), -np.inf), np.zeros((R, H))
    kept = {}
    for i, (s, n) in enumerate(rows):
        if n == 0:
            continue
        if s not in kept:
            L = cache.lens[s]
            t = np.arange(L)
            kept = {s: (cache.rows(s, L, "k"), cache.rows(s, L, "v"),
                        2.0 ** (cache.vs[cache.table[s, t // cache.bs]].astype(np.float64) - 127))}
        k, v, unit = (x[:n] for x in kept[s])
        for h in range(H):
            g = h // r
            z = scale * (k[:, g] @ q[i, h])
            m = z.max()
            e = np.exp(z - m)
            w = e / e.sum()
            out[i, h] = w @ v[:, g]
            lse[i, h] = m + np.log(e.sum())
            ds = 2.0 ** -18 * abs(scale) * (np.abs(k[:, g]) @ np.abs(q[i, h])).max() + 2.0 ** -20
            if parts:
                ds += 2.0 ** -17 * abs(scale) * np.abs(q[i, h]).max() * np.abs(k[:, g]).sum(axis=1).max()
            B = 2.0 ** -39 * (w * unit[:, g]).max() * (np.abs(v[:, g]) / unit[:, g, None]).sum(axis=0)
            tol[i, h] = (2 * ds + p_step + 2.0 ** -16) * (w @ np.abs(v[:, g])) + B
            ltol[i, h] = ds + 2.0 ** -21 * abs(lse[i, h])
    return out, tol, lse, ltol


def check(got, ref, tol, dtype, what):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), f"{what}: non-finite values"
    bound = tol + np.abs(ref) * (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) + 1e-37
    worst = np.unravel_index(np.argmax(np.abs(g - ref) - bound), g.shape)
    assert (np.abs(g - ref) <= bound).all(), \
        f"{what}: off by {abs(g - ref)[worst]:.3e} at {worst}, bound {bound[worst]:.3e}"


def check_lse(got, ref, tol):
    g = got.double().cpu().numpy()
    fin = np.isfinite(ref)
    assert np.array_equal(g[~fin], ref[~fin])
    assert (np.abs(g[fin] - ref[fin]) <= tol[fin]).all(), f"lse off by {np.abs(g[fin] - ref[fin]).max():.3e}"


# ---------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------
def write_case(rng, spans, G, D, bs, dtype, size=1.0, tail=0):
    """spans: (cached tokens with the new ones, new ones) per sequence; `tail` rows behind the last sequence."""
    lens = [n for n, _ in spans]
    table, nb = deal(rng, lens, bs)
    cu = np.concatenate([[0], np.cumsum([q for _, q in spans])])
    x = []
    for _ in range(2):
        t = rng.standard_normal((int(cu[-1]) + tail, G, D)) * size * 2.0 ** rng.uniform(-3, 3, (int(cu[-1]) + tail, G, 1))
        x.append(torch.from_numpy(t).to(dtype))
    caches = [pool(rng, nb, bs, G, D) for _ in range(2)]
    return table, cu, lens, x, caches


def run_write(table, cu, lens, x, caches):
    dev = [gpu(caches[0][0]), gpu(caches[1][0]), gpu(caches[0][1]), gpu(caches[1][1])]
    pa.metis_reshape_and_cache_fp8(gpu(x[0]), gpu(x[1]), *dev, i32(cu), i32(table), i32(lens))
    return dev


def check_write(dev, table, cu, lens, x, caches):
    for w in range(2):
        codes, b = oracle.write_cache(x[w], *caches[w], cu, table, lens)
        assert np.array_equal(dev[2 + w].cpu().numpy(), b), "scale bytes"
        assert np.array_equal(dev[w].cpu().numpy(), codes), "codes"


@pytest.mark.parametrize("G,D,bs,dtype", [
    (8, 128, 16, BF16), (1, 64, 16, F32), (3, 64, 32, BF16), (4, 128, 64, F32), (5, 128, 32, F32), (2, 64, 64, BF16),
    (17, 128, 16, BF16), (1, 128, 64, BF16),
])
def test_write_parity_bitwise(G, D, bs, dtype):
    rng = np.random.default_rng(G * D + bs)
    spans = [(5, 5), (1, 1), (0, 0), (bs, bs), (bs + 1, 1), (2 * bs + 3, bs + 7), (0, 0), (100, 37), (3 * bs - 1, 1),
             (77, 77), (bs - 1, 1), (200, 128), (64, 0)]
    case = write_case(rng, spans, G, D, bs, dtype, tail=3)
    pa.metis_read_status(clear=True)
    dev = run_write(*case)
    check_write(dev, *case)
    assert pa.metis_read_status() == 0


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 30, 2.0 ** -118])
def test_write_of_rows_far_smaller_or_larger_than_the_page(size):
    """Scales that grow by 2^30 (every earlier code becomes zero) or stay; fp32 subnormal-sized rows."""
    rng = np.random.default_rng(7)
    case = write_case(rng, [(20, 3), (40, 40), (17, 1)], 2, 64, 32, F32, size=size)
    check_write(run_write(*case), *case)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_of_non_finite_and_zero_rows(dtype):
    rng = np.random.default_rng(8)
    table, cu, lens, x, caches = write_case(rng, [(30, 12), (6, 6), (33, 1)], 2, 128, 16, dtype)
    for t in x:
        t[3, 0, 5] = float("nan")
        t[4, 1, 6] = float("inf")
        t[5, 1, 7] = -float("inf")
        t[12:18, 1] = 0.0
        t[18, 0] = float("inf")  # a row without a finite value in its page
    check_write(run_write(table, cu, lens, x, caches), table, cu, lens, x, caches)


def test_write_in_several_calls():
    """A prompt written in odd pieces: each call's result feeds the next."""
    rng = np.random.default_rng(9)
    bs, G, D = 32, 3, 64
    full = [(150, 150), (61, 61)]
    table, cu, lens, x, caches = write_case(rng, full, G, D, bs, BF16)
    dev = [gpu(caches[0][0]), gpu(caches[1][0]), gpu(caches[0][1]), gpu(caches[1][1])]
    ref = caches
    done = np.zeros(2, int)
    for step in ([1, 1], [30, 0], [1, 31], [45, 2], [73, 27]):
        rows = [torch.cat([x[w][cu[s] + done[s]:cu[s] + done[s] + step[s]] for s in range(2)]) for w in range(2)]
        done += step
        c = np.concatenate([[0], np.cumsum(step)])
        pa.metis_reshape_and_cache_fp8(gpu(rows[0]), gpu(rows[1]), *dev, i32(c), i32(table), i32(done))
        ref = [oracle.write_cache(rows[w], *ref[w], c, table, done) for w in range(2)]
        for w in range(2):
            assert np.array_equal(dev[w].cpu().numpy(), ref[w][0]) and np.array_equal(dev[2 + w].cpu().numpy(), ref[w][1])
    assert (done == lens).all()


def test_write_of_many_sequences():
    """More sequences than one round of the item search covers (32 * 32 < 1100)."""
    rng = np.random.default_rng(10)
    spans = [(int(n), int(min(n, q))) for n, q in zip(rng.integers(0, 40, 1100), rng.integers(0, 25, 1100))]
    case = write_case(rng, spans, 1, 64, 16, BF16)
    check_write(run_write(*case), *case)


def test_write_bad_contents_are_flagged_and_not_written():
    rng = np.random.default_rng(11)
    bs, G, D = 16, 2, 64
    table, cu, lens, x, caches = write_case(rng, [(20, 5), (18, 4), (40, 7), (9, 9)], G, D, bs, BF16)
    good = (table.copy(), cu.copy(), list(lens))

    def attempt(bit, table, cu, lens, keep):
        """`keep`: the sequences that must still be written."""
        pa.metis_read_status(clear=True)
        dev = run_write(table, cu, lens, x, caches)
        assert pa.metis_read_status(clear=True) & bit
        for w in range(2):
            ref = caches[w]
            for s in keep:
                n = good[1][s + 1] - good[1][s]
                ref = oracle.write_cache(x[w][good[1][s]:good[1][s + 1]], *ref, [0, n], good[0][s:s + 1], good[2][s:s + 1])
            assert np.array_equal(dev[w].cpu().numpy(), ref[0]) and np.array_equal(dev[2 + w].cpu().numpy(), ref[1])

    t = table.copy()
    t[1, 0] = caches[0][0].shape[0]  # past the pool: sequence 1's first page is lost, its second is written
    pa.metis_read_status(clear=True)
    run_write(t, cu, lens, x, caches)
    assert pa.metis_read_status(clear=True) & pa.STATUS_BAD_BLOCK_ID
    t[1] = -1
    attempt(pa.STATUS_BAD_BLOCK_ID, t, cu, lens, [0, 2, 3])
    attempt(pa.STATUS_BAD_Q_LEN, table, cu, [20, 3, 40, 9], [0, 2, 3])
    attempt(pa.STATUS_SEQ_TOO_LONG, table, cu, [20, 18, 49, 9], [0, 1, 3])
    attempt(pa.STATUS_BAD_OFFSETS, table, np.array([0, 5, 9, 16, 26]), [20, 18, 40, 10], [0, 1, 2])


# ---------------------------------------------------------------------------
# read back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("G,D,bs,dtype", [(8, 128, 16, BF16), (1, 64, 16, F32), (3, 64, 32, BF16), (5, 128, 64, F32)])
def test_gather_parity_bitwise(G, D, bs, dtype):
    rng = np.random.default_rng(G + D + bs)
    lens = [0, 1, 15, 16, 17, bs, bs + 1, 0, 333, 2 * bs]
    c = Cache(rng, lens, G, D, bs, spread=20.0)
    # rows in another order than the sequences, with gaps
    order = rng.permutation(len(lens))
    offs, at = np.zeros(len(lens), int), 2
    for s in order:
        offs[s] = at
        at += lens[s] + 3
    outs = [torch.full((at, G, D), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    pa.metis_read_status(clear=True)
    pa.metis_gather_cache_fp8(*c.dev, c.bt, c.sl, i32(offs), k_out=outs[0], v_out=outs[1])
    for w, out in zip("kv", outs):
        ref = np.full((at, G, D), 7.0)
        for s, n in enumerate(lens):
            ref[offs[s]:offs[s] + n] = c.rows(s, n, w)
        assert torch.equal(out.cpu(), torch.from_numpy(ref).to(dtype))
    assert pa.metis_read_status() == 0


def test_gather_bad_contents():
    rng = np.random.default_rng(3)
    c = Cache(rng, [40, 33, 50], 2, 64, 16)
    bad = c.table.copy()
    bad[1, 1] = c.nb
    offs = [0, 40, 73]
    pa.metis_read_status(clear=True)
    k, v = pa.metis_gather_cache_fp8(*c.dev, i32(bad), c.sl, i32(offs), num_rows=123, out_dtype=F32)
    assert pa.metis_read_status(clear=True) == pa.STATUS_BAD_BLOCK_ID
    ref = np.concatenate([c.rows(s, n, "k") for s, n in enumerate(c.lens)])
    ref[40 + 16:40 + 32] = 0.0
    assert np.array_equal(k.double().cpu().numpy(), ref)
    # rows past the end, and before the start, are not written
    out = [torch.full((60, 2, 64), 7.0, device=DEV) for _ in range(2)]
    pa.metis_gather_cache_fp8(*c.dev, c.bt, c.sl, i32([20, -4, 1 << 30]), k_out=out[0], v_out=out[1], max_seq_len=64)
    assert pa.metis_read_status(clear=True) == pa.STATUS_BAD_OFFSETS
    ref = np.full((60, 2, 64), 7.0)
    ref[0:29] = c.rows(1, 33, "v")[4:]
    ref[29:60] = c.rows(0, 40, "v")[9:]
    got = out[1].double().cpu().numpy()
    # rows 20 .. 28 belong to two sequences here
    assert np.array_equal(got[:20], ref[:20]) and np.array_equal(got[29:], ref[29:])
    # tokens past max_seq_len are not read
    k, _ = pa.metis_gather_cache_fp8(*c.dev, c.bt, c.sl, i32(offs), num_rows=123, out_dtype=F32, max_seq_len=35)
    assert pa.metis_read_status(clear=True) == pa.STATUS_SEQ_TOO_LONG
    assert np.array_equal(k[73:73 + 35].double().cpu().numpy(), c.rows(2, 35, "k"))


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 65, 127, 129, 200, 511, 700]


def decode_case(rng, lens, r, G, D, bs, dtype, scale=None, spread=2.0, partition=0, max_len=None, workspace=None):
    c = Cache(rng, lens, G, D, bs, spread)
    q = torch.from_numpy(rng.standard_normal((len(lens), G * r, D))).to(dtype)
    scale = D ** -0.5 if scale is None else scale
    pa.metis_read_status(clear=True)
    out, lse = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, c.sl, scale, partition_size=partition,
                                              max_seq_len=max_len, workspace=workspace, want_lse=True)
    ref, tol, rl, lt = attention(c, q.double().numpy(), list(enumerate(lens)), scale,
                                 STEP[dtype])
    check(out, ref, tol, dtype, "out")
    check_lse(lse, rl, lt)
    assert pa.metis_read_status() == 0
    return out


@pytest.mark.parametrize("r,G,D,bs,dtype", [
    (4, 8, 128, 16, BF16), (1, 1, 64, 16, BF16), (2, 3, 128, 32, BF16), (3, 2, 64, 64, BF16), (5, 1, 128, 64, BF16),
    (6, 2, 64, 32, BF16), (7, 4, 128, 32, BF16), (8, 2, 128, 16, BF16), (8, 1, 64, 64, BF16),
    (4, 1, 64, 16, F32), (7, 2, 128, 32, F32), (8, 1, 128, 64, F32), (1, 3, 64, 32, F32), (3, 2, 128, 16, F32),
])
@pytest.mark.parametrize("partition", [0, 48, 256])
def test_decode_parity(r, G, D, bs, dtype, partition):
    decode_case(np.random.default_rng(r * 100 + G + D + bs + partition), LENS, r, G, D, bs, dtype, partition=partition)


def test_decode_unranked_batch():
    """More sequences than the longest-first ranking takes."""
    rng = np.random.default_rng(2)
    decode_case(rng, list(rng.integers(0, 90, 200)), 2, 1, 64, 16, BF16)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (128, F32), (64, F32)])
@pytest.mark.parametrize("partition", [0, 16, 256])
def test_decode_more_items_than_sms(D, dtype, partition):
    """The plans for large batches: several warps per item, and (many partitions) one."""
    rng = np.random.default_rng(D + partition)
    lens = [0, 1, 1100] + [int(n) for n in rng.integers(1, 400, 20)]
    decode_case(rng, lens, 2, 8, D, 16, dtype, partition=partition)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (128, F32), (64, F32)])
@pytest.mark.parametrize("S", [1, 3, 12])
def test_decode_unsplit_with_sms_to_spare(D, dtype, S):
    """8 to 96 items: several CTAs for each of them (lengths far below the bound, and above them all), or one."""
    rng = np.random.default_rng(S + D)
    for lens, max_len in (([2100] + [257] * (S - 1), None), ([700, 0, 1][:S] + [31] * (S - 3), 5000),
                          ([127, 255, 256][:S] + [100] * (S - 3), None)):
        decode_case(rng, lens, 2, 8, D, 32, dtype, max_len=max_len)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (128, F32), (64, F32)])
@pytest.mark.parametrize("partition", [16, 80, 1024])
def test_decode_few_partitions_joined_in_one_launch(D, dtype, partition):
    """Up to eight partitions of few items: none, one, a part of one, all of them, and a bound on the
    lengths that leaves the last ones empty."""
    rng = np.random.default_rng(partition + D)
    P = partition
    for lens, parts in (([0, 1, P - 1, P, P + 1], 2), ([2 * P + 5, 0, 5 * P - 1], 8), ([7 * P + 3], 8), ([P // 2, 3], 1)):
        for r in (1, 3, 8):
            decode_case(rng, lens, r, 2, D, 16, dtype, partition=P, max_len=parts * P)


def test_decode_joined_partitions_of_a_sequence_past_the_bound():
    rng = np.random.default_rng(77)
    lens, D = [300, 90], 64
    c = Cache(rng, lens, 1, D, 16)
    q = torch.from_numpy(rng.standard_normal((2, 4, D))).to(BF16)
    pa.metis_read_status(clear=True)
    out, lse = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, c.sl, 0.125, partition_size=64, max_seq_len=256,
                                              want_lse=True)
    assert pa.metis_read_status(clear=True) == pa.STATUS_SEQ_TOO_LONG  # the first 256 tokens are read
    c.lens = [256, 90]
    ref, tol, rl, lt = attention(c, q.double().numpy(), [(0, 256), (1, 90)], 0.125, STEP[BF16])
    check(out, ref, tol, BF16, "out")
    check_lse(lse, rl, lt)


def test_decode_windows_of_32_units():
    """Sequences whose warps walk several windows of block ids (one warp: 32 units of 32 tokens each)."""
    rng = np.random.default_rng(15)
    for bs in (16, 64):
        decode_case(rng, [9000, 8192, 8191, 1], 1, 1, 64, bs, BF16)
        decode_case(rng, [5000, 4100], 2, 1, 128, bs, BF16, partition=4096)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bs", [16, 32])
def test_decode_scales_of_any_spread(dtype, bs):
    """Pages that differ by up to 2^60: each page's factor is applied in fp32."""
    decode_case(np.random.default_rng(4), [400, 90, 33], 4, 2, 128, bs, dtype, scale=2.0 ** -30, spread=30.0)


@pytest.mark.parametrize("partition", [0, 512])
def test_decode_long_flat_tail_beside_one_large_weight(partition):
    """One token 2^18 times as heavy as each of 6,000 others: their sum still counts."""
    rng = np.random.default_rng(14)
    n, D, bs = 6000, 64, 16
    c = Cache(rng, [n], 1, D, bs, spread=0.0)
    t = np.arange(n)
    page = c.table[0, t // bs]
    c.k[page, t % bs, 0] = 0
    c.k[page[0], 0, 0] = oracle.encode_e4m3(np.full(D, 1.0))
    c.ks[:] = 127
    c.put()
    q = torch.full((1, 4, D), 18.0 * np.log(2) / D).to(BF16)
    for dtype in (BF16, F32):
        out, lse = pa.metis_paged_attn_decode_fp8(gpu(q, dtype), *c.dev, c.bt, c.sl, 1.0, partition_size=partition,
                                                  want_lse=True)
        ref, tol, rl, lt = attention(c, q.double().numpy(), [(0, n)], 1.0, STEP[dtype])
        check(out, ref, tol, dtype, "out")
        check_lse(lse, rl, lt)


@pytest.mark.parametrize("big", [127, 200])
@pytest.mark.parametrize("partition", [0, 512, 8192])
def test_decode_many_pages_of_zero_values_beside_one_of_large_ones(partition, big):
    """8,000 tokens whose V is zero (scale 2^-126) and whose weight is e^-11 of the first one's
    take part in the sum, whatever the scale of the page in front of, between or behind them."""
    rng = np.random.default_rng(big)
    n, D, bs = 8000, 128, 16
    for first in (0, 300, 499):
        c = Cache(rng, [n], 1, D, bs, spread=0.0)
        t = np.arange(n)
        page = c.table[0, t // bs]
        c.k[page, t % bs, 0] = 0
        c.k[page[first * bs], 0, 0, 0] = oracle.encode_e4m3(np.full(1, 11.0))[0]
        c.ks[:] = 127
        others = np.delete(c.table[0, :n // bs], first)
        c.v[others] = 0
        c.vs[others] = 1
        c.vs[page[first * bs]] = big
        c.put()
        q = torch.zeros((1, 4, D)).to(BF16)
        q[:, :, 0] = 1.0
        for dtype in (BF16, F32):
            out, lse = pa.metis_paged_attn_decode_fp8(gpu(q, dtype), *c.dev, c.bt, c.sl, 1.0, partition_size=partition,
                                                      want_lse=True)
            ref, tol, rl, lt = attention(c, q.double().numpy(), [(0, n)], 1.0, STEP[dtype])
            check(out, ref, tol, dtype, "out")
            check_lse(lse, rl, lt)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_decode_softmax_scales(scale):
    decode_case(np.random.default_rng(5), [300, 1, 40], 4, 2, 64, 16, BF16, scale=scale, spread=0.5)


def test_decode_query_of_any_size():
    """Rows of zeros, of 1e30 and 1e-30: the power of two that brings a row into fp16's range is undone."""
    rng = np.random.default_rng(6)
    lens = [50, 60, 70, 80]
    c = Cache(rng, lens, 2, 128, 16, spread=0.0)
    q = rng.standard_normal((4, 8, 128)) * np.array([1e30, 1e-30, 0.0, 1.0])[:, None, None]
    q[3, 2, 5] = 4096.0  # one large element beside small ones
    for dtype in (BF16, F32):
        qt = torch.from_numpy(q).to(dtype)
        for s, scale in ((0, 1e-31), (1, 1e29), (2, 1.0), (3, 0.01)):
            out, lse = pa.metis_paged_attn_decode_fp8(gpu(qt[s:s + 1]), *c.dev, c.bt[s:s + 1].contiguous(),
                                                      c.sl[s:s + 1].contiguous(), scale, want_lse=True)
            one = Cache.__new__(Cache)
            one.__dict__.update(c.__dict__)
            one.table, one.lens = c.table[s:s + 1], lens[s:s + 1]
            ref, tol, rl, lt = attention(one, qt[s:s + 1].double().numpy(), [(0, lens[s])], scale,
                                         STEP[dtype])
            check(out, ref, tol, dtype, "out")
            check_lse(lse, rl, lt)


def test_decode_nan_code_of_a_live_token_reaches_the_output():
    rng = np.random.default_rng(7)
    c = Cache(rng, [40, 40], 1, 64, 16)
    c.k[c.table[0, 1], 3, 0, 9] = 0x7F
    c.v[c.table[1, 2], 2, 0, 11] = 0xFF
    c.put()
    q = gpu(torch.from_numpy(rng.standard_normal((2, 4, 64))).to(BF16))
    out, _ = pa.metis_paged_attn_decode_fp8(q, *c.dev, c.bt, c.sl, 0.125)
    o = out.float().cpu()
    assert torch.isnan(o[0]).all()
    assert torch.isnan(o[1, :, 11]).all() and torch.isfinite(o[1, :, :11]).all() and torch.isfinite(o[1, :, 12:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("partition", [0, 16, 64, 512])
def test_decode_nan_wherever_it_stands(partition, dtype):
    """NaN codes in K and V, pages whose scale is NaN, whole units of NaN scores and a NaN query reach
    the outputs of the heads (and, of V's codes, the columns) that use them, and no others."""
    rng = np.random.default_rng(partition)
    lens, G, r, D, bs = [200, 70, 333, 16, 300, 129], 2, 3, 128, 16
    c = Cache(rng, lens, G, D, bs)
    c.k[c.table[0, 4:8], :, 0, 5] = 0x7F        # two whole units of one warp
    c.v[c.table[1, 3], 7, 1, 99] = 0xFF
    c.ks[c.table[2, 20], 1] = 255               # the last, partial page
    c.vs[c.table[4, 9], 0] = 255
    c.k[c.table[5, 8], 0, 1, 0] = 0x7F          # the last token
    c.put()
    c.k[c.table[2, 20], :, 1], c.ks[c.table[2, 20], 1] = 0x7F, 127  # the reference's view of a NaN scale
    c.v[c.table[4, 9], :, 0], c.vs[c.table[4, 9], 0] = 0x7F, 127
    q = torch.from_numpy(rng.standard_normal((len(lens), G * r, D))).to(dtype)
    q[3, 4, 17] = float("nan")
    out, lse = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, c.sl, D ** -0.5, partition_size=partition,
                                              want_lse=True)
    with np.errstate(invalid="ignore"):
        ref, tol, rl, lt = attention(c, q.double().numpy(), list(enumerate(lens)), D ** -0.5, STEP[dtype])
    o, ln = out.double().cpu().numpy(), lse.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(o), np.isnan(ref))
    np.testing.assert_array_equal(np.isnan(ln), np.isnan(rl))
    good = ~np.isnan(ref)
    assert (np.abs(o - ref)[good] <= (tol + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * np.abs(ref))[good]).all()
    assert (np.abs(ln - rl)[~np.isnan(rl)] <= lt[~np.isnan(rl)]).all()
    if dtype == BF16 and partition == 0:  # the same rows as decodes of a chunked call (ratio 3 has no chunks)
        q4 = torch.cat([q.view(-1, G, r, D), q.view(-1, G, r, D)[:, :, :1]], 2).reshape(-1, G * 4, D)
        out4, lse4 = pa.metis_paged_attn_prefill_chunk_fp8(gpu(q4), i32(np.arange(len(lens) + 1)), *c.dev, c.bt, c.sl,
                                                           D ** -0.5, want_lse=True)
        o4 = out4.double().cpu().numpy().reshape(-1, G, 4, D)[:, :, :3].reshape(o.shape)
        np.testing.assert_array_equal(np.isnan(o4), np.isnan(ref))
        assert (np.abs(o4 - ref)[good] <= (tol + 2.0 ** -8 * np.abs(ref))[good]).all()


def test_decode_bad_contents():
    rng = np.random.default_rng(8)
    lens = [70, 40]
    c = Cache(rng, lens, 2, 64, 16)
    q = torch.from_numpy(rng.standard_normal((2, 8, 64))).to(BF16)
    bad = c.table.copy()
    bad[0, 2] = -5
    pa.metis_read_status(clear=True)
    out, _ = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, i32(bad), c.sl, 0.125)
    assert pa.metis_read_status(clear=True) == pa.STATUS_BAD_BLOCK_ID
    b = c.table[0, 2]
    c.k[b], c.v[b], c.ks[b], c.vs[b] = 0, 0, 127, 127  # the page reads as zeros
    ref, tol, _, _ = attention(c, q.double().numpy(), list(enumerate(lens)), 0.125, STEP[BF16])
    check(out, ref, tol, BF16, "out")
    # longer than the table row: clamped to it
    out, _ = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, i32([999, 40]), 0.125, max_seq_len=1000,
                                            partition_size=32)
    assert pa.metis_read_status(clear=True) & pa.STATUS_SEQ_TOO_LONG
    assert torch.isfinite(out[1].float()).all()


# ---------------------------------------------------------------------------
# chunked prefill
# ---------------------------------------------------------------------------
def prefill_case(rng, spans, r, G, D, bs, scale=None, spread=2.0):
    lens = [n for n, _ in spans]
    c = Cache(rng, lens, G, D, bs, spread)
    cu = np.concatenate([[0], np.cumsum([q for _, q in spans])])
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), G * r, D))).to(BF16)
    scale = D ** -0.5 if scale is None else scale
    pa.metis_read_status(clear=True)
    out, lse = pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32(cu), *c.dev, c.bt, c.sl, scale, want_lse=True)
    rows = [(s, n - m + i + 1) for s, (n, m) in enumerate(spans) for i in range(m)]
    ref, tol, rl, lt = attention(c, q.double().numpy(), rows, scale, CHUNK_STEP, parts=True)
    check(out, ref, tol, BF16, "out")
    check_lse(lse, rl, lt)
    assert pa.metis_read_status() == 0


@pytest.mark.parametrize("r,G,D,bs", [
    (4, 2, 128, 16), (1, 2, 64, 16), (2, 1, 128, 32), (8, 1, 64, 64), (16, 1, 128, 16), (16, 1, 64, 32), (4, 1, 128, 64),
])
def test_prefill_parity(r, G, D, bs):
    rng = np.random.default_rng(r + G + D + bs)
    prefill_case(rng, [(1, 1), (130, 130), (0, 0), (300, 1), (129, 2), (260, 64), (64, 33), (17, 17), (400, 129)], r, G,
                 D, bs)


@pytest.mark.parametrize("r,G,D,bs", [(4, 8, 128, 16), (16, 8, 64, 32), (1, 8, 128, 64)])
def test_prefill_more_units_than_sms(r, G, D, bs):
    """Every SM walks several units, some with one query tile and some with two; rows sampled."""
    rng = np.random.default_rng(r + D)
    spans = [(int(n) + int(q), int(q)) for n, q in zip(rng.integers(0, 500, 12), rng.integers(60, 420, 12))]
    spans += [(300, 1), (5, 5), (33, 1)]
    lens = [n for n, _ in spans]
    c = Cache(rng, lens, G, D, bs)
    cu = np.concatenate([[0], np.cumsum([q for _, q in spans])])
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), G * r, D))).to(BF16)
    pa.metis_read_status(clear=True)
    call = lambda: pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32(cu), *c.dev, c.bt, c.sl, 0.1, want_lse=True)
    out, lse = call()
    rows = [(s, n - m + i + 1) for s, (n, m) in enumerate(spans) for i in range(m)]
    at = np.sort(rng.choice(len(rows), 40, replace=False))
    ref, tol, rl, lt = attention(c, q[torch.from_numpy(at)].double().numpy(), [rows[i] for i in at], 0.1, CHUNK_STEP,
                                 parts=True)
    check(out[torch.from_numpy(at).to(DEV)], ref, tol, BF16, "out")
    check_lse(lse[torch.from_numpy(at).to(DEV)], rl, lt)
    again, _ = call()  # the units land on other SMs: the same bits
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert pa.metis_read_status() == 0


@pytest.mark.parametrize("r,G,D,bs", [(4, 2, 128, 16), (1, 1, 64, 32), (8, 1, 64, 16), (2, 3, 128, 64), (16, 2, 128, 16)])
def test_prefill_few_chunks_split_over_their_keys(r, G, D, bs):
    """Chunks that leave most SMs idle, behind prefixes that end at, before and behind a tile's and a
    part's edge, beside short ones and decodes."""
    rng = np.random.default_rng(r + D)
    for spans in ([(3000, 70)], [(1025, 1024)], [(2560, 128), (90, 1), (700, 33)], [(1024 + 17, 17), (513, 2), (40, 40)],
                  [(4500, 3), (1300, 1), (0, 0), (5, 2)]):
        prefill_case(rng, spans, r, G, D, bs)


@pytest.mark.parametrize("r,G,D,bs,spans", [
    (8, 8, 64, 16, [(2900, 800)]),                            # 200 units: a round of whole ones, 48 in parts
    (4, 8, 128, 32, [(3700, 640)]),                           # 80 units: parts in two rounds
    (4, 8, 128, 16, [(2500, 900), (2300, 500), (90, 60), (700, 1), (40, 1)]),
])
def test_prefill_last_round_split_over_its_keys(r, G, D, bs, spans):
    rng = np.random.default_rng(D + bs)
    lens = [n for n, _ in spans]
    c = Cache(rng, lens, G, D, bs)
    cu = np.concatenate([[0], np.cumsum([q for _, q in spans])])
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), G * r, D))).to(BF16)
    pa.metis_read_status(clear=True)
    call = lambda: pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32(cu), *c.dev, c.bt, c.sl, D ** -0.5, want_lse=True)
    out, lse = call()
    rows = [(s, n - m + i + 1) for s, (n, m) in enumerate(spans) for i in range(m)]
    at = np.sort(rng.choice(len(rows), 40, replace=False))
    ref, tol, rl, lt = attention(c, q[torch.from_numpy(at)].double().numpy(), [rows[i] for i in at], D ** -0.5,
                                 CHUNK_STEP, parts=True)
    check(out[torch.from_numpy(at).to(DEV)], ref, tol, BF16, "out")
    check_lse(lse[torch.from_numpy(at).to(DEV)], rl, lt)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    for _ in range(3):  # the parts land on other SMs: the same bits
        again, lse2 = call()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    assert pa.metis_read_status() == 0


def test_prefill_split_and_whole_agree_and_repeat():
    """The same call with and without the memory for parts, and twice with it."""
    rng = np.random.default_rng(31)
    c = Cache(rng, [2900, 64, 1500], 2, 128, 16)
    q_lens = [100, 1, 300]
    cu = i32(np.concatenate([[0], np.cumsum(q_lens)]))
    q = gpu(torch.from_numpy(rng.standard_normal((401, 8, 128))).to(BF16))
    small, full = pa.metis_prefill_workspace_bytes(3, 401, 8, 2), pa.metis_prefill_fp8_workspace_bytes(3, 401, 8, 2, 128, 2900)
    assert full > small
    outs = [pa.metis_paged_attn_prefill_chunk_fp8(
        q, cu, *c.dev, c.bt, c.sl, 0.088, max_seq_len=2900, want_lse=True,
        workspace=torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV)) for n in (small, full, full)]
    assert torch.equal(outs[1][0].view(torch.int16), outs[2][0].view(torch.int16)) and torch.equal(outs[1][1], outs[2][1])
    a, b = outs[0][0].double(), outs[1][0].double()
    # each is within its bound of the exact row, 2^-7 of a weighted mean of |v| (at most 2^2 * 4.5 here) and a rounding
    assert ((a - b).abs() <= 2 * (2.0 ** -7 * 18 + 2.0 ** -8 * a.abs())).all()
    assert (outs[0][1] - outs[1][1]).abs().max() <= 1e-3


def test_prefill_chunks_only_and_decodes_only():
    rng = np.random.default_rng(20)
    prefill_case(rng, [(520, 257), (3, 3)], 4, 2, 128, 16)
    prefill_case(rng, [(n, 1) for n in (1, 16, 40, 333)], 4, 2, 128, 16)


def test_prefill_scales_of_any_spread():
    prefill_case(np.random.default_rng(21), [(300, 70), (90, 1)], 4, 2, 128, 16, scale=2.0 ** -30, spread=30.0)


def test_prefill_nan_code_of_a_live_token_reaches_the_output():
    rng = np.random.default_rng(22)
    c = Cache(rng, [40, 40], 1, 64, 16)
    c.k[c.table[0, 1], 3, 0, 9] = 0x7F
    c.v[c.table[1, 2], 2, 0, 11] = 0xFF
    c.put()
    q = gpu(torch.from_numpy(rng.standard_normal((80, 4, 64))).to(BF16))
    out, _ = pa.metis_paged_attn_prefill_chunk_fp8(q, i32([0, 40, 80]), *c.dev, c.bt, c.sl, 0.125)
    o = out.float().cpu()
    assert torch.isnan(o[19:40]).all()
    assert torch.isnan(o[40 + 34:, :, 11]).all()
    assert torch.isfinite(o[40:, :, :11]).all() and torch.isfinite(o[40:, :, 12:]).all()


@pytest.mark.parametrize("r,D,bs", [(4, 128, 16), (1, 64, 32), (8, 64, 16), (2, 128, 64)])
def test_prefill_nan_of_a_token_reaches_only_the_rows_that_see_it(r, D, bs):
    """NaN codes in K and V, and pages whose scale is NaN, of tokens that earlier rows of the same
    chunk must not see: NaN appears in the rows at and behind them alone, of V in its column alone."""
    rng = np.random.default_rng(r * 10 + D)
    spans = [(400, 300), (170, 170), (333, 130), (90, 1), (260, 5), (2100, 60)]
    lens, q_lens = [n for n, _ in spans], [n for _, n in spans]
    G = 2
    c = Cache(rng, lens, G, D, bs)

    def at(s, t):
        return c.table[s, t // bs], t % bs

    v_nans = [(0, 101, 0, 3), (0, 130, 0, 3), (0, 140, 1, 60), (0, 377, 0, 7), (0, 399, 1, 0), (1, 5, 1, 33), (1, 6, 1, 33),
              (1, 127, 0, 63), (1, 128, 0, 62), (2, 250, 1, 1), (2, 20, 1, 40), (4, 258, 0, 9), (5, 700, 0, 11), (5, 2041, 1, 12), (5, 2099, 0, 0), (5, 2048, 0, 8)]
    for s, t, g, d in v_nans:
        c.v[(*at(s, t), g, d)] = rng.choice([0x7F, 0xFF])
    c.k[(*at(1, 150), 1, 4)] = 0x7F
    c.ks[at(2, 320)[0], 0] = 255
    c.vs[at(0, 384)[0], 1] = 255
    c.put()
    # the reference's view of a NaN scale: every code of the page is NaN
    c.k[at(2, 320)[0], :, 0], c.ks[at(2, 320)[0], 0] = 0x7F, 127
    c.v[at(0, 384)[0], :, 1], c.vs[at(0, 384)[0], 1] = 0x7F, 127
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), G * r, D))).to(BF16)
    out, lse = pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32(cu), *c.dev, c.bt, c.sl, D ** -0.5, want_lse=True)
    rows = [(s, n - m + i + 1) for s, (n, m) in enumerate(spans) for i in range(m)]
    with np.errstate(invalid="ignore"):
        ref, tol, rl, lt = attention(c, q.double().numpy(), rows, D ** -0.5, CHUNK_STEP, parts=True)
    o = out.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(o), np.isnan(ref))
    # B of the bound counts every V code a row sees: its NaN columns do not matter, those beside them do
    good = ~np.isnan(ref)
    assert good.mean() > 0.5 and (~good).any()
    assert (np.abs(o - ref)[good] <= (tol + 2.0 ** -8 * np.abs(ref))[good]).all()
    ln = lse.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(ln), np.isnan(rl))
    assert (np.abs(ln - rl)[~np.isnan(rl)] <= (lt + 2.0 ** -21 * np.abs(rl))[~np.isnan(rl)]).all()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_steps_of_a_serving_loop():
    """Prompts written and prefilled in chunks beside decodes, then decode steps: every step writes its
    rows, attends over the codes, and the codes read back agree with the oracle's."""
    rng = np.random.default_rng(30)
    bs, G, r, D = 16, 2, 4, 128
    S, total = 3, [150, 60, 90]
    c = Cache(rng, total, G, D, bs, poisoned=False)
    done = np.array([0, 37, 0])
    scale = D ** -0.5
    for step in ([64, 1, 0], [64, 1, 50], [1, 1, 1], [1, 1, 1]):
        done = done + step
        cu = np.concatenate([[0], np.cumsum(step)])
        T = int(cu[-1])
        kv = [torch.from_numpy(rng.standard_normal((T, G, D)) * 2.0 ** rng.uniform(-2, 2, (T, G, 1))).to(BF16)
              for _ in range(2)]
        q = torch.from_numpy(rng.standard_normal((T, G * r, D))).to(BF16)
        sl = i32(done)
        pa.metis_reshape_and_cache_fp8(gpu(kv[0]), gpu(kv[1]), *c.dev, i32(cu), c.bt, sl)
        out, lse = pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32(cu), *c.dev, c.bt, sl, scale, want_lse=True,
                                                         max_seq_len=160)
        c.k, c.ks = oracle.write_cache(kv[0], c.k, c.ks, cu, c.table, done)
        c.v, c.vs = oracle.write_cache(kv[1], c.v, c.vs, cu, c.table, done)
        c.lens = [int(n) for n in done]
        rows = [(s, int(done[s]) - m + i + 1) for s, m in enumerate(step) for i in range(m)]
        ref, tol, rl, lt = attention(c, q.double().numpy(), rows, scale, CHUNK_STEP, parts=True)
        check(out, ref, tol, BF16, "prefill")
        check_lse(lse, rl, lt)
        if max(step) == 1:
            o2, _ = pa.metis_paged_attn_decode_fp8(gpu(q), *c.dev, c.bt, sl, scale, max_seq_len=160, partition_size=32)
            ref, tol, _, _ = attention(c, q.double().numpy(), list(enumerate(c.lens)), scale, STEP[BF16])
            check(o2, ref, tol, BF16, "decode")
    # read back as pages of a bf16 cache, and attend over those
    pages = [-(-n // bs) for n in c.lens]
    first = np.concatenate([[0], np.cumsum(pages)])
    k, v = (t.zero_() for t in (torch.empty(int(first[-1]) * bs, G, D, dtype=BF16, device=DEV) for _ in range(2)))
    pa.metis_gather_cache_fp8(*c.dev, c.bt, i32(c.lens), i32(first[:-1] * bs), k_out=k, v_out=v)
    bt = np.full((S, max(pages)), -1)
    for s in range(S):
        bt[s, :pages[s]] = np.arange(first[s], first[s + 1])
    o3, _ = pa.metis_paged_attn_decode(gpu(q), k.view(-1, bs, G, D), v.view(-1, bs, G, D), i32(bt), i32(c.lens), scale)
    # (that kernel's weights are bf16: 2^-8)
    ref, tol, _, _ = attention(c, q.double().numpy(), list(enumerate(c.lens)), scale, 2.0 ** -8)
    check(o3, ref, tol, BF16, "bf16 decode over the pages read back")


def test_graph_of_a_decode_step_replayed():
    """Write, decode (split) and read back as one graph, captured once and replayed as the lengths grow."""
    rng = np.random.default_rng(31)
    bs, G, r, D, cap = 32, 2, 7, 64, 192
    c = Cache(rng, [cap, cap, cap], G, D, bs, poisoned=False)
    lens = np.array([40, 1, 96])
    key, value = (torch.zeros(3, G, D, dtype=BF16, device=DEV) for _ in range(2))
    q = torch.zeros(3, G * r, D, dtype=BF16, device=DEV)
    sl, cu = i32(lens), i32([0, 1, 2, 3])
    out = torch.empty_like(q)
    ws = torch.empty(pa.metis_decode_workspace_bytes(3, G * r, D, cap, 64), dtype=torch.uint8, device=DEV)
    k, v = (torch.zeros(3 * cap, G, D, dtype=F32, device=DEV) for _ in range(2))
    ro = i32([0, cap, 2 * cap])

    def step():
        pa.metis_reshape_and_cache_fp8(key, value, *c.dev, cu, c.bt, sl)
        pa.metis_paged_attn_decode_fp8(q, *c.dev, c.bt, sl, 0.125, out=out, partition_size=64, max_seq_len=cap,
                                       workspace=ws)
        pa.metis_gather_cache_fp8(*c.dev, c.bt, sl, ro, k_out=k, v_out=v, max_seq_len=cap)

    def load():
        nonlocal kv, qh
        kv = [torch.from_numpy(rng.standard_normal((3, G, D)) * 2.0 ** rng.uniform(-2, 4)).to(BF16) for _ in range(2)]
        qh = torch.from_numpy(rng.standard_normal((3, G * r, D))).to(BF16)
        key.copy_(kv[0])
        value.copy_(kv[1])
        q.copy_(qh)
        sl.copy_(torch.from_numpy(lens))

    kv = qh = None

    def verify():
        c.k, c.ks = oracle.write_cache(kv[0], c.k, c.ks, [0, 1, 2, 3], c.table, lens)
        c.v, c.vs = oracle.write_cache(kv[1], c.v, c.vs, [0, 1, 2, 3], c.table, lens)
        c.lens = [int(n) for n in lens]
        ref, tol, _, _ = attention(c, qh.double().numpy(), list(enumerate(c.lens)), 0.125, STEP[BF16])
        check(out, ref, tol, BF16, "out")
        for s in range(3):
            assert np.array_equal(v[s * cap:s * cap + c.lens[s]].double().cpu().numpy(), c.rows(s, c.lens[s], "v"))

    load()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # on another stream than the tensors' own
    torch.cuda.current_stream().wait_stream(side)
    verify()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        lens += [1, 1, 33]
        lens = np.minimum(lens, cap)
        load()
        g.replay()
        torch.cuda.synchronize()
        # sequence 2 skips tokens: only its newest row is written, the rest is what the pool held
        verify()


def test_calls_on_another_stream_own_their_memory():
    """Outputs and workspaces allocated by a call for `stream` are not reused by the current stream's work."""
    rng = np.random.default_rng(34)
    c = Cache(rng, [700, 300], 2, 64, 16)
    q = gpu(torch.from_numpy(rng.standard_normal((2, 8, 64))).to(BF16))
    ref, _ = pa.metis_paged_attn_decode_fp8(q, *c.dev, c.bt, c.sl, 0.125, partition_size=64, max_seq_len=700)
    kref, _ = pa.metis_gather_cache_fp8(*c.dev, c.bt, c.sl, i32([0, 700]), num_rows=1000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        outs = []
        for _ in range(8):
            o, _ = pa.metis_paged_attn_decode_fp8(q, *c.dev, c.bt, c.sl, 0.125, partition_size=64, max_seq_len=700,
                                                  stream=stream)
            k, _ = pa.metis_gather_cache_fp8(*c.dev, c.bt, c.sl, i32([0, 700]), num_rows=1000, stream=stream)
            outs.append((o, k))
            torch.full((1 << 20,), 3.0, device=DEV)  # current-stream work that takes freed memory
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) and torch.equal(k, kref) for o, k in outs)


def test_two_streams_at_once():
    """Split prefill, joined and merged decode and the write on two streams, each with its own tensors:
    the bits of the same calls one after another."""
    rng = np.random.default_rng(50)
    cases = []
    for lens, q_lens in (([2600, 300, 70], [200, 1, 70]), ([1900, 2300, 5], [64, 130, 1])):
        c = Cache(rng, lens, 2, 128, 16)
        T = sum(q_lens)
        q = gpu(torch.from_numpy(rng.standard_normal((T, 8, 128))).to(BF16))
        kv = [gpu(torch.from_numpy(rng.standard_normal((T, 2, 128))).to(BF16)) for _ in range(2)]
        cases.append((c, q, kv, i32(np.concatenate([[0], np.cumsum(q_lens)]))))

    def steps(c, q, kv, cu, dev, stream):
        pa.metis_reshape_and_cache_fp8(*kv, *dev, cu, c.bt, c.sl, stream=stream)
        outs = [pa.metis_paged_attn_prefill_chunk_fp8(q, cu, *dev, c.bt, c.sl, 0.09, max_seq_len=2600, stream=stream)[0]]
        for partition in (0, 64, 512):
            outs.append(pa.metis_paged_attn_decode_fp8(q[:3], *dev, c.bt, c.sl, 0.09, partition_size=partition,
                                                       max_seq_len=2600, stream=stream)[0])
        return outs

    alone = []
    for case in cases:
        dev = [x.clone() for x in case[0].dev]
        alone.append((steps(*case, dev, None), dev))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        dev = [[x.clone() for x in case[0].dev] for case in cases]
        torch.cuda.synchronize()
        outs = [steps(*case, d, st) for case, d, st in zip(cases, dev, streams)]
        torch.cuda.synchronize()
        for got, d, (ref, ref_dev) in zip(outs, dev, alone):
            assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, ref))
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(d, ref_dev))


def test_offsets_past_32_bits():
    """Pages at the end of pools of more than 2^32 bytes."""
    bs, G, D, r = 64, 8, 128, 4
    nb = (1 << 32) // (bs * G * D) + 5
    rng = np.random.default_rng(32)
    dev = [torch.empty(nb, bs, G, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
    dev += [torch.full((nb, G), 120, dtype=torch.uint8, device=DEV) for _ in range(2)]
    table = np.array([[nb - 1, 3, nb - 3]])
    n = 150
    kv = [torch.from_numpy(rng.standard_normal((n, G, D))).to(BF16) for _ in range(2)]
    q = torch.from_numpy(rng.standard_normal((n, G * r, D))).to(BF16)
    pa.metis_reshape_and_cache_fp8(gpu(kv[0]), gpu(kv[1]), *dev, i32([0, n]), i32(table), i32([n]))
    c = Cache.__new__(Cache)
    c.bs, c.G, c.D, c.lens, c.table = bs, G, D, [n], np.array([[0, 1, 2]])
    blank = np.zeros((3, bs, G, D), np.uint8), np.zeros((3, G), np.uint8)
    c.k, c.ks = oracle.write_cache(kv[0], *blank, [0, n], c.table, [n])
    c.v, c.vs = oracle.write_cache(kv[1], *blank, [0, n], c.table, [n])
    k, v = pa.metis_gather_cache_fp8(*dev, i32(table), i32([n]), i32([0]), num_rows=n, out_dtype=F32)
    assert np.array_equal(k.double().cpu().numpy(), c.rows(0, n, "k"))
    assert np.array_equal(v.double().cpu().numpy(), c.rows(0, n, "v"))
    out, _ = pa.metis_paged_attn_decode_fp8(gpu(q[-1:]), *dev, i32(table), i32([n]), 0.09)
    ref, tol, _, _ = attention(c, q[-1:].double().numpy(), [(0, n)], 0.09, STEP[BF16])
    check(out, ref, tol, BF16, "decode")
    out, _ = pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), i32([0, n]), *dev, i32(table), i32([n]), 0.09)
    ref, tol, _, _ = attention(c, q.double().numpy(), [(0, i + 1) for i in range(n)], 0.09, CHUNK_STEP, parts=True)
    check(out, ref, tol, BF16, "prefill")


def test_binding_refusals():
    rng = np.random.default_rng(33)
    c = Cache(rng, [20], 2, 64, 16)
    q = torch.zeros(1, 8, 64, dtype=BF16, device=DEV)
    with pytest.raises(TypeError):
        pa.metis_paged_attn_decode_fp8(q, c.dev[0].float(), *c.dev[1:], c.bt, c.sl, 0.1)
    with pytest.raises(ValueError):
        pa.metis_paged_attn_decode_fp8(q, *c.dev[:2], c.dev[2][:1], c.dev[3], c.bt, c.sl, 0.1)
    with pytest.raises(ValueError):
        pa.metis_paged_attn_decode_fp8(q, *c.dev, c.bt, c.sl, 0.1, out=torch.empty(1, 4, 64, dtype=BF16, device=DEV))
    with pytest.raises(ValueError):
        pa.metis_gather_cache_fp8(*c.dev, c.bt, c.sl, i32([0]))  # neither outputs nor num_rows
    with pytest.raises(ValueError):
        pa.metis_gather_cache_fp8(*c.dev, c.bt, c.sl, i32([0]), k_out=torch.empty(20, 2, 64, device=DEV))
    with pytest.raises(ValueError):
        pa.metis_reshape_and_cache_fp8(q, q, *c.dev, i32([0, 1]), c.bt, c.sl)  # 8 heads, the cache has 2
    with pytest.raises(TypeError):
        pa.metis_reshape_and_cache_fp8(q.half(), q.half(), *c.dev, i32([0, 1]), c.bt, c.sl)
