"""Per-head norm and rotation of queries and keys, and their way into the pages, against float64.

Tolerance per element: half a step of the output type (finfo.eps / 2 of the value), plus the fp32
arithmetic in front of it.  The sum of squares is D / lanes <= 8 products added in turn and at most five
additions across lanes (13 roundings of its terms, half of which reach its root), mean and eps one, root
and reciprocal two, the products with factor and weight two, cosine's and sine's one each and their sum one:
below 16 roundings of 2^-24 of the addends' sizes |y_a| + |y_b| -> 2^-20 of them.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clear_status():
    pa.metis_read_status(clear=True)
    yield


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def close(got, ref, add, dtype):
    g = f64(got)
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + 2.0 ** -20 * add + 1e-37
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], g[bad][0], ref[bad][0])


class Rows:
    def __init__(self, seed, T, H, G, D, dtype, R, *, packed=True, norm=True, P=500, bs=16, pad=0.1, scale=3.0):
        g = torch.Generator().manual_seed(seed)
        x = (torch.randn(T, H + 2 * G, D, generator=g) * 2.0 ** torch.empty(T, H + 2 * G, 1).uniform_(-scale, scale,
                                                                                                     generator=g)).to(dtype)
        self.q, self.k, self.v = x[:, :H], x[:, H:H + G], x[:, H + G:]
        if packed:
            d = x.to(DEV)
            self.dev = d[:, :H], d[:, H:H + G], d[:, H + G:]
        else:
            self.dev = tuple(t.contiguous().to(DEV) for t in (self.q, self.k, self.v))
        self.table = pa.rope_table(P, R, device="cpu") if R else None
        self.pos = torch.randint(P, (T,), generator=g, dtype=torch.int32)
        self.w = [(torch.rand(D, generator=g) + 0.5).to(dtype) if norm else None for _ in range(2)]
        self.nb, self.bs = T // bs + 3, bs
        self.slots = torch.randperm(self.nb * bs, generator=g)[:T].to(torch.int64)
        self.slots[torch.rand(T, generator=g) < pad] = -1
        self.dtype = dtype

    def on(self, t):
        return None if t is None else t.to(DEV)

    def kw(self, **more):
        return dict(q_weight=self.on(self.w[0]), k_weight=self.on(self.w[1]), **more)

    def want(self, eps, interleaved):
        turn = None if self.table is None else f64(self.table)
        return [oracle.norm_rope(f64(x), None if w is None else f64(w), turn, self.pos.tolist(), eps, interleaved)
                for x, w in ((self.q, self.w[0]), (self.k, self.w[1]))]


CASES = [  # T, H, G, D, dtype, R, interleaved, packed, norm
    (1, 32, 8, 128, BF16, 128, False, True, True),
    (67, 32, 8, 128, BF16, 128, False, True, True),
    (33, 4, 1, 64, F32, 64, False, False, True),
    (20, 28, 4, 128, BF16, 64, False, True, True),
    (19, 5, 3, 64, BF16, 16, True, False, True),
    (40, 16, 4, 64, F32, 32, True, True, False),
    (12, 7, 7, 128, F32, 48, False, True, True),
    (9, 1, 1, 64, BF16, 64, False, True, False),
    (300, 9, 3, 128, BF16, 96, False, False, True),
    (15, 64, 8, 128, BF16, 128, True, True, True),
    (11, 3, 2, 128, F32, 0, False, True, True),
]


@pytest.mark.parametrize("T,H,G,D,dtype,R,interleaved,packed,norm", CASES)
def test_norm_rope_parity(T, H, G, D, dtype, R, interleaved, packed, norm):
    c = Rows(T + D, T, H, G, D, dtype, R, packed=packed, norm=norm)
    eps = 1e-5
    (rq, aq), (rk, ak) = c.want(eps, interleaved)
    q, k, v = c.dev
    before = [t.clone() for t in (q, k, v)]
    qo, ko = pa.metis_qk_norm_rope(q, k, c.on(c.table), c.pos.to(DEV), eps=eps, interleaved=interleaved, **c.kw())
    close(qo, rq, aq, dtype)
    close(ko, rk, ak, dtype)
    caches = [torch.full((c.nb, c.bs, G, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2)]
    q2 = pa.metis_qk_norm_rope_and_cache(q, k, v, c.on(c.table), c.pos.to(DEV), *caches, c.slots.to(DEV), eps=eps,
                                         interleaved=interleaved, **c.kw())
    assert torch.equal(q2, qo)
    # the pages hold exactly the other call's keys and the values, and nothing else was written
    nan = torch.full((c.nb, c.bs, G, D), float("nan"), dtype=dtype)
    kk, vv = oracle.reshape_and_cache(ko.cpu(), c.v.contiguous(), nan, nan.clone(), c.slots)
    for got, ref in zip(caches, (kk, vv)):
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=12345.0), torch.nan_to_num(ref, nan=12345.0))
    for t, b in zip((q, k, v), before):
        assert torch.equal(t, b)
    assert pa.metis_read_status() == 0


def test_one_weight_only():
    c = Rows(1, 30, 6, 2, 128, BF16, 128)
    for i in range(2):
        w, c.w[i] = c.w[i], None
        (rq, aq), (rk, ak) = c.want(1e-6, False)
        qo, ko = pa.metis_qk_norm_rope(*c.dev[:2], c.on(c.table), c.pos.to(DEV), **c.kw())
        close(qo, rq, aq, BF16)
        close(ko, rk, ak, BF16)
        c.w[i] = w


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place(dtype):
    c = Rows(2, 50, 8, 2, 128, dtype, 64, packed=False)
    q, k = c.dev[:2]
    args = c.on(c.table), c.pos.to(DEV)
    qo, ko = pa.metis_qk_norm_rope(q, k, *args, **c.kw())
    q2, k2 = pa.metis_qk_norm_rope(q, k, *args, q_out=q, k_out=k, **c.kw())
    assert q2 is q and torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("dtype,scale", [(F32, 100.0), (BF16, 100.0)])
def test_values_whose_squares_leave_the_range(dtype, scale):
    """Rows of values near 2^+-100: squares beyond fp32, for which eps is nothing or everything."""
    c = Rows(3, 64, 4, 2, 128, dtype, 128, scale=scale)
    for eps in (1e-6, 0.0):
        (rq, aq), (rk, ak) = c.want(eps, False)
        qo, ko = pa.metis_qk_norm_rope(*c.dev[:2], c.on(c.table), c.pos.to(DEV), eps=eps, **c.kw())
        close(qo, rq, aq, dtype)
        close(ko, rk, ak, dtype)


def test_rows_of_zeros_infinities_and_nan_stay_in_their_rows():
    c = Rows(4, 8, 4, 2, 128, F32, 128)
    q = c.dev[0].clone()
    q[1, 2] = 0
    q[2, 0, 5] = float("inf")
    q[3, 1, 70] = float("nan")
    c.q = q.cpu()
    (rq, aq), _ = c.want(1e-6, False)
    qo, _ = pa.metis_qk_norm_rope(q, c.dev[1], c.on(c.table), c.pos.to(DEV), **c.kw())
    fine = torch.ones(8, 4, dtype=torch.bool)
    fine[2, 0] = fine[3, 1] = False
    g = qo.cpu()[fine]
    assert torch.isfinite(g).all() and (qo[1, 2] == 0).all() and torch.isnan(qo[3, 1]).any()
    ref = rq[fine.numpy()]
    assert (np.abs(f64(g) - ref) <= 2.0 ** -23 * np.abs(ref) + 2.0 ** -20 * aq[fine.numpy()]).all()


def test_positions_and_slots_out_of_range():
    c = Rows(5, 10, 4, 2, 64, BF16, 32, norm=False, pad=0.0)
    c.pos[3], c.pos[7] = -1, 500
    (rq, aq), _ = c.want(1e-6, False)
    qo, _ = pa.metis_qk_norm_rope(*c.dev[:2], c.on(c.table), c.pos.to(DEV), **c.kw())
    close(qo, rq, aq, BF16)
    assert (qo[3, :, :32] == 0).all() and torch.equal(qo[3, :, 32:].cpu(), c.q[3, :, 32:])
    assert pa.metis_read_status() == pa.STATUS_BAD_POSITION
    c.pos[3], c.pos[7] = 0, 499
    c.slots[2] = c.nb * c.bs
    caches = [torch.zeros(c.nb, c.bs, 2, 64, dtype=BF16, device=DEV) for _ in range(2)]
    pa.metis_qk_norm_rope_and_cache(*c.dev, c.on(c.table), c.pos.to(DEV), *caches, c.slots.to(DEV), **c.kw())
    assert pa.metis_read_status() == pa.STATUS_BAD_BLOCK_ID
    live = torch.zeros(c.nb * c.bs, dtype=torch.bool)
    live[c.slots[c.slots < c.nb * c.bs]] = True
    assert (caches[1].cpu().view(-1, 2, 64)[~live] == 0).all()
    assert torch.equal(caches[1].cpu().view(-1, 2, 64)[c.slots[9]], c.v[9])


def test_no_rows_and_refusals():
    c = Rows(6, 4, 4, 2, 64, BF16, 64)
    q, k, v = c.dev
    t, pos = c.on(c.table), c.pos.to(DEV)
    qo, _ = pa.metis_qk_norm_rope(q[:0], k[:0], t, pos[:0])
    assert qo.shape == (0, 4, 64)
    with pytest.raises(ValueError):
        pa.metis_qk_norm_rope(q.transpose(1, 2).contiguous().transpose(1, 2), k, t, pos)
    with pytest.raises(ValueError):
        pa.metis_qk_norm_rope(q, k, t, pos[:3])
    with pytest.raises(TypeError):
        pa.metis_qk_norm_rope(q, k.float(), t, pos)
    with pytest.raises(TypeError):
        pa.metis_qk_norm_rope(q, k, t, pos.long())
    with pytest.raises(TypeError):
        pa.metis_qk_norm_rope(q, k, t, None)
    with pytest.raises(TypeError):
        pa.metis_qk_norm_rope(q, k, t, pos, q_weight=torch.ones(64, device=DEV))
    with pytest.raises(pa.MetisError):  # the queries of an odd slice are not 16-byte aligned
        x = torch.zeros(4 * 8 * 64 + 1, dtype=BF16, device=DEV)[1:].view(4, 8, 64)
        pa.metis_qk_norm_rope(x[:, :4], x[:, 4:6], t, pos)
    with pytest.raises(pa.MetisError):
        pa.metis_qk_norm_rope(q, k, t[:, :24].contiguous(), pos)


def test_captured_and_replayed_on_another_stream():
    c = Rows(7, 64, 8, 2, 128, BF16, 128)
    q, k, v = (t.clone() for t in c.dev)
    t, pos, slots = c.on(c.table), c.pos.to(DEV), c.slots.to(DEV)
    w = c.kw()
    caches = [torch.zeros(c.nb, c.bs, 2, 128, dtype=BF16, device=DEV) for _ in range(2)]
    out = torch.empty(64, 8, 128, dtype=BF16, device=DEV)
    call = lambda: pa.metis_qk_norm_rope_and_cache(q, k, v, t, pos, *caches, slots, q_out=out, **w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for i in range(3):
        for x in (q, k, v):
            x.mul_(-1.25)
        pos.copy_((pos + 17) % 500)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            g.replay()
        side.synchronize()
        got = [out.clone()] + [x.clone() for x in caches]
        call()
        for a, b in zip(got, [out] + caches):
            assert torch.equal(a, b)
