"""Decodes whose sequences share prefixes against the float64 oracle, which knows nothing of sharing: it
attends over every sequence's own table row.

Slots of no sequence and the workspace start as NaN.  Tolerance of an output per element: the weights of each
part are rounded to bf16 in front of the product with V (eps / 2 = 2^-8 of the sum of weight * |v|, which a
weighted mean of parts keeps), the output once more (2^-8 of its value), and scores, exponentials, sums and the
join in fp32 come to less than 2^-14 of that sum.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from helpers import BF16_LSE_ATOL
from test_gpu_window import compare, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _clear_status():
    pa.metis_read_status(clear=True)
    yield


class Batch:
    """groups: (shared tokens, tokens of each member); `after`: sequences behind the last group."""

    def __init__(self, seed, groups, H, G, D, bs, after=(), extra=2):
        rng = np.random.default_rng(seed)
        self.lens = np.array([n for _, m in groups for n in m] + list(after))
        self.cu = np.concatenate([[0], np.cumsum([len(m) for _, m in groups])])
        self.shared = np.array([p for p, _ in groups], dtype=np.int64)
        S = len(self.lens)
        width = max(1, int((-(-self.lens // bs)).max())) + 1
        total = int(sum(-(-n // bs) for n in self.lens)) + sum(-(-p // bs) for p, _ in groups) + extra
        order = list(rng.permutation(total))
        self.table = np.full((S, width), -1)
        k, v = (rng.standard_normal((total, bs, G, D)) for _ in range(2))
        used = np.zeros((total, bs), dtype=bool)
        s = 0
        for p, members in groups:
            whole = p // bs
            common = [order.pop() for _ in range(whole)] if any(n >= p for n in members) else []
            tail = None  # the tokens of a shared partial page: every member has a copy
            for n in members:
                if n >= p:
                    own = [order.pop() for _ in range(-(-n // bs) - whole)]
                    self.table[s, : whole + len(own)] = common + own
                    if p % bs:
                        if tail is None:
                            tail = own[0]
                        k[own[0], : p % bs], v[own[0], : p % bs] = k[tail, : p % bs], v[tail, : p % bs]
                else:
                    own = [order.pop() for _ in range(-(-n // bs))]
                    self.table[s, : len(own)] = own
                s += 1
        for n in after:
            own = [order.pop() for _ in range(-(-n // bs))]
            self.table[s, : len(own)] = own
            s += 1
        for i, n in enumerate(self.lens):
            t = np.arange(n)
            used[self.table[i, t // bs], t % bs] = True
        k[~used] = np.nan
        v[~used] = np.nan
        self.k, self.v = torch.from_numpy(k).to(BF16), torch.from_numpy(v).to(BF16)
        self.q = torch.from_numpy(rng.standard_normal((S, H, D))).to(BF16)
        self.scale = D ** -0.5

    def want(self):
        o, l = oracle.paged_decode(self.q, self.k, self.v, self.table, self.lens, self.scale)
        _, _, size = oracle.paged_window_decode(self.q, self.k, self.v, self.table, self.lens, self.scale, 2 ** 31, 0)
        return o, l, size

    def args(self):
        return [self.q.to(DEV), self.k.to(DEV), self.v.to(DEV), i32(self.table), i32(self.lens), i32(self.cu),
                i32(self.shared), self.scale]

    def workspace(self):
        S, H, D = self.q.shape
        n = pa.metis_shared_workspace_bytes(S, H, self.k.shape[2], D, len(self.shared))
        return torch.full((n // 4,), float("nan"), device=DEV)

    def run(self, **kw):
        kw.setdefault("max_seq_len", max(1, int(self.lens.max())))
        return pa.metis_paged_attn_decode_shared(*self.args(), workspace=self.workspace(), want_lse=True, **kw)

    def check(self, status=0, **kw):
        out, lse = self.run(**kw)
        torch.cuda.synchronize()
        assert pa.metis_read_status() == status
        compare(out, lse, self.want(), BF16)


def members(rng, p, n, hi):
    return [p + int(x) for x in rng.integers(0, hi + 1, n)]


@pytest.mark.parametrize("H,G,D,bs", [(8, 2, 128, 16), (4, 4, 64, 32), (16, 2, 128, 64), (2, 1, 64, 16)])
@pytest.mark.parametrize("p", [1, 16, 100, 128, 129, 640])
def test_one_group(H, G, D, bs, p):
    rng = np.random.default_rng(p)
    Batch(p + H, [(p, members(rng, p, 5, 90))], H, G, D, bs).check()


@pytest.mark.parametrize("H,G,D,bs,n", [(32, 8, 128, 16, 64), (8, 1, 128, 16, 33), (4, 2, 64, 16, 200), (2, 2, 128, 32, 300)])
def test_many_members(H, G, D, bs, n):
    """Several query tiles per group, with one and with two in the last pair."""
    rng = np.random.default_rng(n)
    Batch(n, [(700, members(rng, 700, n, 60))], H, G, D, bs).check()


def test_groups_of_all_kinds():
    """Nothing shared, one member, members shorter than the prefix and empty ones (first, last, all), own tokens
    of none; sequences behind the groups."""
    rng = np.random.default_rng(1)
    groups = [(0, [30, 1]), (48, [80]), (64, [0, 10, 64, 100, 0]), (200, [3, 0]), (130, members(rng, 130, 20, 200)), (16, []),
              (33, [33, 40, 32]), (512, [600, 512, 0])]
    for seed, (H, G, D, bs) in enumerate([(8, 2, 128, 16), (4, 4, 64, 16), (8, 1, 64, 32)]):
        Batch(seed, groups, H, G, D, bs, after=[50, 0, 7]).check()


@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (4, 1, 64)])
def test_many_short_members_in_front(H, G, D):
    """The first member with the whole prefix stands behind up to a few hundred padded or shorter ones, or there is none."""
    groups = [(48, [3] * n + [50, 48]) for n in (7, 8, 9, 39, 40, 41, 135, 136, 137, 300)]
    groups += [(130, [0] * n + [131]) for n in (8, 136, 264)] + [(16, [15] * 200), (16, []), (33, [0] * 9), (20, [21])]
    Batch(15, groups, H, G, D, 16, after=[5]).check()
    Batch(16, [(40, [0] * 30 + [60, 41])] * 520, 2, 1, 64, 16).check()  # more groups than threads


def test_short_members_in_front_cost_no_load_each():
    """20,000 padded rows in front of a group's members or behind them: the same work."""
    S, live, p, bs = 20000, 64, 512, 16
    b = Batch(17, [(p, [p + 20] * live)], 4, 1, 64, bs)
    q = torch.randn(S, 4, 64, device=DEV).to(BF16)
    ws = torch.empty(pa.metis_shared_workspace_bytes(S, 4, 1, 64, 1), dtype=torch.uint8, device=DEV)
    times, outs = [], []
    for at in (0, S - live):
        lens, table = np.zeros(S, dtype=np.int64), np.full((S, b.table.shape[1]), -1)
        lens[at:at + live], table[at:at + live] = b.lens, b.table
        qa = q.clone()
        qa[at:at + live] = b.q.to(DEV)
        args = [qa, b.k.to(DEV), b.v.to(DEV), i32(table), i32(lens), i32([0, S]), i32([p]), b.scale]
        call = lambda: pa.metis_paged_attn_decode_shared(*args, max_seq_len=600, workspace=ws)[0]
        outs.append(call()[at:at + live].clone())
        call()
        took = []
        for _ in range(9):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            call()
            end.record()
            end.synchronize()
            took.append(start.elapsed_time(end))
        times.append(sorted(took)[4])
    assert pa.metis_read_status() == 0
    o, _, size = b.want()
    for out in outs:
        d = np.abs(out.double().cpu().numpy() - o)
        assert (d <= (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * np.abs(o)).all()
    assert times[1] < 4 * times[0], times  # (16 times with a load in series for each, 2.5 by warps)


def test_more_groups_than_threads():
    rng = np.random.default_rng(2)
    groups = [(int(p), members(rng, int(p), int(n), 20)) for p, n in zip(rng.integers(0, 200, 1100), rng.integers(0, 3, 1100))]
    Batch(3, groups, 4, 2, 64, 16).check()


def test_few_sequences_behind_a_long_prefix():
    """Own tokens shared by a cluster's CTAs; a unit's prefix in many parts."""
    Batch(4, [(20000, [20003, 21000, 20000, 23000])], 8, 2, 128, 16).check()


def test_long_own_tokens():
    Batch(5, [(128, [5000, 130, 4000])], 8, 2, 128, 16).check()


@pytest.mark.parametrize("shared,S", [(39000, 512), (17000, 1100)])
def test_lengths_that_add_up_past_fp32s_whole_numbers(shared, S):
    """More than 2^24 tokens over a few pages that every table row names again and again: the CTAs have to agree on
    their shares whatever the lengths.  Against the decode that shares nothing: a tile left out or taken twice moves
    lse by 0.003 and more."""
    rng = np.random.default_rng(S)
    H, G, D, bs, pages, hi = 4, 1, 64, 16, 64, shared + 3000
    k, v = (torch.from_numpy(rng.standard_normal((pages, bs, G, D))).to(BF16).to(DEV) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((S, H, D))).to(BF16).to(DEV)
    table = i32(np.broadcast_to(np.arange(-(-hi // bs)) % pages, (S, -(-hi // bs))).copy())
    ws = torch.empty(pa.metis_shared_workspace_bytes(S, H, G, D, 1), dtype=torch.uint8, device=DEV)
    for _ in range(20):
        p = int(rng.integers(shared, shared + 999))
        lens = rng.integers(p, hi, S)
        assert lens.sum() > 2 ** 24
        kw = dict(max_seq_len=hi, want_lse=True)
        call = lambda: pa.metis_paged_attn_decode_shared(q, k, v, table, i32(lens), i32([0, S]), i32([p]), 0.125, workspace=ws,
                                                         **kw)
        out, lse = call()
        want, wl = pa.metis_paged_attn_decode(q, k, v, table, i32(lens), 0.125, **kw)
        size, _ = pa.metis_paged_attn_decode(q, k, v.abs(), table, i32(lens), 0.125, **kw)
        assert (lse - wl).abs().max() <= 2 * BF16_LSE_ATOL
        # both are within the tolerance above of the exact values
        tol = 2 * ((2.0 ** -8 + 2.0 ** -14) * size.double() * (1 + 2.0 ** -6) + 2.0 ** -8 * want.double().abs() * (1 + 2.0 ** -6))
        assert ((out.double() - want.double()).abs() <= tol).all()
        again = call()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert pa.metis_read_status() == 0


def test_no_groups():
    Batch(6, [], 8, 2, 128, 16, after=[40, 700, 0, 1]).check()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    rng = np.random.default_rng(7)
    b = Batch(7, [(300, members(rng, 300, 9, 100))], 8, 2, 128, 16)
    b.scale = scale
    b.check()


def test_contents_that_are_flagged():
    rng = np.random.default_rng(8)
    b = Batch(8, [(64, members(rng, 64, 6, 50)), (128, members(rng, 128, 6, 50)), (32, members(rng, 32, 4, 9))], 8, 2, 64, 16)
    keep = b.shared.copy(), b.cu.copy()
    b.shared[1] = -5
    b.check(status=pa.STATUS_BAD_Q_LEN)
    b.shared[1] = 2 ** 31 - 1
    b.check(status=pa.STATUS_SEQ_TOO_LONG)
    b.shared[1] = 100000
    b.check(status=pa.STATUS_SEQ_TOO_LONG)
    b.shared = keep[0].copy()
    b.cu[0] = -4  # the first group is left out: its sequences are decoded by themselves
    b.check(status=pa.STATUS_BAD_OFFSETS)
    b.cu = keep[1].copy()
    b.cu[-1] = 400
    b.check(status=pa.STATUS_BAD_OFFSETS)
    for cu in ([0, 16, 0, 16], [16, 0, 16, 0], [2 ** 31 - 1, -(2 ** 31), 5, 3]):  # decreasing: no fault
        b.cu = np.array(cu)
        b.run()
        torch.cuda.synchronize()
        assert pa.metis_read_status() == pa.STATUS_BAD_OFFSETS
    b.cu = keep[1].copy()
    b.table[0, 1] = b.k.shape[0]
    b.run()
    assert pa.metis_read_status() == pa.STATUS_BAD_BLOCK_ID


def test_length_beyond_the_bound():
    b = Batch(9, [(64, [100, 90, 164])], 8, 2, 64, 16)
    out, _ = b.run(max_seq_len=120)
    assert pa.metis_read_status() == pa.STATUS_SEQ_TOO_LONG
    b.lens[2] = 120
    o, _, size = b.want()
    assert (np.abs(out.double().cpu().numpy() - o) <= (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * np.abs(o)).all()


def test_captured_twice_and_replayed_at_once():
    """Two captured calls with workspaces of their own on two streams; lengths and prefixes change in between."""
    rng = np.random.default_rng(10)
    runs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        b = Batch(11 + i, [(256, members(rng, 256, 20, 300)), (512, members(rng, 512, 12, 100))], 8, 2, 128, 16)
        a, ws = b.args(), b.workspace()
        out = torch.empty_like(a[0])
        runs.append((b, a, out, lambda a=a, ws=ws, out=out: pa.metis_paged_attn_decode_shared(
            *a, out=out, max_seq_len=700, workspace=ws)))
    torch.cuda.synchronize()
    graphs = []
    for (b, a, out, call), st in zip(runs, streams):
        with torch.cuda.stream(st):
            call()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        graphs.append(g)
    for step in range(3):
        for b, a, out, _ in runs:
            b.shared -= 16 * step
            b.lens -= 3
            b.lens = np.maximum(b.lens, b.shared.repeat(np.diff(b.cu)))
            a[4].copy_(i32(b.lens))
            a[6].copy_(i32(b.shared))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for b, a, out, call in runs:
            o, _, size = b.want()
            d = np.abs(out.double().cpu().numpy() - o)
            assert (d <= (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * np.abs(o)).all()
            seen = out.clone()
            call()
            assert torch.equal(seen, out)
    assert pa.metis_read_status() == 0


def test_on_another_stream_with_memory_of_the_call():
    rng = np.random.default_rng(12)
    b = Batch(13, [(300, members(rng, 300, 30, 50))], 8, 2, 128, 16)
    want, side = b.want(), torch.cuda.Stream()
    a = b.args()
    torch.cuda.synchronize()
    for _ in range(3):
        out, lse = pa.metis_paged_attn_decode_shared(*a, max_seq_len=400, want_lse=True, stream=side)
        side.synchronize()
        compare(out, lse, want, BF16)


def test_refusals():
    b = Batch(14, [(32, [40, 50])], 8, 2, 64, 16)
    a = b.args()
    kw = dict(max_seq_len=50)
    with pytest.raises(pa.MetisError):
        pa.metis_paged_attn_decode_shared(a[0].float(), a[1].float(), a[2].float(), *a[3:], **kw)
    with pytest.raises(ValueError):
        pa.metis_paged_attn_decode_shared(*a[:5], i32([0, 1, 2]), *a[6:], **kw)
    with pytest.raises(TypeError):
        pa.metis_paged_attn_decode_shared(*a[:6], a[6].long(), a[7], **kw)
    with pytest.raises(pa.MetisError):
        pa.metis_paged_attn_decode_shared(*a, workspace=torch.empty(1024, dtype=torch.uint8, device=DEV), **kw)
    with pytest.raises(pa.MetisError):  # ratio 3
        pa.metis_paged_attn_decode_shared(a[0][:, :6].contiguous(), *a[1:], **kw)
    empty, _ = pa.metis_paged_attn_decode_shared(a[0][:0], a[1], a[2], a[3][:0], a[4][:0], i32([0, 0]), i32([32]), 0.1, **kw)
    assert empty.shape == (0, 8, 64)
