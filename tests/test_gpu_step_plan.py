"""A step's index arrays against the oracle's token-by-token rule: whole numbers, compared exactly."""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make(rng, S, cached_hi, new_hi, bs, slack=2, spare=3, idle=0.2):
    """A batch whose cached tokens have pages, and a stack with the others."""
    cached = rng.integers(0, cached_hi + 1, S)
    new = np.where(rng.random(S) < idle, 0, rng.integers(0, new_hi + 1, S))
    held = -(-cached // bs)
    after = -(-(cached + new) // bs)
    width = int(after.max(initial=0)) + slack
    nb = int(np.maximum(after, held).sum()) + spare
    order = rng.permutation(nb)
    table = np.full((S, max(width, 1)), -1)
    at = 0
    for s in range(S):
        table[s, : held[s]] = order[at : at + held[s]]
        at += held[s]
    return new, cached, table, order[at:], nb


def check(new, cached, table, stack, nb, bs, T, *, depth=None, held=None, refs=True, in_place=False, stream=None):
    depth = len(stack) if depth is None else depth
    refcount = np.zeros(nb, dtype=np.int64) if refs else None
    ref = oracle.plan_step(new, cached, table, stack, depth, bs, T, nb, held=held, refcount=refcount)
    pa.metis_read_status(clear=True)
    bt, sl, fc = i32(table), i32(cached), i32([depth])
    hb = None if held is None else i32(held)
    rc = i32(refcount) if refs else None
    kw = dict(seq_lens=sl, free_count_out=fc, held_blocks_out=hb) if in_place else {}
    got = pa.metis_plan_step(i32(new), sl, bt, i32(stack), fc, block_size=bs, num_tokens=T, num_blocks=nb, held_blocks=hb,
                             refcount=rc, **kw)
    torch.cuda.synchronize()
    for name in ("cu_q_lens", "seq_lens", "positions", "slot_mapping"):
        a, b = getattr(got, name).cpu().numpy(), ref[name]
        assert np.array_equal(a, b), (name, np.flatnonzero(a != b)[:5], a[a != b][:5], b[a != b][:5])
    assert np.array_equal(bt.cpu().numpy(), ref["block_table"])
    assert int(got.free_count) == ref["free_count"]
    if refs:
        assert np.array_equal(rc.cpu().numpy(), ref["refcount"])
    if held is not None:
        assert np.array_equal(got.held_blocks.cpu().numpy(), ref["held_blocks"])
    assert pa.metis_read_status() == ref["status"]
    if not in_place:
        assert np.array_equal(sl.cpu().numpy(), cached) and int(fc) == depth
    return ref


@pytest.mark.parametrize("S,cached_hi,new_hi,bs", [
    (1, 0, 1, 16), (1, 40, 1, 16), (64, 4096, 1, 16), (7, 100, 300, 64), (33, 500, 40, 32), (130, 3, 2, 1),
    (1000, 64, 40, 16), (4096, 100, 3, 16), (4097, 100, 3, 32), (9000, 20, 6, 16), (3, 1000, 30000, 16), (5, 7, 9, 24),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_parity(S, cached_hi, new_hi, bs, in_place):
    rng = np.random.default_rng(S + bs)
    new, cached, table, stack, nb = make(rng, S, cached_hi, new_hi, bs)
    check(new, cached, table, stack, nb, bs, int(new.sum()) + int(rng.integers(0, 3)) * 50, in_place=in_place,
          refs=not in_place or S % 2 == 0)


def test_all_idle_and_no_rows():
    rng = np.random.default_rng(3)
    new, cached, table, stack, nb = make(rng, 20, 100, 0, 16)
    check(new, cached, table, stack, nb, 16, 0)
    check(new, cached, table, stack, nb, 16, 40)


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_that_the_row_names_already(in_place):
    """A prefix lookup dealt out the prompt's full pages: they are not taken again."""
    rng = np.random.default_rng(4)
    bs, S = 16, 50
    new, cached, table, stack, nb = make(rng, S, 200, 90, bs)
    held = -(-cached // bs)
    extra = np.minimum((cached + new) // bs - held, rng.integers(0, 4, S)).clip(min=0)
    stack = list(stack)
    for s in range(S):
        for j in range(extra[s]):
            table[s, held[s] + j] = stack.pop(0)
    want = held + extra
    want[::7] = 0  # (raised to what the cached tokens need)
    extra_gone = [s for s in range(0, S, 7) if extra[s]]
    for s in extra_gone:
        table[s, held[s]:] = -1
    check(new, cached, table, stack, nb, bs, int(new.sum()), held=want, in_place=in_place)


def test_contents_that_are_flagged():
    rng = np.random.default_rng(5)
    bs = 16
    new, cached, table, stack, nb = make(rng, 40, 200, 90, bs)
    T = int(new.sum())
    neg = new.copy()
    neg[[3, 9]] = [-5, -(2 ** 31)]
    assert check(neg, cached, table, stack, nb, bs, T)["status"] == 8
    few = check(new, cached, table, stack, nb, bs, T, depth=5)
    assert few["status"] == 32 and few["free_count"] == 0
    assert check(new, cached, table, stack, nb, bs, T, depth=0)["status"] == 32
    assert check(new, cached, table, stack, nb, bs, T, depth=-3)["status"] == 32
    assert check(new, cached, table, stack, nb, bs, T, depth=len(stack) + 9)["status"] == 0  # clamped
    assert check(new, cached, table, stack, nb, bs, T // 2)["status"] == 64
    assert check(new, cached, table, stack, nb, bs, 0)["status"] == 64
    bad = np.array(stack)
    bad[-3] = nb
    bad[-4] = -7
    assert check(new, cached, table, bad, nb, bs, T)["status"] == 1
    narrow = table[:, : table.shape[1] // 2]
    assert check(new, cached, narrow, stack, nb, bs, T)["status"] & 2
    huge = new.copy()
    huge[20:] = 2 ** 31 - 1  # sums past 2^31
    assert check(huge, cached, table, stack, nb, bs, T)["status"] & 64


def test_lengths_at_the_end_of_int32():
    check(np.array([5, 3]), np.array([2 ** 31 - 4, 2 ** 31 - 1]), np.array([[1, 2], [3, 4]]), np.array([0]), 8, 16, 8)


def test_bad_held_entry():
    pa.metis_read_status(clear=True)
    bt = i32([[99]])
    got = pa.metis_plan_step(i32([2]), i32([3]), bt, i32([1]), i32([1]), block_size=16, num_tokens=2, num_blocks=8)
    assert got.slot_mapping.tolist() == [-1, -1] and bt.tolist() == [[99]] and pa.metis_read_status() == 1


def test_captured_steps_advance_by_themselves():
    """In place, a captured decode step is replayed: lengths, table and stack advance as in an eager loop."""
    rng = np.random.default_rng(6)
    S, bs, steps = 37, 16, 40
    _, cached, table, stack, nb = make(rng, S, 100, 0, bs, slack=4, spare=S * 4)
    new = np.ones(S, dtype=np.int64)
    sl, bt, fc, q = i32(cached), i32(table), i32([len(stack)]), i32(new)
    free = i32(stack)
    outs = dict(seq_lens=sl, free_count_out=fc, cu_q_lens=i32(np.zeros(S + 1)), positions=i32(np.zeros(S)),
                slot_mapping=torch.zeros(S, dtype=torch.int64, device=DEV))
    call = lambda: pa.metis_plan_step(q, sl, bt, free, fc, block_size=bs, num_tokens=S, num_blocks=nb, **outs)
    keep = [x.clone() for x in (sl, bt, fc)]
    call()  # the first call on a device raises the kernel's shared memory limit
    for x, y in zip((sl, bt, fc), keep):
        x.copy_(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x, y in zip((sl, bt, fc), keep):
        x.copy_(y)
    depth = len(stack)
    for _ in range(steps):
        g.replay()
        ref = oracle.plan_step(new, cached, table, stack, depth, bs, S, nb)
        cached, table, depth = ref["seq_lens"], ref["block_table"], ref["free_count"]
        assert np.array_equal(outs["slot_mapping"].cpu().numpy(), ref["slot_mapping"])
        assert np.array_equal(sl.cpu().numpy(), cached) and int(fc) == depth
    assert np.array_equal(bt.cpu().numpy(), table) and pa.metis_read_status() == 0


def test_on_another_stream_and_refusals():
    rng = np.random.default_rng(7)
    new, cached, table, stack, nb = make(rng, 30, 100, 10, 16)
    ref = oracle.plan_step(new, cached, table, stack, len(stack), 16, int(new.sum()), nb)
    side = torch.cuda.Stream()
    args = [i32(new), i32(cached), i32(table), i32(stack), i32([len(stack)])]
    torch.cuda.synchronize()
    got = pa.metis_plan_step(*args, block_size=16, num_tokens=int(new.sum()), num_blocks=nb, stream=side)
    side.synchronize()
    assert np.array_equal(got.slot_mapping.cpu().numpy(), ref["slot_mapping"])
    kw = dict(block_size=16, num_tokens=8, num_blocks=nb)
    with pytest.raises(TypeError):
        pa.metis_plan_step(args[0].long(), *args[1:], **kw)
    with pytest.raises(ValueError):
        pa.metis_plan_step(args[0], args[1][:-1], *args[2:], **kw)
    with pytest.raises(ValueError):
        pa.metis_plan_step(*args, refcount=i32([0]), **kw)
    with pytest.raises(ValueError):
        pa.metis_plan_step(args[0], args[1], args[2].t(), *args[3:], **kw)
    with pytest.raises(pa.MetisError):
        pa.metis_plan_step(*args, block_size=0, num_tokens=8, num_blocks=nb)
