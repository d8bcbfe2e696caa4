"""Refusals of the step-planning and norm/rotation calls, on the host (no GPU; nothing is launched)."""
import ctypes

import pytest
import torch

import paged_attention_kv_decode_gb300 as pa
from test_abi import FAKE, lib  # noqa: F401

vp = lambda x: None if x is None else ctypes.c_void_p(x)


def plan(lib, **kw):
    a = dict(q=FAKE, cached=FAKE, held=None, bt=FAKE, stack=FAKE, cap=8, count=FAKE, refs=None, sl=FAKE, ho=None,
             left=FAKE, cu=FAKE, slots=FAKE, pos=FAKE, S=4, T=16, bs=16, mb=8, nb=64)
    a.update(kw)
    return lib.metis_plan_step(vp(a["q"]), vp(a["cached"]), vp(a["held"]), vp(a["bt"]), vp(a["stack"]), a["cap"],
                               vp(a["count"]), vp(a["refs"]), vp(a["sl"]), vp(a["ho"]), vp(a["left"]), vp(a["cu"]),
                               vp(a["slots"]), vp(a["pos"]), a["S"], a["T"], a["bs"], a["mb"], a["nb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(bt=None), -1), (dict(stack=None), -1), (dict(count=None), -1), (dict(cu=None), -1),
    (dict(slots=None), -1), (dict(left=None), -1), (dict(S=-1), -2), (dict(T=-1), -2), (dict(bs=0), -2), (dict(mb=0), -2),
    (dict(nb=0), -2), (dict(cap=-1), -2), (dict(mb=1 << 28, bs=16), -2), (dict(slots=FAKE + 4), -4),
    (dict(held=FAKE + 2), -4), (dict(refs=FAKE + 1), -4), (dict(bt=FAKE + 2), -4),
])
def test_plan_rejects(lib, kw, code):  # noqa: F811
    assert plan(lib, **kw) == code
    assert pa.metis_last_error() != ""


def test_plan_of_no_sequences_is_a_no_op(lib):  # noqa: F811
    assert plan(lib, S=0) == 0


def rope(lib, cache=True, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, cs=FAKE, pos=FAKE, qo=FAKE + 4096, kc=FAKE, vc=FAKE, slots=FAKE, n=4,
             H=8, G=2, D=128, qs=1024, ks=256, vs=256, R=128, P=100, il=0, eps=1e-6, bs=16, nb=64, dt=pa.METIS_BF16)
    a.update(kw)
    head = (vp(a["q"]), vp(a["k"]))
    mid = (vp(a["qw"]), vp(a["kw"]), vp(a["cs"]), vp(a["pos"]), vp(a["qo"]), vp(a["kc"]))
    size = (a["n"], a["H"], a["G"], a["D"], a["qs"], a["ks"])
    tail = (a["R"], a["P"], a["il"], a["eps"])
    if cache:
        return lib.metis_qk_norm_rope_and_cache(*head, vp(a["v"]), *mid, vp(a["vc"]), vp(a["slots"]), *size, a["vs"], *tail,
                                                a["bs"], a["nb"], a["dt"], None)
    return lib.metis_qk_norm_rope(*head, *mid, *size, *tail, a["dt"], None)


@pytest.mark.parametrize("cache", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(cs=None), -1), (dict(pos=None), -1), (dict(qo=None), -1), (dict(n=-1), -2),
    (dict(H=0), -2), (dict(P=0), -2), (dict(D=96), -3), (dict(R=24), -3), (dict(R=144), -3), (dict(dt=3), -3),
    (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2), (dict(qs=1020), -2), (dict(qs=1028), -4), (dict(ks=8), -2),
    (dict(q=FAKE + 8), -4), (dict(qw=FAKE + 2), -4), (dict(pos=FAKE + 1), -4), (dict(qo=FAKE, qs=2048), -2),
])
def test_norm_rope_rejects(lib, cache, kw, code):  # noqa: F811
    assert rope(lib, cache, **kw) == code
    assert pa.metis_last_error() != ""


@pytest.mark.parametrize("kw,code", [(dict(v=None), -1), (dict(slots=None), -1), (dict(vc=None), -1), (dict(bs=0), -2),
                                     (dict(nb=0), -2), (dict(vs=8), -2), (dict(slots=FAKE + 4), -4)])
def test_norm_rope_and_cache_rejects(lib, kw, code):  # noqa: F811
    assert rope(lib, True, **kw) == code


def test_norm_rope_of_no_rows_is_a_no_op(lib):  # noqa: F811
    assert rope(lib, True, n=0) == 0 and rope(lib, False, n=0) == 0


def test_binding_refuses_cpu_tensors(lib):  # noqa: F811
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.metis_plan_step(i, i, i.view(1, 2), i, i[:1], block_size=16, num_tokens=2, num_blocks=4)
    x = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.metis_qk_norm_rope(x, x, None, None)


def test_rope_table_on_the_host():
    t = pa.rope_table(100, 16, base=500.0, device="cpu")
    assert t.shape == (100, 16) and t.dtype == torch.float32
    angle = 99 * 500.0 ** (-2 * 5 / 16)
    assert abs(t[99, 5].item() - torch.tensor(angle, dtype=torch.float64).cos().item()) <= 2 ** -24
    assert abs(t[99, 13].item() - torch.tensor(angle, dtype=torch.float64).sin().item()) <= 2 ** -24


def window(lib, prefill, **kw):
    a = dict(q=FAKE, cu=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, out=FAKE, lse=None, S=4, T=8, H=32, G=8, D=128, bs=16, mb=8,
             nb=64, dt=pa.METIS_BF16, scale=0.1, W=100, K=4, max_len=128, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    tail = (a["H"], a["G"], a["D"], a["bs"], a["mb"], a["nb"], a["dt"], a["scale"], a["W"], a["K"], a["max_len"])
    ptrs = (vp(a["k"]), vp(a["v"]), vp(a["bt"]), vp(a["sl"]), vp(a["out"]), vp(a["lse"]), a["S"])
    if prefill:
        return lib.metis_paged_attn_prefill_chunk_window(vp(a["q"]), vp(a["cu"]), *ptrs, a["T"], *tail, vp(a["ws"]),
                                                         a["ws_bytes"], None)
    return lib.metis_paged_attn_decode_window(vp(a["q"]), *ptrs, *tail, None)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(bt=None), -1), (dict(out=None), -1), (dict(S=-1), -2), (dict(W=0), -2), (dict(W=-5), -2),
    (dict(K=-1), -2), (dict(H=30), -2), (dict(D=96), -3), (dict(bs=8), -3), (dict(dt=7), -3), (dict(q=FAKE + 2), -4),
    (dict(sl=FAKE + 1), -4), (dict(scale=float("nan")), -2), (dict(mb=1 << 28, bs=64), -2), (dict(max_len=0), -2),
])
def test_window_rejects(lib, prefill, kw, code):  # noqa: F811
    assert window(lib, prefill, **kw) == code
    assert pa.metis_last_error() != ""


def test_window_limits_of_each_call(lib):  # noqa: F811
    assert window(lib, False, H=72, G=8) == -3 and window(lib, False, S=70000) == -2
    assert window(lib, True, H=24, G=8) == -3 and window(lib, True, ws=None) == -5 and window(lib, True, dt=pa.METIS_F32) == -3
    assert window(lib, False, S=0) == 0 and window(lib, True, S=0) == 0 and window(lib, True, T=0) == 0


def shared(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, cu=FAKE, pl=FAKE, out=FAKE, lse=None, S=4, n=2, H=32, G=8, D=128,
             bs=16, mb=8, nb=64, dt=pa.METIS_BF16, scale=0.1, max_len=128, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return lib.metis_paged_attn_decode_shared(
        *(vp(a[x]) for x in ("q", "k", "v", "bt", "sl", "cu", "pl", "out", "lse")),
        *(a[x] for x in ("S", "n", "H", "G", "D", "bs", "mb", "nb", "dt", "scale", "max_len")), vp(a["ws"]), a["ws_bytes"],
        None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(cu=None), -1), (dict(pl=None), -1), (dict(out=None), -1), (dict(S=-1), -2), (dict(n=-1), -2),
    (dict(H=30), -2), (dict(H=24), -3), (dict(H=128), -3), (dict(D=96), -3), (dict(bs=8), -3), (dict(dt=pa.METIS_F32), -3),
    (dict(q=FAKE + 2), -4), (dict(cu=FAKE + 2), -4), (dict(scale=float("nan")), -2), (dict(S=70000), -2),
    (dict(mb=1 << 26, nb=1 << 26, max_len=1 << 30, S=4000, n=4000), -2),  # more tiles than fit in int32
])
def test_shared_rejects(lib, kw, code):  # noqa: F811
    assert shared(lib, **kw) == code
    assert pa.metis_last_error() != ""


def test_shared_of_no_sequences_and_workspace(lib):  # noqa: F811
    assert shared(lib, S=0) == 0
    assert pa.metis_shared_workspace_bytes(0, 8, 2, 64, 1) == 0 and pa.metis_shared_workspace_bytes(4, 9, 2, 64, 1) == 0
