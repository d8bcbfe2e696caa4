"""Block tables that the kernel directly in front writes: a prefix lookup's page ids are the table of
the call behind it, in one graph, and change between replays."""
import numpy as np
import pytest
import torch

import paged_attention_kv_decode_gb300 as pa
from test_gpu_cache_fp8 import BF16, DEV, F32, Cache, gpu, i32

pytestmark = pytest.mark.gpu


def test_lookup_then_each_call_replayed():
    rng = np.random.default_rng(1)
    S, mb, bs, G, r, D = 4, 6, 16, 2, 4, 64
    n = S * mb
    c = Cache(rng, [mb * bs] * S, G, D, bs, poisoned=False, extra=8)
    lens = i32([96, 50, 17, 81])
    cu = i32([0, 40, 41, 51, 81])
    q = gpu(torch.from_numpy(rng.standard_normal((81, G * r, D))).to(BF16))
    rows = [gpu(torch.from_numpy(rng.standard_normal((81, G, D))).to(BF16)) for _ in range(2)]
    kf, vf = (torch.from_numpy(rng.standard_normal((c.nb, bs, G, D))).to(DEV, F32) for _ in range(2))
    kb, vb = kf.to(BF16), vf.to(BF16)
    offsets = i32([0, 96, 192, 288])
    keys = torch.from_numpy(rng.integers(1, 1 << 60, n)).to(DEV)
    pool = keys.clone()
    hash_table = pa.prefix_table_alloc(256)
    free, count = i32(np.arange(c.nb)), i32([c.nb])
    refs = torch.zeros(c.nb, dtype=torch.int32, device=DEV)
    bt = torch.zeros(S, mb, dtype=torch.int32, device=DEV)
    hits = torch.zeros(n, dtype=torch.uint8, device=DEV)
    ws = torch.empty(max(256, pa.metis_prefix_lookup_workspace_bytes(n)), dtype=torch.uint8, device=DEV)

    def look():
        pa.metis_prefix_lookup(keys, hash_table, free, count, refs, pages_out=bt.view(-1), hits_out=hits, workspace=ws)

    def outputs(table, in_front):
        """Every call that takes a table, `in_front` launched directly before it."""
        outs = []
        in_front()
        outs.append(pa.metis_paged_attn_decode(q[:S].float(), kf, vf, table, lens, 0.1, max_seq_len=96)[0])
        for partition in (0, 32):
            in_front()
            outs.append(pa.metis_paged_attn_decode(q[:S], kb, vb, table, lens, 0.1, max_seq_len=96,
                                                   partition_size=partition)[0])
        in_front()
        outs.append(pa.metis_paged_attn_prefill_chunk(q, cu, kb, vb, table, lens, 0.1, max_seq_len=96)[0])
        cache8 = [x.clone() for x in c.dev]
        for partition in (0, 16, 48):
            in_front()
            outs.append(pa.metis_paged_attn_decode_fp8(q[:S], *cache8, table, lens, 0.1, max_seq_len=96,
                                                       partition_size=partition)[0])
        in_front()
        outs.append(pa.metis_paged_attn_prefill_chunk_fp8(q, cu, *cache8, table, lens, 0.1, max_seq_len=96)[0])
        k, v = (torch.zeros(384, G, D, dtype=BF16, device=DEV) for _ in range(2))
        in_front()
        pa.metis_gather_cache_fp8(*cache8, table, lens, offsets, k_out=k, v_out=v, max_seq_len=96)
        in_front()
        pa.metis_reshape_and_cache_fp8(*rows, *cache8, cu, table, lens)
        return outs + [k, v] + cache8

    look()  # the pages are handed out once; later lookups find them
    torch.cuda.synchronize()
    pa.metis_read_status(clear=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = outputs(bt, look)
    for _ in range(4):
        keys.copy_(pool[torch.from_numpy(rng.permutation(n)).to(DEV)])
        graph.replay()
        torch.cuda.synchronize()
        ref = outputs(bt.clone(), lambda: None)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, ref)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
    assert sorted(bt.view(-1).tolist()) == sorted(set(bt.view(-1).tolist()))
    assert pa.metis_read_status(clear=True) == 0
