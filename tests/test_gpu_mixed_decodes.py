"""Many decodes on few SMs beside chunks: each group of warps walks several items through one ring."""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from helpers import assert_lse, assert_parity
from test_gpu_cache_fp8 import BF16, STEP, Cache, attention, check, check_lse, gpu, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 32)])
def test_groups_walk_several_items(D, bs):
    """60 decodes x 4 heads beside 1,500 queries that take nearly all SMs, over the 8-bit cache and over
    the same values in bf16; twenty runs give the same bits."""
    rng = np.random.default_rng(D)
    lens = [int(n) for n in rng.integers(1, 400, 60)] + [1500]
    q_lens = [1] * 60 + [1500]
    G, r = 4, 2
    c = Cache(rng, lens, G, D, bs, spread=0.0, poisoned=False)
    q = torch.from_numpy(rng.standard_normal((sum(q_lens), G * r, D))).to(BF16)
    cu = i32(np.concatenate([[0], np.cumsum(q_lens)]))
    pa.metis_read_status(clear=True)
    call = lambda: pa.metis_paged_attn_prefill_chunk_fp8(gpu(q), cu, *c.dev, c.bt, c.sl, 0.1, max_seq_len=1500, want_lse=True)
    out, lse = call()
    rows = [(s, lens[s]) for s in range(60)]
    ref, tol, rl, lt = attention(c, q[:60].double().numpy(), rows, 0.1, STEP[BF16])
    check(out[:60], ref, tol, BF16, "decodes")
    check_lse(lse[:60], rl, lt)
    for _ in range(20):
        again, _ = call()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    # the same values as a bf16 cache (codes times a power of two are exact in bf16)
    k, v = (torch.from_numpy(oracle.dequantize(a, b)).to(BF16) for a, b in ((c.k, c.ks), (c.v, c.vs)))
    kd, vd = gpu(k), gpu(v)
    call = lambda: pa.metis_paged_attn_prefill_chunk(gpu(q), cu, kd, vd, c.bt, c.sl, 0.1, max_seq_len=1500, want_lse=True)
    out, lse = call()
    assert_parity(out[:60], ref, BF16)
    assert_lse(lse[:60], rl, BF16)
    for _ in range(20):
        again, _ = call()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert pa.metis_read_status() == 0
