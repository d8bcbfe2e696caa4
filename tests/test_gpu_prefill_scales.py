"""bf16 chunked prefill: softmax scales far below 1e-30 and of zero, beside query rows as far above one."""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from paged_attention_kv_decode_gb300 import workloads as wl
from helpers import assert_lse, assert_parity, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,scale", [(1e30, 1e-31), (1e30, -1e-31), (1e30, 0.0), (1e35, 2e-36), (1e-30, 1e29)])
def test_scale_and_queries_far_apart(size, scale):
    case = wl.make_prefill_case(9, [40, 0, 300], [130, 33, 1], H=8, G=2, D=128, bs=16, dtype=torch.bfloat16, scale=scale)
    q = (case.q.double() * size).to(torch.bfloat16)
    ref, lse_ref = oracle.paged_prefill(q, case.cu_q_lens, case.k_cache, case.v_cache, case.block_table, case.seq_lens, scale)
    out, lse = pa.metis_paged_attn_prefill_chunk(dev(q), dev(case.cu_q_lens), dev(case.k_cache), dev(case.v_cache),
                                                 dev(case.block_table), dev(case.seq_lens), scale,
                                                 max_seq_len=case.max_seq_len, want_lse=True)
    assert_parity(out, ref, torch.bfloat16)
    assert_lse(lse, lse_ref, torch.bfloat16)
    assert np.isfinite(ref).all()
