"""The plan of a batch without sequences: rows of padding, offsets and depth, as of any other batch."""
import pytest
import torch

import paged_attention_kv_decode_gb300 as pa
from test_gpu_step_plan import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    pa.metis_read_status(clear=True)
    yield


def dirty(T):
    """Outputs that hold anything."""
    return dict(seq_lens=i32([]), cu_q_lens=i32([77]), positions=torch.full((T,), 99, dtype=torch.int32, device=DEV),
                slot_mapping=torch.full((T,), 5, dtype=torch.int64, device=DEV), free_count_out=i32([123456]))


@pytest.mark.parametrize("T", [0, 1, 40, 100000])
@pytest.mark.parametrize("depth,want", [(3, 3), (0, 0), (-4, 0), (9, 5)])
@pytest.mark.parametrize("passed", [True, False])
def test_rows_are_padding_and_the_depth_is_kept(T, depth, want, passed):
    # (memory that the call is then given holds something else)
    for _ in range(4):
        torch.full((max(T, 1),), 12, dtype=torch.int64, device=DEV)
    stack, count = i32([4, 3, 2, 1, 0]), i32([depth])
    got = pa.metis_plan_step(i32([]), i32([]), i32([]).view(0, 8), stack, count, block_size=16, num_tokens=T, num_blocks=9,
                             **(dirty(T) if passed else {}))
    torch.cuda.synchronize()
    assert got.slot_mapping.tolist() == [-1] * T and got.positions.tolist() == [0] * T
    assert got.cu_q_lens.tolist() == [0] and got.free_count.tolist() == [want] and got.seq_lens.shape == (0,)
    assert count.tolist() == [depth] and pa.metis_read_status() == 0


def test_in_place_on_another_stream_and_captured():
    side, count, out = torch.cuda.Stream(), i32([9]), dirty(20)
    out["free_count_out"] = count
    call = lambda **kw: pa.metis_plan_step(i0, i0, t0, stack, count, block_size=16, num_tokens=20, num_blocks=9, **out, **kw)
    i0, t0, stack = i32([]), i32([]).view(0, 8), i32([4, 3, 2, 1, 0])
    torch.cuda.synchronize()
    got = call(stream=side)
    side.synchronize()
    assert got.slot_mapping.tolist() == [-1] * 20 and count.tolist() == [5]
    got = call(stream=side.cuda_stream)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out["slot_mapping"].fill_(3)
    out["cu_q_lens"].fill_(3)
    g.replay()
    torch.cuda.synchronize()
    assert out["slot_mapping"].tolist() == [-1] * 20 and out["cu_q_lens"].tolist() == [0] and count.tolist() == [5]
