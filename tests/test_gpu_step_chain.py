"""The calls of a serving step one behind another, as a layer would make them: index arrays, norm and rotation
into the pages, attention.  Every array between them is the one before's output, nothing waits in between; each is
checked afterwards against its oracle on what it was given."""
import numpy as np
import pytest
import torch

import oracle
import paged_attention_kv_decode_gb300 as pa
from test_gpu_qk_norm_rope import close, f64
from test_gpu_window import compare, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
H, G, D, BS = 8, 2, 128, 16


class Layer:
    """One layer's cache, page stack and tables; every call goes to `stream`."""

    def __init__(self, rng, S, width, pages, max_position=4000):
        self.S, self.pages = S, pages
        self.k, self.v = (torch.full((pages, BS, G, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
        self.table = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(S, dtype=torch.int32, device=DEV)
        self.free = i32(rng.permutation(pages))
        self.count = i32([pages])
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.turn = pa.rope_table(max_position, D)
        self.w = [torch.from_numpy(rng.uniform(0.5, 1.5, D)).to(BF16).to(DEV) for _ in range(2)]
        self.scale = D ** -0.5

    def rows(self, x):
        return x[:, :H], x[:, H:H + G], x[:, H + G:]

    def step(self, q_lens, x, **held):
        """Plan and write the step's rows x [T, H + 2 G, D]; returns the plan and the queries."""
        plan = pa.metis_plan_step(q_lens, self.lens, self.table, self.free, self.count, block_size=BS,
                                  num_tokens=x.shape[0], num_blocks=self.pages, refcount=self.refs, seq_lens=self.lens,
                                  free_count_out=self.count, **held)
        q = pa.metis_qk_norm_rope_and_cache(*self.rows(x), self.turn, plan.positions, self.k, self.v, plan.slot_mapping,
                                            q_weight=self.w[0], k_weight=self.w[1])
        return plan, q

    def check_rows(self, x, plan, q):
        """Queries, keys and values of the step against the oracle of norm and rotation."""
        xq, xk, xv = (f64(t) for t in self.rows(x))
        pos, slots = plan.positions.tolist(), plan.slot_mapping.cpu().numpy()
        want, add = oracle.norm_rope(xq, f64(self.w[0]), f64(self.turn), pos, 1e-6, False)
        close(q, want, add, BF16)
        live = slots >= 0
        want, add = oracle.norm_rope(xk, f64(self.w[1]), f64(self.turn), pos, 1e-6, False)
        close(self.k.view(-1, G, D)[torch.from_numpy(slots[live]).to(DEV)], want[live], add[live], BF16)
        assert np.array_equal(f64(self.v.view(-1, G, D)[torch.from_numpy(slots[live]).to(DEV)]), xv[live])


def rows(rng, T):
    return torch.from_numpy(rng.standard_normal((T, H + 2 * G, D)) * 2).to(BF16).to(DEV)


@pytest.mark.parametrize("window,sinks", [(50, 4), (10 ** 6, 0)])
def test_prompts_then_captured_decode_steps(window, sinks):
    """Two chunked-prefill steps with decodes and padding, then a captured decode step replayed: lengths, pages and
    the stack advance on the GPU."""
    rng = np.random.default_rng(window % 100)
    S, padding = 6, 5
    lay = Layer(rng, S, 30, 140)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cached, table, depth = np.zeros(S, np.int64), np.full((S, 30), -1), lay.pages
    with torch.cuda.stream(side):
        for new in ([100, 0, 37, 1, 200, 64], [60, 90, 1, 1, 33, 1]):
            x = rows(rng, sum(new) + padding)
            plan, q = lay.step(i32(new), x)
            out = torch.full_like(q, 7.0)
            _, lse = pa.metis_paged_attn_prefill_chunk_window(q, plan.cu_q_lens, lay.k, lay.v, lay.table, lay.lens,
                                                              lay.scale, window, sinks, out=out, max_seq_len=480,
                                                              want_lse=True)
            side.synchronize()
            ref = oracle.plan_step(new, cached, table, lay.free.tolist(), depth, BS, x.shape[0], lay.pages)
            cached, table, depth = ref["seq_lens"], ref["block_table"], ref["free_count"]
            assert np.array_equal(lay.table.cpu().numpy(), table) and int(lay.count) == depth
            assert np.array_equal(plan.slot_mapping.cpu().numpy(), ref["slot_mapping"]) and ref["status"] == 0
            lay.check_rows(x, plan, q)
            T = sum(new)
            compare(out[:T], lse[:T], oracle.paged_window(q[:T].cpu(), ref["cu_q_lens"], lay.k.cpu(), lay.v.cpu(), table,
                                                          cached, lay.scale, window, sinks), BF16)
            assert (out[T:] == 7).all()

        x, ones = rows(rng, S), i32([1] * S)
        outs = dict(cu_q_lens=i32([0] * (S + 1)), positions=i32([0] * S),
                    slot_mapping=torch.zeros(S, dtype=torch.int64, device=DEV))
        qo, out = torch.empty(S, H, D, dtype=BF16, device=DEV), torch.empty(S, H, D, dtype=BF16, device=DEV)
        lse = torch.empty(S, H, device=DEV)

        def decode():
            pa.metis_plan_step(ones, lay.lens, lay.table, lay.free, lay.count, block_size=BS, num_tokens=S,
                               num_blocks=lay.pages, refcount=lay.refs, seq_lens=lay.lens, free_count_out=lay.count, **outs)
            pa.metis_qk_norm_rope_and_cache(*lay.rows(x), lay.turn, outs["positions"], lay.k, lay.v, outs["slot_mapping"],
                                            q_weight=lay.w[0], k_weight=lay.w[1], q_out=qo)
            pa.metis_paged_attn_decode_window(qo, lay.k, lay.v, lay.table, lay.lens, lay.scale, window, sinks, out=out,
                                              lse_out=lse, max_seq_len=480)

        state = [t.clone() for t in (lay.lens, lay.table, lay.count, lay.refs)]
        decode()  # the first call on a device raises the kernels' limits
        for t, s in zip((lay.lens, lay.table, lay.count, lay.refs), state):
            t.copy_(s)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            decode()
        for t, s in zip((lay.lens, lay.table, lay.count, lay.refs), state):
            t.copy_(s)
        for _ in range(20):
            x.copy_(rows(rng, S))
            g.replay()
            side.synchronize()
            ref = oracle.plan_step([1] * S, cached, table, lay.free.tolist(), depth, BS, S, lay.pages)
            cached, table, depth = ref["seq_lens"], ref["block_table"], ref["free_count"]
            assert np.array_equal(lay.lens.cpu().numpy(), cached) and np.array_equal(lay.table.cpu().numpy(), table)
            compare(out, lse, oracle.paged_window_decode(qo.cpu(), lay.k.cpu(), lay.v.cpu(), table, cached, lay.scale,
                                                         window, sinks), BF16)
    assert pa.metis_read_status() == 0


def test_prompts_behind_cached_system_prompts_then_shared_decodes():
    """Two system prompts' pages come from the prefix cache; the members' prompts and first decode share them."""
    rng = np.random.default_rng(3)
    members, system = [5, 4], [96, 160]
    prompts = [np.concatenate([np.full(system[g], 100 + g) + np.arange(system[g]), rng.integers(0, 1000, rng.integers(3, 60))])
               for g in range(2) for _ in range(members[g])]
    S = len(prompts)
    lay = Layer(rng, S, 20, 120)
    pages = [len(p) // BS for p in prompts]
    cu_tokens = np.concatenate([[0], np.cumsum([len(p) for p in prompts])])
    cu_pages = np.concatenate([[0], np.cumsum(pages)])
    keys = pa.metis_prefix_block_hashes(i32(np.concatenate(prompts)), i32(cu_tokens), i32(cu_pages), BS, int(cu_pages[-1]))
    hashed = pa.prefix_table_alloc(1024)
    got, hits = pa.metis_prefix_lookup(keys, hashed, lay.free, lay.count, lay.refs)
    # the scheduler: full pages are dealt out, of which hits need no computing (of the first member: all do)
    hit = hits.cpu().numpy().astype(bool)
    cached = [int(np.argmin(np.append(hit[cu_pages[s]:cu_pages[s + 1]], False))) * BS for s in range(S)]
    cached = [min(c, len(p) - 1) // BS * BS for c, p in zip(cached, prompts)]
    for s in range(S):
        lay.table[s, :pages[s]] = got[cu_pages[s]:cu_pages[s + 1]]
    lay.lens.copy_(i32(cached))
    new = [len(p) - c for p, c in zip(prompts, cached)]
    # a token's row depends on the token and its position alone, as the first layer's does
    embed = rows(rng, 1100)
    x = torch.cat([embed[torch.from_numpy(p[c:]).to(DEV)] for p, c in zip(prompts, cached)])
    plan, q = lay.step(i32(new), x, held_blocks=i32(pages))
    assert plan.held_blocks.tolist() == [-(-len(p) // BS) for p in prompts]
    out, lse = pa.metis_paged_attn_prefill_chunk(q, plan.cu_q_lens, lay.k, lay.v, lay.table, lay.lens, lay.scale,
                                                 max_seq_len=320, want_lse=True)
    lay.check_rows(x, plan, q)
    table, lens = lay.table.cpu().numpy(), lay.lens.cpu().numpy()
    assert lens.tolist() == [len(p) for p in prompts]
    assert all((table[s, :system[g] // BS] == table[a, :system[g] // BS]).all()
               for g, (a, b) in enumerate([(0, 5), (5, 9)]) for s in range(a, b))
    x = rows(rng, S)
    plan, q = lay.step(i32([1] * S), x)
    shared, ls = pa.metis_paged_attn_decode_shared(q, lay.k, lay.v, lay.table, lay.lens, i32([0, 5, 9]), i32(system),
                                                   lay.scale, max_seq_len=320, want_lse=True)
    torch.cuda.synchronize()
    args = q.cpu(), lay.k.cpu(), lay.v.cpu(), lay.table.cpu().numpy(), lay.lens.cpu().numpy(), lay.scale
    o, l = oracle.paged_decode(*args)
    compare(shared, ls, (o, l, oracle.paged_window_decode(*args, 2 ** 31, 0)[2]), BF16)
    plain, pl = pa.metis_paged_attn_decode(q, lay.k, lay.v, lay.table, lay.lens, lay.scale, max_seq_len=320, want_lse=True)
    assert (ls - pl).abs().max() <= 2e-3
    assert pa.metis_read_status() == 0
