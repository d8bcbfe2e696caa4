"""The operators around a step of paged attention, as measured: cases, plain forms, exact values.

* ``plan``     the index arrays of a step, from the requests' lengths: pages for the new tokens from
               the top of a stack of free pages (sequence by sequence), block-table entries, slots,
               positions, offsets.
* ``rotate``   queries and keys of the new tokens normalised per head (RMS norm with a weight per
               dimension), rotated by their positions, and keys and values written into their pages.
* ``window``   decode and chunked prefill in which a query at position p sees the last ``window``
               tokens (p among them) and the first ``sinks`` tokens.
* ``shared``   decode of a batch whose sequences share their first tokens in groups: the members of
               group g (neighbours in the batch) have the same first ``prefix_lens[g]`` tokens.

Caches are ``[num_blocks, block_size, kv_heads, head_dim]``, token t of sequence s in block
``block_table[s, t // block_size]``, slot ``t % block_size``.  Lengths come from the case alone
(``lengths`` seeds them), every value from the seed.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _plan(*, seqs, cached_lo, cached_hi, new_lo, new_hi, idle=0, block=16, padding=0, lengths=1):
    return dict(op="plan", seqs=seqs, cached_lo=cached_lo, cached_hi=cached_hi, new_lo=new_lo, new_hi=new_hi,
                idle=idle, block=block, padding=padding, lengths=lengths)


def _rotate(*, rows, padding=0, heads=32, kv_heads=8, dim=128, rotary=None, norm=True, interleaved=False, block=16,
            dtype="bf16", positions=8192, packed=True):
    return dict(op="rotate", rows=rows, padding=padding, heads=heads, kv_heads=kv_heads, dim=dim,
                rotary=dim if rotary is None else rotary, norm=norm, interleaved=interleaved, block=block, dtype=dtype,
                positions=positions, packed=packed)


def _window(op, *, window, sinks, chunks=0, chunk_lo=1, chunk_hi=1, singles=0, empty=0, prefix_lo=0, prefix_hi=0,
            heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", lengths=1):
    return dict(op=op, window=window, sinks=sinks, chunks=chunks, chunk_lo=chunk_lo, chunk_hi=chunk_hi,
                singles=singles, empty=empty, prefix_lo=prefix_lo, prefix_hi=prefix_hi, heads=heads,
                kv_heads=kv_heads, dim=dim, block=block, dtype=dtype, lengths=lengths)


def _shared(*, groups, members_lo, members_hi, prefix_lo, prefix_hi, own_lo, own_hi, empty=0, heads=32, kv_heads=8,
            dim=128, block=16, lengths=1):
    return dict(op="shared", groups=groups, members_lo=members_lo, members_hi=members_hi, prefix_lo=prefix_lo,
                prefix_hi=prefix_hi, own_lo=own_lo, own_hi=own_hi, empty=empty, heads=heads, kv_heads=kv_heads,
                dim=dim, block=block, lengths=lengths)


def listed():
    return [
        # one decode step of a batch of 64: a token each, now and then a new page
        dict(_plan(seqs=64, cached_lo=511, cached_hi=4095, new_lo=1, new_hi=1, lengths=2), name="plan_step_64"),
        # 4,096 prompts behind cached system prompts, with a padded token count
        dict(_plan(seqs=4096, cached_lo=576, cached_hi=640, new_lo=32, new_hi=160, idle=40, padding=1000, lengths=9),
             name="plan_prompts_4096"),
        # the new rows of a decode step of 64
        dict(_rotate(rows=64), name="rotate_step_64"),
        # the new rows of a chunked-prefill step: 16 chunks of 512 and 48 single rows
        dict(_rotate(rows=8240), name="rotate_chunks"),
        # a ragged fp32 batch: 64-dim heads rotated in their first 32 dims by neighbouring pairs, padded rows, no norm
        dict(_rotate(rows=1789, padding=259, heads=16, kv_heads=4, dim=64, rotary=32, norm=False, interleaved=True,
                     block=64, dtype="fp32", packed=False), name="rotate_ragged_fp32"),
        # the batched decode step with a window of 4,096 over contexts of 512..32,768 tokens
        dict(_window("window_decode", window=4096, sinks=4, singles=64, prefix_lo=511, prefix_hi=32767, lengths=2),
             name="window_decode_batch_64"),
        # few sequences with long contexts and a short window
        dict(_window("window_decode", window=1024, sinks=16, singles=8, prefix_lo=32767, prefix_hi=131071, lengths=3),
             name="window_decode_long_8"),
        # four short sequences in fp32
        dict(_window("window_decode", window=16, sinks=2, singles=4, prefix_hi=63, heads=4, kv_heads=1, dim=64,
                     dtype="fp32", lengths=1), name="window_decode_tiny_fp32"),
        # the chunked-prefill step: 16 chunks of 512 over prefixes up to 4,096, with 48 decodes
        dict(_window("window_prefill", window=1024, sinks=4, chunks=16, chunk_lo=512, chunk_hi=512, singles=48,
                     prefix_hi=4096, lengths=4), name="window_prefill_mixed"),
        # one long chunk over a long prefix
        dict(_window("window_prefill", window=4096, sinks=64, chunks=1, chunk_lo=2048, chunk_hi=2048, prefix_lo=14336,
                     prefix_hi=14336, lengths=7), name="window_prefill_long_chunk"),
        # a batch of 64 behind one long document
        dict(_shared(groups=1, members_lo=64, members_hi=64, prefix_lo=16384, prefix_hi=16384, own_lo=16, own_hi=1024,
                     lengths=10), name="shared_document_64"),
        # 1,024 sequences behind 16 system prompts
        dict(_shared(groups=16, members_lo=64, members_hi=64, prefix_lo=576, prefix_hi=640, own_lo=32, own_hi=160,
                     lengths=11), name="shared_prompts_1024"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rotate", "window_decode", "window_prefill", "shared"])
    block = rng.choice([16, 32, 64])
    lengths = rng.randrange(1 << 20)
    if op == "plan":
        seqs = _log(rng, 1, 4096)
        cached = _log(rng, 1, 8192)
        new = _log(rng, 1, max(1, 400000 // seqs))
        return _plan(seqs=seqs, cached_lo=rng.choice([0, cached]), cached_hi=cached, new_lo=rng.choice([0, 1, new]),
                     new_hi=new, idle=rng.choice([0, 1, 5]), block=block, padding=rng.choice([0, 0, 1, 77]),
                     lengths=lengths)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128])
    if op == "rotate":
        return _rotate(rows=_log(rng, 1, 8192), padding=rng.choice([0, 0, 3, 64]), kv_heads=kv_heads,
                       heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 8]) if kv_heads < 8 else 32, dim=dim,
                       rotary=rng.choice([dim, dim, dim // 2, 16]), norm=rng.random() < 0.7,
                       interleaved=rng.random() < 0.3, block=block, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                       positions=_log(rng, 1, 131072), packed=rng.random() < 0.7)
    if op == "shared":
        ratio = rng.choice([1, 2, 4, 8])
        groups = _log(rng, 1, 16)
        members = _log(rng, 1, 512 // groups)
        return _shared(groups=groups, members_lo=rng.choice([1, members]), members_hi=members,
                       prefix_lo=rng.choice([0, 16]), prefix_hi=_log(rng, 16, 8192 // groups),
                       own_lo=1, own_hi=_log(rng, 1, max(2, 32768 // (groups * members))), empty=rng.choice([0, 0, 2]),
                       heads=kv_heads * ratio, kv_heads=kv_heads, dim=dim, block=block, lengths=lengths)
    window = _log(rng, 1, 4096)
    sinks = rng.choice([0, 0, 1, 4, 17, 130])
    at = dict(window=window, sinks=sinks, kv_heads=kv_heads, dim=dim, block=block, empty=rng.choice([0, 0, 1, 3]),
              lengths=lengths)
    if op == "window_decode":
        at["heads"] = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        at["dtype"] = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        at["singles"] = _log(rng, 1, 64)
        at["prefix_hi"] = _log(rng, 1, 32767)
    else:
        at["heads"] = kv_heads * rng.choice([1, 2, 4, 8] if kv_heads > 4 else [1, 2, 4, 8, 16])
        at["chunks"] = _log(rng, 1, 16)
        at["chunk_hi"] = _log(rng, 2, 2048 // at["chunks"])
        at["chunk_lo"] = rng.choice([1, at["chunk_hi"]])
        at["singles"] = rng.choice([0, 0, _log(rng, 1, 32)])
        at["prefix_hi"] = _log(rng, 1, 8192)
        # the plain form holds every sequence's padded score matrix: keep it below the listed ones'
        seqs = at["chunks"] + at["singles"]
        most = 1_000_000_000 // (seqs * at["heads"] * at["chunk_hi"])
        at["prefix_hi"] = max(1, min(at["prefix_hi"], most - at["chunk_hi"]))
    return _window(op, **at)


def _lengths(case):
    """Per sequence (cached tokens with the queried or new ones, queried or new tokens), in batch order."""
    rng = random.Random(case["lengths"])
    got = []
    if case["op"] == "plan":
        for _ in range(case["seqs"]):
            new = rng.randint(case["new_lo"], case["new_hi"])
            got.append((rng.randint(case["cached_lo"], case["cached_hi"]) + new, new))
        got += [(0, 0)] * case["idle"]
    else:
        for _ in range(case["chunks"]):
            q = rng.randint(case["chunk_lo"], case["chunk_hi"])
            got.append((rng.randint(case["prefix_lo"], case["prefix_hi"]) + q, q))
        for _ in range(case["singles"]):
            got.append((rng.randint(case["prefix_lo"], case["prefix_hi"]) + 1, 1))
        got += [(0, 0)] * case["empty"]
    rng.shuffle(got)
    return got


def _groups(case):
    """Per group (tokens shared, [tokens of each member]): whole pages are shared, empty members have none."""
    rng = random.Random(case["lengths"])
    got = []
    for _ in range(case["groups"]):
        shared = rng.randint(case["prefix_lo"], case["prefix_hi"]) // case["block"] * case["block"]
        members = [shared + rng.randint(case["own_lo"], case["own_hi"])
                   for _ in range(rng.randint(case["members_lo"], case["members_hi"]))]
        members += [0] * case["empty"]
        rng.shuffle(members)
        got.append((shared, members))
    return got


def _seen(case, n, q):
    """(query, key) pairs and different keys of a sequence of n tokens whose last q are queried."""
    w, k = case["window"], case["sinks"]
    pairs = 0
    for p in range(n - q, n):
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(k, lo)
    lo = max(0, n - q - w + 1)
    return pairs, (n - lo + min(k, lo) if q else 0)


def work(case):
    op = case["op"]
    if op == "plan":
        seqs = _lengths(case)
        bs = case["block"]
        rows = sum(q for _, q in seqs)
        new = sum(-(-n // bs) - -(-(n - q) // bs) for n, q in seqs)
        # a table entry read for the page a sequence is in; entry, stack and count of a new page; 12 bytes a row
        return {"bytes": 16 * len(seqs) + 4 * len(seqs) + 12 * new + 12 * (rows + case["padding"]), "flops": 4.0 * rows}
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    size = 4 if case.get("dtype") == "fp32" else 2
    if op == "rotate":
        rows = case["rows"]
        angles = 4 * case["rotary"] * min(rows, case["positions"])
        return {"bytes": 2 * rows * (H + 2 * G) * D * size + angles + 12 * (rows + case["padding"]) + 2 * D * size,
                "flops": 8.0 * rows * (H + G) * D}
    if op == "shared":
        keys = pairs = S = pages = 0
        for shared, members in _groups(case):
            live = [n for n in members if n]
            keys += (shared if live else 0) + sum(n - shared for n in live)
            pairs += sum(live)
            S += len(members)
            pages += sum(-(-(n - shared) // case["block"]) for n in live) + shared // case["block"]
        return {"bytes": 4 * keys * G * D + 4 * S * H * D + 4 * S * H + 4 * (pages + S), "flops": 4.0 * pairs * H * D}
    keys = pairs = rows = pages = 0
    seqs = _lengths(case)
    for n, q in seqs:
        p, k = _seen(case, n, q)
        pairs, keys, rows, pages = pairs + p, keys + k, rows + q, pages + -(-k // case["block"])
    return {"bytes": 2 * keys * G * D * size + 2 * rows * H * D * size + 4 * rows * H + 4 * (pages + 2 * len(seqs)),
            "flops": 4.0 * pairs * H * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _cu(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


def _prepare_plan(case, gen):
    seqs = _lengths(case)
    bs = case["block"]
    held = [-(-(n - q) // bs) for n, q in seqs]
    after = [-(-n // bs) for n, _ in seqs]
    nb, wide = sum(after) + 5, max(1, max(after)) + 1
    order = torch.randperm(nb, device=DEV, generator=gen)
    first = _ints(_cu(held)[:-1], torch.int64)
    at = torch.arange(wide, device=DEV)
    table = order[(first[:, None] + at).clamp(max=nb - 1)].where(at < _ints(held)[:, None], torch.full_like(at, -1))
    free = order[sum(held):].to(torch.int32)
    count = torch.zeros(nb, dtype=torch.int32, device=DEV)
    count[order[: sum(held)]] = 1
    rows = sum(q for _, q in seqs)
    return dict(op="plan", block=bs, rows=rows, tokens=rows + case["padding"], num_blocks=nb,
                q_lens=_ints([q for _, q in seqs]), cached_lens=_ints([n - q for n, q in seqs]),
                block_table=table.to(torch.int32).contiguous(), free_stack=free.contiguous(),
                free_count=_ints([free.numel()]), refcount=count)


def _prepare_rotate(case, gen):
    rows, tokens = case["rows"], case["rows"] + case["padding"]
    H, G, D, bs, R = case["heads"], case["kv_heads"], case["dim"], case["block"], case["rotary"]
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16

    def rand(*shape):
        x = torch.randn(*shape, device=DEV, generator=gen)
        return x.mul_(2.0 ** torch.empty(*shape[:2], 1, device=DEV).uniform_(-2.0, 3.0, generator=gen)).to(dtype)

    if case["packed"]:  # the output of one projection, queries, keys and values side by side
        x = rand(tokens, H + 2 * G, D)
        q, k, v = x[:, :H], x[:, H : H + G], x[:, H + G :]
    else:
        q, k, v = rand(tokens, H, D), rand(tokens, G, D), rand(tokens, G, D)
    turn = torch.arange(case["positions"], device=DEV, dtype=torch.float64)[:, None]
    turn = turn * 10000.0 ** (-2.0 * torch.arange(R // 2, device=DEV, dtype=torch.float64) / R)
    nb = -(-tokens // bs) + 4
    slot = torch.randperm(nb * bs, device=DEV, generator=gen)[:tokens]
    slot[rows:] = -1  # padded rows are not written
    st = dict(op="rotate", q=q, k=k, v=v, interleaved=case["interleaved"], slot_mapping=slot.contiguous(), R=R,
              cos_sin=torch.cat([turn.cos(), turn.sin()], 1).float().contiguous(), eps=1e-6, q_weight=None,
              k_weight=None,
              positions=torch.randint(case["positions"], (tokens,), device=DEV, generator=gen, dtype=torch.int32))
    if case["norm"]:
        for x in ("q_weight", "k_weight"):
            st[x] = torch.empty(D, device=DEV).uniform_(0.5, 1.5, generator=gen).to(dtype)
    for x in ("k_cache", "v_cache"):
        st[x] = torch.randn(nb, bs, G, D, device=DEV, generator=gen).to(dtype)
    return st


def _pool(case, gen, slots):
    """K and V pages in use: values whose size differs by head; slots that no token owns (True) hold NaN."""
    nb, bs = slots.shape
    G, D = case["kv_heads"], case["dim"]
    out = []
    for _ in range(2):
        x = torch.randn(nb, bs, G, D, device=DEV, generator=gen)
        x.mul_(2.0 ** torch.empty(1, 1, G, 1, device=DEV).uniform_(-1.0, 1.0, generator=gen))
        x[slots] = math.nan
        out.append(x.to(torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16))
    return out


def _prepare_window(case, gen):
    seqs = _lengths(case)
    H, D, bs, W, K = case["heads"], case["dim"], case["block"], case["window"], case["sinks"]
    wide = max(1, max(-(-n // bs) for n, _ in seqs))
    lens, counts = _ints([n for n, _ in seqs]), _ints([q for _, q in seqs])
    # pages that no query of the step sees have been given back: their entries hold -1
    t = torch.arange(wide, device=DEV) * bs
    oldest = (lens - counts - W + 1).clamp(min=0)[:, None]
    held = (t < lens[:, None]) & ((t + bs > oldest) | (t < K)) & (counts > 0)[:, None]
    total = int(held.sum())
    nb = total + 3
    table = torch.full((len(seqs), wide), -1, dtype=torch.int32, device=DEV)
    table[held] = torch.randperm(nb, device=DEV, generator=gen)[:total].to(torch.int32)
    # tokens behind the last one, and those in kept pages that no query sees, may hold anything
    free = torch.ones(nb, bs, dtype=torch.bool, device=DEV)
    pos = torch.arange(wide * bs, device=DEV)
    seen = ((pos < lens[:, None]) & ((pos >= oldest) | (pos < K))).view(len(seqs), wide, bs)
    free[table[held].long()] = ~seen[held]
    k_cache, v_cache = _pool(case, gen, free)
    decode = case["op"] == "window_decode"
    rows = len(seqs) if decode else sum(q for _, q in seqs)
    q = torch.randn(rows, H, D, device=DEV, generator=gen).to(k_cache.dtype)
    return dict(op=case["op"], window=W, sinks=K, q=q, k_cache=k_cache, v_cache=v_cache, block_table=table,
                seq_lens=lens, cu_q_lens=_ints(_cu([q for _, q in seqs])), scale=1.0 / math.sqrt(D),
                len_max=max(1, max(n for n, _ in seqs)), q_max=max(q for _, q in seqs), rows=rows)


def _prepare_shared(case, gen):
    groups = _groups(case)
    H, D, bs = case["heads"], case["dim"], case["block"]
    wide = max(1, max(-(-n // bs) for _, members in groups for n in members))
    nb = sum(shared // bs + sum(-(-(n - shared) // bs) for n in members if n) for shared, members in groups) + 3
    order = torch.randperm(nb, device=DEV, generator=gen).to(torch.int32)
    lens = [n for _, members in groups for n in members]
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device=DEV)
    free = torch.ones(nb, bs, dtype=torch.bool, device=DEV)
    at = s = 0
    for shared, members in groups:
        common = order[at : at + shared // bs]
        at += shared // bs
        free[common.long()] = False
        for n in members:
            if n:
                mine = -(-(n - shared) // bs)
                table[s, : shared // bs] = common
                table[s, shared // bs : shared // bs + mine] = order[at : at + mine]
                free[order[at : at + mine].long()] = (torch.arange(mine * bs, device=DEV) >= n - shared).view(mine, bs)
                at += mine
            s += 1
    k_cache, v_cache = _pool(case, gen, free)
    q = torch.randn(len(lens), H, D, device=DEV, generator=gen).to(torch.bfloat16)
    return dict(op="shared", q=q, k_cache=k_cache, v_cache=v_cache, block_table=table, seq_lens=_ints(lens),
                cu_group_seqs=_ints(_cu([len(members) for _, members in groups])),
                prefix_lens=_ints([shared for shared, _ in groups]), scale=1.0 / math.sqrt(D), len_max=max(1, max(lens)),
                groups=[(shared, len(members), max(members)) for shared, members in groups])


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    make = {"plan": _prepare_plan, "rotate": _prepare_rotate, "shared": _prepare_shared}
    return make.get(case["op"], _prepare_window)(case, gen)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_plan(st):
    bs, T, table = st["block"], st["tokens"], st["block_table"]
    S, wide = table.shape
    q, before = st["q_lens"].long(), st["cached_lens"].long()
    after = before + q
    held, want = (before + bs - 1) // bs, (after + bs - 1) // bs
    take = (want - held) * (q > 0)
    first = take.cumsum(0) - take  # pages taken by the sequences in front
    lp = torch.arange(wide, device=DEV)
    fresh = (lp >= held[:, None]) & (lp < (held + take)[:, None])
    depth = st["free_count"].long()
    rank = (first - held)[:, None] + lp
    page = st["free_stack"].long()[(depth - 1 - rank).clamp(0, st["free_stack"].numel() - 1)]
    table.copy_(page.to(torch.int32).where(fresh, table))
    refcount = st["refcount"]
    refcount[page[fresh]] = 1
    cu = torch.zeros(S + 1, dtype=torch.int64, device=DEV)
    cu[1:] = q.cumsum(0)
    n = torch.arange(T, device=DEV)
    seq = (torch.searchsorted(cu, n, right=True) - 1).clamp(max=S - 1)
    live = n < cu[-1]
    pos = (before[seq] + n - cu[seq]).where(live, torch.zeros_like(n))
    slot = table[seq, pos // bs].long() * bs + pos % bs
    return {"seq_lens": after.to(torch.int32), "cu_q_lens": cu.to(torch.int32),
            "slot_mapping": slot.where(live, torch.full_like(slot, -1)), "positions": pos.to(torch.int32),
            "free_count": (depth - take.sum()).to(torch.int32), "block_table": table, "refcount": refcount}


def _plain_rotate_one(st, x, weight):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(2, keepdim=True) + st["eps"]) * weight.float()
    R = st["R"]
    turn = st["cos_sin"][st["positions"].long()][:, None]
    c, s = turn[..., : R // 2], turn[..., R // 2 :]
    out = y.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if st["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out.to(x.dtype)


def _plain_rotate(st):
    q = _plain_rotate_one(st, st["q"], st["q_weight"])
    k = _plain_rotate_one(st, st["k"], st["k_weight"])
    slot = st["slot_mapping"]
    live = slot >= 0
    for cache, x in ((st["k_cache"], k), (st["v_cache"], st["v"])):
        cache.view(-1, *cache.shape[2:])[slot[live]] = x[live]
    return q


def _gather(st, at, live):
    """K and V of the tokens `at` of every sequence [S, N], in fp32, zeros where not `live`."""
    bs = st["k_cache"].shape[1]
    at = at.where(live, torch.zeros_like(at))
    page = st["block_table"].long().gather(1, at // bs).where(live, torch.zeros_like(at))
    return [c[page, at % bs].float().masked_fill_(~live[..., None, None], 0.0) for c in (st["k_cache"], st["v_cache"])]


def _softmax(s, v):
    """s [S, G, rows, N] scores (-inf: hidden), v [S, N, G, D]: outputs [S, G, rows, D] and lse [S, G, rows]."""
    m = s.amax(3, keepdim=True)
    p = s.sub_(m.where(torch.isfinite(m), torch.zeros_like(m))).exp_()
    l = p.sum(3, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3))
    return (o / l).masked_fill_(l == 0, 0.0), (m + l.log()).squeeze(3)


def _plain_window_decode(st):
    q, (S, H, D), G = st["q"], st["q"].shape, st["k_cache"].shape[2]
    lens = st["seq_lens"].long()[:, None]
    sinks = torch.arange(min(st["sinks"], st["len_max"]), device=DEV)
    recent = torch.arange(min(st["window"], st["len_max"]), device=DEV)
    lo = (lens - st["window"]).clamp(min=0)
    at = torch.cat([sinks.expand(S, -1), lo + recent], 1)
    live = torch.cat([sinks < torch.minimum(lo, lens), lo + recent < lens], 1)
    k, v = _gather(st, at, live)
    s = torch.matmul(q.float().view(S, G, H // G, D), k.permute(0, 2, 3, 1)).mul_(st["scale"])
    o, lse = _softmax(s.masked_fill_(~live[:, None, None], -math.inf), v)
    return o.view(S, H, D).to(q.dtype), lse.view(S, H)


def _plain_window_prefill(st):
    q, (T, H, D), G, Q, L = st["q"], st["q"].shape, st["k_cache"].shape[2], st["q_max"], st["len_max"]
    S = st["seq_lens"].numel()
    lens, cu = st["seq_lens"].long(), st["cu_q_lens"].long()
    count = cu[1:] - cu[:-1]
    t = torch.arange(L, device=DEV)
    oldest = (lens - count - st["window"] + 1)[:, None]
    k, v = _gather(st, t.expand(S, -1), (t < lens[:, None]) & ((t >= oldest) | (t < st["sinks"])) & (count > 0)[:, None])
    i = torch.arange(Q, device=DEV)
    x = q[(cu[:-1, None] + i).clamp(max=T - 1)].float().view(S, Q, G, H // G, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(x.reshape(S, G, -1, D), k.permute(0, 2, 3, 1)).mul_(st["scale"]).view(S, H, Q, L)
    at = ((lens - count)[:, None] + i)[..., None]  # the position of each query
    seen = (t < lens[:, None, None]) & (t <= at) & ((t > at - st["window"]) | (t < st["sinks"]))
    s.masked_fill_(~seen[:, None], -math.inf)
    o, lse = _softmax(s.view(S, G, -1, L), v)
    seq = torch.repeat_interleave(torch.arange(S, device=DEV), count, output_size=T)
    at = torch.arange(T, device=DEV) - cu[seq]
    o, lse = o.view(S, H, Q, D).transpose(1, 2), lse.view(S, H, Q).transpose(1, 2)
    return o[seq, at].to(q.dtype), lse[seq, at]


def _plain_shared(st):
    q, (S, H, D), (nb, bs, G, _) = st["q"], st["q"].shape, st["k_cache"].shape
    outs, lses, a = [], [], 0
    for shared, n, longest in st["groups"]:
        lens = st["seq_lens"][a : a + n].long()[:, None]
        x = q[a : a + n].float().view(n, G, H // G, D)
        mine = dict(st, block_table=st["block_table"][a : a + n])
        t = torch.arange(shared, max(shared, longest), device=DEV).expand(n, -1)
        k, v = _gather(mine, t, t < lens)
        s = torch.matmul(x, k.permute(0, 2, 3, 1)).mul_(st["scale"]).masked_fill_(~(t < lens)[:, None, None], -math.inf)
        # the shared tokens once for the whole group, by the table of its longest member
        t = torch.arange(shared, device=DEV)
        page = mine["block_table"][lens.argmax(), t // bs].long()
        there = longest > 0
        k0 = st["k_cache"][page * there, t % bs].float()
        v0 = st["v_cache"][page * there, t % bs].float()
        s0 = torch.matmul(x.transpose(0, 1).reshape(G, n * (H // G), D), k0.permute(1, 2, 0)).mul_(st["scale"])
        s0 = s0.view(G, n, H // G, shared).transpose(0, 1).masked_fill(~(t < lens)[:, None, None], -math.inf)
        m = torch.cat([s0.amax(3, keepdim=True) if shared else s0.new_full((n, G, H // G, 1), -math.inf),
                       s.amax(3, keepdim=True) if s.shape[3] else s.new_full((n, G, H // G, 1), -math.inf)], 3)
        m = m.amax(3, keepdim=True)
        base = m.where(torch.isfinite(m), torch.zeros_like(m))
        p0, p = (s0 - base).exp_(), (s - base).exp_()
        l = p0.sum(3, keepdim=True) + p.sum(3, keepdim=True)
        o = torch.matmul(p0.transpose(0, 1).reshape(G, n * (H // G), shared), v0.transpose(0, 1))
        o = o.view(G, n, H // G, D).transpose(0, 1) + torch.matmul(p, v.permute(0, 2, 1, 3))
        outs.append((o / l).masked_fill_(l == 0, 0.0).reshape(n, H, D))
        lses.append((m + l.log()).view(n, H))
        a += n
    return torch.cat(outs).to(q.dtype), torch.cat(lses)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["op"]
    if own:
        import paged_attention_kv_decode_gb300 as pa

        if op == "plan":
            step = pa.metis_plan_step(st["q_lens"], st["cached_lens"], st["block_table"], st["free_stack"],
                                      st["free_count"], block_size=st["block"], num_tokens=st["tokens"],
                                      num_blocks=st["num_blocks"], refcount=st["refcount"])
            return {"seq_lens": step.seq_lens, "cu_q_lens": step.cu_q_lens, "slot_mapping": step.slot_mapping,
                    "positions": step.positions, "free_count": step.free_count, "block_table": st["block_table"],
                    "refcount": st["refcount"]}
        if op == "rotate":
            q = pa.metis_qk_norm_rope_and_cache(st["q"], st["k"], st["v"], st["cos_sin"], st["positions"],
                                                st["k_cache"], st["v_cache"], st["slot_mapping"],
                                                q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"],
                                                interleaved=st["interleaved"])
            return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        cache = (st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"])
        if op == "window_decode":
            o, lse = pa.metis_paged_attn_decode_window(st["q"], *cache, st["scale"], st["window"], st["sinks"],
                                                       max_seq_len=st["len_max"], want_lse=True)
        elif op == "window_prefill":
            o, lse = pa.metis_paged_attn_prefill_chunk_window(st["q"], st["cu_q_lens"], *cache, st["scale"],
                                                              st["window"], st["sinks"], max_seq_len=st["len_max"],
                                                              want_lse=True)
        else:
            o, lse = pa.metis_paged_attn_decode_shared(st["q"], *cache, st["cu_group_seqs"], st["prefix_lens"],
                                                       st["scale"], max_seq_len=st["len_max"], want_lse=True)
        return {"out": o, "lse": lse}
    if op == "plan":
        return _plain_plan(st)
    if op == "rotate":
        return {"q": _plain_rotate(st), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    plain = {"window_decode": _plain_window_decode, "window_prefill": _plain_window_prefill, "shared": _plain_shared}
    o, lse = plain[op](st)
    return {"out": o, "lse": lse}


# ---------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _exact_rotate(case, st):
    R = case["rotary"]
    turn = st["cos_sin"][st["positions"].long()].double()
    z = torch.complex(turn[:, : R // 2], turn[:, R // 2 :])[:, None]  # a rotation of a pair is a complex product
    got = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        y = x.double()
        if w is not None:
            y = y / (y.square().sum(2, keepdim=True) / y.shape[2] + st["eps"]).sqrt() * w.double()
        pair = y[..., :R].unflatten(2, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        pair = pair if case["interleaved"] else pair.transpose(2, 3)
        pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        pair = pair if case["interleaved"] else pair.transpose(2, 3)
        got.append(torch.cat([pair.flatten(2), y[..., R:]], 2))
    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    bs = k_cache.shape[1]
    for n, slot in enumerate(st["slot_mapping"].tolist()):
        if slot >= 0:
            k_cache[slot // bs, slot % bs] = got[1][n]
            v_cache[slot // bs, slot % bs] = st["v"][n].double()
    return {"q": got[0], "k_cache": k_cache, "v_cache": v_cache}


def _exact_rows(st, s, x, n, tokens, seen):
    """Rows x [q, H, D] of sequence s over its tokens `tokens`, of which row i sees seen[i]."""
    bs, G = st["k_cache"].shape[1:3]
    page = st["block_table"][s, tokens // bs].long()
    k = st["k_cache"][page, tokens % bs].double()
    v = st["v_cache"][page, tokens % bs].double()
    k, v = (c.where(seen.any(0)[:, None, None], torch.zeros_like(c)) for c in (k, v))
    o = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(x.shape[:2], dtype=torch.float64, device=DEV)
    r = x.shape[1] // G
    for g in range(G):
        z = torch.einsum("qhd,td->qht", x[:, g * r : g * r + r].double(), k[:, g]) * st["scale"]
        z = z.masked_fill(~seen[:, None], -math.inf)
        lse[:, g * r : g * r + r] = torch.logsumexp(z, 2)
        o[:, g * r : g * r + r] = torch.einsum("qht,td->qhd", torch.softmax(z, 2), v[:, g])
    return o, lse


def exact(case, seed):
    if case["op"] == "plan":  # whole numbers: the plain form is held to be equal
        return None
    st = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(case, st)
    outs, lses = [], []
    H, D = case["heads"], case["dim"]
    if case["op"] == "shared":
        seqs = [(n, 1) for _, members in _groups(case) for n in members]
    else:
        seqs = _lengths(case)
    row = 0
    for s, (n, q) in enumerate(seqs):
        if case["op"] != "window_prefill":
            q = 1  # a row for every sequence, those without tokens too
        x = st["q"][row : row + q]
        row += q
        if n == 0:
            outs.append(torch.zeros(q, H, D, dtype=torch.float64, device=DEV))
            lses.append(torch.full((q, H), -math.inf, dtype=torch.float64, device=DEV))
            continue
        at = torch.arange(n - q, n, device=DEV)[:, None]
        if case["op"] == "shared":
            tokens = torch.arange(n, device=DEV)
            seen = torch.ones(1, n, dtype=torch.bool, device=DEV)
        else:
            lo = max(0, n - q - case["window"] + 1)
            tokens = torch.cat([torch.arange(min(case["sinks"], lo), device=DEV), torch.arange(lo, n, device=DEV)])
            seen = (tokens <= at) & ((tokens > at - case["window"]) | (tokens < case["sinks"]))
        o, lse = _exact_rows(st, s, x, n, tokens, seen)
        outs.append(o)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
