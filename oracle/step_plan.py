"""CPU oracle for a step's index arrays -- TEST INFRASTRUCTURE ONLY.

The rule written out with Python integers, a sequence, a page and a token at a time: sequence s
has ``cached[s]`` tokens and gets ``q_lens[s]`` new ones; pages that its table row lacks come from
the top of the free stack; a token at position p of a page b has slot ``b * block_size + p %
block_size``.  Also returned: the status bits that such inputs set.
"""

from __future__ import annotations

import numpy as np

BAD_BLOCK_ID, SEQ_TOO_LONG, BAD_Q_LEN, OUT_OF_PAGES, BAD_OFFSETS = 1, 2, 8, 32, 64
INT_MAX = 2 ** 31 - 1


def plan_step(q_lens, cached, block_table, free_stack, free_count, block_size, num_tokens, num_blocks, held=None,
              refcount=None):
    table = np.array(block_table, dtype=np.int64, copy=True)
    refs = None if refcount is None else np.array(refcount, dtype=np.int64, copy=True)
    S, width = table.shape
    stack = [int(x) for x in free_stack]
    depth = min(max(int(free_count), 0), len(stack))
    status = taken = row = 0
    seq_lens, held_out, cu, slots, positions = [], [], [0], [], []
    for s in range(S):
        n, before = int(q_lens[s]), int(cached[s])
        if n < 0 or before < 0:
            status |= BAD_Q_LEN
        n, before = max(n, 0), max(before, 0)
        if row + n > num_tokens:
            status |= BAD_OFFSETS
            n = num_tokens - row
        names = max(0 if held is None else int(held[s]), -(-before // block_size))
        names = min(max(names, 0), width)
        for i in range(n):
            p = before + i
            page, off = divmod(p, block_size)
            block = -1
            if page >= width:
                status |= SEQ_TOO_LONG
            else:
                if page >= names:  # the next page of the sequence
                    assert page == names and off == 0
                    names += 1
                    if taken < depth:
                        block = stack[depth - 1 - taken]
                        if not 0 <= block < num_blocks:
                            status |= BAD_BLOCK_ID
                            block = -1
                    else:
                        status |= OUT_OF_PAGES
                    taken += 1
                    table[s, page] = block
                    if refs is not None and block >= 0:
                        refs[block] = 1
                block = int(table[s, page])
                if not 0 <= block < num_blocks:
                    block = -1
            slots.append(-1 if block < 0 else block * block_size + off)
            positions.append(min(p, INT_MAX))
        row += n
        cu.append(row)
        seq_lens.append(min(before + n, INT_MAX))
        held_out.append(names)
    slots += [-1] * (num_tokens - row)
    positions += [0] * (num_tokens - row)
    return dict(seq_lens=np.array(seq_lens), cu_q_lens=np.array(cu), slot_mapping=np.array(slots, dtype=np.int64),
                positions=np.array(positions, dtype=np.int64), held_blocks=np.array(held_out), block_table=table,
                refcount=refs, free_count=max(depth - taken, 0), status=status)
