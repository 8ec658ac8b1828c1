"""Whole-number CPU oracle of the tables of a batch (test infrastructure
only): one token at a time, from the definition."""

from __future__ import annotations

import numpy as np


def batch_tables(context, query, table, page_size, num_tokens, axes=1, free=None, cursor=0,
                 delta=None):
    """The tables of a step whose requests fit their rows, the list and the
    token rows: (table, query_start, seq_lens, positions [axes, T], slots,
    next cursor)."""
    S = len(context)
    table = np.array(table, dtype=np.int64, copy=True)
    start = np.zeros(S + 1, dtype=np.int64)
    lens = np.zeros(S, dtype=np.int64)
    pos = np.zeros((axes, num_tokens), dtype=np.int64)
    slots = np.full(num_tokens, -1, dtype=np.int64)
    t = 0
    for s in range(S):
        start[s] = t
        have = -(-int(context[s]) // page_size)
        for i in range(int(query[s])):
            p = int(context[s]) + i
            j = p // page_size
            if free is not None and j >= have:
                have = j + 1
                table[s, j] = free[cursor]
                cursor += 1
            pos[:, t] = p + (int(delta[s]) if delta is not None else 0)
            slots[t] = table[s, j] * page_size + p % page_size
            t += 1
        lens[s] = int(context[s]) + int(query[s])
    start[S] = t
    return table, start, lens, pos, slots, cursor
