"""Cases of the calls of paged_step.h for the tests."""

from __future__ import annotations

import dataclasses

import numpy as np
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import workloads as W


def hide(case, sinks):
    """The case with NaN in every key and value that no row of its request
    sees, and -1 in the table for every page without a visible one (as after
    a cache manager has taken those pages back)."""
    P = case.page_size
    table = case.block_table.clone()
    kc, vc = case.k_cache, case.v_cache
    nhd = case.layout == W.NHD
    for s, L in enumerate(case.seq_lens_host):
        m = case.query_len(s)
        lo = max(0, L - m + 1 - case.window) if case.window else 0
        if m == 0:
            lo = L
        seen = np.zeros(table.shape[1] * P, dtype=bool)
        seen[lo:L] = True
        seen[:min(sinks, L) if m else 0] = True
        for j in range(table.shape[1]):
            page = int(table[s, j])
            mine = seen[j * P:(j + 1) * P]
            if j * P >= L or not mine.any():
                table[s, j] = -1
            if j * P < L:
                off = torch.from_numpy(np.nonzero(~mine)[0])
                for c in (kc, vc):
                    if nhd:
                        c[page, off] = float("nan")
                    else:
                        c[page, :, off] = float("nan")
    return dataclasses.replace(case, block_table=table)


def run_sinks(case, sinks, scratch=None, opts=None, out=None, stream=None):
    """paged_decode_attn_sinks on a case (tensors on the GPU)."""
    out = torch.empty_like(case.q) if out is None else out
    pd.paged_decode_attn_sinks(case.q, case.k_cache, case.v_cache, case.block_table,
                               case.seq_lens, out, case.num_q_heads, case.num_kv_heads,
                               case.head_size, case.page_size, case.max_query_len, case.window,
                               sinks, case.scale, case.layout, scratch,
                               query_start=case.query_start, opts=opts, stream=stream)
    return out


def run_prefill_sinks(case, sinks, scratch=None, num_sms=0, plan=None, out=None):
    """paged_prefill_attn_sinks on a case, with its own plan or another."""
    if plan is None:
        plan = pd.paged_prefill_plan_sinks(case.query_start_host, case.seq_lens_host,
                                           case.num_q_heads, case.num_kv_heads, case.head_size,
                                           case.window, sinks, num_sms)
    items, info = plan
    out = torch.empty_like(case.q) if out is None else out
    pd.paged_prefill_attn_sinks(case.q, case.k_cache, case.v_cache, case.block_table,
                                case.seq_lens, case.query_start, items.to(case.q.device), info,
                                out, case.num_q_heads, case.num_kv_heads, case.head_size,
                                case.page_size, case.window, sinks, case.scale, case.layout,
                                scratch)
    return out


def batch(S, P, seed, q_hi=4, c_hi=900, empty=0.1, slack=3):
    """(contexts, query lengths, table, free list, pages in the pool) of a
    step: every request's pages so far in its row, the other entries -1."""
    g = np.random.default_rng(seed)
    c = g.integers(0, c_hi + 1, S)
    q = np.where(g.random(S) < empty, 0, g.integers(1, q_hi + 1, S))
    if S:
        c[0] = 0
        c[-1] = (c[-1] // P) * P  # new pages from the first token on
    have, need = -(-c // P), -(-(c + q) // P)
    width = int(need.max()) + 1 if S else 1
    pages = int(need.sum()) + slack
    ids = g.permutation(pages)
    table = np.full((S, width), -1)
    table[np.arange(width)[None] < have[:, None]] = ids[:int(have.sum())]
    return c, q, table, ids[int(have.sum()):], pages
