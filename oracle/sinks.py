"""fp64 CPU oracle of attention over a window with sinks (test infrastructure
only), one row at a time from its definition; it shares nothing with the CUDA
path."""

from __future__ import annotations

import numpy as np
import torch


def widen(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def visible(n: int, window: int, sinks: int) -> np.ndarray:
    """The keys a row of n keys sees: all of [0, n) without a window, else
    those of the newest ``window`` and of the first ``sinks``."""
    k = np.arange(max(n, 0))
    if window <= 0:
        return k
    return k[(k >= n - window) | (k < sinks)]


def attention(case, sinks: int, rows=None) -> np.ndarray:
    """Outputs [T, Hq, D] of a ``workloads.DecodeCase`` (or of the rows (t,
    hq) asked for, [len(rows), D]) with ``sinks`` beside its window."""
    P, M, Hq, Hkv, D = (case.page_size, case.max_query_len, case.num_q_heads, case.num_kv_heads,
                        case.head_size)
    G = Hq // Hkv
    table = case.block_table.cpu().numpy()
    lens = case.seq_lens.cpu().numpy()
    T = case.q.shape[0]
    out = np.zeros((T, Hq, D))
    want = None if rows is None else {}
    for t, h in rows or []:
        want.setdefault(int(t), []).append(int(h))
    kc, vc = (c if case.layout == 0 else c.permute(0, 2, 1, 3) for c in (case.k_cache, case.v_cache))
    kc, vc = kc.cpu(), vc.cpu()
    for s, L in enumerate(lens):
        if case.query_start_host is None:
            t0, m = s * M, M
        else:
            t0 = case.query_start_host[s]
            m = case.query_start_host[s + 1] - t0
        for i in range(m):
            t = t0 + i
            heads = range(Hq) if want is None else want.get(t, [])
            keys = visible(int(L) - m + i + 1, case.window, sinks)
            if not len(keys) or not len(heads):
                continue
            page = torch.from_numpy(table[s, keys // P].astype(np.int64))
            tok = torch.from_numpy(keys % P)
            kk, vv = widen(kc[page, tok]), widen(vc[page, tok])  # [keys, Hkv, D]
            for hq in heads:
                h = hq // G
                x = case.scale * (kk[:, h] @ widen(case.q[t, hq]))
                p = np.exp(x - x.max())
                out[t, hq] = p @ vv[:, h] / p.sum()
    if rows is None:
        return out
    return np.stack([out[t, h] for t, h in rows])
