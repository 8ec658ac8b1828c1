"""Early reads over a window with sinks: the kernel ahead on the stream (the
rotary + cache write) makes q and the newest keys and values while the attention
call reads the older pages.  Every step has inputs of its own, written over
other ones of the same size, and its outputs are checked by themselves; outputs
of the q, keys or values before them would fail the same check."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W
from gpu_helpers import check, sample_rows, scratch_for
from step_cases import run_sinks

pytestmark = pytest.mark.gpu


def _path(case, sinks, sc, opts):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return pd.paged_decode_plan_sinks(case.num_seqs, case.num_q_heads, case.num_kv_heads, case.head_size,
                                      case.page_size, case.max_query_len, case.window, sinks,
                                      case.block_table.shape[1], sms, scratch=sc, opts=opts)["path"]


@pytest.mark.parametrize("path", [6, 1])
@pytest.mark.parametrize("D,S,Hq,Hkv,M", [(128, 40, 32, 8, 2), (64, 70, 8, 8, 1), (256, 30, 16, 2, 4),
                                          (128, 40, 32, 8, 1)])
@pytest.mark.parametrize("captured", [False, True])
def test_every_step_reads_its_own_tokens(captured, path, D, S, Hq, Hkv, M):
    pd.build()
    pd.paged_decode_device_status(reset=True)
    sinks, P = 4, 16
    lens = [int(x) for x in np.random.default_rng(D + S).integers(M, 2500, S)]
    lens[:3] = [M, M + 1, 2500]
    case = W.make_case("early", seed=D, dtype=torch.bfloat16, head_size=D, num_q_heads=Hq, num_kv_heads=Hkv,
                       page_size=P, max_query_len=M, seq_lens=lens, window=60)
    slots, pos = [], []
    for s, L in enumerate(lens):
        for k in range(L - M, L):
            slots.append(int(case.block_table[s, k // P]) * P + k % P)
            pos.append(k)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    g = case.to("cuda")
    slots, pos, table = i32(slots), i32([pos] * 3), W.rope_cos_sin_table(2600, D).cuda()
    axis = bytes([0, 1, 2, 0] * (D // 8))
    sc, opts = scratch_for(case, 16), pd.options(early_reads=1, path=path)
    assert _path(case, sinks, sc, opts) == path
    gen = torch.Generator().manual_seed(D + 7)
    q_rot = torch.empty_like(g.q)
    new = [[torch.randn(S * M, h, D, generator=gen).to(case.dtype).cuda() for h in (Hq, Hkv, Hkv)] for _ in range(6)]
    kept = [[torch.full_like(g.q, 7.0)] + [torch.empty_like(t) for t in (q_rot, g.k_cache, g.v_cache)] for _ in new]

    def run():
        for (q, k, v), (out, *copies) in zip(new, kept):
            pd.paged_rope_axes_cache_write(q, k, v, pos, slots, table, axis, q_rot, g.k_cache, g.v_cache, Hq, Hkv, D,
                                           D, P, W.HND, True)
            run_sinks(dataclasses.replace(g, q=q_rot), sinks, sc, opts, out=out)
            for to, at in zip(copies, (q_rot, g.k_cache, g.v_cache)):
                to.copy_(at)

    torch.cuda.synchronize()
    run()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for out, *_ in kept:
            out.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert pd.paged_decode_device_status(reset=True) == 0
    rows = sample_rows(case, 150)
    # (rows of a few keys keep values of V's own size: half a step of the weights
    # and of the output, 2^-8 max |V| each; relative to the row, no bound)
    before = None
    for out, q, k, v in kept:
        now = dataclasses.replace(case, q=q.cpu(), k_cache=k.cpu(), v_cache=v.cpu())
        ref = O.attention(now, sinks, rows)
        tol = 2 * 2.0 ** -8 * float(now.v_cache[torch.isfinite(now.v_cache)].float().abs().max())
        check(now, out, rows=rows, ref=ref, tol=tol, rel_tol=1.0)
        if before is not None:
            for stale in (dict(q=before.q), dict(k_cache=before.k_cache), dict(v_cache=before.v_cache)):
                other = O.attention(dataclasses.replace(now, **stale), sinks, rows)
                assert np.abs(other - ref).max() > 4 * tol, stale.keys()
        before = now
