"""A serving step of the calls of paged_step.h together: the tables from the
lengths, new keys rotated on three axes into the pages taken, attention over a
window with sinks; prompts first, then captured decode steps, each against the
oracles on the caches as written."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import batch_tables as B
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W
from gpu_helpers import check, sample_rows

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("early", [0, 1])
def test_a_step_builds_writes_and_attends(early):
    pd.build()
    pd.paged_decode_device_status(reset=True)
    S, P, Hq, Hkv, D, width, pages, window, sinks = 5, 16, 8, 2, 128, 40, 160, 90, 6
    axis, dt = pd.rope_pair_axis((24, 20, 20)), torch.bfloat16
    gen = torch.Generator().manual_seed(31)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dt).cuda()  # noqa: E731
    cos_sin = W.rope_cos_sin_table(700, D).cuda()
    kc, vc = (torch.full((pages, Hkv, P, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    free = _i32(np.random.default_rng(1).permutation(pages))
    cur, nxt, table = _i32([0]), _i32([0]), _i32(np.full((S, width), -1))
    ctx, lens, start = _i32(np.zeros(S)), _i32(np.zeros(S)), _i32(np.zeros(S + 1))
    delta = _i32(np.zeros(S))
    host = dict(table=np.full((S, width), -1), ctx=np.zeros(S, dtype=int), cursor=0)

    def tables(qd, pos, slots):
        pd.paged_batch_tables(ctx, qd, table, start, lens, pos, slots, P, pages, free_pages=free,
                              cursor=cur, next_cursor=nxt, position_delta=delta)

    def rope(q, k, v, pos, slots, q_rot):
        pd.paged_rope_axes_cache_write(q, k, v, pos, slots, cos_sin, axis, q_rot, kc, vc, Hq, Hkv,
                                       D, D, P, W.HND, True)

    def expect(q_rot, out, qd, M, pos, slots):
        want = B.batch_tables(host["ctx"], qd.tolist(), host["table"], P, q_rot.shape[0], 3,
                              free.tolist(), host["cursor"], delta.tolist())
        for a, b in zip((table, start, lens, pos, slots), want):
            assert np.array_equal(a.cpu().numpy(), b)
        assert int(nxt) == want[5]
        host.update(table=want[0], ctx=want[2], cursor=want[5])
        case = W.DecodeCase("step", dt, D, Hq, Hkv, P, M, window, D ** -0.5, W.HND, q_rot.cpu(),
                            kc.cpu(), vc.cpu(), table.cpu(), lens.cpu(), seq_lens_host=lens.tolist(),
                            query_start=start.cpu(), query_start_host=start.tolist())
        rows = sample_rows(case, 120)
        rows = [(t, h) for t, h in rows if t < int(start[-1])]
        check(case, out, rows=rows, ref=O.attention(case, sinks, rows))
        assert float(out[int(start[-1]):].abs().sum()) == 0.0
        assert pd.paged_decode_device_status(reset=True) == 0

    # the prompts
    q_lens = [300, 17, 1, 120, 64]
    T = sum(q_lens)
    qd = _i32(q_lens)
    pos, slots = torch.zeros((3, T), dtype=torch.int32, device="cuda"), _i32(np.zeros(T))
    tables(qd, pos, slots)
    q, k, v = rnd(T, Hq, D), rnd(T, Hkv, D), rnd(T, Hkv, D)
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    rope(q, k, v, pos, slots, q_rot)
    items, info = pd.paged_prefill_plan_sinks([0] + list(np.cumsum(q_lens)), q_lens, Hq, Hkv, D,
                                              window, sinks)
    pd.paged_prefill_attn_sinks(q_rot, kc, vc, table, lens, start, items.cuda(), info, out, Hq, Hkv,
                                D, P, window, sinks, D ** -0.5, W.HND, pd.prefill_scratch(Hkv, D))
    torch.cuda.synchronize()
    expect(q_rot, out, qd, max(q_lens), pos, slots)

    # decode steps of 0..2 tokens per request in a batch padded to 10 rows
    delta.copy_(torch.tensor([0, -3, 0, -60, 5], dtype=torch.int32))
    T, M = 10, 2
    qd = _i32([1, 1, 2, 0, 1])
    pos, slots = torch.zeros((3, T), dtype=torch.int32, device="cuda"), _i32(np.zeros(T))
    q, k, v = rnd(T, Hq, D), rnd(T, Hkv, D), rnd(T, Hkv, D)
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    sc = pd.Scratch(S, Hq, Hkv, D, M, max_splits=16)
    opts = pd.options(early_reads=early)

    def step():
        ctx.copy_(lens)
        cur.copy_(nxt)
        tables(qd, pos, slots)
        rope(q, k, v, pos, slots, q_rot)
        pd.paged_decode_attn_sinks(q_rot, kc, vc, table, lens, out, Hq, Hkv, D, P, M, window, sinks,
                                   D ** -0.5, W.HND, sc, query_start=start, opts=opts)

    step()
    torch.cuda.synchronize()
    expect(q_rot, out, qd, M, pos, slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(20):
        for x in (q, k, v):
            x.copy_(rnd(*x.shape))
        qd.copy_(torch.tensor([n % 3, 1, 2, (n + 1) % 2, 1], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        expect(q_rot, out, qd, M, pos, slots)
