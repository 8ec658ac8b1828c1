"""Prefill over a window with sinks at head sizes 64 and 128, tile after tile
(plans of 256-row tiles without a split), against the fp64 oracle.

Bounds: those of gpu_helpers.  Keys that no row sees are NaN, pages without a
visible key -1 in the table.  A plan for one SM has such tiles."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W
from gpu_helpers import check, sample_rows
from step_cases import hide, run_prefill_sinks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _plan(case, sinks, num_sms=1):  # (one SM: whole tiles)
    plan = pd.paged_prefill_plan_sinks(case.query_start_host, case.seq_lens_host, case.num_q_heads,
                                       case.num_kv_heads, case.head_size, case.window, sinks, num_sms)
    G = case.num_q_heads // case.num_kv_heads
    if num_sms == 1:
        assert plan[1].num_split_tiles == 0
        padded = 1 << (G - 1).bit_length()
        rows = (128 if case.head_size == 256 else 256) // padded * G
        assert plan[1].tile_rows == (256 if case.head_size == 128 and 8 * G < 5 * padded else rows)
    return plan


def _run(case, sinks, rows=300, **kw):
    hidden = hide(case, sinks)
    g = hidden.to("cuda")
    out = torch.full_like(g.q, 7.0)
    run_prefill_sinks(g, sinks, None, plan=_plan(case, sinks), out=out)
    torch.cuda.synchronize()
    rows = sample_rows(case, rows)
    rows = [(t, h) for t, h in rows if t < case.query_start_host[-1]]
    check(hidden, out, rows=rows, ref=O.attention(hidden, sinks, rows), **kw)
    assert float(out[case.query_start_host[-1]:].abs().sum()) == 0.0
    return hidden, g, out


def _case(seed, q_lens, contexts, **kw):
    base = dict(num_q_heads=8, num_kv_heads=2, window=200)
    base.update(kw)
    return W.make_prefill_case("tiles", seed=seed, q_lens=q_lens, contexts=contexts, **base)


both = pytest.mark.parametrize("D", [64, 128, 256])


@both
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window,sinks", [(200, 4), (17, 40), (64, 64), (1, 16), (1000, 130)])
def test_tiles_types_and_windows(dtype, window, sinks, D):
    _run(_case(window, [300, 1, 77, 0, 160, 64], [0, 700, 333, 50, 16, 2000], dtype=dtype, window=window,
               pad_tokens=3, head_size=D), sinks)


@both
@pytest.mark.parametrize("heads", [(2, 2), (4, 2), (32, 8), (16, 2), (32, 1), (6, 2), (20, 4), (128, 1), (256, 2), (7, 1), (3, 1), (21, 3), (18, 2)])
def test_tiles_heads(heads, D):
    """1 .. 128 q heads to a kv head; 3, 5, 7 and 9 padded to 4, 8 and 16 (9 not
    at head size 128); one kv head, past whose heads q ends."""
    _run(_case(heads[0], [70, 9, 130], [150, 0, 600], num_q_heads=heads[0], num_kv_heads=heads[1],
               head_size=D), 20)


@both
def test_tiles_many_to_a_cta(D):
    """Some eight rounds over the SMs, of tiles of one to ten stages."""
    g = np.random.default_rng(1)
    q = [int(x) for x in g.integers(1, 900, 24)]
    c = [int(x) for x in g.integers(0, 1500, 24)]
    _run(_case(2, q, c, num_q_heads=32, num_kv_heads=8, window=500, pad_tokens=1, head_size=D), 7, rows=400)


@both
def test_tiles_of_single_tokens(D):
    g = np.random.default_rng(2)
    c = [int(x) for x in g.integers(0, 400, 90)]
    _run(_case(3, [1] * 90, c, num_q_heads=32, num_kv_heads=8, window=100, head_size=D), 3, rows=400)


@both
@pytest.mark.parametrize("layout", [W.NHD, W.HND])
@pytest.mark.parametrize("P", [48, 784])
def test_tiles_layouts_and_pages(layout, P, D):
    _run(_case(P, [500, 33], [900, 5], layout=layout, page_size=P, window=300, head_size=D), 21)


@both
@pytest.mark.parametrize("std,scale", [(4.0, None), (3.0, -0.09)])
def test_tiles_large_scores(std, scale, D):
    """Scores far apart and of either sign: O rescaled, stages taken again."""
    case = _case(7, [256, 300], [500, 40], window=400, std=std, head_size=D)
    if scale is not None:
        case = dataclasses.replace(case, scale=scale)
    v = 2 * 2.0 ** -8 * float(case.v_cache[torch.isfinite(case.v_cache)].float().abs().max())
    # (rows of one or two keys that matter: half a step of P and of the output
    # each, of V's own size)
    _run(case, 10, tol=v, rel_tol=2.0 ** -6)


@both
@pytest.mark.parametrize("slope", [0.02, -0.02, 0.3])
def test_tiles_scores_along_the_keys(slope, D):
    """Scores that rise (or fall) from key to key, past every reference in
    masked and unmasked stages, on every other head the other way round."""
    case = _case(8, [150, 200], [900, 60], window=300, head_size=D)
    q, k = case.q.clone(), case.k_cache.clone()
    q[:] = 1.0
    q[:, 1::2] = -1.0
    for s, L in enumerate(case.seq_lens_host):
        for p in range(L):
            k[int(case.block_table[s, p // 16]), :, p % 16] = slope * p
    case = dataclasses.replace(case, q=q, k_cache=k)
    # (as above: a few keys matter to a row)
    v = 2 * 2.0 ** -8 * float(case.v_cache[torch.isfinite(case.v_cache)].float().abs().max())
    _run(case, 10, tol=v, rel_tol=2.0 ** -6)


@both
def test_tiles_scale_zero(D):
    """The mean of the visible V."""
    _run(dataclasses.replace(_case(9, [150, 200], [900, 60], window=300, head_size=D), scale=0.0), 10)


def test_tiles_strided_q_and_out():
    case = hide(_case(8, [100, 200], [90, 300]), 4)
    g = case.to("cuda")
    T = 300
    wide_q = torch.full((T, 14, 128), 7.0, dtype=case.dtype, device="cuda")
    wide_q[:, 3:11] = g.q
    wide_o = torch.full((T, 10, 160), 7.0, dtype=case.dtype, device="cuda")
    out = wide_o[:, 1:9, 16:144]
    run_prefill_sinks(dataclasses.replace(g, q=wide_q[:, 3:11]), 4, None, plan=_plan(case, 4), out=out)
    torch.cuda.synchronize()
    rows = sample_rows(case, 300)
    check(case, out, rows=rows, ref=O.attention(case, 4, rows))
    wide_o[:, 1:9, 16:144] = 7.0
    assert bool((wide_o == 7.0).all())
    # heads outermost
    by_head = g.q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = run_prefill_sinks(dataclasses.replace(g, q=by_head), 4, None, plan=_plan(case, 4))
    torch.cuda.synchronize()
    check(case, out, rows=rows, ref=O.attention(case, 4, rows))
    # every head the same row (a stride that TMA does not take: another way)
    one = g.q[:, :1].expand(-1, 8, -1)
    same = dataclasses.replace(case, q=case.q[:, :1].expand(-1, 8, -1).contiguous())
    out = run_prefill_sinks(dataclasses.replace(g, q=one), 4, None, plan=_plan(case, 4))
    torch.cuda.synchronize()
    check(same, out, rows=rows, ref=O.attention(same, 4, rows))


@both
def test_tiles_rows_of_other_requests_hold_nan(D):
    """A tile's box of q reads on into the next request's rows and past the
    batch: NaN and infinities there stay where they are."""
    case = _case(9, [30, 50, 20], [400, 10, 60], pad_tokens=2, head_size=D)
    hidden, g, want = _run(case, 5)
    for value in (float("nan"), float("inf")):
        q = g.q.clone()
        q[30:80] = value
        out = run_prefill_sinks(dataclasses.replace(g, q=q), 5, None, plan=_plan(case, 5))
        torch.cuda.synchronize()
        assert torch.equal(out[:30], want[:30]) and torch.equal(out[80:], want[80:])


@both
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tiles_other_heads_hold_nan(bad, D):
    """The rows that pad a token's heads are the next kv head's: whatever q holds
    there, a kv head's outputs are its own."""
    case = _case(14, [90, 40], [300, 0], num_q_heads=9, num_kv_heads=3, head_size=D)
    q = case.q.clone()
    q[:, 3:6] = bad
    hidden = hide(case, 6)
    g = dataclasses.replace(hidden.to("cuda"), q=q.cuda())
    out = run_prefill_sinks(g, 6, None, plan=_plan(case, 6))
    torch.cuda.synchronize()
    rows = [(t, h) for t, h in sample_rows(case, 400) if not 3 <= h < 6]
    out[:, 3:6] = 0
    check(hidden, out, rows=rows, ref=O.attention(hidden, 6, rows))


@both
def test_tiles_a_request_longer_than_its_keys(D):
    """Rows before the sequence's start see nothing and are zero."""
    case = _case(10, [90, 40], [100, 0], head_size=D)
    g = case.to("cuda")
    lens = torch.tensor([30, 0], dtype=torch.int32)
    out = run_prefill_sinks(dataclasses.replace(g, seq_lens=lens.cuda()), 4, None, plan=_plan(case, 4))
    torch.cuda.synchronize()
    now = dataclasses.replace(case, seq_lens=lens, seq_lens_host=lens.tolist())
    check(now, out, ref=O.attention(now, 4))
    assert float(out[:60].abs().sum()) == 0.0 and float(out[90:].abs().sum()) == 0.0


def test_tiles_repeat_bit_for_bit_and_replay():
    case = _case(11, [400, 90, 250], [800, 0, 64], num_q_heads=32, num_kv_heads=8)
    g = case.to("cuda")
    items, info = _plan(case, 6)
    work = items.cuda()
    out, again = torch.empty_like(g.q), torch.empty_like(g.q)

    def call(o):
        pd.paged_prefill_attn_sinks(g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, g.query_start, work,
                                    info, o, 32, 8, 128, 16, 200, 6, case.scale, W.HND)
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(again)
        call(again)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    # other lengths and queries under the same plan
    lens = torch.tensor([1100, 90, 300], dtype=torch.int32)
    g.seq_lens.copy_(lens)
    q = torch.randn(case.q.shape, generator=torch.Generator().manual_seed(1)).to(case.dtype)
    g.q.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    now = dataclasses.replace(case, q=q, seq_lens=lens, seq_lens_host=lens.tolist())
    rows = sample_rows(now, 300)
    check(now, again, rows=rows, ref=O.attention(now, 6, rows))


def _status():
    torch.cuda.synchronize()
    return pd.paged_decode_device_status(reset=True)


@both
def test_tiles_report_bad_inputs(D):
    case = _case(12, [200, 100, 64], [300, 0, 900], num_q_heads=32, num_kv_heads=8, head_size=D)
    hidden, g, want = _run(case, 4)
    plan = _plan(case, 4)
    # work items out of range, or of a segment: skipped, the rest runs
    for col, value in ((0, 3), (0, -1), (1, -2), (2, 1), (3, 2)):
        items = plan[0].clone()
        k = int((items[:, 0] == 1).nonzero()[0])
        tile = int(items[k, 1])
        items[k, col] = value
        out = torch.full_like(g.q, 7.0)
        run_prefill_sinks(g, 4, None, plan=(items, plan[1]), out=out)
        assert _status() == pd.DEV_BAD_WORK
        n = plan[1].tile_rows // 4  # tokens of a tile
        skipped = slice(200 + n * tile, min(300, 200 + n + n * tile))
        assert bool((out[skipped] == 7.0).all())
        out[skipped] = want[skipped]
        assert torch.equal(out, want)
    # a page outside the pool, a length past the table, a start out of order
    table = g.block_table.clone()
    table[1] = g.k_cache.shape[0]
    out = run_prefill_sinks(dataclasses.replace(g, block_table=table), 4, None, plan=plan)
    assert _status() == pd.DEV_BAD_PAGE
    assert torch.equal(out[:200], want[:200]) and torch.equal(out[300:], want[300:])
    lens = g.seq_lens.clone()
    lens[0] = case.block_table.shape[1] * 16 + 5
    run_prefill_sinks(dataclasses.replace(g, seq_lens=lens), 4, None, plan=plan)
    assert _status() & pd.DEV_BAD_SEQLEN
    start = g.query_start.clone()
    start[2] = 10 ** 6
    run_prefill_sinks(dataclasses.replace(g, query_start=start), 4, None, plan=plan)
    assert _status() & pd.DEV_BAD_QSTART
    assert torch.equal(run_prefill_sinks(g, 4, None, plan=plan), want)


@pytest.mark.parametrize("D,wide_rows", [(64, 256), (256, 128)])
def test_tiles_under_either_plan(D, wide_rows):
    """Plans of the tile kernel's rows and of 64-row tiles (the plan made
    without sinks), under calls without sinks or without a window too."""
    case = _case(13, [300, 77], [500, 0], head_size=D)
    g = case.to("cuda")
    sc = pd.prefill_scratch(2, D, num_sms=160)
    rows = sample_rows(case, 300)
    wide = _plan(case, 9)
    narrow = pd.paged_prefill_plan(case.query_start_host, case.seq_lens_host, 8, 2, D, 200, 152)
    assert (wide[1].tile_rows, narrow[1].tile_rows) == (wide_rows, 64)
    for sinks, window in ((9, 200), (0, 200), (9, 0)):
        c = dataclasses.replace(case, window=window)
        ref = O.attention(c, sinks, rows)
        for plan in (wide, narrow):
            out = run_prefill_sinks(dataclasses.replace(g, window=window), sinks, sc, plan=plan)
            torch.cuda.synchronize()
            check(c, out, rows=rows, ref=ref)
    out = pd.prefill_case(g, plan=wide)
    torch.cuda.synchronize()
    check(case, out, rows=rows, ref=O.attention(case, 0, rows))
    # strides that TMA does not take are refused under this plan
    one = dataclasses.replace(g, q=g.q[:, :1].expand(-1, 8, -1))
    with pytest.raises(pd.PagedDecodeError, match="PD_EALIGN"):
        run_prefill_sinks(one, 9, sc, plan=wide)
    run_prefill_sinks(one, 9, sc, plan=narrow)
    # the split of a 64-row plan is not for these tiles
    info = pd.PdPrefillPlanInfo.from_buffer_copy(narrow[1])
    info.tile_rows, info.num_split_tiles = wide_rows, 1
    with pytest.raises(pd.PagedDecodeError, match="PD_EINVAL"):
        run_prefill_sinks(g, 9, sc, plan=(narrow[0], info))
