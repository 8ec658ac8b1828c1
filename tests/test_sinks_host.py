"""Attention over a window with sinks on the CPU: exported symbols, refusals
(checked on the host before any launch), the launch plans, and the oracle's
pins."""

import numpy as np
import pytest
import torch

import oracle
import paged_split_kv_02_gb300 as pd
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W
from step_cases import hide

PASSES = -8  # a call that passes every check reaches the missing device


@pytest.fixture(scope="module", autouse=True)
def _built():
    if torch.cuda.is_available():
        pytest.skip("host tensors: for machines without a GPU")
    pd.build()
    oracle.build()


def test_exports_every_declared_symbol():
    names = pd.declared_symbols(pd.STEP_HEADER)
    assert {"paged_decode_attn_sinks", "paged_decode_plan_sinks", "paged_prefill_plan_sinks",
            "paged_prefill_attn_sinks"} <= set(names)
    for n in names:
        assert hasattr(pd.lib(), n), n


def test_arguments_that_are_not_what_they_should_be():
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(AttributeError):
        _attn(q="no tensor")
    with pytest.raises(OverflowError):
        _attn(window=2 ** 31)
    with pytest.raises(TypeError):
        _attn(sinks=1.5)
    assert _attn(q=None) == -1 and _attn(out=None) == -1
    assert _attn(q=torch.zeros(1, 1, 1, 4, 8, 128, dtype=torch.bfloat16)) == -1   # six dims
    assert _attn(q=q.double()) == -2


def _attn(**kw):
    c = W.make_case("refuse", seed=1, dtype=torch.bfloat16, head_size=128, num_q_heads=8,
                    num_kv_heads=2, page_size=16, max_query_len=2, seq_lens=[100, 40], window=32)
    a = dict(q=c.q, k=c.k_cache, v=c.v_cache, bt=c.block_table, sl=c.seq_lens,
             out=torch.empty_like(c.q), Hq=8, Hkv=2, D=128, P=16, M=2, window=32, sinks=4, scale=0.1,
             layout=W.HND, qs=None, opts=None)
    a.update(kw)
    return pd.paged_decode_attn_sinks(a["q"], a["k"], a["v"], a["bt"], a["sl"], a["out"], a["Hq"],
                                      a["Hkv"], a["D"], a["P"], a["M"], a["window"], a["sinks"],
                                      a["scale"], a["layout"], None, query_start=a["qs"],
                                      opts=a["opts"], check=False)


def test_decode_sinks_refusals():
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    assert _attn() == PASSES
    assert _attn(qs=torch.tensor([0, 2, 3], dtype=torch.int32)) == PASSES
    for kw, rc in [(dict(sinks=-1), -1), (dict(window=-1), -1), (dict(sinks=-1, window=0), -1),
                   (dict(scale=float("nan")), -1), (dict(D=96), -3), (dict(M=9), -4), (dict(M=0), -4),
                   (dict(P=24), -1), (dict(Hq=7), -1), (dict(layout=2), -1), (dict(q=q[:3]), -1),
                   (dict(q=q.float()), -2), (dict(q=q.half()), -2), (dict(bt=torch.zeros(2, 7)), -2),
                   (dict(bt=torch.zeros(3, 7, dtype=torch.int32)), -1),
                   (dict(qs=torch.zeros(2, dtype=torch.int32)), -1), (dict(qs=torch.zeros(3)), -2)]:
        assert _attn(**kw) == rc, kw
    with pytest.raises(pd.PagedDecodeError):
        pd.paged_decode_attn_sinks(q, q, q, q, q, q, 8, 2, 128, 16, 2, 32, 4, 0.1, W.HND)


def test_plan_sinks():
    def plan(window, sinks, width=2048, S=1, **kw):
        sd = pd.PdScratch()
        sd.data, sd.bytes = 1 << 30, pd.paged_decode_scratch_bytes(S, 32, 8, 128, 4, 256)
        sd.counter_slots = S * 8 * pd.COUNTERS_PER_PAIR
        return pd.paged_decode_plan_sinks(S, 32, 8, 128, 16, 4, window, sinks, width, 152,
                                          scratch_desc=sd, opts=pd.options(**kw) if kw else None)
    for S in (1, 7, 64):
        for window in (1, 100, 4096, 2 ** 31 - 1):
            for sinks in (0, 1, 16, 500, 2 ** 31 - 1):
                p = plan(window, sinks, S=S)
                # the segments cover the blocks of the window, a partial one
                # at its start, and the sinks, or the whole table
                need = min(2048, -(-(window + 3) // 16) + 1 + -(-sinks // 16))
                assert p["seg_blocks"] * p["max_segments"] >= need
                assert p["path"] in ((1, 6) if S > 1 and sinks else (1,)) and p["smem_bytes"] <= 232448
                assert p["scratch_needed"] <= pd.paged_decode_scratch_bytes(S, 32, 8, 128, 4, 256)
                if p["path"] == 1 and S > 1 and sinks:   # one wave
                    assert p["grid_x"] * p["grid_y"] <= 152
    assert (pd.paged_decode_plan_sinks(1, 32, 8, 128, 16, 4, 512, 0, 2048, 152)
            == pd.paged_decode_plan(1, 32, 8, 128, 16, 4, 512, 2048, 152))
    # without a window every key is visible, whatever the sinks
    assert plan(0, 9) == plan(0, 0)
    assert plan(0, 9, path=3)["path"] == 3
    for bad in (dict(window=64, sinks=-1), dict(window=-1, sinks=1), dict(window=64, sinks=1, path=2),
                dict(window=64, sinks=1, path=3)):
        with pytest.raises(pd.PagedDecodeError):
            plan(**bad)


def test_decode_plan_window_kernel():
    """Batches of more than a wave take the window kernel, but for few blocks to
    a CTA, or many of four n-tiles."""
    scratch = pd.PdScratch(data=1 << 40, bytes=1 << 30, counter_slots=1 << 20)
    def plan(S, D, M, window, Hq=32, Hkv=8, sinks=4, opts=None):
        return pd.paged_decode_plan_sinks(S, Hq, Hkv, D, 16, M, window, sinks, 1000, 152,
                                          scratch_desc=scratch, opts=opts)
    def path(*args, **kw):
        return plan(*args, **kw)["path"]
    # asked for
    six = pd.options(path=6)
    assert path(16, 128, 1, 128, opts=six) == 6 and path(2, 256, 8, 128, Hq=56, opts=six) == 6
    for bad in (dict(S=1), dict(S=1025), dict(D=512), dict(M=8, Hq=64), dict(window=0), dict(sinks=0)):
        with pytest.raises(pd.PagedDecodeError):
            plan(**{**dict(S=16, D=128, M=1, window=128, opts=six), **bad})
    with pytest.raises(pd.PagedDecodeError):
        plan(16, 128, 1, 128, opts=pd.options(path=6, stages=4))
    # one wave where it is not taken
    for S, M in ((4, 1), (16, 4), (64, 1)):
        p = plan(S, 512, M, 1024, Hq=16, Hkv=2)
        assert 100 < p["grid_x"] * p["grid_y"] <= 152
    assert path(64, 128, 4, 1024) == 6 and path(64, 128, 7, 1024) == 1 and path(64, 128, 7, 100) == 1
    assert path(64, 128, 8, 1024, Hq=20, Hkv=4) == 6 and path(64, 64, 4, 128, Hq=20, Hkv=4) == 1
    assert path(2, 128, 1, 128) == 1 and path(64, 512, 1, 1024) == 1
    # few blocks to a CTA: one wave of the other kernel
    assert path(16, 128, 1, 128) == 1 and path(16, 128, 1, 1024) == 1 and path(16, 128, 1, 4096) == 6


def test_prefill_plan_sinks():
    def plan(q_lens, lens, window, sinks, D=128, sms=152):
        qs = [0] + list(np.cumsum(q_lens))
        return pd.paged_prefill_plan_sinks(qs, lens, 8, 2, D, window, sinks, sms)
    for D, rows in ((64, None), (128, 256), (512, 64)):
        for window, sinks in ((100, 4), (64, 300), (1, 1), (0, 50)):
            q_lens, lens = [300, 1, 0, 90], [1300, 1, 40, 3000]
            items, info = plan(q_lens, lens, window, sinks, D)
            rows = info.tile_rows if D == 64 else rows   # 64 or 256 there
            blocks = {(int(i[0]), int(i[1])): int(i[6]) for i in items}
            for s, (m, L) in enumerate(zip(q_lens, lens)):
                for t in range(-(-m * 4 // rows)):
                    first, last = t * rows // 4, min(m - 1, ((t + 1) * rows - 1) // 4)
                    seen = set()
                    for i in range(first, last + 1):
                        seen |= {k // 16 for k in O.visible(L - m + i + 1, window, sinks)}
                    # (the sinks' last block and the window's first may be one)
                    assert len(seen) <= blocks[s, t] <= len(seen) + 1, (s, t)
            assert info.num_items == len(items)
    a, b = plan([300], [900], 128, 0), pd.paged_prefill_plan([0, 300], [900], 8, 2, 128, 128, 152)
    assert torch.equal(a[0], b[0])
    for bad in ((-1, 4), (4, -1)):
        with pytest.raises(pd.PagedDecodeError):
            plan([3], [3], *bad)
    with pytest.raises(pd.PagedDecodeError):
        pd.paged_prefill_plan_sinks([0, 3, 1], [3, 3], 8, 2, 128, 16, 4, 152)


def test_prefill_plan_whole_tiles():
    """Whole tiles of 256 rows at head sizes 64 and 128, of 128 at 256, but for
    few long ones."""
    def plan(q_lens, window, D, sinks=4, Hq=8, Hkv=2, sms=152):
        qs = [0] + list(np.cumsum(q_lens))
        info = pd.paged_prefill_plan_sinks(qs, [60000] * len(q_lens), Hq, Hkv, D, window, sinks, sms)[1]
        assert info.tile_rows == (256 if D == 128 else info.tile_rows)
        return info.tile_rows, info.num_split_tiles > 0
    # up to 288 blocks: whole (at 64, or with up to 64 rows, 96)
    assert plan([64], 4000, 128) == (256, False) and plan([64], 5000, 128) == (256, True)
    assert plan([16], 1400, 128) == (256, False) and plan([16], 1600, 128) == (256, True)
    assert plan([16, 17], 4000, 128) == (256, False)
    assert plan([4], 500, 256) == (128, False) and plan([4], 700, 256) == (64, True)
    assert plan([64], 1400, 64) == (256, False) and plan([64], 1600, 64) == (64, True)
    # half the SMs (a fifth at 64) filled: whole at any length
    assert plan([64 * 38], 30000, 128) == (256, False) and plan([64 * 37], 30000, 128) == (256, True)
    assert plan([64 * 16], 30000, 64) == (256, False) and plan([64 * 15], 30000, 64)[0] == 64
    assert plan([64 * 25], 30000, 128, sms=100) == (256, False)
    # one long request among short ones is cut
    lens = [60000] + [16] * 100
    qs = list(range(0, 16 * 102, 16))
    for window, split in ((1000, 0), (30000, 2)):
        info = pd.paged_prefill_plan_sinks(qs, lens, 8, 2, 128, window, 4, 152)[1]
        assert (info.num_split_tiles > 0) == (split > 0), window
    # at 256: 128 rows, or 64
    assert plan([64], 4000, 256) == (128, False) and plan([64], 5000, 256) == (64, True)
    assert plan([32 * 16], 30000, 256) == (128, False) and plan([32 * 15], 30000, 256) == (64, True)
    # three heads to a kv head, padded to four; five to eight; nine not at 128
    assert [plan([6400], 1000, D, Hq=6) for D in (64, 256)] == [(192, False), (96, False)]
    assert [plan([6400], 1000, D, Hq=10) for D in (64, 256)] == [(160, False), (80, False)]
    def rows128(q):
        return pd.paged_prefill_plan_sinks([0, 6400], [60000], q, 2, 128, 1000, 4, 152)[1].tile_rows
    assert [rows128(q) for q in (2, 6, 10, 14, 18, 24, 256, 258)] == [256, 192, 160, 224, 256, 192, 256, 256]
    assert plan([6400], 1000, 128, Hq=18) == (256, False) and plan([6400], 1000, 64, Hq=258)[0] == 64
    # without sinks or a window, the plan of those calls
    for kw in (dict(window=1000, sinks=0), dict(window=0, sinks=4)):
        assert plan([640], D=64, **kw)[0] == 64 and plan([64], D=128, **kw) == (256, True)
    assert plan([], 1000, 64) == (256, False)


def test_prefill_sinks_refusals():
    c = W.make_prefill_case("refuse", seed=1, q_lens=[20, 3], contexts=[10, 0], num_q_heads=8,
                            num_kv_heads=2, window=16)
    items, info = pd.paged_prefill_plan_sinks(c.query_start_host, c.seq_lens_host, 8, 2, 128, 16, 4,
                                              1000)

    def call(window=16, sinks=4, scale=0.1, work=items, out=None, D=128, qs=c.query_start):
        return pd.paged_prefill_attn_sinks(c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, qs,
                                           work, info, torch.empty_like(c.q) if out is None else out,
                                           8, 2, D, 16, window, sinks, scale, W.HND, None, check=False)
    assert call() == PASSES
    for kw, rc in [(dict(sinks=-1), -1), (dict(window=-2), -1), (dict(scale=float("inf")), -1),
                   (dict(work=items[:0]), -1), (dict(work=items.long()), -2), (dict(out=c.q.float()), -2),
                   (dict(D=256), -1), (dict(D=100), -3), (dict(qs=c.query_start[:-1]), -1)]:
        assert call(**kw) == rc, kw


# ---- pins of the oracle -----------------------------------------------------

def _pin(**kw):
    return W.make_case("pin", **{**dict(seed=3, dtype=torch.float16, head_size=64, num_q_heads=4,
                                        num_kv_heads=2, page_size=16, max_query_len=3,
                                        seq_lens=[90, 0, 2], window=20), **kw})


def test_oracle_against_the_window_and_full_oracles():
    c, full = _pin(), _pin(window=0)
    assert np.allclose(O.attention(c, 0), oracle.attention(c), rtol=1e-12, atol=1e-12)
    # sinks up to the window's start, or past the sequence: every key
    for sinks in (70, 90, 1000):
        assert np.allclose(O.attention(c, sinks), oracle.attention(full), rtol=1e-12, atol=1e-12)


def test_oracle_as_a_merge_of_two_ranges():
    c = _pin(num_kv_heads=1, max_query_len=1, seq_lens=[200], window=0)
    want = oracle.merge([oracle.partial(c, 0, 7), oracle.partial(c, 150, 200)])
    got = O.attention(W.DecodeCase(**{**c.__dict__, "window": 50}), 7)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_hidden_cases_hold_nan_only_where_no_row_looks():
    c = _pin(max_query_len=2, seq_lens=[300], window=40)
    before = O.attention(c, 5)
    after = hide(c, 5)
    assert np.array_equal(O.attention(after, 5), before)
    assert after.block_table[0].eq(-1).nonzero()[:, 0].tolist() == list(range(1, 16))
    assert np.isnan(O.attention(after, 6)).any()
