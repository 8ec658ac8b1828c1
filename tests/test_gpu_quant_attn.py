"""paged_decode_attn_quant against the fp64 oracle on the values that the codes
stand for (bounds: quant_cases.near)."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from gpu_helpers import sample_rows
from paged_split_kv_02_gb300 import workloads as W
from quant_cases import near, quant_case, run
from step_cases import hide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _case(lens, D=128, heads=(8, 2), P=16, M=1, dtype=torch.bfloat16, layout=W.HND, window=0, seed=1, q_lens=None,
          pad=0, **kw):
    if q_lens is not None:
        return W.make_varlen_case("quant", seed=seed, q_lens=q_lens, pad_tokens=pad, dtype=dtype, head_size=D,
                                  num_q_heads=heads[0], num_kv_heads=heads[1], page_size=P, seq_lens=lens,
                                  layout=layout, window=window, **kw)
    return W.make_case("quant", seed=seed, dtype=dtype, head_size=D, num_q_heads=heads[0], num_kv_heads=heads[1],
                       page_size=P, max_query_len=M, seq_lens=lens, layout=layout, window=window, **kw)


def _scratch(c, splits=64):
    return pd.Scratch(c.num_seqs, c.num_q_heads, c.num_kv_heads, c.head_size, c.max_query_len, max_splits=splits)


def _checked(case, sinks=0, splits=64, packed=False, factors=(None, None), rows=None):
    qc = quant_case(case, factors, packed)
    sc = None if splits is None else _scratch(case, splits)
    out = run(qc, sinks, sc)
    torch.cuda.synchronize()
    near(qc, out, sinks, rows)
    if sc is not None:
        assert int(sc.counters().abs().sum()) == 0
    return qc, out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [0, 300, 33, 1]])
def test_short_contexts(dtype, D, lens):
    _checked(_case(lens, D=D, dtype=dtype))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (16, 1), (15, 5), (24, 3)])
@pytest.mark.parametrize("M", [1, 3, 8])
def test_head_groups_and_query_tokens(D, heads, M):
    _checked(_case([700, 5, 210], D=D, heads=heads, M=M, dtype=torch.float16 if M == 3 else torch.bfloat16))


@pytest.mark.parametrize("layout", [W.NHD, W.HND])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("P", [16, 48, 64, 1056])
@pytest.mark.parametrize("D", [64, 256])
def test_layouts_and_pages(layout, packed, P, D):
    _checked(_case([1500, 47, 48, 49], D=D, P=P, layout=layout, heads=(6, 3), M=2), packed=packed)


@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 0), (40, 5), (100, 16), (16, 130), (700, 33), (5000, 3)])
@pytest.mark.parametrize("D", [64, 128, 512])
def test_windows(window, sinks, D):
    # (what no row sees is NaN, its pages are gone from the table)
    case = hide(_case([900, 3, 57, 1400], D=D, M=4, window=window), sinks)
    _checked(case, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 7)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_query_lengths_and_padding(window, sinks, D):
    case = _case([500, 9, 40, 260, 0, 2], q_lens=[3, 0, 1, 4, 0, 2], pad=3, D=D, window=window)
    qc = quant_case(case)
    out = torch.full_like(case.q, float("nan"), device="cuda")
    run(qc, sinks, _scratch(case), out=out)
    torch.cuda.synchronize()
    near(qc, out, sinks)
    assert float(out[-3:].abs().sum()) == 0.0


def test_more_query_tokens_than_keys():
    _checked(_case([2, 1, 0, 5], M=4))


@pytest.mark.parametrize("splits", [None, 0, 2, 8, 256])
@pytest.mark.parametrize("D,heads,M", [(128, (8, 2), 1), (64, (32, 1), 4), (512, (4, 1), 8)])
def test_any_scratch(splits, D, heads, M):
    _checked(_case([2100, 13, 800], D=D, heads=heads, M=M), splits=splits)


@pytest.mark.parametrize("D,heads,M", [(128, (8, 2), 2), (256, (8, 2), 2), (512, (8, 1), 1), (64, (4, 1), 8), (128, (32, 1), 1)])
@pytest.mark.parametrize("splits", [20, 256])
def test_one_long_context(D, heads, M, splits):
    # (up to 152 parts of a unit, merged in groups)
    case = _case([20000], D=D, heads=heads, M=M)
    _checked(case, splits=splits, rows=sample_rows(case, 12))


def test_scales_of_any_size():
    # fp32 scales that are no powers of two, from block to block 2^-40 to 2^20 apart
    rng = np.random.default_rng(5)
    case = _case([333, 70], heads=(8, 2), M=2)
    shape = (case.k_cache.shape[0], 1, 2)
    small = rng.uniform(0.6, 1.9, shape)  # (a code may pass 448 and saturate: it is what it is)
    _checked(case, factors=(small, np.exp2(rng.uniform(-20, 0, shape))))
    v = case.v_cache * torch.exp2(torch.randint(-40, 20, (case.v_cache.shape[0], 1, 1, 1)).float())
    wide = dataclasses.replace(case, v_cache=v.to(torch.bfloat16))
    _checked(wide, factors=(small, small))


def test_a_block_of_zeros_keeps_its_weight():
    # (its scale is 2^-64: the sum of the weights must not lose it)
    case = _case([64], heads=(4, 1))
    v = case.v_cache.clone()
    v[:2] = 0
    _checked(dataclasses.replace(case, v_cache=v))


@pytest.mark.parametrize("size", [1e-6, 3e4])
def test_queries_of_any_size(size):
    case = _case([150, 31], heads=(8, 2), M=2)
    _checked(dataclasses.replace(case, q=(case.q.float() * size).to(case.dtype), scale=case.scale / size))


def test_one_key_takes_the_weight_of_a_long_tail():
    # a first key far above the others, whose small weights sum to a quarter
    case = _case([8000], heads=(4, 1), v_mean=1.0)
    page = int(case.block_table[0, 0])
    top = torch.zeros(128)
    top[0] = 440.0
    case.k_cache[page, 0, 0] = top.to(case.dtype)
    case.q[..., 0] = 11.0 / case.scale / 440.0
    _checked(case, splits=64)


def test_many_sequences():
    # past the sequences of one line, with lengths that leave some without a key
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, 2500).tolist()
    case = _case(lens, D=64, heads=(2, 1))
    rows = [(int(t), int(t) % 2) for t in rng.integers(0, 2500, 300)] + [(0, 0), (447, 1), (448, 0), (2499, 1)]
    for splits in (1, None):
        _checked(case, splits=splits, rows=rows)


def test_offsets_past_32_bits():
    # a pool of 5 GiB whose last pages are used, scales of a wide stride
    free = torch.cuda.mem_get_info()[0]
    if free < 24 << 30:
        pytest.skip("needs 24 GiB")
    case = _case([200], heads=(4, 2))
    small = quant_case(case)
    n = (5 << 30) // (2 * 16 * 128)
    used = small.k.shape[0]
    k = torch.empty((n, 2, 16, 128), dtype=torch.uint8, device="cuda")
    k[n - used:] = small.k.view(torch.uint8)
    v = torch.empty_like(k)
    v[n - used:] = small.v.view(torch.uint8)
    s = torch.empty((2, n, 1, 2 * 520), device="cuda")[..., ::520]
    s[0, n - used:] = small.ks
    s[1, n - used:] = small.vs
    moved = dataclasses.replace(case, block_table=case.block_table + (n - used))
    qc = dataclasses.replace(small, case=moved, k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn),
                             ks=s[0], vs=s[1])
    out = run(qc, 0, _scratch(case))
    torch.cuda.synchronize()
    near(small, out)


def test_strided_tensors():
    case = _case([130, 17], heads=(8, 2), M=2, P=32)
    qc = quant_case(case)
    wide = lambda t, d: torch.cat([t, torch.full_like(t, 0)], d)  # noqa: E731
    k = wide(wide(qc.k.view(torch.uint8), 2), 0)[:qc.k.shape[0], :, :32]
    ks = wide(qc.ks, 2)[..., :2]
    q = wide(case.q.cuda(), 1)[:, :8]
    out = torch.full((4, 16, 128), 7.0, dtype=case.dtype, device="cuda")
    table = torch.cat([case.block_table, case.block_table], 1).cuda()[:, :case.block_table.shape[1]]
    pd.paged_decode_attn_quant(q, k.view(torch.float8_e4m3fn), qc.v, ks, qc.vs, table, case.seq_lens.cuda(),
                               out[:, 4:12], 8, 2, 128, 32, 2, 0, 0, case.scale, case.layout, _scratch(case))
    torch.cuda.synchronize()
    near(qc, out[:, 4:12])
    assert bool((out[:, :4] == 7).all() and (out[:, 12:] == 7).all())


def test_captured_and_replayed_on_another_stream():
    case = _case([900, 40, 3000], heads=(8, 2), M=2)
    qc = quant_case(case)
    sc = _scratch(case)
    args = [t.cuda() for t in (case.q, case.block_table, case.seq_lens)]
    outs = [torch.empty_like(args[0]) for _ in range(2)]

    def call(out, window):
        pd.paged_decode_attn_quant(args[0], qc.k, qc.v, qc.ks, qc.vs, args[1], args[2], out, 8, 2, 128, 16, 2, window,
                                   0, case.scale, case.layout, sc)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for out, window in zip(outs, (0, 500)):
            call(out, window)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                for _ in range(3):
                    call(out, window)
            graphs.append(g)
        for _ in range(20):
            for g in graphs:  # one scratch, one stream
                g.replay()
    side.synchronize()
    near(qc, outs[0])
    near(dataclasses.replace(qc, case=case, exact=dataclasses.replace(qc.exact, window=500)), outs[1])
    first = outs[0].clone()
    args[2].copy_(torch.tensor([33, 900, 7], dtype=torch.int32))
    # (shorter lengths: the tables still hold their pages)
    args[2].clamp_(max=40)
    graphs[0].replay()
    torch.cuda.synchronize()
    short = dataclasses.replace(qc.exact, seq_lens=args[2].cpu(), seq_lens_host=args[2].tolist())
    near(dataclasses.replace(qc, exact=short), outs[0])
    assert not torch.equal(first, outs[0])


def test_the_same_call_gives_the_same_bits():
    case = _case([3000, 1, 777, 90], heads=(16, 2), M=4)
    qc = quant_case(case)
    sc = _scratch(case)
    outs = [run(qc, 0, sc) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_bad_pages_and_lengths_are_reported():
    case = _case([60, 60], heads=(4, 2))
    qc = quant_case(case)
    table = case.block_table.clone()
    table[0, 1] = 10 ** 6
    table[1, 3] = -5
    run(dataclasses.replace(qc, case=dataclasses.replace(case, block_table=table)), 0, _scratch(case))
    assert pd.paged_decode_device_status(reset=True) == pd.DEV_BAD_PAGE
    lens = torch.tensor([60, 600], dtype=torch.int32)
    run(dataclasses.replace(qc, case=dataclasses.replace(case, seq_lens=lens)), 0, _scratch(case))
    assert pd.paged_decode_device_status(reset=True) & pd.DEV_BAD_SEQLEN
    case = _case([60, 60], q_lens=[1, 1], heads=(4, 2))
    bad = dataclasses.replace(case, query_start=torch.tensor([0, 5, 2], dtype=torch.int32))
    run(dataclasses.replace(quant_case(case), case=bad), 0, _scratch(case))
    assert pd.paged_decode_device_status(reset=True) & pd.DEV_BAD_QSTART


def test_a_batch_without_requests_zeroes_its_padding():
    case = _case([40], q_lens=[1], heads=(4, 2))
    qc = quant_case(case)
    out = torch.full((3, 4, 128), 5.0, dtype=case.dtype, device="cuda")
    none = dataclasses.replace(case, q=torch.zeros((3, 4, 128), dtype=case.dtype), block_table=case.block_table[:0],
                               seq_lens=case.seq_lens[:0], query_start=torch.zeros(1, dtype=torch.int32))
    run(dataclasses.replace(qc, case=none), 0, None, out=out)
    torch.cuda.synchronize()
    assert float(out.abs().sum()) == 0.0


@pytest.mark.parametrize("D,M", [(64, 4), (128, 1), (512, 2)])
def test_pages_shared_and_pages_before_a_window(D, M):
    # two requests begin with the same pages; pages that a window has left are gone from the table
    case = _case([700, 500, 90], D=D, heads=(8, 2), M=M)
    table, pool = case.block_table.clone(), case.k_cache.shape[0]
    table[1, :20] = table[0, :20]
    assert int(table.max()) < pool
    _checked(dataclasses.replace(case, block_table=table))
    for window, sinks in ((100, 0), (100, 20)):
        cut = table.clone()
        for s, L in enumerate((700, 500, 90)):
            first = max(0, L - M + 1 - window) // 16
            cut[s, -(-sinks // 16):first] = -1
        qc = quant_case(dataclasses.replace(case, window=window, block_table=table))
        out = run(dataclasses.replace(qc, case=dataclasses.replace(qc.case, block_table=cut)), sinks, _scratch(case))
        torch.cuda.synchronize()
        near(qc, out, sinks)


def test_two_streams_at_once():
    # calls on two streams, each with scratch of its own
    case = _case([2000, 30, 900], heads=(16, 2), M=2)
    qc = quant_case(case)
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    scratch = [_scratch(case) for _ in streams]
    tensors = [case.q.cuda(), case.block_table.cuda(), case.seq_lens.cuda()]
    torch.cuda.synchronize()
    for _ in range(15):
        for st, sc in zip(streams, scratch):
            out = torch.zeros_like(tensors[0])
            st.wait_stream(torch.cuda.current_stream())
            pd.paged_decode_attn_quant(tensors[0], qc.k, qc.v, qc.ks, qc.vs, tensors[1], tensors[2], out, 16, 2, 128, 16,
                                       2, 0, 0, case.scale, case.layout, sc, stream=st)
            outs.append(out)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    near(qc, outs[0])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("heads,M", [((8, 2), 8), ((16, 2), 3), ((8, 2), 3), ((24, 2), 8), ((4, 2), 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 20)])
def test_many_rows_of_many_requests(D, heads, M, window, sinks):
    # (few units take fewer rows a CTA: these have all that fit, in cut and in whole units)
    rng = np.random.default_rng(D + M)
    lens = rng.integers(0, 120, 50).tolist()
    lens[7], lens[31] = 900, 700
    case = _case(lens, D=D, heads=heads, M=M, window=window)
    R = heads[0] // heads[1] * M
    full = min(-(-R // 8), 4 if D == 64 else 512 // D)
    plan = pd.paged_decode_plan_quant(50, *heads, D, 16, M, window, sinks, case.block_table.shape[1], 152, _scratch(case))
    assert plan["n_tiles"] >= full
    rows = [(int(t), int(t) % heads[0]) for t in rng.integers(0, 50 * M, 150)] + [(7 * M, 0), (32 * M - 1, heads[0] - 1)]
    _checked(case, sinks, rows=rows)


@pytest.mark.parametrize("D,M", [(64, 8), (128, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("L", [300, 9000, 40000])
def test_rows_of_a_few_long_requests(D, M, L):
    # the rows a CTA are the plan's choice, by the table's width
    case = _case([L], D=D, heads=(8, 2), M=M)
    _checked(case, rows=[(t, h) for t in range(M) for h in (0, 3, 7)], splits=256)
