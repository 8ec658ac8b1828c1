"""The calls on the 8-bit cache: blocks that are written again, scales further than
2^31 elements away, tables much wider than their requests, row groups that have
no row of a request."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from gpu_helpers import sample_rows
from oracle import quant_cache as Q
from paged_split_kv_02_gb300 import workloads as W
from quant_cases import near, quant_case, run
from test_gpu_quant_cache import RUNS, Cache, _i32, _slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _scratch(c, splits=64):
    return pd.Scratch(c.num_seqs, c.num_q_heads, c.num_kv_heads, c.head_size, c.max_query_len, max_splits=splits)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_a_block_written_again_with_what_it_holds(D):
    g = np.random.default_rng(D)
    pages = sum((a + n - 1) // 16 - a // 16 + 1 for a, n in RUNS) + 2
    c = Cache(D, pages, 16, 2, D, W.HND)
    slots = _slots(g, RUNS, pages, 16)
    codes0, scale0 = [x.copy() for x in c.codes], [x.copy() for x in c.scale]
    back = [Q.dequantised(a, s).reshape(-1, 2, D)[slots] for a, s in zip(codes0, scale0)]
    k, v = (torch.from_numpy(b).to(torch.bfloat16).cuda() for b in back)
    for x, b in zip((k, v), back):
        assert np.array_equal(x.double().cpu().numpy(), b)

    def write():
        pd.paged_rope_quant_cache_write(None, k, v, None, _i32(slots), None, None, None, c.k, c.v, c.ks, c.vs, 0, 2, D,
                                        0, 16, W.HND)
        torch.cuda.synchronize()
        return c.got()

    codes, scale = write()
    for i in range(2):
        # what tokens hold is the same, but for codes below the scale that their block now has
        Q.store(back[i], slots, codes0[i], scale0[i])
        assert np.array_equal(codes[i], codes0[i]) and np.array_equal(scale[i], scale0[i])
    again, scale2 = write()
    assert all(np.array_equal(a, b) for a, b in zip(codes + scale, again + scale2))


def _far_scales(scale, buf, at):
    """Scales as a view whose last pages lie past 2^31 elements, block and head apart."""
    view = buf.as_strided(scale.shape, (1 << 29, 7001, 37), at)
    view.copy_(scale)
    return view


def test_scales_past_32_bits():
    pages, P, H, D = 6, 32, 2, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    buf = torch.empty(pages << 29, device="cuda")
    c = Cache(4, pages, P, H, D, W.NHD)
    codes0, scale0 = [x.copy() for x in c.codes], [x.copy() for x in c.scale]
    ks, vs = (_far_scales(s, buf, at) for s, at in ((c.ks, 11), (c.vs, 100003)))
    assert 5 * ks.stride(0) > 1 << 31
    slots = np.array([0, 1, 33, 34, 5 * P + 7, 5 * P + 8, 5 * P + 16, 4 * P + 31])
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((2, 8, H, D))).bfloat16()
    pd.paged_rope_quant_cache_write(None, x[0].cuda(), x[1].cuda(), None, _i32(slots), None, None, None, c.k, c.v, ks,
                                    vs, 0, H, D, 0, P, W.NHD)
    c.ks, c.vs = ks, vs
    codes, scale = c.got()
    for j in range(2):
        Q.store(x[j].double().numpy(), slots, codes0[j], scale0[j])
        assert np.array_equal(codes[j], codes0[j]) and np.array_equal(scale[j], scale0[j])
    out = [torch.zeros((pages, P, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = _i32(np.arange(pages)[None])
    pd.paged_quant_cache_read(c.k, c.v, ks, vs, table, _i32([pages * P]), table, *out, H, D, P, W.NHD)
    for j in range(2):
        assert torch.equal(out[j].cpu(), torch.from_numpy(Q.dequantised(codes0[j], scale0[j])).bfloat16())
    # the attention over the last two pages
    case = W.make_case("quant", seed=1, dtype=torch.bfloat16, head_size=D, num_q_heads=4, num_kv_heads=H, page_size=P,
                       max_query_len=2, seq_lens=[50], layout=W.NHD)
    case = dataclasses.replace(case, block_table=torch.tensor([[5, 4]], dtype=torch.int32))
    values = [torch.from_numpy(Q.dequantised(a, s)) for a, s in zip(codes0, scale0)]
    top = max(float(v.abs().max()) for v in values)  # (random codes are large: scores below 30)
    case = dataclasses.replace(case, scale=case.scale / top, k_cache=values[0], v_cache=values[1])
    qc = dataclasses.replace(quant_case(dataclasses.replace(case, k_cache=values[0] * 0, v_cache=values[1] * 0)),
                             case=case, exact=case, k=c.k, v=c.v, ks=ks, vs=vs)
    got = run(qc, 0, _scratch(case))
    torch.cuda.synchronize()
    near(qc, got)


@pytest.mark.parametrize("D,layout", [(64, W.NHD), (128, W.HND), (256, W.HND)])
def test_tables_much_wider_than_the_requests(D, layout):
    # what stands behind a request's pages in a table is not looked at
    lens, P, width = [70, 1, 0, 333], 16, 5000
    case = W.make_case("quant", seed=2, dtype=torch.float16, head_size=D, num_q_heads=8, num_kv_heads=2, page_size=P,
                       max_query_len=1, seq_lens=lens, layout=layout)
    wide = torch.full((4, width), 10 ** 8, dtype=torch.int32)
    wide[:, 1::2] = -3
    for s, L in enumerate(lens):
        n = -(-L // P)
        wide[s, :n] = case.block_table[s, :n]
    case = dataclasses.replace(case, block_table=wide)
    qc = quant_case(case)
    out = run(qc, 0, _scratch(case))
    torch.cuda.synchronize()
    near(qc, out)
    pages = qc.k.shape[0]
    staged = [torch.full(qc.k.shape, 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    pd.paged_quant_cache_read(qc.k, qc.v, qc.ks, qc.vs, wide.cuda(), _i32(lens), wide.cuda(), *staged, 2, D, P, layout)
    torch.cuda.synchronize()
    for got, codes, s in zip(staged, (qc.k, qc.v), (qc.ks, qc.vs)):
        want = np.full((pages, P, 2, D), 9.0)
        Q.read(Q.dequantised(Q.by_token(codes, layout), s.cpu().numpy()), wide.tolist(), lens, wide.tolist(), want)
        got = got if layout == W.NHD else got.permute(0, 2, 1, 3)
        assert torch.equal(got.cpu(), torch.from_numpy(want).half())


@pytest.mark.parametrize("D,heads,M", [(512, (8, 1), 8), (256, (16, 2), 8), (256, (16, 2), 4), (128, (32, 4), 8),
                                       (64, (32, 1), 8)])
@pytest.mark.parametrize("splits", [None, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (80, 9)])
def test_row_groups_without_a_row_of_a_request(D, heads, M, splits, window, sinks):
    # requests of one token beside one that has them all: most of the groups have no row of them
    q_lens = [1, M, 0, 1, 2, 1]
    case = W.make_varlen_case("quant", seed=D + M, q_lens=q_lens, pad_tokens=2, dtype=torch.bfloat16, head_size=D,
                              num_q_heads=heads[0], num_kv_heads=heads[1], page_size=16,
                              seq_lens=[300, 45, 80, 1, 700, 128], layout=W.HND, window=window)
    qc = quant_case(case)
    out = torch.full_like(case.q, float("nan"), device="cuda")
    run(qc, sinks, None if splits is None else _scratch(case, splits), out=out)
    torch.cuda.synchronize()
    near(qc, out, sinks, rows=sample_rows(case, 200))
    assert float(out[-2:].abs().sum()) == 0.0 and bool(torch.isfinite(out).all())
