"""Scales of the 8-bit cache at and past the range that the attention takes."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import workloads as W
from quant_cases import near, quant_case, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _case(lens, D=128, heads=(8, 2), M=2, **kw):
    return W.make_case("quant", seed=3, dtype=torch.bfloat16, head_size=D, num_q_heads=heads[0], num_kv_heads=heads[1],
                       page_size=16, max_query_len=M, seq_lens=lens, layout=W.HND, **kw)


def _scratch(c):
    return pd.Scratch(c.num_seqs, c.num_q_heads, c.num_kv_heads, c.head_size, c.max_query_len, max_splits=64)


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 0.0, -1.0, 2.0 ** 33, 2.0 ** -65, 2.0 ** 32 * 1.001])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_a_visible_scale_out_of_range_is_reported(D, value, which):
    # the block that every row sees whole, and the last one, of which some rows see a key
    case = _case([400, 33], D=D)
    for s, j in ((0, 7), (1, 2)):
        qc = quant_case(case)
        getattr(qc, which)[int(case.block_table[s, j]), 0, 1] = value
        run(qc, 0, _scratch(case))
        assert pd.paged_decode_device_status(reset=True) == pd.DEV_BAD_SCALE, (s, j)


@pytest.mark.parametrize("value", [float("nan"), 0.0, 2.0 ** 60])
def test_a_scale_that_no_row_sees_is_not(value):
    case = _case([400, 33], window=40)
    qc = quant_case(case)
    for t in (qc.ks, qc.vs):
        t[case.block_table[0, 3:20].long().cuda()] = value
    out = run(qc, 20, _scratch(case))
    torch.cuda.synchronize()
    near(qc, out, 20)


@pytest.mark.parametrize("size", [2.0 ** -64, 2.0 ** 32])
def test_the_ends_of_the_range_are_taken(size):
    # (times a power of two: of every value scale, and of the output; the least or the largest at the end)
    case = _case([300, 17])
    qc = quant_case(case, (None, np.ones((case.k_cache.shape[0], 1, 2))))
    seen = torch.cat([case.block_table[0, :19], case.block_table[1, :2]]).long().cuda()
    held = qc.vs[seen]
    end = float(held.min() if size < 1 else held.max())
    out = run(dataclasses.replace(qc, vs=qc.vs * (size / end)), 0, _scratch(case))
    torch.cuda.synchronize()
    near(qc, out.double() * (end / size))


def test_values_past_the_range_are_written_and_then_reported():
    # 448 x 2^32 is the largest that the attention takes; the write stores what it gets
    case = _case([48], D=64, heads=(2, 1), M=1)
    kc, vc, ks, vs = pd.quant_cache(case.k_cache.shape[0], 1, 64, 16, W.HND)
    page = case.block_table[0].long()
    slots = (page[:3, None] * 16 + torch.arange(16)).reshape(-1).int().cuda()
    k = torch.randn(48, 1, 64).bfloat16().cuda()
    for top, status in ((448 * 2.0 ** 32, 0), (450 * 2.0 ** 32, pd.DEV_BAD_SCALE)):
        v = k.clone()
        v[20, 0, 3] = top
        pd.paged_rope_quant_cache_write(None, k, v, None, slots, None, None, None, kc, vc, ks, vs, 0, 1, 64, 0, 16, W.HND)
        assert float(vs.max()) == (2.0 ** 32 if not status else 2.0 ** 33)
        out = torch.empty((1, 2, 64), dtype=torch.bfloat16, device="cuda")
        pd.paged_decode_attn_quant(case.q.cuda(), kc, vc, ks, vs, case.block_table.cuda(), case.seq_lens.cuda(), out, 2, 1,
                                   64, 16, 1, 0, 0, case.scale, W.HND, _scratch(case))
        assert pd.paged_decode_device_status(reset=True) == status
