"""paged_rope_quant_cache_write with slots that break its rules: what is left out
is reported, whatever the window of tokens a CTA has, and nothing else changes."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import quant_cache as Q
from paged_split_kv_02_gb300 import workloads as W
from quant_cases import to_pools

pytestmark = pytest.mark.gpu

D, P, PAGES = 64, 32, 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


# (tokens, kv heads) by which the write has 1, 4, 16, 32 and 64 tokens a CTA on 152 SMs
SIZES = [(40, 1), (1200, 8), (9000, 4), (30000, 1), (110000, 1)]


def _check(T, H, at, slots, kept, status):
    """A write of T tokens, padding but for ``slots`` from token ``at`` on."""
    g = np.random.default_rng(at)
    codes = [g.integers(0, 0x7F, (PAGES, P, H, D)).astype(np.uint8) for _ in range(2)]
    scale = [np.exp2(g.integers(-14, 2, (PAGES, P // 16, H))).astype(np.float32) for _ in range(2)]
    pools = to_pools(*codes, W.HND, False)
    scales = [torch.from_numpy(s).cuda() for s in scale]
    every = np.full(T, -1, dtype=np.int32)
    every[at:at + len(slots)] = slots
    x = [torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rows = [torch.from_numpy(g.standard_normal((len(slots), H, D))).bfloat16() for _ in range(2)]
    for a, b in zip(x, rows):
        a[at:at + len(slots)] = b.cuda()
    pd.paged_rope_quant_cache_write(None, *x, None, torch.from_numpy(every).cuda(), None, None, None, *pools, *scales,
                                    0, H, D, 0, P, W.HND)
    assert pd.paged_decode_device_status(reset=True) == status, (T, H, at, slots)
    for c, s, c0, s0, r in zip(pools, scales, codes, scale, rows):
        Q.store(r.double().numpy(), kept, c0, s0)
        assert np.array_equal(Q.by_token(c, W.HND), c0) and np.array_equal(s.cpu().numpy(), s0), (T, H, at, slots)


@pytest.mark.parametrize("T,H", SIZES)
def test_a_slot_that_comes_again_after_a_whole_run(T, H):
    # at every place of the CTAs' tokens
    for at in range(0, 18 if T < 100 else 64):
        slots = list(range(16, 32)) + [16, 40]
        _check(T, H, at, slots, slots[:16] + [-1, 40], pd.DEV_BAD_SLOT)


@pytest.mark.parametrize("T,H", SIZES)
def test_a_whole_run_and_the_next_blocks(T, H):
    for at in (0, 1, 14, 15, 16, 20):
        slots = list(range(16, 36))
        _check(T, H, at, slots, slots, 0)


@pytest.mark.parametrize("T,H", SIZES)
def test_a_block_in_two_runs(T, H):
    # the first one is written; beside it, with padding or another block between, and as far away as is looked
    cases = [([16, 17, -1, 18], [16, 17, -1, -1]), ([0, 16, 1], [0, 16, -1]), ([35, 70, 32, 33, 20], [35, 70, -1, -1, 20]),
             ([5, 3, 40, 6], [5, -1, 40, -1]), ([7, 20, 9, 21, 10], [7, 20, -1, -1, -1])]
    for gap in (2, 16, 17, 33, 64, 80, pd.RUN_DISTANCE):
        between = [-1] * (gap - 1)
        cases.append(([16] + between + [17, 18, 50], [16] + between + [-1, -1, 50]))
    for at in (0, 1, 14, 16, 31, 47, 63):
        for slots, kept in cases:
            if at + len(slots) <= T:
                _check(T, H, at, slots, kept, pd.DEV_BAD_SLOT)


@pytest.mark.parametrize("T,H", SIZES)
def test_one_run_each_of_many_blocks(T, H):
    for at in (0, 5, 16):
        slots = [20, 3, -1, 40, 41, -1, 64, 100, 101, 150]
        _check(T, H, at, slots, slots, 0)
