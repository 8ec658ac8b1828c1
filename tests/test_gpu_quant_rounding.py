"""The calls on the 8-bit cache with scales that are no powers of two: what is
rounded is rounded once, also where fp32 lies between.  The values here sit
next to the midpoint of two neighbours, nearer than fp32 can tell."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import quant_cache as Q
from paged_split_kv_02_gb300 import workloads as W
from quant_cases import to_pools

pytestmark = pytest.mark.gpu

D, P, PAGES = 64, 16, 3000
BITS = {torch.float16: (11, -14), torch.bfloat16: (8, -126)}  # of a significand, and the least exponent


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def rounded(x: np.ndarray, dtype) -> np.ndarray:
    """x, fp64, to the nearest value of the type, ties to even."""
    bits, least = BITS[dtype]
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 1, least) - bits + 1.0)
    return np.rint(x / step) * step


def _codes(g, shape):
    c = g.integers(0, 256, shape).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] = 0x3C
    return c


def _pools(codes, scale):
    return to_pools(*codes, W.NHD, False), [torch.from_numpy(s).cuda() for s in scale]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_value_read_is_rounded_once(dtype):
    g = np.random.default_rng(1)
    bits = BITS[dtype][0]
    codes = [_codes(g, (PAGES, P, 1, D)) for _ in range(2)]
    scale = []
    for c in codes:
        # c[., 0, 0, 0] x scale within half a step of fp32 of a midpoint, 2^(bits + 1) being one more bit
        c[:, 0, 0, 0] = g.choice([0x39, 0x3B, 0x3D, 0x3F, 0xB9], PAGES)
        mid = (2 * g.integers(2 ** (bits - 1), 2 ** bits, PAGES) + 1) * np.exp2(g.integers(-20, 2, PAGES) - bits)
        scale.append((mid / np.abs(Q.values(c[:, 0, 0, 0]))).astype(np.float32).reshape(PAGES, 1, 1))
    (k, v), (ks, vs) = _pools(codes, scale)
    out = [torch.empty((PAGES, P, 1, D), dtype=dtype, device="cuda") for _ in range(2)]
    table = torch.arange(PAGES, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([PAGES * P], dtype=torch.int32, device="cuda")
    pd.paged_quant_cache_read(k, v, ks, vs, table, lens, table, *out, 1, D, P, W.NHD)
    for o, c, s in zip(out, codes, scale):
        want = rounded(Q.dequantised(c, s), dtype)
        assert np.isfinite(want).all() and np.abs(want).max() < 65504
        bad = o.double().cpu().numpy() != want
        assert not bad.any(), int(bad.sum())
