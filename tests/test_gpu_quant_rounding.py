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


def _append(codes, scale, x, offset):
    """Token ``offset`` of every page written, fp16 rows x [PAGES, 1, D], K and V."""
    pools, scales = _pools(codes, scale)
    slots = np.arange(PAGES) * P + offset
    dev = [torch.from_numpy(a).half().cuda() for a in x]
    assert all(np.array_equal(a.double().cpu().numpy(), b) for a, b in zip(dev, x))
    pd.paged_rope_quant_cache_write(None, *dev, None, torch.from_numpy(slots.astype(np.int32)).cuda(), None, None, None,
                                    *pools, *scales, 0, 1, D, 0, P, W.NHD)
    for c, s, c0, s0, a in zip(pools, scales, codes, scale, x):
        Q.store(a, slots, c0, s0)
        assert np.array_equal(s.cpu().numpy(), s0)
        bad = Q.by_token(c, W.NHD) != c0
        assert not bad.any(), int(bad.sum())


def test_a_code_of_an_old_scale_is_rounded_once():
    g = np.random.default_rng(2)
    mids = (Q.MAGNITUDES[1:] + Q.MAGNITUDES[:-1]) / 2
    codes, scale, x = [], [], []
    for _ in range(2):
        # x[., 0, 0] / scale next to a midpoint of two codes, x below a quarter of 448 x scale
        top = g.integers(1024, 2048, PAGES) * 2.0 ** -8
        mid = g.choice(mids[(mids > 2.0 ** -5) & (mids < 100)], PAGES)
        s = (top / mid).astype(np.float32)
        a = np.zeros((PAGES, 1, D))
        a[:, 0, 0] = top
        a[:, 0, 1:] = (g.standard_normal((PAGES, D - 1)) * top[:, None] / 4).astype(np.float16)
        a[:, 0, 1] = -top
        codes.append(_codes(g, (PAGES, P, 1, D)))
        scale.append(s.reshape(PAGES, 1, 1))
        x.append(a)
    _append(codes, scale, x, 5)


def test_the_codes_of_a_grown_scale_are_rounded_once():
    g = np.random.default_rng(3)
    mids = (Q.MAGNITUDES[1:] + Q.MAGNITUDES[:-1]) / 2
    codes, scale, x = [], [], []
    for _ in range(2):
        # code 0 of token 3 x old / new next to a midpoint, the new scale 2^-5 .. 2^2
        c = _codes(g, (PAGES, P, 1, D))
        c[:, 3, 0, 0] = g.integers(0x20, 0x7F, PAGES)
        c[:, 3, 0, 1] = c[:, 3, 0, 0] | 0x80
        held = Q.values(c[:, 3, 0, 0])
        new = np.exp2(g.integers(-5, 3, PAGES))
        below = np.maximum(np.searchsorted(mids, held) - 1 - g.integers(0, 12, PAGES), 0)
        s = (mids[below] * new / held).astype(np.float32)
        s = np.where(s < new, s, new / 2).astype(np.float32)
        a = np.zeros((PAGES, 1, D))
        a[:, 0, :] = (g.uniform(-1, 1, (PAGES, D)) * new[:, None] * 100).astype(np.float16)
        a[:, 0, 7] = 400 * new
        codes.append(c)
        scale.append(s.reshape(PAGES, 1, 1))
        x.append(a)
    _append(codes, scale, x, 9)
