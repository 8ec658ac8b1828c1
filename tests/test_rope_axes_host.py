"""paged_rope_axes_cache_write on the CPU: refusals (checked on the host before
any launch), the pairs' axes, and its oracle's pins."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import rope_cache as R
from oracle.rope_axes import rope_axes
from paged_split_kv_02_gb300 import workloads as W

PASSES = -8  # a call that passes every check reaches the missing device


@pytest.fixture(scope="module", autouse=True)
def _built():
    if torch.cuda.is_available():
        pytest.skip("host tensors: for machines without a GPU")
    pd.build()


def _rope(axis=None, sections=(12, 10, 10), **kw):
    c = W.make_rope_case("refuse", seed=1, dtype=torch.bfloat16, num_tokens=6, num_q_heads=4,
                         num_kv_heads=2, head_size=128, rot_dim=64, page_size=16, num_pages=3)
    a = dict(q=c.q, k=c.k, v=c.v, pos=torch.zeros(3, 6, dtype=torch.int32), slots=c.slot_mapping,
             cs=c.cos_sin, out=torch.empty_like(c.q), kc=c.k_cache, vc=c.v_cache, Hq=4, Hkv=2, D=128,
             rot=64, P=16, layout=W.HND, neox=True)
    a.update(kw)
    return pd.paged_rope_axes_cache_write(
        a["q"], a["k"], a["v"], a["pos"], a["slots"], a["cs"],
        pd.rope_pair_axis(sections) if axis is None else axis, a["out"], a["kc"], a["vc"], a["Hq"],
        a["Hkv"], a["D"], a["rot"], a["P"], a["layout"], a["neox"], check=False)


def test_rope_axes_refusals():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for kw in [dict(), dict(pos=i(6).expand(3, 6)), dict(pos=i(8, 6)), dict(pos=i(3, 9)[:, 1:7]),
               dict(neox=False)]:
        assert _rope(**kw) == PASSES, kw
    for kw, rc in [(dict(pos=i(6)), -1), (dict(pos=i(2, 6)), -1), (dict(pos=i(9, 6)), -1),
                   (dict(pos=i(0, 6)), -1), (dict(pos=i(3, 5)), -1), (dict(pos=i(3, 6).long()), -2),
                   (dict(pos=i(3, 12)[:, ::2]), -5), (dict(slots=i(5)), -1), (dict(slots=i(6).long()), -2),
                   (dict(D=96), -3), (dict(P=0), -1), (dict(rot=24, axis=bytes(12)), -1),
                   (dict(rot=0, axis=b""), -1), (dict(Hq=3), -1), (dict(cs=torch.zeros(10, 60)), -1),
                   (dict(cs=torch.zeros(10, 64).double()), -2), (dict(axis=bytes([3] * 32)), -1),
                   (dict(layout=5), -1), (dict(k=torch.zeros(6, 2, 128)), -2)]:
        assert _rope(**kw) == rc, kw
    with pytest.raises(ValueError):
        _rope(axis=bytes(31))
    with pytest.raises(pd.PagedDecodeError):
        pd.paged_rope_axes_cache_write(*[i(3)] * 6, bytes(8), i(3), i(3), i(3), 1, 1, 64, 16, 16, 0)


def test_rope_pair_axis():
    assert list(pd.rope_pair_axis([2, 1, 3])) == [0, 0, 1, 2, 2, 2]
    assert list(pd.rope_pair_axis([4, 2, 2], interleaved=True)) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert list(pd.rope_pair_axis([5], interleaved=True)) == [0] * 5
    for sections in ([24, 20, 20], [16, 16, 16, 16], [44, 20]):
        m = pd.rope_pair_axis(sections, interleaved=True)
        assert [m.count(a) for a in range(len(sections))] == sections
    for bad in ([1, 3, 0], [], [3, -1], [1] * 9):
        with pytest.raises(ValueError):
            pd.rope_pair_axis(bad, interleaved=True)


def test_oracle_of_one_position():
    c = W.make_rope_case("pin", seed=6, dtype=torch.float16, num_tokens=5, num_q_heads=3,
                         num_kv_heads=1, head_size=64, rot_dim=32, page_size=16, num_pages=1)
    x, table = c.q.double().numpy(), c.cos_sin.double().numpy()
    pos = c.positions.numpy()
    for neox in (True, False):
        want = R.rope(x, pos, table, 32, neox)
        assert np.array_equal(rope_axes(x, np.stack([pos, pos]), table, [0, 1] * 8, 32, neox), want)
        # a pair turned by the other axis's position alone
        two = rope_axes(x, np.stack([pos, pos * 0]), table, [1] * 15 + [0], 32, neox)
        a, b = R.pair_index(32, neox)
        same = np.ones(64, dtype=bool)
        same[[a[15], b[15]]] = False
        assert np.array_equal(two[..., same], x[..., same])
        assert np.array_equal(two[..., ~same], want[..., ~same])
