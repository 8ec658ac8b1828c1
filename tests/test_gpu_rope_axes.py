"""paged_rope_axes_cache_write against its fp64 oracle, through the C ABI.

Bounds: an fp32 computation rounded once, half a step of the input type (2^-8
of the value for bf16, 2^-11 for fp16) plus the fp32 arithmetic (2^-22 of |x1|
+ |x2|); v is copied bit for bit, the slots the call does not name keep their
bits."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import rope_cache as R
from oracle.rope_axes import rope_axes
from paged_split_kv_02_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _inputs(seed, dtype, T, Hq, Hkv, D, rot, P, layout, axes, max_pos=3000, pad=0, packed=False,
            neox=True):
    c = W.make_rope_case("axes", seed=seed, dtype=dtype, num_tokens=T, num_q_heads=Hq,
                         num_kv_heads=Hkv, head_size=D, rot_dim=rot, page_size=P,
                         num_pages=-(-T // P) + 2, layout=layout, is_neox=neox, max_pos=max_pos,
                         pad_tokens=pad, packed=packed)
    return c, np.random.default_rng(seed).integers(0, max_pos, (axes, T)).astype(np.int32)


def _pair_magnitude(x, rot, neox):
    a, b = R.pair_index(rot, neox)
    m = np.zeros_like(x)
    m[..., a] = m[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return m


def _near(gpu, ref, x, rot, neox, dtype, what):
    eps = 2.0 ** -22 * _pair_magnitude(x, rot, neox)
    tol = HALF_ULP[dtype] * (np.abs(ref) + eps) + eps + 2.0 ** -24
    bad = np.abs(gpu.double().cpu().numpy() - ref) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values off"


def _call(g, pos, axis, q_out, stream=None):
    pd.paged_rope_axes_cache_write(g.q, g.k, g.v, pos, g.slot_mapping, g.cos_sin, axis, q_out,
                                   g.k_cache, g.v_cache, g.num_q_heads, g.num_kv_heads, g.head_size,
                                   g.rot_dim, g.page_size, g.layout, g.is_neox, stream=stream)


def _rope(c, pos, axis, inplace=False):
    g = c.to("cuda")
    q_out = g.q if inplace else torch.empty_like(g.q)
    _call(g, torch.from_numpy(pos).cuda(), axis, q_out)
    torch.cuda.synchronize()
    table = c.cos_sin.double().numpy()
    qr, kr = (rope_axes(x.double().numpy(), pos, table, axis, c.rot_dim, c.is_neox)
              for x in (c.q, c.k))
    _near(q_out, qr, c.q.double().numpy(), c.rot_dim, c.is_neox, c.dtype, "q")
    by = (lambda x: x) if c.layout == W.NHD else (lambda x: x.permute(0, 2, 1, 3))
    want_k, want_v = by(c.k_cache).clone(), by(c.v_cache).clone()
    got_k, got_v = by(g.k_cache).cpu(), by(g.v_cache).cpu()
    slots = c.slot_mapping.numpy()
    on = np.nonzero(slots >= 0)[0]
    page = torch.from_numpy(slots[on] // c.page_size).long()
    tok = torch.from_numpy(slots[on] % c.page_size).long()
    _near(got_k[page, tok], kr[on], c.k.double().numpy()[on], c.rot_dim, c.is_neox, c.dtype, "k")
    want_k[page, tok] = got_k[page, tok]
    want_v[page, tok] = c.v[torch.from_numpy(on)]
    assert torch.equal(got_v, want_v), "v copied, the other slots as they were"
    assert torch.equal(got_k, want_k), "the other slots as they were"
    return g, q_out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("D,rot,sections,inter", [
    (128, 128, (16, 24, 24), False), (128, 128, (24, 20, 20), True), (64, 64, (11, 10, 11), False),
    (256, 64, (8, 12, 12), False), (512, 512, (100, 78, 78), True), (128, 96, (48, 0), False),
    (64, 32, (1, 2, 3, 10), False), (256, 256, (128,), False), (512, 16, (4, 2, 2), True)])
def test_rope_axes_match_the_oracle(dtype, neox, D, rot, sections, inter):
    c, pos = _inputs(D + rot, dtype, 37, 8, 2, D, rot, 16, W.HND, len(sections), pad=3, neox=neox)
    _rope(c, pos, pd.rope_pair_axis(sections, inter))


@pytest.mark.parametrize("layout", [W.NHD, W.HND])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,heads", [(1, (32, 8)), (50, (6, 6)), (1400, (20, 4))])
def test_rope_axes_layouts_and_sizes(layout, packed, T, heads):
    c, pos = _inputs(T, torch.bfloat16, T, *heads, 128, 64, 48, layout, 3, packed=packed)
    _rope(c, pos, pd.rope_pair_axis((12, 10, 10)), inplace=T == 50)


@pytest.mark.parametrize("T,pad,neox,rot", [(6000, 5, True, 128), (5003, 0, False, 64), (9000, 9000, True, 96)])
def test_rope_axes_many_tokens(T, pad, neox, rot):
    c, pos = _inputs(T, torch.float16, T, 10, 2, 128, rot, 16, W.HND, 3, pad=pad, neox=neox)
    half = rot // 2
    _rope(c, pos, pd.rope_pair_axis((half - 2 * (half // 3), half // 3, half // 3), neox),
          inplace=not neox)


def test_rope_axes_no_tokens():
    c, pos = _inputs(1, torch.bfloat16, 0, 4, 2, 64, 64, 16, W.HND, 3)
    _rope(c, pos, pd.rope_pair_axis((12, 10, 10)))


def test_rope_axes_strided_rows():
    """q, k and v as slices of one fused projection's output."""
    c, pos = _inputs(7, torch.bfloat16, 40, 8, 2, 128, 128, 16, W.NHD, 3)
    fused = torch.cat([c.q, c.k, c.v], 1).cuda()
    g = c.to("cuda")
    axis = pd.rope_pair_axis((24, 20, 20), True)
    want = torch.empty_like(g.q)
    _call(g, torch.from_numpy(pos).cuda(), axis, want)
    s = c.to("cuda")
    wide = torch.from_numpy(np.pad(pos, ((0, 0), (3, 9)))).cuda()
    s = dataclasses.replace(s, q=fused[:, :8], k=fused[:, 8:10], v=fused[:, 10:])
    _call(s, wide[:, 3:43], axis, s.q)
    torch.cuda.synchronize()
    assert torch.equal(fused[:, :8], want) and torch.equal(s.k_cache, g.k_cache)
    assert torch.equal(s.v_cache, g.v_cache) and torch.equal(fused[:, 8:10], g.k)


def test_rope_axes_of_one_position_are_the_one_axis_call():
    c, pos = _inputs(3, torch.float16, 90, 8, 2, 128, 128, 16, W.HND, 1, pad=2)
    g, q_out = _rope(c, pos, bytes(64))
    one = dataclasses.replace(c, positions=torch.from_numpy(pos[0].copy())).to("cuda")
    q1 = pd.rope_case(one)
    assert torch.equal(q_out, q1) and torch.equal(g.k_cache, one.k_cache)
    # the same position on every axis, as a broadcast row
    two = c.to("cuda")
    q4 = torch.empty_like(q1)
    _call(two, torch.from_numpy(pos).cuda().expand(4, -1), pd.rope_pair_axis((16, 16, 16, 16)), q4)
    torch.cuda.synchronize()
    assert torch.equal(q4, q1) and torch.equal(two.k_cache, g.k_cache)


def test_rope_axes_report_positions_and_slots():
    c, pos = _inputs(5, torch.float16, 8, 4, 2, 64, 64, 16, W.HND, 3, max_pos=100)
    pos[1, 2], pos[2, 3] = 100, -4
    slots = c.slot_mapping.clone()
    slots[5] = c.k_cache.shape[0] * 16
    bad = dataclasses.replace(c, slot_mapping=slots)
    g = bad.to("cuda")
    q_out = torch.empty_like(g.q)
    axis = pd.rope_pair_axis((12, 10, 10))
    _call(g, torch.from_numpy(pos).cuda(), axis, q_out)
    torch.cuda.synchronize()
    assert pd.paged_decode_device_status(reset=True) == pd.DEV_BAD_POSITION | pd.DEV_BAD_SLOT
    ref = rope_axes(c.q.double().numpy(), pos.clip(0, 99), c.cos_sin.double().numpy(), axis, 64, True)
    _near(q_out, ref, c.q.double().numpy(), 64, True, torch.float16, "q")


def test_rope_axes_captured_and_on_another_stream():
    c, pos = _inputs(9, torch.bfloat16, 33, 8, 2, 128, 128, 16, W.HND, 3, pad=1)
    axis = pd.rope_pair_axis((24, 20, 20))
    g = c.to("cuda")
    p = torch.from_numpy(pos).cuda()
    q_out = torch.zeros_like(g.q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _call(g, p, axis, q_out, stream=st)
    st.synchronize()
    table = c.cos_sin.double().numpy()
    x = c.q.double().numpy()
    _near(q_out, rope_axes(x, pos, table, axis, 128, True), x, 128, True, c.dtype, "q")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(g, p, axis, q_out)
    p.copy_(torch.from_numpy(pos[::-1].copy()))
    graph.replay()
    torch.cuda.synchronize()
    _near(q_out, rope_axes(x, pos[::-1], table, axis, 128, True), x, 128, True, c.dtype, "q")
