"""The calls of paged_quant.h on the CPU: refusals (checked on the host before any
launch), the plan, and the oracle's pins."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import quant_cache as Q
from paged_split_kv_02_gb300 import workloads as W

PASSES = -8  # a call that passes every check reaches the missing device
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("host tensors: for machines without a GPU")


def _cache(pages=3, H=2, D=128, P=32, layout=W.HND, **kw):
    return pd.quant_cache(pages, H, D, P, layout, device="cpu", **kw)


def _attn(**kw):
    k, v, ks, vs = _cache(packed=kw.pop("packed", False))
    a = dict(q=torch.zeros(2, 4, 128).half(), k=k, v=v, ks=ks, vs=vs, bt=torch.zeros(2, 3, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32), qs=None, out=torch.zeros(2, 4, 128).half(), Hq=4, Hkv=2, D=128,
             P=32, M=1, w=0, sinks=0, scale=1.0, layout=W.HND)
    a.update(kw)
    return pd.paged_decode_attn_quant(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["lens"], a["out"], a["Hq"],
                                      a["Hkv"], a["D"], a["P"], a["M"], a["w"], a["sinks"], a["scale"], a["layout"],
                                      query_start=a["qs"], check=False)


def test_symbols_and_constants():
    names = pd.declared_symbols(pd.QUANT_HEADER)
    assert len(names) == 4 and all(hasattr(pd.lib(), n) for n in names)
    text = open(pd.QUANT_HEADER).read()
    assert f"#define PD_SCALE_TOKENS {pd.SCALE_TOKENS}" in text and "#define PD_E4M3 4" in text
    assert pd._DTYPES[E4M3] == 4


def test_attn_refusals(no_gpu):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f16 = lambda *s: torch.zeros(s).half()  # noqa: E731
    k, v, ks, vs = _cache()
    for kw in [dict(), dict(packed=True), dict(w=7, sinks=3), dict(qs=i(3)), dict(qs=i(3), q=f16(5, 4, 128), out=f16(5, 4, 128)),
               dict(ks=torch.zeros(3, 2, 4)[..., ::2])]:
        assert _attn(**kw) == PASSES, kw
    u8 = k.view(torch.uint8)
    for kw, rc in [
            (dict(q=None), -1), (dict(out=None), -1), (dict(ks=None), -1), (dict(Hq=3), -1), (dict(D=96), -3), (dict(M=0), -4),
            (dict(M=9), -4), (dict(P=24), -1), (dict(P=16), -1), (dict(w=-1), -1), (dict(sinks=-1), -1),
            (dict(scale=float("nan")), -1), (dict(layout=2), -1), (dict(layout=W.NHD), -1),
            (dict(q=f16(3, 4, 128)), -1), (dict(q=torch.zeros(2, 4, 128)), -2), (dict(out=torch.zeros(2, 4, 128).bfloat16()), -2),
            (dict(k=u8), -2), (dict(v=v.half()), -2), (dict(k=k[:, :1]), -1), (dict(k=k.view(torch.uint8)[:2].view(E4M3)), -1),
            (dict(ks=ks.double()), -2), (dict(ks=ks[:2]), -1), (dict(ks=ks[..., :1]), -1), (dict(ks=ks.reshape(6, 2)), -1),
            (dict(vs=vs.expand(3, 2, 2).new_zeros(3, 1, 2).expand(3, 2, 2)), -1),
            (dict(k=torch.zeros(3, 2, 32, 136, dtype=torch.uint8)[..., 1:129].view(E4M3)), -5),
            (dict(bt=i(2, 3).long()), -2), (dict(lens=i(2).long()), -2), (dict(bt=i(1, 3)), -1), (dict(bt=i(2, 0)), -1),
            (dict(qs=i(2)), -1), (dict(qs=i(3).long()), -2), (dict(q=f16(2, 4, 132)[..., 4:]), -5)]:
        assert _attn(**kw) == rc, kw
    # no rows: nothing to do
    assert _attn(q=f16(0, 4, 128), out=f16(0, 4, 128), lens=i(0), bt=i(0, 3)) == 0
    with pytest.raises(pd.PagedDecodeError):
        pd.paged_decode_attn_quant(*[i(3)] * 8, 1, 1, 64, 16, 1, 0, 0, 1.0, 0)
    with pytest.raises(OverflowError):
        _attn(w=2 ** 31)


def _read(**kw):
    k, v, ks, vs = _cache()
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    a = dict(k=k, v=v, ks=ks, vs=vs, bt=i(2, 3), lens=i(2), to=i(2, 3), ko=torch.zeros(5, 2, 32, 128).half(),
             vo=torch.zeros(5, 2, 32, 128).half(), H=2, D=128, P=32, layout=W.HND)
    a.update(kw)
    return pd.paged_quant_cache_read(a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["lens"], a["to"], a["ko"], a["vo"],
                                     a["H"], a["D"], a["P"], a["layout"], check=False)


def test_read_refusals(no_gpu):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    o = lambda *s: torch.zeros(s).half()  # noqa: E731
    assert _read() == PASSES and _read(bt=i(0, 3), to=i(0, 3), lens=i(0)) == 0
    for kw, rc in [(dict(to=None), -1), (dict(H=0), -1), (dict(D=100), -3), (dict(P=8), -1), (dict(layout=3), -1), (dict(to=i(2, 2)), -1),
                   (dict(to=i(3, 3)), -1), (dict(to=i(2, 3).long()), -2), (dict(lens=i(3)), -1), (dict(lens=i(2).long()), -2),
                   (dict(ko=o(5, 2, 32, 64)), -1), (dict(ko=o(4, 2, 32, 128)), -1), (dict(ko=o(5, 2, 32, 128).float()), -2),
                   (dict(vo=o(5, 2, 32, 128).bfloat16()), -2), (dict(k=o(3, 2, 32, 128)), -2), (dict(ko=_cache()[0]), -2)]:
        assert _read(**kw) == rc, kw


def _write(**kw):
    k, v, ks, vs = _cache()
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    a = dict(q=torch.zeros(6, 4, 128).bfloat16(), k=torch.zeros(6, 2, 128).bfloat16(), v=torch.zeros(6, 2, 128).bfloat16(),
             pos=i(6), slots=i(6), cs=torch.zeros(10, 64), axis=None, out=torch.zeros(6, 4, 128).bfloat16(), kc=k, vc=v,
             ks=ks, vs=vs, Hq=4, Hkv=2, D=128, rot=64, P=32, layout=W.HND, neox=True)
    a.update(kw)
    return pd.paged_rope_quant_cache_write(a["q"], a["k"], a["v"], a["pos"], a["slots"], a["cs"], a["axis"], a["out"],
                                           a["kc"], a["vc"], a["ks"], a["vs"], a["Hq"], a["Hkv"], a["D"], a["rot"],
                                           a["P"], a["layout"], a["neox"], check=False)


def test_write_refusals(no_gpu):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = lambda *s: torch.zeros(s).bfloat16()  # noqa: E731
    k, v, ks, vs = _cache()
    for kw in [dict(), dict(pos=i(3, 6), axis=[0, 1, 2, 0] * 8), dict(pos=i(6).expand(3, 6)), dict(q=None, out=None, Hq=0),
               dict(rot=0, pos=None, cs=None), dict(neox=False, rot=8, axis=bytes(4)), dict(pos=i(1, 6))]:
        assert _write(**kw) == PASSES, kw
    for kw, rc in [(dict(q=None), -1), (dict(out=None), -1), (dict(k=None), -1), (dict(vs=None), -1), (dict(rot=0), -1),
                   (dict(pos=None), -1), (dict(cs=None), -1), (dict(rot=136, cs=torch.zeros(10, 136)), -1), (dict(rot=24), -1),
                   (dict(rot=-16), -1), (dict(D=96), -3), (dict(P=24), -1), (dict(layout=4), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1),
                   (dict(slots=i(5)), -1), (dict(slots=i(6).long()), -2), (dict(pos=i(5)), -1), (dict(pos=i(6).long()), -2),
                   (dict(pos=i(9, 6)), -1), (dict(pos=i(3, 12)[:, ::2]), -5), (dict(axis=bytes([1] * 32)), -1),
                   (dict(k=b(6, 2, 128).half()), -2), (dict(v=b(6, 2, 128).half()), -2), (dict(q=b(6, 4, 128).half()), -2),
                   (dict(k=b(6, 2, 132)[..., 4:]), -5), (dict(cs=torch.zeros(10, 60)), -1), (dict(cs=torch.zeros(10, 64).double()), -2),
                   (dict(kc=b(3, 2, 32, 128)), -2), (dict(kc=k[:, :, :16]), -1), (dict(ks=ks[:, :1]), -1), (dict(vs=vs.half()), -2)]:
        assert _write(**kw) == rc, kw
    with pytest.raises(ValueError):
        _write(axis=bytes(31))
    none = dict(q=b(0, 4, 128), k=b(0, 2, 128), v=b(0, 2, 128), pos=i(0), slots=i(0), out=b(0, 4, 128))
    assert _write(**none) == 0


def test_quant_cache():
    for layout, shape in ((W.NHD, (3, 32, 2, 64)), (W.HND, (3, 2, 32, 64))):
        for packed in (False, True):
            k, v, ks, vs = pd.quant_cache(3, 2, 64, 32, layout, packed, "cpu")
            assert k.shape == v.shape == shape and k.dtype == E4M3 and ks.shape == vs.shape == (3, 2, 2)
            assert (v.data_ptr() - k.data_ptr() == 64) == packed
    for bad in (dict(page_size=24), dict(page_size=0), dict(layout=7)):
        with pytest.raises(pd.PagedDecodeError):
            pd.quant_cache(**{**dict(num_blocks=1, num_kv_heads=1, head_size=64, page_size=16, layout=0, device="cpu"), **bad})


@pytest.mark.parametrize("S,Hq,Hkv,D,M,width,splits", [
    (1, 32, 8, 128, 1, 2048, 256), (64, 16, 2, 256, 2, 1024, 64), (5, 8, 1, 512, 8, 313, 200), (1, 16, 4, 64, 1, 19, 64),
    (3000, 8, 8, 64, 1, 100, 8), (2, 512, 1, 512, 8, 4, 8), (4, 32, 1, 64, 8, 500, 0), (1, 8, 8, 128, 1, 2 ** 27 - 1, 64)])
@pytest.mark.parametrize("window", [0, 300])
def test_plan(S, Hq, Hkv, D, M, width, splits, window):
    sd = pd.PdScratch()
    sd.data = 1 << 30
    sd.bytes = pd.paged_decode_scratch_bytes(S, Hq, Hkv, D, M, splits)
    sd.counter_slots = S * Hkv * pd.COUNTERS_PER_PAIR
    for scratch in (sd, None):
        p = pd.paged_decode_plan_quant(S, Hq, Hkv, D, 16, M, window, 4, width, 152, scratch_desc=scratch)
        assert p["path"] == 7 and p["rows"] == Hq // Hkv * M
        assert p["rows_per_cta"] * p["row_groups"] >= p["rows"] > p["rows_per_cta"] * (p["row_groups"] - 1)
        assert p["rows_per_cta"] <= 8 * p["n_tiles"] and p["smem_bytes"] <= 232448
        assert 4 <= p["key_groups"] <= 12 and p["block_threads"] == 32 * p["key_groups"]
        units = S * Hkv * p["row_groups"]
        if p["merge"]:
            # two parts of a CTA, behind the counters
            assert p["grid_x"] <= 152 and units <= sd.counter_slots
            assert p["scratch_needed"] + 4 * sd.counter_slots <= sd.bytes + 256
        else:
            assert p["scratch_needed"] == 0 and p["grid_x"] * p["grid_y"] >= units
    assert pd.paged_decode_plan_quant(1, 32, 8, 128, 16, 1, 0, 0, 2048, 152)["merge"] == 0


def test_plan_rows_of_a_cta():
    def tiles(S, Hq, Hkv, D, M, keys, scratch=True):
        sd = pd.PdScratch()
        sd.data, sd.counter_slots = 1 << 30, S * Hkv * pd.COUNTERS_PER_PAIR
        sd.bytes = pd.paged_decode_scratch_bytes(S, Hq, Hkv, D, M, 256)
        return pd.paged_decode_plan_quant(S, Hq, Hkv, D, 16, M, 0, 0, keys // 16, 152,
                                          scratch_desc=sd if scratch else None)["n_tiles"]

    # as many rows as there are, up to what fits, for many units or without scratch; fewer for few
    assert tiles(64, 32, 8, 128, 8, 4096) == 4 and tiles(64, 32, 8, 128, 1, 4096) == 1
    assert tiles(1, 32, 8, 128, 8, 320, scratch=False) == 4
    assert tiles(1, 32, 8, 128, 8, 320) == 1 and tiles(1, 32, 8, 128, 8, 32768) == 2
    assert tiles(1, 32, 8, 128, 4, 32768) == 2 and tiles(1, 32, 8, 128, 4, 4096) == 1
    assert tiles(1, 16, 2, 256, 2, 32768) == 1 and tiles(10, 16, 2, 256, 2, 8000) == 2
    # (rows past the counters of the scratch)
    assert tiles(1, 512, 1, 128, 8, 4096) == 4


def test_plan_refusals():
    ok = [2, 8, 2, 128, 16, 1, 0, 0, 10, 152]
    for at, value, rc in [(0, 0, -1), (1, 7, -1), (2, 0, -1), (3, 80, -3), (4, 8, -1), (5, 9, -4), (6, -1, -1), (7, -1, -1),
                          (8, 0, -1), (9, 0, -1), (8, 2 ** 28, -1)]:
        args = list(ok)
        args[at] = value
        with pytest.raises(pd.PagedDecodeError) as e:
            pd.paged_decode_plan_quant(*args)
        assert e.value.code == rc, (at, value)


def test_oracle_rounding():
    # torch's own conversion, on every code, the midpoints between and around them
    mags = Q.MAGNITUDES
    assert torch.equal(torch.arange(127, dtype=torch.uint8).view(E4M3).double(), torch.from_numpy(mags))
    mid = (mags[1:] + mags[:-1]) / 2
    x = np.concatenate([mags, mid, np.nextafter(mid, 0), np.nextafter(mid, 999), [0.0, 2.0 ** -30]])
    x = np.concatenate([x, -x])
    near32 = x[x == x.astype(np.float32)]
    want = torch.from_numpy(near32.astype(np.float32)).to(E4M3).view(torch.uint8).numpy()
    assert np.array_equal(Q.encode(near32), want)
    up, down = Q.values(Q.encode(np.nextafter(mid, 999))), Q.values(Q.encode(np.nextafter(mid, 0)))
    assert np.array_equal(up, mags[1:]) and np.array_equal(down, mags[:-1])
    assert Q.encode(np.array([500.0, np.inf, -np.inf, np.nan])).tolist() == [0x7E, 0x7E, 0xFE, 0x7F]


def test_oracle_scales_and_store():
    assert Q.least_scale(0.0) == 2.0 ** -64 and Q.least_scale(448.0) == 1.0 and Q.least_scale(448.5) == 2.0
    assert Q.least_scale(449.0 / 256) == 2.0 ** -7 and Q.least_scale(448.0 / 256) == 2.0 ** -8
    codes, scale = np.zeros((1, 32, 1, 2), dtype=np.uint8), np.zeros((1, 2, 1))
    Q.store(np.array([[[448.0, 1.0]]]), [16], codes, scale)
    assert scale.tolist() == [[[0.0], [1.0]]] and Q.values(codes[0, 16, 0]).tolist() == [448.0, 1.0]
    Q.store(np.array([[[0.5, 896.0]]]), [17], codes, scale)       # grows: the first token's codes follow
    assert scale[0, 1, 0] == 2.0 and Q.dequantised(codes, scale)[0, 16:18, 0].tolist() == [[448.0, 1.0], [0.5, 896.0]]
    Q.store(np.array([[[3.0, 3.0]]]), [18], codes, scale)         # does not shrink
    assert scale[0, 1, 0] == 2.0
    Q.store(np.array([[[3.0, 3.0]]]), [16], codes, scale)         # starts anew
    assert scale[0, 1, 0] == 2.0 ** -7 and Q.dequantised(codes, scale)[0, 16, 0].tolist() == [3.0, 3.0]
