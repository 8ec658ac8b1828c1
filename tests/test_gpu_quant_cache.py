"""paged_rope_quant_cache_write and paged_quant_cache_read against their fp64
oracle, and a serving step over the 8-bit cache.

Without a rotation every code and scale is the oracle's.  A rotated key is
off by the fp32 arithmetic, 2^-22 of |x1| + |x2|, before it is quantised, which
adds half a step: 2^-4 of the value, or 2^-10 of the scale below 2^-6 of it."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from gpu_helpers import sample_rows
from oracle import quant_cache as Q
from oracle import rope_cache as R
from oracle.rope_axes import rope_axes
from paged_split_kv_02_gb300 import workloads as W
from quant_cases import E4M3, HALF_STEP, QuantCase, near, to_pools

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Cache:
    """A cache of seeded codes and scales, on the host and the GPU."""

    def __init__(self, seed, pages, P, H, D, layout, packed=False):
        g = np.random.default_rng(seed)
        self.layout, self.P = layout, P
        self.codes = [g.integers(0, 256, (pages, P, H, D)).astype(np.uint8) for _ in range(2)]
        for c in self.codes:
            c[(c & 0x7F) == 0x7F] = 0x3C  # (a NaN stays one: tested apart)
        self.scale = [np.exp2(g.integers(-14, 2, (pages, P // 16, H))).astype(np.float32) for _ in range(2)]
        self.k, self.v = to_pools(*self.codes, layout, packed)
        self.ks, self.vs = (torch.from_numpy(s).cuda() for s in self.scale)

    def got(self):
        return ([Q.by_token(c, self.layout) for c in (self.k, self.v)],
                [s.cpu().numpy() for s in (self.ks, self.vs)])


def _slots(g, runs, pages, P):
    """Slots of tokens, run after run of (first token of its sequence, tokens):
    each sequence in pages of its own, any order."""
    ids = iter(g.permutation(pages))
    out = []
    for first, n in runs:
        held = {}
        for p in range(first, first + n):
            if p // P not in held:
                held[p // P] = int(next(ids))
            out.append(held[p // P] * P + p % P)
    return np.array(out)


def _check_write(cache, slots, k, v, k_slack, codes0, scale0, exact_k):
    """The caches after a write of k and v [T, H, D] (fp64; k to k_slack)."""
    (gk, gv), (gks, gvs) = cache.got()
    want, sc = codes0[1].copy(), scale0[1].copy()
    Q.store(v, slots, want, sc)
    assert np.array_equal(gvs, sc) and np.array_equal(gv, want), "v"
    want, sc = codes0[0].copy(), scale0[0].copy()
    Q.store(k, slots, want, sc)
    if exact_k:
        assert np.array_equal(gks, sc) and np.array_equal(gk, want), "k"
        return
    # a scale may be the next power of two only where the largest value is within the slack
    P = cache.P
    lower, upper = scale0[0].copy(), scale0[0].copy()
    Q.store(np.sign(k) * np.maximum(np.abs(k) - k_slack, 0), slots, codes0[0].copy(), lower)
    Q.store(np.sign(k) * (np.abs(k) + k_slack), slots, codes0[0].copy(), upper)
    assert ((gks >= lower) & (gks <= upper)).all(), "k scales"
    named = np.zeros(gk.shape[0] * P, dtype=bool)
    on = np.nonzero(slots >= 0)[0]
    named[slots[on]] = True
    page, tok = slots[on] // P, slots[on] % P
    s = gks[page, tok // 16].astype(np.float64)[..., None]
    off = np.abs(Q.values(gk[page, tok]) * s - k[on])
    a = np.abs(k[on]) + k_slack[on]
    assert (off <= np.maximum(2.0 ** -4 * a, 2.0 ** -10 * s) + k_slack[on]).all(), "k codes"
    same = np.repeat(gks == sc, 16, axis=1) & ~named.reshape(gk.shape[:2])[..., None]
    assert np.array_equal(gk[same], want[same]), "the other tokens of k"


def _write(seed, dtype, D, runs, P=16, heads=(8, 2), rot=None, neox=True, axes=1, layout=W.HND, packed=False, pad=0,
           q=True, scale=1.0, inplace=False, edit=None):
    g = np.random.default_rng(seed)
    rot = D if rot is None else rot
    Hq, H = heads
    pages = sum((a + n - 1) // P - a // P + 1 for a, n in runs) + 2
    slots = np.concatenate([_slots(g, runs, pages, P), np.full(pad, -1, dtype=int)])
    T = len(slots)
    cache = Cache(seed, pages, P, H, D, layout, packed)
    codes0, scale0 = [c.copy() for c in cache.codes], [s.copy() for s in cache.scale]
    rnd = lambda h: torch.from_numpy(g.standard_normal((T, h, D)) * scale).to(dtype)  # noqa: E731
    xq, xk, xv = rnd(Hq), rnd(H), rnd(H)
    # heads of other sizes, and values that need every scale
    xk = (xk * torch.exp2(torch.from_numpy(g.integers(-6, 6, (1, H, 1))).float())).to(dtype)
    if edit:
        edit(xk, xv)
    table = W.rope_cos_sin_table(3000, max(rot, 8))
    pos = g.integers(0, 3000, (axes, T)).astype(np.int32)
    sections = [rot // 2 - (axes - 1) * (rot // 2 // axes)] + [rot // 2 // axes] * (axes - 1)
    axis = pd.rope_pair_axis(sections) if rot else None
    dq = xq.cuda()
    out = dq if inplace else torch.empty_like(dq)
    p = _i32(pos if axes > 1 else pos[0])
    pd.paged_rope_quant_cache_write(dq if q else None, xk.cuda(), xv.cuda(), p if rot else None, _i32(slots),
                                    table.cuda() if rot else None, axis if axes > 1 else None, out if q else None,
                                    cache.k, cache.v, cache.ks, cache.vs, Hq, H, D, rot, P, layout, neox)
    torch.cuda.synchronize()
    fq, fk, fv = (x.double().numpy() for x in (xq, xk, xv))
    if rot:
        turn = lambda x: rope_axes(x, pos, table.double().numpy(), axis, rot, neox)  # noqa: E731
        a, b = R.pair_index(rot, neox)

        def pairs(x):
            m = np.zeros_like(x)
            m[..., a] = m[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
            return m
        rq, rk, sq, sk = turn(fq), turn(fk), 2.0 ** -22 * pairs(fq), 2.0 ** -22 * pairs(fk)
    else:
        rq, rk, sq, sk = fq, fk, np.zeros_like(fq), np.zeros_like(fk)
    if q:
        off = np.abs(out.double().cpu().numpy() - rq)
        assert (off <= HALF_STEP[dtype] * (np.abs(rq) + sq) + sq + 2.0 ** -25).all(), "q"
    _check_write(cache, slots, rk, fv, sk, codes0, scale0, rot == 0)
    return cache


RUNS = [(0, 40), (5, 1), (15, 1), (16, 1), (31, 3), (7, 9), (3, 60), (0, 1), (0, 16), (12, 4)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("D,rot,axes", [(64, 64, 1), (64, 32, 3), (128, 128, 1), (128, 96, 4), (128, 0, 1),
                                        (256, 64, 3), (256, 256, 1), (512, 512, 2), (512, 16, 1), (512, 0, 1)])
def test_write(dtype, neox, D, rot, axes):
    _write(D + rot, dtype, D, RUNS, rot=rot, neox=neox, axes=axes, pad=3)


@pytest.mark.parametrize("layout", [W.NHD, W.HND])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("P,heads", [(16, (6, 6)), (48, (20, 4)), (1056, (15, 5)), (128, (4, 1))])
def test_write_layouts(layout, packed, P, heads):
    _write(P, torch.bfloat16, 128, RUNS, P=P, heads=heads, rot=64, layout=layout, packed=packed, inplace=P == 48)


@pytest.mark.parametrize("D,rot", [(64, 0), (128, 128), (256, 0), (512, 64)])
@pytest.mark.parametrize("T", [1, 700, 5000, 12000])
def test_write_sizes(D, rot, T):
    T = min(T, 3_000_000 // D)  # (the oracle takes its time)
    # (batches of one token each, and prompts; windows of 1 to 16 tokens a CTA)
    runs = [(11, T)] if T != 700 else [(i % 23, 1) for i in range(T)]
    _write(T, torch.float16, D, runs, rot=rot, heads=(2, 1), q=D != 256)


@pytest.mark.parametrize("D", [128, 512])
def test_write_many_short_runs(D):
    g = np.random.default_rng(9)
    _write(1, torch.bfloat16, D, [(int(g.integers(0, 40)), int(g.integers(1, 5))) for _ in range(900)], rot=0,
           heads=(1, 1))


@pytest.mark.parametrize("D,H,rot,axes,neox", [(64, 1, 64, 1, True), (64, 2, 0, 1, True), (128, 1, 96, 4, False),
                                               (256, 1, 16, 1, True), (512, 1, 8, 2, False)])
def test_write_few_heads_of_many_tokens(D, H, rot, axes, neox):
    # windows of up to 64 tokens a CTA: runs of every length in them, at every place
    g = np.random.default_rng(D)
    T, runs = 55_000 if D == 64 else 27_000 if D == 128 else 14_000, []
    while sum(n for _, n in runs) < T:
        runs.append((int(g.integers(0, 40)), int(g.choice([1, 2, 15, 16, 17, 63, 64, 65, 300, 1000]))))
    _write(D + H, torch.bfloat16, D, runs, rot=rot, neox=neox, axes=axes, heads=(1 if H == 1 else 2, H), q=D == 64)


def test_write_extremes():
    inf, nan = float("inf"), float("nan")

    def edit(k, v):
        v[:40] = 0            # blocks of zeros: the least scale
        v[40, 0, :8] = torch.tensor([inf, -inf, nan, 1.0, -2.0, 0.0, -0.0, 3e38])
        v[41, 1] = nan        # no finite value at all
        v[42] = 1e-38
        k[0, 0, 0], k[1, 1, 1] = inf, nan
        k[41, 0] = 448.0      # the border of a scale, and just past it
        k[41, 1] = 450.0

    _write(4, torch.bfloat16, 128, [(0, 40), (0, 1), (3, 1), (0, 1), (9, 16)], rot=0, edit=edit)


def test_write_to_pools_that_were_never_written():
    # NaN scales and codes: a first write starts the block, an append counts them as nothing
    c = Cache(1, 4, 32, 2, 128, W.HND)
    for t in (c.ks, c.vs):
        t.fill_(float("nan"))
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x7F)
    slots = np.array([0, 1, 2, 37, 64 + 16])
    x = torch.randn((2, 5, 2, 128), dtype=torch.bfloat16)
    pd.paged_rope_quant_cache_write(None, x[0].cuda(), x[1].cuda(), None, _i32(slots), None, None, None, c.k, c.v,
                                    c.ks, c.vs, 0, 2, 128, 0, 32, W.HND)
    torch.cuda.synchronize()
    for i, (codes, s) in enumerate(zip(*c.got())):
        want, sc = np.full_like(codes, 0x7F), np.full_like(s, np.nan)
        Q.store(x[i].double().numpy(), slots, want, sc)
        assert np.array_equal(codes, want) and np.array_equal(s, sc, equal_nan=True)


def test_write_twice_changes_nothing_more():
    c = _write(6, torch.bfloat16, 128, RUNS, rot=0)
    codes, scale = c.got()
    slots = _slots(np.random.default_rng(6), RUNS, c.k.shape[0], 16)
    back = [Q.dequantised(a, s).reshape(-1, 2, 128)[slots] for a, s in zip(codes, scale)]
    k, v = (torch.from_numpy(b).to(torch.bfloat16).cuda() for b in back)
    pd.paged_rope_quant_cache_write(None, k, v, None, _i32(slots), None, None, None, c.k, c.v, c.ks, c.vs, 0, 2, 128,
                                    0, 16, W.HND)
    torch.cuda.synchronize()
    again, scale2 = c.got()
    # (codes of values that the cache holds are those it holds; a restarted block's
    # scale may be smaller than one that its old content asked for)
    for a, b, s, s2 in zip(codes, again, scale, scale2):
        assert (s2 <= s).all()
        assert np.array_equal(Q.dequantised(a, s), Q.dequantised(b, s2)) or (s2 < s).any()


def test_write_grows_a_scale_token_by_token():
    c = Cache(2, 2, 16, 1, 64, W.NHD)
    codes0, scale0 = [x.copy() for x in c.codes], [x.copy() for x in c.scale]
    g = np.random.default_rng(2)
    for i in range(16):
        x = torch.from_numpy(g.standard_normal((2, 1, 1, 64)) * 1.7 ** i).half()
        pd.paged_rope_quant_cache_write(None, x[0].cuda(), x[1].cuda(), None, _i32([16 + i]), None, None, None, c.k,
                                        c.v, c.ks, c.vs, 0, 1, 64, 0, 16, W.NHD)
        for j in range(2):
            Q.store(x[j].double().numpy(), [16 + i], codes0[j], scale0[j])
    torch.cuda.synchronize()
    codes, scale = c.got()
    assert all(np.array_equal(a, b) for a, b in zip(codes + scale, codes0 + scale0))


def test_bad_slots_and_positions():
    c = Cache(3, 3, 16, 2, 64, W.HND)
    codes0, scale0 = [x.copy() for x in c.codes], [x.copy() for x in c.scale]
    x = torch.randn((2, 6, 2, 64)).half()

    def write(slots, pos=None):
        pd.paged_rope_quant_cache_write(None, x[0].cuda(), x[1].cuda(), None if pos is None else _i32(pos),
                                        _i32(slots), None if pos is None else W.rope_cos_sin_table(8, 16).cuda(), None,
                                        None, c.k, c.v, c.ks, c.vs, 0, 2, 64, 0 if pos is None else 16, 16, W.HND)
        return pd.paged_decode_device_status(reset=True)

    # the same slot twice, and one that goes back: they and the rest of the run are left out
    for slots, ok in (([3, 4, 4, 5, 17, 18], [0, 1, 4, 5]), ([40, 39, 41, 3, 5, 6], [0, 3, 4, 5]),
                      ([1, 2, 48, 1000, 20, 21], [0, 1, 4, 5])):
        assert write(slots) == pd.DEV_BAD_SLOT
        kept = np.array([s if i in ok else -1 for i, s in enumerate(slots)])
        for j in range(2):
            Q.store(x[j].double().numpy(), kept, codes0[j], scale0[j])
        codes, scale = c.got()
        assert all(np.array_equal(a, b) for a, b in zip(codes + scale, codes0 + scale0)), slots
    assert write([-1] * 6) == 0 and write(list(range(6)), [0, 1, 2, 3, 4, 7]) == 0
    assert write(list(range(6)), [0, 1, 2, 3, 4, 8]) == pd.DEV_BAD_POSITION


def _far(codes, layout, pages):
    """The same pool, small, and as the last pages of one of 5 GiB."""
    used = codes.shape[0]
    big = torch.empty((pages,) + tuple(codes.shape[1:]), dtype=torch.uint8, device="cuda")
    big[pages - used:] = codes.view(torch.uint8)
    return big.view(E4M3)


def test_offsets_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    D, H, P, used = 128, 2, 16, 6
    pages = (5 << 30) // (P * H * D)
    c = Cache(8, used, P, H, D, W.HND)
    codes0, scale0 = [x.copy() for x in c.codes], [x.copy() for x in c.scale]
    k, v = (_far(t, W.HND, pages) for t in (c.k, c.v))
    ks, vs = (torch.empty((pages, 1, 2 * 600), device="cuda")[..., ::600] for _ in range(2))
    for big, s in ((ks, c.ks), (vs, c.vs)):
        big[pages - used:] = s
    slots = np.array([0, 1, 2, 30, 31, 80, 81, 82])
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((2, 8, H, D))).bfloat16()
    pd.paged_rope_quant_cache_write(None, x[0].cuda(), x[1].cuda(), None, _i32(slots + (pages - used) * P), None, None,
                                    None, k, v, ks, vs, 0, H, D, 0, P, W.HND)
    k_out, v_out = (torch.zeros((pages, H, P, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = np.arange(pages - used, pages)[None]
    pd.paged_quant_cache_read(k, v, ks, vs, _i32(table), _i32([used * P]), _i32(table), k_out, v_out, H, D, P, W.HND)
    torch.cuda.synchronize()
    for j, (codes, s, out) in enumerate(((k, ks, k_out), (v, vs, v_out))):
        Q.store(x[j].double().numpy(), slots, codes0[j], scale0[j])
        assert np.array_equal(Q.by_token(codes[pages - used:], W.HND), codes0[j])
        assert np.array_equal(s[pages - used:].cpu().numpy(), scale0[j])
        want = torch.from_numpy(Q.dequantised(codes0[j], scale0[j])).bfloat16().permute(0, 2, 1, 3)
        assert torch.equal(out[pages - used:].cpu(), want)


def test_write_from_one_projection_and_strided_scales():
    # q, k, v as views of one tensor of rows, rotated in place; pools and scales as views of wider ones
    g = np.random.default_rng(12)
    T, Hq, H, D, P = 37, 8, 2, 128, 32
    qkv = torch.from_numpy(g.standard_normal((T, Hq + 2 * H, D))).half()
    dev = qkv.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + H], dev[:, Hq + H:]
    c = Cache(12, 4, P, H, D, W.NHD)
    codes0, scale0 = [x.copy() for x in c.codes], [x.copy() for x in c.scale]
    wide = [torch.full((8, P, H + 3, D + 16), 0x41, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pools = [w[::2, :, 1:1 + H, 16:] for w in wide]
    for a, b in zip(pools, (c.k, c.v)):
        a.copy_(b.view(torch.uint8))
    ks, vs = (torch.stack([s, s.new_full(s.shape, 5.0)], 1)[:, 0] for s in (c.ks, c.vs))
    slots = np.arange(5, 5 + T)
    pos = g.integers(0, 90, T).astype(np.int32)
    table = W.rope_cos_sin_table(90, D)
    pd.paged_rope_quant_cache_write(q, k, v, _i32(pos), _i32(slots), table.cuda(), None, q, *(a.view(E4M3) for a in pools),
                                    ks, vs, Hq, H, D, D, P, W.NHD)
    torch.cuda.synchronize()
    x = qkv.double().numpy()
    axis = pd.rope_pair_axis([D // 2])
    turned = rope_axes(x, pos[None], table.double().numpy(), axis, D, True)
    slack = 2.0 ** -22 * (np.abs(x) + np.abs(np.roll(x, D // 2, -1)))
    got = q.double().cpu().numpy()
    off = np.abs(got - turned[:, :Hq])
    assert (off <= 2.0 ** -11 * (np.abs(turned) + slack)[:, :Hq] + slack[:, :Hq] + 2.0 ** -25).all()
    assert torch.equal(dev[:, Hq:].cpu(), qkv[:, Hq:])
    c.k, c.v, c.ks, c.vs = (*(a.view(E4M3) for a in pools), ks, vs)
    _check_write(c, slots, turned[:, Hq:Hq + H], x[:, Hq + H:], slack[:, Hq:Hq + H], codes0, scale0, False)
    for w, a in zip(wide, pools):
        a.fill_(0x41)
        assert bool((w == 0x41).all())


# ---------------------------------------------------------------------------
# The read.

def _read(seed, dtype, D, lens, P=16, H=2, layout=W.HND, packed=False, drop=()):
    g = np.random.default_rng(seed)
    need = [-(-L // P) for L in lens]
    width, pages = max(need + [1]) + 1, sum(need) + 3
    c = Cache(seed, pages, P, H, D, layout, packed)
    src, dst = g.permutation(pages), g.permutation(pages + 5)
    table, to = (np.full((len(lens), width), -1) for _ in range(2))
    n = 0
    for s, m in enumerate(need):
        table[s, :m], to[s, :m] = src[n:n + m], dst[n:n + m]
        n += m
    for i, (s, j) in enumerate(drop):
        (table if i % 2 else to)[s, j] = -1
    shape = (pages + 5, P, H, D) if layout == W.NHD else (pages + 5, H, P, D)
    pool = torch.full(shape[:3] + (2 * D,), 9.0, dtype=dtype, device="cuda")
    k, v = (pool[..., :D], pool[..., D:]) if packed else (pool[..., :D].clone(), pool[..., D:].clone())
    pd.paged_quant_cache_read(c.k, c.v, c.ks, c.vs, _i32(table), _i32(lens), _i32(to), k, v, H, D, P, layout)
    torch.cuda.synchronize()
    for x, codes, s in zip((k, v), c.codes, c.scale):
        want = np.full((pages + 5, P, H, D), 9.0)
        Q.read(Q.dequantised(codes, s), table, lens, to, want)
        want = torch.from_numpy(want).to(dtype)
        got = (x if layout == W.NHD else x.permute(0, 2, 1, 3)).cpu()
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("layout,packed", [(W.NHD, True), (W.HND, False), (W.HND, True)])
def test_read(dtype, D, layout, packed):
    _read(D, dtype, D, [40, 0, 1, 15, 16, 17, 300], layout=layout, packed=packed, drop=[(0, 1), (6, 3), (6, 4)])


@pytest.mark.parametrize("P,H", [(16, 1), (48, 3), (1056, 5), (64, 8)])
def test_read_pages(P, H):
    _read(P, torch.bfloat16, 128, [5000, 3, 1100], P=P, H=H, layout=W.NHD)


def test_read_many_requests():
    _read(1, torch.float16, 64, np.random.default_rng(1).integers(0, 90, 3000).tolist(), H=1)


def test_read_shares_pages_and_is_captured():
    # two requests with the same first pages, staged apart; a graph of it, on another stream
    c = Cache(5, 9, 48, 2, 128, W.HND)
    table = np.array([[7, 3, 1, -1], [7, 3, 8, 0]])
    to = np.array([[0, 4, 2, 9], [1, 5, 3, 6]])
    lens = [100, 150]
    k, v = (torch.full((10, 2, 48, 128), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    args = [_i32(a) for a in (table, lens, to)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pd.paged_quant_cache_read(c.k, c.v, c.ks, c.vs, *args, k, v, 2, 128, 48, W.HND)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, codes, s in zip((k, v), c.codes, c.scale):
        want = np.full((10, 48, 2, 128), 9.0)
        Q.read(Q.dequantised(codes, s), table, lens, to, want)
        assert torch.equal(x.permute(0, 2, 1, 3).cpu(), torch.from_numpy(want).half())


def test_read_reports():
    c = Cache(1, 3, 16, 1, 64, W.HND)
    k, v = (torch.zeros((2, 1, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    for table, to, lens, bit in (([[0, 1]], [[0, 2]], [32], pd.DEV_BAD_PAGE), ([[0, 9]], [[0, 1]], [32], pd.DEV_BAD_PAGE),
                                 ([[0, 1]], [[0, 1]], [33], pd.DEV_BAD_SEQLEN), ([[0, 1]], [[0, 1]], [-3], 0)):
        pd.paged_quant_cache_read(c.k, c.v, c.ks, c.vs, _i32(table), _i32(lens), _i32(to), k, v, 1, 64, 16, W.HND)
        assert pd.paged_decode_device_status(reset=True) == bit


# ---------------------------------------------------------------------------
# A run of them together.

@pytest.mark.parametrize("P,D,layout", [(16, 128, W.HND), (48, 64, W.NHD), (32, 256, W.HND)])
def test_serving_steps_over_the_cache(P, D, layout):
    """Prompts written and read back for prefill, then captured decode steps:
    tables, rotary write, attention; the oracles take the caches as written."""
    S, Hq, H, width, pages, dt = 5, 8, 2, 60, 240, torch.bfloat16
    gen = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dt).cuda()  # noqa: E731
    cos_sin = W.rope_cos_sin_table(900, D).cuda()
    kc, vc, ks, vs = pd.quant_cache(pages, H, D, P, layout, packed=layout == W.NHD)
    free, cur, nxt = _i32(np.random.default_rng(1).permutation(pages)), _i32([0]), _i32([0])
    table, ctx, lens, start = _i32(np.full((S, width), -1)), _i32(np.zeros(S)), _i32(np.zeros(S)), _i32(np.zeros(S + 1))

    def write(qd, q, k, v, q_rot, pos, slots):
        pd.paged_batch_tables(ctx, qd, table, start, lens, pos, slots, P, pages, free_pages=free, cursor=cur,
                              next_cursor=nxt)
        pd.paged_rope_quant_cache_write(q, k, v, pos, slots, cos_sin, None, q_rot, kc, vc, ks, vs, Hq, H, D, D, P,
                                        layout)

    def expect(q_rot, out, M):
        codes = [Q.by_token(c, layout) for c in (kc, vc)]
        back = [torch.from_numpy(Q.dequantised(c, s.cpu().numpy())) for c, s in zip(codes, (ks, vs))]
        back = [b if layout == W.NHD else b.permute(0, 2, 1, 3) for b in back]
        case = W.DecodeCase("step", dt, D, Hq, H, P, M, 0, D ** -0.5, layout, q_rot.cpu(), *back, table.cpu(),
                            lens.cpu(), seq_lens_host=lens.tolist(), query_start=start.cpu(),
                            query_start_host=start.tolist())
        rows = [(t, h) for t, h in sample_rows(case, 60) if t < int(start[-1])]
        assert pd.paged_decode_device_status(reset=True) == 0
        return QuantCase(case, case, kc, vc, ks, vs), rows

    q_lens = [300, 17, 1, 120, 64]
    T = sum(q_lens)
    qd, pos, slots = _i32(q_lens), torch.zeros((1, T), dtype=torch.int32, device="cuda"), _i32(np.zeros(T))
    q, k, v = rnd(T, Hq, D), rnd(T, H, D), rnd(T, H, D)
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    write(qd, q, k, v, q_rot, pos, slots)
    # prefill over staged pages
    shape = (pages, P, H, D) if layout == W.NHD else (pages, H, P, D)
    k16, v16 = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
    to = torch.where(table >= 0, pages - 1 - table, -1)
    pd.paged_quant_cache_read(kc, vc, ks, vs, table, lens, to, k16, v16, H, D, P, layout)
    items, info = pd.paged_prefill_plan([0] + list(np.cumsum(q_lens)), q_lens, Hq, H, D, 0)
    pd.paged_prefill_attn(q_rot, k16, v16, to, lens, start, items.cuda(), info, out, Hq, H, D, P, 0, D ** -0.5, layout,
                          pd.prefill_scratch(H, D))
    torch.cuda.synchronize()
    qc, rows = expect(q_rot, out, max(q_lens))
    from gpu_helpers import check
    from oracle import sinks as O
    check(qc.case, out, rows=rows, ref=O.attention(qc.case, 0, rows))

    T, M = 10, 2
    qd, pos, slots = _i32([1, 1, 2, 0, 1]), torch.zeros((1, T), dtype=torch.int32, device="cuda"), _i32(np.zeros(T))
    q, k, v = rnd(T, Hq, D), rnd(T, H, D), rnd(T, H, D)
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    sc = pd.Scratch(S, Hq, H, D, M, max_splits=32)

    def step():
        ctx.copy_(lens)
        cur.copy_(nxt)
        write(qd, q, k, v, q_rot, pos, slots)
        pd.paged_decode_attn_quant(q_rot, kc, vc, ks, vs, table, lens, out, Hq, H, D, P, M, 0, 0, D ** -0.5, layout, sc,
                                   query_start=start)

    step()
    torch.cuda.synchronize()
    qc, rows = expect(q_rot, out, M)
    near(qc, out, rows=rows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(12):
        for x in (q, k, v):
            x.copy_(rnd(*x.shape) * 1.3 ** n)
        q.div_(1.3 ** (2 * n))
        qd.copy_(torch.tensor([n % 3, 1, 2, (n + 1) % 2, 1], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        qc, rows = expect(q_rot, out, M)
        near(qc, out, rows=rows)
        assert float(out[int(start[-1]):].abs().sum()) == 0.0
