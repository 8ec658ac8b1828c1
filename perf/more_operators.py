"""Measured cases of the 8-bit paged cache: the write that quantises, the read
back to 16 bits, and the attention of decode steps over it.

``run`` makes one pass through an operator: where ``own`` is true the calls of
``paged_split_kv_02_gb300``, else the same computation in elementary torch
operations, in 32 bits, rounded once at the end.

The cache holds e4m3 codes and, for every 16 tokens of a page and kv head, one
fp32 scale: a value is code x scale.  A written scale is the smallest power of
two (2^-64 at least) under which no value of the block passes 448.

Operators
* ``write``: rotary embedding of q and k and the store of k and v as codes.  A
  call that writes the first token of a block starts it anew; else the block's
  scale grows where the new tokens need it, and its other codes are rounded to
  the new scale;
* ``read``: pages of requests as 16-bit pages of a staging pool;
* ``decode``: attention of 1..8 query tokens a request, over every key or over a
  window beside which the first keys stay visible.
"""

import math
import random

import numpy as np
import torch

own = False

NHD, HND = 0, 1
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
BLOCK = 16  # tokens of a scale
LEAST = -64  # the least scale's exponent


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------
# The cases.

def listed():
    write = dict(op="write", layout=HND, packed=False, pad=0, axes=1, neox=True, max_pos=32768, mix=1)
    read = dict(op="read", layout=HND, packed=False, window=0, mix=1)
    decode = dict(op="decode", layout=HND, packed=False, varlen=False, pad=0, window=0, sinks=0, mix=1)
    return [
        # the new tokens of one user's speculative step: the smallest write,
        # where latency is all
        dict(write, name="write_one_spec", dtype="fp16", D=256, Hq=8, Hkv=1, P=32, rot=256, S=1, q_lo=4, q_hi=4),
        # a serving batch, one token each, most of them appended to a block
        dict(write, name="write_decode64", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, rot=128, S=64, q_lo=1, q_hi=1,
             pad=3),
        # long prompts in the usual shapes: the largest write
        dict(write, name="write_prompt16384", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, rot=128, S=4, q_lo=4096,
             q_hi=4096),
        # a mixed batch with images: ragged lengths, three position axes, a
        # partly rotated head in pairs of neighbours, a token-major pool with K
        # and V side by side
        dict(write, name="write_ragged_axes", dtype="fp16", D=64, Hq=16, Hkv=4, P=48, rot=32, S=37, q_lo=1, q_hi=700,
             pad=9, axes=3, neox=False, layout=NHD, packed=True),
        # one request's context, staged for its next prompt chunk
        dict(read, name="read_one4096", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, S=1, lo=4090, hi=4090),
        # the contexts of a prefill batch: the largest read
        dict(read, name="read_batch16", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, S=16, lo=2000, hi=16384),
        # the windows of a batch alone (older pages were given back), on the
        # pages of hybrid models
        dict(read, name="read_window_d256", dtype="fp16", D=256, Hq=16, Hkv=2, P=1056, S=24, lo=1, hi=16384,
             window=2000, layout=NHD, packed=True),
        # a short chat on narrow heads: the smallest decode step
        dict(decode, name="decode_one300_d64", dtype="fp16", D=64, Hq=16, Hkv=4, P=48, S=1, M=1, lo=300, hi=300),
        # one user's long document
        dict(decode, name="decode_one32768", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, S=1, M=1, lo=32768, hi=32768),
        # speculative decoding over a captured batch: 1..4 draft tokens, a
        # request without a token, padding rows; the largest decode step
        dict(decode, name="decode_spec32", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, S=32, M=4, lo=1024, hi=16384,
             varlen=True, pad=7),
        # a window beside which the first keys stay, pages of hybrid models
        dict(decode, name="decode_window48_d256", dtype="bf16", D=256, Hq=16, Hkv=2, P=1056, S=48, M=2, lo=1, hi=16384,
             window=2000, sinks=130, layout=NHD, packed=True),
        # wide heads, all their rows to one kv head
        dict(decode, name="decode_wide_d512", dtype="fp16", D=512, Hq=8, Hkv=1, P=64, S=5, M=8, lo=500, hi=20000),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    if hi <= lo:
        return lo
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 0.5)))))))


def _draw(rng):
    op = rng.choice(["write", "write", "read", "decode", "decode", "decode"])
    heads = rng.choice([(32, 8), (8, 2), (8, 1), (16, 2), (16, 4), (24, 8), (6, 6), (20, 4), (15, 5)])
    D = rng.choice([64, 128, 128, 256, 512])
    base = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), D=D, Hq=heads[0], Hkv=heads[1],
                P=rng.choice([16, 16, 32, 48, 64, 128, 528, 784, 1056]), layout=rng.choice([NHD, HND]),
                packed=rng.random() < 0.25, mix=rng.randrange(1 << 30))
    if op == "write":
        neox = rng.random() < 0.6
        S, q_hi = _spread(rng, 1, 256), _spread(rng, 1, 4096)
        return dict(base, S=S, q_lo=_spread(rng, 1, q_hi), q_hi=q_hi, neox=neox, axes=rng.choice([1, 1, 3, 4]),
                    rot=rng.choice([r for r in (0, 32, 64, 96, 128, 256, 512) if r <= D]), pad=rng.choice([0, 0, 5]),
                    max_pos=rng.choice([8192, 32768]))
    hi = _spread(rng, 1, 32768)
    window = rng.choice([0, 0, _spread(rng, 1, 8192)])
    base.update(S=_spread(rng, 1, 64), lo=_spread(rng, 1, hi), hi=hi, window=window)
    if op == "read":
        return base
    varlen = rng.random() < 0.5
    return dict(base, M=rng.randint(1, 8), sinks=_spread(rng, 1, 300) if window and rng.random() < 0.7 else 0,
                varlen=varlen, pad=rng.choice([0, 5]) if varlen else 0)


def _padded(case):
    """Values that a form with rectangular blocks holds at once."""
    if case["op"] == "write":
        return 0
    c, q = _lengths(case)
    longest = max(a + b for a, b in zip(c, q))
    if case["op"] == "read":
        return case["S"] * longest * case["Hkv"] * case["D"]
    keys = min(case["window"] + 16, longest) + case["sinks"] if case["window"] else longest
    return case["S"] * keys * max(case["M"] * case["Hq"], case["Hkv"] * case["D"])


def draw(rng):
    cases = listed()
    top = [work(c) for c in cases]
    most = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    padded = max(_padded(c) for c in cases)
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and _padded(case) <= padded:
            return case


# ---------------------------------------------------------------------------
# Lengths of a case's requests: of the case alone, so that work() knows them.

def _lengths(case):
    """(contexts, new tokens) of the requests: tokens cached before the step
    and in it.  Of a read, every token is in the cache."""
    rng = random.Random(case["mix"])
    S = case["S"]
    if case["op"] == "write":
        q = [_spread(rng, case["q_lo"], case["q_hi"]) for _ in range(S)]
        return [rng.randint(0, 3000) if case["q_hi"] < 1000 else 16 * rng.randint(0, 100) for _ in range(S)], q
    lens = [_spread(rng, case["lo"], case["hi"]) for _ in range(S)]
    if case["op"] == "read":
        return lens, [0] * S
    if case["varlen"]:
        q = [rng.randint(1, case["M"]) for _ in range(S)]
        if S >= 8:
            q[S // 3] = 0  # a request that gets no token in this step
    else:
        q = [case["M"]] * S
        if S >= 8:
            lens[S // 3] = 0  # an empty slot of the batch
    return [L - m for L, m in zip(lens, q)], q


def _visible(n, window, sinks):
    """Keys that a row of n keys sees."""
    if not window:
        return max(0, n)
    lo = max(0, n - window)
    return max(0, n) - max(0, lo - min(sinks, lo))


def _union(L, q, window, sinks):
    """Keys that the rows of a request see between them."""
    if L <= 0 or q <= 0:
        return 0
    if not window:
        return L
    lo = max(0, min(L, L - q + 1) - window)
    return L - max(0, lo - min(sinks, lo))


def _first(case, L):
    """The first token of a request of L tokens that a read brings back."""
    return max(0, L - case["window"]) // case["P"] * case["P"] if case["window"] else 0


def work(case):
    c, q = _lengths(case)
    D, Hq, Hkv, P, S = (case[x] for x in ("D", "Hq", "Hkv", "P", "S"))
    if case["op"] == "write":
        T, live = sum(q) + case["pad"], sum(q)
        blocks = sum(-(-(a + b) // BLOCK) - a // BLOCK for a, b in zip(c, q))
        appended = sum(1 for a in c if a % BLOCK)
        # q in and out, k and v in, codes and scales out (of an appended block
        # the old scales in), angles, positions, slots
        return {"bytes": 4 * T * Hq * D + 4 * live * Hkv * D + 2 * live * Hkv * D + 8 * Hkv * (blocks + appended)
                + 4 * T * (case["rot"] + case["axes"] * (case["rot"] > 0) + 1),
                "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * live * Hkv * D}
    if case["op"] == "read":
        toks = sum(L - _first(case, L) for L in c)
        pages = sum(-(-L // P) for L in c)
        return {"bytes": 6 * toks * Hkv * D + 8 * Hkv * -(-toks // BLOCK) + 8 * pages + 4 * S,
                "flops": 2 * toks * Hkv * D}
    w, k = case["window"], case["sinks"]
    keys = sum(_union(a + b, b, w, k) for a, b in zip(c, q))
    T = sum(q) + case["pad"] if case["varlen"] else S * case["M"]
    seen = sum(_visible(a + i + 1, w, k) for a, b in zip(c, q) for i in range(b))
    return {"bytes": 2 * keys * Hkv * D + 8 * Hkv * -(-keys // BLOCK) + 4 * T * Hq * D + 4 * keys // P + 8 * S,
            "flops": 4 * D * Hq * seen}


# ---------------------------------------------------------------------------
# Inputs.

def _gen(seed, dev, stream):
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + stream * 7919 + 31)
    return g


def _normal(shape, dtype, gen, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)


def _to(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def _by_slot(pool, layout):
    """A pool as [page, token, kv head, d]."""
    return pool if layout == NHD else pool.permute(0, 2, 1, 3)


def _new_pools(case, pages, dtype, dev):
    """Empty K and V pools in the case's layout."""
    P, Hkv, D = case["P"], case["Hkv"], case["D"]
    shape = (pages, P, Hkv, D) if case["layout"] == NHD else (pages, Hkv, P, D)
    if case["packed"]:
        pool = torch.zeros(shape[:3] + (2 * D,), dtype=torch.uint8 if dtype == E4M3 else dtype, device=dev)
        k, v = pool[..., :D], pool[..., D:]
    else:
        k, v = (torch.zeros(shape, dtype=torch.uint8 if dtype == E4M3 else dtype, device=dev) for _ in range(2))
    return (k.view(E4M3), v.view(E4M3)) if dtype == E4M3 else (k, v)


def _scale_of(amax):
    """The smallest power of two, 2^LEAST at least, under which amax is at most
    448 = 0.875 x 2^9."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    e = torch.where(amax > 0, e, LEAST).clamp(min=LEAST)
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _fill(case, codes, scale, seed, stream, dev, lean=None):
    """A quantised pool of seeded values, some heads' channels larger than
    others; ``lean``: (pages, tokens, [kv head, d]) that these tokens lean
    towards."""
    pages, per = scale.shape[0], case["P"] // BLOCK
    gen = _gen(seed, dev, stream)
    wide = torch.exp(0.4 * torch.randn((case["Hkv"], case["D"]), generator=gen, device=dev))
    for a in range(0, pages, max(1, (1 << 26) // (case["P"] * case["Hkv"] * case["D"]))):
        b = min(pages, a + max(1, (1 << 26) // (case["P"] * case["Hkv"] * case["D"])))
        x = torch.randn((b - a, case["P"], case["Hkv"], case["D"]), generator=gen, device=dev) * wide
        if lean is not None:
            on = (lean[0] >= a) & (lean[0] < b)
            x[lean[0][on] - a, lean[1][on]] += lean[2]
        x = x.reshape(b - a, per, BLOCK, case["Hkv"], case["D"])
        s = _scale_of(x.abs().amax((2, 4)))
        scale[a:b] = s
        x = (x / s[:, :, None, :, None]).reshape(b - a, case["P"], case["Hkv"], case["D"])
        _by_slot(codes, case["layout"])[a:b].view(torch.uint8).copy_(x.to(E4M3).view(torch.uint8))


def _cache(case, pages, seed, dev, lean=None):
    k, v = _new_pools(case, pages, E4M3, dev)
    ks, vs = (torch.empty((pages, case["P"] // BLOCK, case["Hkv"]), device=dev) for _ in range(2))
    _fill(case, k, ks, seed, 1, dev, lean)
    _fill(case, v, vs, seed, 2, dev)
    return k, v, ks, vs


def _never_written(case, st, tables, lens):
    """NaN in the slots past each request's last token, and in the scales of
    blocks that hold none."""
    P = case["P"]
    at = [(int(tables[s, L // P]), i) for s, L in enumerate(lens) if L % P for i in range(L % P, P)]
    if at:
        at = torch.tensor(at, device=st["k"].device)
        for c in (st["k"], st["v"]):
            _by_slot(c, case["layout"]).view(torch.uint8)[at[:, 0], at[:, 1]] = 0x7F
    at = [(int(tables[s, L // P]), i) for s, L in enumerate(lens) if L % P for i in range(-(-(L % P) // BLOCK), P // BLOCK)]
    if at:
        at = torch.tensor(at, device=st["k"].device)
        for c in (st["ks"], st["vs"]):
            c[at[:, 0], at[:, 1]] = float("nan")


def _decode_inputs(case, seed):
    """Queries and a cache that holds the visible pages alone (the others were
    given back: -1 in the table), with first keys that draw much of the weight,
    as the first tokens of a trained model do."""
    dev = _device()
    dt = DTYPES[case["dtype"]]
    P, S, D, Hq, Hkv = case["P"], case["S"], case["D"], case["Hq"], case["Hkv"]
    c, q = _lengths(case)
    lens = [max(a + b, 0) for a, b in zip(c, q)]
    W = max(1, max(-(-L // P) for L in lens))
    held = np.zeros((S, W), dtype=bool)
    for s, (L, m) in enumerate(zip(lens, q)):
        if L:
            lo = max(0, L - m + 1 - case["window"]) if case["window"] else 0
            held[s, lo // P:-(-L // P)] = True
            held[s, :-(-min(case["sinks"], L) // P)] = True
    pages = max(1, int(held.sum()))
    ids = np.random.RandomState((seed * 7919 + 11) % (1 << 32)).permutation(pages)
    table = np.full((S, W), -1, dtype=np.int32)
    table[held] = ids[:int(held.sum())]
    u = torch.randn((Hkv, D), generator=_gen(seed, dev, 4), device=dev) * 0.6
    first = [(int(table[s, i // P]), i % P) for s, L in enumerate(lens) for i in range(min(L, 4)) if table[s, i // P] >= 0]
    lean = None
    if first:
        at = torch.tensor(first, device=dev)
        lean = (at[:, 0], at[:, 1], u)
    st = dict(zip(("k", "v", "ks", "vs"), _cache(case, pages, seed, dev, lean)))
    _never_written(case, st, table, lens)
    start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    T = int(start[-1]) + case["pad"] if case["varlen"] else S * case["M"]
    qs = torch.randn((T, Hkv, Hq // Hkv, D), generator=_gen(seed, dev, 3), device=dev)
    qs = (qs + u[None, :, None, :]).to(dt).reshape(T, Hq, D)
    return dict(st, q=qs, table=_to(table, dev), lens=_to(lens, dev), start=_to(start, dev), lens_host=lens,
                start_host=start.tolist(), scale=1.0 / math.sqrt(D), out=torch.empty_like(qs))


def _read_inputs(case, seed):
    """Requests' pages in the cache and pages of a staging pool for them; a
    window's older pages in neither."""
    dev = _device()
    P, S = case["P"], case["S"]
    lens, _ = _lengths(case)
    lens = np.array(lens)[np.random.RandomState((seed * 7919 + 3) % (1 << 32)).permutation(S)]
    W = max(1, max(-(-L // P) for L in lens))
    held = np.zeros((S, W), dtype=bool)
    for s, L in enumerate(lens):
        held[s, _first(case, L) // P:-(-L // P)] = True
    pages = int(held.sum())
    rs = np.random.RandomState((seed * 7919 + 13) % (1 << 32))
    table, to = (np.full((S, W), -1, dtype=np.int32) for _ in range(2))
    table[held] = rs.permutation(pages)
    to[held] = rs.permutation(pages)
    st = dict(zip(("k", "v", "ks", "vs"), _cache(case, pages, seed, dev)))
    _never_written(case, st, table, lens)
    k_out, v_out = _new_pools(case, pages, DTYPES[case["dtype"]], dev)
    return dict(st, table=_to(table, dev), to=_to(to, dev), lens=_to(lens, dev), k_out=k_out, v_out=v_out)


def _sections(case):
    """Pairs of each axis."""
    half, axes = case["rot"] // 2, case["axes"]
    return [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)


def _write_inputs(case, seed):
    """New tokens of requests, laid out one after the other, and a cache whose
    appended blocks hold the tokens before them."""
    dev = _device()
    dt = DTYPES[case["dtype"]]
    D, Hq, Hkv, P, rot = (case[x] for x in ("D", "Hq", "Hkv", "P", "rot"))
    c, q = _lengths(case)
    rs = np.random.RandomState((seed * 7919 + 17) % (1 << 32))
    order = rs.permutation(case["S"])  # other requests for another seed
    c, q = np.array(c)[order], np.array(q)[order]
    live, T = int(q.sum()), int(q.sum()) + case["pad"]
    # the pages that hold new tokens
    pages = int(sum(-(-(a + b) // P) - a // P for a, b in zip(c, q)))
    ids = rs.permutation(pages)
    slots, n = np.full(T, -1, dtype=np.int64), 0
    pos, t = np.zeros((case["axes"], T), dtype=np.int64), 0
    for a, b in zip(c, q):
        p = a + np.arange(b)
        slots[t:t + b] = ids[n + p // P - a // P] * P + p % P
        grid = [p, a + (p - a) // 7, a + (p - a) % 7, a + (p - a) % 3]  # text, then an image's rows
        for x in range(case["axes"]):
            pos[x, t:t + b] = np.where(p - a < b // 2, p, grid[x])
        n += -(-(a + b) // P) - a // P
        t += b
    k_cache, v_cache, ks, vs = _cache(case, pages, seed, dev)
    # appended blocks whose old tokens were small: their scale has to grow
    ks *= torch.where(torch.rand(ks.shape, generator=_gen(seed, dev, 9), device=dev) < 0.3, 0.25, 1.0)
    wide = torch.exp(0.4 * torch.randn((Hkv, D), generator=_gen(seed, dev, 8), device=dev))
    qs = _normal((T, Hq, D), dt, _gen(seed, dev, 5), dev)
    k, v = ((torch.randn((T, Hkv, D), generator=_gen(seed, dev, 6 + j), device=dev) * wide).to(dt) for j in range(2))
    st = dict(q=qs, k=k, v=v, slots=_to(slots, dev), live=live, kc=k_cache, vc=v_cache, ks=ks, vs=vs,
              q_out=torch.empty_like(qs), positions=None, table=None, axis=None)
    if rot:
        pos = np.minimum(pos, case["max_pos"] - 1)
        f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=dev) / rot)
        ang = torch.arange(case["max_pos"], dtype=torch.float64, device=dev)[:, None] * f[None, :]
        axis = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
        st.update(positions=_to(pos, dev), table=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(),
                  axis=bytes(axis), axis_dev=torch.tensor(axis, dtype=torch.int64, device=dev))
    return st


def prepare(case, seed):
    st = {"write": _write_inputs, "read": _read_inputs, "decode": _decode_inputs}[case["op"]](case, seed)
    st["case"] = case
    if own and case["op"] == "decode":
        # what a program keeps for its calls
        import paged_split_kv_02_gb300 as pd

        st["scratch"] = pd.Scratch(case["S"], case["Hq"], case["Hkv"], case["D"], case["M"],
                                   max_splits=max(8, 1024 // (case["S"] * case["Hkv"])))
    return st


# ---------------------------------------------------------------------------
# One pass.

def run(st):
    if own:
        return _run_own(st)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode}[st["case"]["op"]](st)


def _run_own(st):
    import paged_split_kv_02_gb300 as pd

    c = st["case"]
    if c["op"] == "write":
        pd.paged_rope_quant_cache_write(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["table"],
                                        st["axis"], st["q_out"], st["kc"], st["vc"], st["ks"], st["vs"], c["Hq"],
                                        c["Hkv"], c["D"], c["rot"], c["P"], c["layout"], c["neox"])
        return [st["q_out"], st["kc"], st["vc"], st["ks"], st["vs"]]
    if c["op"] == "read":
        pd.paged_quant_cache_read(st["k"], st["v"], st["ks"], st["vs"], st["table"], st["lens"], st["to"],
                                  st["k_out"], st["v_out"], c["Hkv"], c["D"], c["P"], c["layout"])
        return [st["k_out"], st["v_out"]]
    pd.paged_decode_attn_quant(st["q"], st["k"], st["v"], st["ks"], st["vs"], st["table"], st["lens"], st["out"],
                               c["Hq"], c["Hkv"], c["D"], c["P"], c["M"], c["window"], c["sinks"], st["scale"],
                               c["layout"], st["scratch"], query_start=st["start"] if c["varlen"] else None)
    return st["out"]


def _rotate(x, cos, sin, rot, neox):
    y = x.float()
    half = rot // 2
    a, b = (y[..., :half], y[..., half:rot]) if neox else (y[..., 0:rot:2], y[..., 1:rot:2])
    c, s = cos[:, None], sin[:, None]
    p, r = a * c - b * s, b * c + a * s
    z = torch.cat([p, r], -1) if neox else torch.stack([p, r], -1).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1)


def _store(x, slot, cache, scale, c):
    """Rows x [n, kv head, d] in 32 bits into the cache at slot [n]."""
    P, per = c["P"], c["P"] // BLOCK
    pages, Hkv, D = scale.shape[0], c["Hkv"], c["D"]
    block = slot // P * per + slot % P // BLOCK
    every = block[:, None].expand(-1, Hkv)
    flat = scale.reshape(-1, Hkv)
    amax = torch.zeros_like(flat).scatter_reduce(0, every, x.abs().amax(-1), "amax")
    first = torch.full((flat.shape[0],), BLOCK, device=x.device).scatter_reduce(0, block, slot % BLOCK, "amin")
    need = _scale_of(amax)
    first = first[:, None]
    new = torch.where(first == BLOCK, flat, torch.where(first == 0, need, torch.maximum(flat, need)))
    # other tokens of a block whose scale grew, rounded to the new one
    by_slot = _by_slot(cache, c["layout"])
    ratio = torch.where((first > 0) & (first < BLOCK), flat / new, 1.0).reshape(pages, per, 1, Hkv, 1)
    old = by_slot.float().reshape(pages, per, BLOCK, Hkv, D) * ratio
    by_slot.view(torch.uint8).copy_(old.reshape(pages, P, Hkv, D).to(E4M3).view(torch.uint8))
    by_slot.view(torch.uint8)[slot // P, slot % P] = (x / new[block][..., None]).to(E4M3).view(torch.uint8)
    scale.copy_(new.reshape(scale.shape))


def _plain_write(st):
    c = st["case"]
    rot, live = c["rot"], st["live"]
    if rot:
        pos = st["positions"].long()[st["axis_dev"]].t()                  # [T, rot / 2]
        pair = torch.arange(rot // 2, device=pos.device)
        cos, sin = st["table"][pos, pair], st["table"][pos, rot // 2 + pair]
        q, k = (_rotate(x, cos, sin, rot, c["neox"]) for x in (st["q"], st["k"]))
    else:
        q, k = st["q"].float(), st["k"].float()
    slot = st["slots"][:live].long()                                      # padding comes last
    _store(k[:live], slot, st["kc"], st["ks"], c)
    _store(st["v"][:live].float(), slot, st["vc"], st["vs"], c)
    st["q_out"].copy_(q)
    return [st["q_out"], st["kc"], st["vc"], st["ks"], st["vs"]]


def _plain_read(st):
    c = st["case"]
    P, per, Hkv, D = c["P"], c["P"] // BLOCK, c["Hkv"], c["D"]
    src, dst, dev = st["table"].long(), st["to"].long(), st["lens"].device
    S, W = src.shape
    page = torch.arange(W, device=dev).expand(S, W)
    n = (st["lens"].long()[:, None] - page * P).clamp(0, P)               # tokens of a page
    there = (src >= 0) & (dst >= 0) & (n > 0)
    # of every staging page, the page that it gets (the last entry: of none)
    N = st["k_out"].shape[0]
    dst = torch.where(there, dst, N).reshape(-1)
    at = torch.full((N + 1,), -1, device=dev).scatter(0, dst, torch.arange(S * W, device=dev))[:N]
    from_page = torch.where(at >= 0, src.reshape(-1)[at], 0)
    count = torch.where(at >= 0, n.reshape(-1)[at], 0)
    live = (torch.arange(P, device=dev) < count[:, None])[:, :, None, None]
    for cache, scale, out in ((st["k"], st["ks"], st["k_out"]), (st["v"], st["vs"], st["v_out"])):
        x = _by_slot(cache, c["layout"]).view(torch.uint8)[from_page].view(E4M3).float()
        x = (x.reshape(N, per, BLOCK, Hkv, D) * scale[from_page][:, :, None, :, None]).reshape(N, P, Hkv, D)
        to = _by_slot(out, c["layout"])
        to.copy_(torch.where(live, x, to.float()))
    return [st["k_out"], st["v_out"]]


def _plain_decode(st):
    """The keys of a request (its first ones, then the window of its first row
    up to its last row) gathered beside one another, softmax over the masked
    scores."""
    c = st["case"]
    P, B, Hq, Hkv, D, w, sinks = c["P"], c["M"], c["Hq"], c["Hkv"], c["D"], c["window"], c["sinks"]
    S, G, T, dev = c["S"], Hq // Hkv, st["q"].shape[0], st["q"].device
    L = st["lens"].long()
    q0 = st["start"].long()[:-1] if c["varlen"] else torch.arange(S, device=dev) * B
    qn = st["start"].long()[1:] - q0 if c["varlen"] else torch.full((S,), B, device=dev)
    i = torch.arange(B, device=dev).expand(S, B)                       # token of the request
    row = torch.where(i < qn[:, None], q0[:, None] + i, T)             # T: no row
    n = (L - qn)[:, None] + i + 1                                      # keys of the row
    lo = (n - w).clamp(min=0) if w else torch.zeros_like(n)
    far = torch.maximum(lo[:, :1], torch.tensor(sinks, device=dev))    # first gathered key of the window
    K = int(st["table"].shape[1]) * P
    K = min(w + B - 1, K) if w else K
    key = torch.cat([torch.arange(sinks, device=dev).expand(S, -1), far + torch.arange(K, device=dev)], 1)
    there = key < L[:, None]
    page = torch.gather(st["table"].long(), 1, torch.where(there, key // P, 0))
    there &= page >= 0
    page = torch.where(there, page, 0)
    on = there[:, :, None, None]

    def gathered(cache, scale):
        x = _by_slot(cache, c["layout"]).view(torch.uint8)[page, key % P].view(E4M3).float()
        return torch.where(on, x * scale[page, key % P // BLOCK][..., None], 0.0)

    q = torch.cat([st["q"], st["q"].new_zeros((1, Hq, D))])[row].float()
    q = q.reshape(S, B, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * B, D)
    x = (q @ gathered(st["k"], st["ks"]).permute(0, 2, 3, 1)).reshape(S, Hkv, G, B, -1) * st["scale"]
    k = key[:, None]
    seen = there[:, None] & (k < n[..., None]) & ((k >= lo[..., None]) | (k < sinks))
    # a key below the window's first row is one of the first, counted once in its own place
    seen = (seen & ((k >= far[..., None]) | (torch.arange(k.shape[-1], device=dev) < sinks)))[:, None, None]
    x = torch.where(seen, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    s = p.sum(-1)
    o = (p.reshape(S, Hkv, G * B, -1) @ gathered(st["v"], st["vs"]).permute(0, 2, 1, 3)).reshape(S, Hkv, G, B, D)
    o = torch.where(s[..., None] > 0, o / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    out = st["q"].new_zeros((T + 1, Hq, D))
    out[row.reshape(-1)] = o.permute(0, 3, 1, 2, 4).reshape(S * B, Hq, D).to(out.dtype)
    return out[:T]


# ---------------------------------------------------------------------------
# The definitions in 64 bits.  Of codes, the quotients that are rounded to them.

def exact(case, seed):
    return {"write": _exact_write, "read": _exact_read, "decode": _exact_decode}[case["op"]](case, seed)


def _exact_write(case, seed):
    st = _write_inputs(case, seed)
    P, rot, half = case["P"], case["rot"], case["rot"] // 2
    turned = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        for j in range(half):
            a, b = (j, j + half) if case["neox"] else (2 * j, 2 * j + 1)
            p = st["positions"][st["axis"][j]].long()
            c, s = st["table"][p, j].double()[:, None], st["table"][p, half + j].double()[:, None]
            y[..., a], y[..., b] = (x[..., a].double() * c - x[..., b].double() * s,
                                    x[..., b].double() * c + x[..., a].double() * s)
        turned.append(y)
    slots = st["slots"].cpu().numpy()
    # rows of the batch by the block that they are written to
    rows, place = {}, {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            rows.setdefault(slot // BLOCK, []).append(t)
    touched = sorted(rows)
    dev = st["q"].device
    table = np.full((len(touched), BLOCK), -1, dtype=np.int64)
    for i, b in enumerate(touched):
        for t in rows[b]:
            table[i, slots[t] % BLOCK] = t
    table = torch.from_numpy(table).to(dev)
    blocks = torch.tensor(touched, device=dev)
    page, sub = blocks * BLOCK // P, blocks * BLOCK % P // BLOCK
    tok = sub[:, None] * BLOCK + torch.arange(BLOCK, device=dev)
    new = (table >= 0)[:, :, None, None]
    fresh = (table[:, 0] >= 0)[:, None]
    out = []
    for x, cache, scale in ((turned[1], st["kc"], st["ks"]), (st["v"].double(), st["vc"], st["vs"])):
        codes, scales = _by_slot(cache, case["layout"]).to(torch.float64), scale.double()
        val = torch.where(new, x[table.clamp(min=0)], 0.0)                # [block, 16, kv head, d]
        top = val.abs().amax((1, 3))
        need = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(min=LEAST))
        need = torch.where(top <= 448.0 * need / 2, need / 2, need).clamp(min=2.0 ** LEAST)
        need = torch.where(top > 448.0 * need, need * 2, need)
        was = scales[page, sub]
        now = torch.where(fresh, need, torch.maximum(was, need))
        kept = codes[page[:, None], tok]
        kept = torch.where(fresh[:, :, None, None], kept, kept * (was / now)[:, None, :, None])
        codes[page[:, None], tok] = torch.where(new, val / now[:, None, :, None], kept)
        scales[page, sub] = now
        out.append((codes if case["layout"] == NHD else codes.permute(0, 2, 1, 3), scales))
    return [turned[0], out[0][0], out[1][0], out[0][1], out[1][1]]


def _exact_read(case, seed):
    st = _read_inputs(case, seed)
    P, out = case["P"], []
    table, to, lens = (st[x].cpu().numpy() for x in ("table", "to", "lens"))
    for cache, scale in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        codes = _by_slot(cache, case["layout"])
        got = torch.zeros(codes.shape, dtype=torch.float64, device=codes.device)
        for s, L in enumerate(lens):
            on = [j for j in range(-(-int(L) // P)) if table[s, j] >= 0]
            if on:
                # every token of the request's pages, then those that it has
                src, dst = (torch.tensor(x[s, on].astype(np.int64), device=codes.device) for x in (table, to))
                val = codes[src].double() * scale[src].double().repeat_interleave(BLOCK, 1)[..., None]
                tok = torch.tensor(on, device=codes.device)[:, None] * P + torch.arange(P, device=codes.device)
                got[dst] = torch.where((tok < int(L))[..., None, None], val, 0.0)
        out.append(got if case["layout"] == NHD else got.permute(0, 2, 1, 3))
    return out


def _exact_decode(case, seed):
    st = _decode_inputs(case, seed)
    P, Hq, Hkv, D = case["P"], case["Hq"], case["Hkv"], case["D"]
    G, T, dev = Hq // Hkv, st["q"].shape[0], st["q"].device
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    kc, vc = _by_slot(st["k"], case["layout"]), _by_slot(st["v"], case["layout"])
    for s in range(case["S"]):
        L = st["lens_host"][s]
        if case["varlen"]:
            t0, m = st["start_host"][s], st["start_host"][s + 1] - st["start_host"][s]
        else:
            t0, m = s * case["M"], case["M"]
        if L <= 0 or m <= 0:
            continue
        k_all, i = torch.arange(L, device=dev), torch.arange(m, device=dev)
        n = L - m + i + 1
        seen = k_all[None] < n[:, None]
        if case["window"]:
            seen &= (k_all[None] >= n[:, None] - case["window"]) | (k_all[None] < case["sinks"])
        some = seen.any(0).nonzero()[:, 0]  # keys that a row sees
        if not len(some):
            continue
        page, tok = st["table"][s].long()[some // P], some % P
        kk = kc[page, tok].double() * st["ks"][page, tok // BLOCK].double()[..., None]
        vv = vc[page, tok].double() * st["vs"][page, tok // BLOCK].double()[..., None]
        for h in range(Hkv):
            q = st["q"][t0:t0 + m, h * G:(h + 1) * G].double()
            x = torch.einsum("igd,kd->gik", q, kk[:, h]) * st["scale"]
            x = x.masked_fill(~seen[:, some], float("-inf"))
            p = torch.softmax(x, -1).nan_to_num(0.0)
            out[t0:t0 + m, h * G:(h + 1) * G] = torch.einsum("gik,kd->igd", p, vv[:, h])
    return out
