"""Measured cases of the sink-window attention, the block tables built on the
GPU and the rotary embedding with several position axes.

``run`` makes one pass through an operator: where ``own`` is true the calls of
``paged_split_kv_02_gb300``, else the same computation in elementary torch
operations, in 32 bits, rounded once at the end.

Operators
* ``attn`` (decode and prefill): paged attention whose rows see the first
  ``sinks`` keys of their sequence and a sliding window of the newest ones;
* ``tables``: block tables, query starts, lengths, positions and cache slots
  of a batch, made from the requests' lengths;
* ``rope``: rotary embedding with one position per axis (time, height, width)
  and the store of k and v into the paged cache.
"""

import math
import random

import numpy as np
import torch

own = False

NHD, HND = 0, 1
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------
# The cases.

def listed():
    decode = dict(op="attn", kind="decode", layout=HND, packed=False, varlen=False, pad=0, mix=1)
    prefill = dict(op="attn", kind="prefill", layout=HND, packed=False, varlen=True, pad=0, mix=1)
    return [
        # one user's chat on a model with wide heads and a short window: the
        # smallest call, where latency is all
        dict(decode, name="decode_one_d256_w512", dtype="fp16", D=256, Hq=8, Hkv=1, P=32, S=1, M=1,
             lo=32768, hi=32768, window=512, sinks=4),
        # a serving batch of ordinary chats, one token each
        dict(decode, name="decode_batch64_w1024", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, S=64, M=1,
             lo=300, hi=16384, window=1024, sinks=4),
        # speculative decoding over a captured batch: 1..4 draft tokens, an
        # empty request, padding rows, a window that long contexts leave
        dict(decode, name="decode_spec32_w4096", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, S=32, M=4,
             lo=1024, hi=16384, window=4096, sinks=16, varlen=True, pad=7),
        # the pages of hybrid models, whose end falls inside a 16-key tile of
        # nothing else; token-major pool with K and V side by side
        dict(decode, name="decode_hybrid48_w2000", dtype="bf16", D=256, Hq=16, Hkv=2, P=1056, S=48, M=2,
             lo=1, hi=16384, window=2000, sinks=130, layout=NHD, packed=True),
        # prompts that continue a conversation, in the usual chunk
        dict(prefill, name="prefill_4x2048_w1024", dtype="bf16", D=128, Hq=32, Hkv=8, P=16,
             q_lo=2048, q_hi=2048, S=4, lo=2048, hi=2048, window=1024, sinks=4),
        # two long documents, the window of a long-context model: the largest
        dict(prefill, name="prefill_2x8192_w4096", dtype="bf16", D=128, Hq=32, Hkv=8, P=16,
             q_lo=8192, q_hi=8192, S=2, lo=0, hi=0, window=4096, sinks=64),
        # chunked prefill of a mixed batch: ragged lengths, other head sizes
        dict(prefill, name="prefill_ragged_d64_w700", dtype="fp16", D=64, Hq=16, Hkv=4, P=48,
             q_lo=1, q_hi=1500, S=9, lo=0, hi=3500, window=700, sinks=33, pad=5, layout=NHD),
        # the tables of a decode step: every request grows by 1..4 tokens
        dict(op="tables", name="tables_decode256", S=256, q_lo=1, q_hi=4, lo=1, hi=16384, P=16,
             axes=1, pad=40, alloc=True, delta=False, mix=1),
        # the tables of a step that mixes long prompts with decoding
        dict(op="tables", name="tables_mixed1500", S=1500, q_lo=0, q_hi=1200, lo=0, hi=9000, P=32,
             axes=3, pad=0, alloc=True, delta=True, mix=1),
        # the new tokens of a decode batch
        dict(op="rope", name="rope_decode64", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, T=64, pad=3,
             rot=128, neox=True, sections="16,24,24", inter=False, layout=HND, packed=False, max_pos=32768),
        # a prompt with images and text
        dict(op="rope", name="rope_prompt16384", dtype="bf16", D=128, Hq=32, Hkv=8, P=16, T=16384, pad=0,
             rot=128, neox=True, sections="24,20,20", inter=True, layout=HND, packed=False, max_pos=32768),
        # a partly rotated head in pairs of neighbours
        dict(op="rope", name="rope_partial5001", dtype="fp16", D=256, Hq=16, Hkv=2, P=784, T=5001, pad=9,
             rot=64, neox=False, sections="8,12,12", inter=False, layout=NHD, packed=True, max_pos=16384),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    if hi <= lo:
        return lo
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 0.5)))))))


def _draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "tables", "rope"])
    heads = rng.choice([(32, 8), (8, 2), (8, 1), (16, 2), (16, 4), (24, 8), (6, 6), (20, 4)])
    P = rng.choice([16, 16, 32, 48, 64, 128, 528, 784, 1056])
    mix = rng.randrange(1 << 30)
    base = dict(P=P, mix=mix)
    if op == "tables":
        q_hi = _spread(rng, 1, 2000)
        return dict(base, op="tables", S=_spread(rng, 1, 2000), q_lo=rng.choice([0, 1]), q_hi=q_hi,
                    lo=rng.choice([0, 1, 100]), hi=_spread(rng, 200, 16384), axes=rng.choice([1, 1, 3, 4]),
                    pad=rng.choice([0, 3, 100]), alloc=rng.random() < 0.75, delta=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "fp16"])
    layout = rng.choice([NHD, HND])
    packed = rng.random() < 0.25
    D = rng.choice([64, 128, 128, 256, 512])
    base.update(dtype=dtype, layout=layout, packed=packed, D=D, Hq=heads[0], Hkv=heads[1])
    if op == "rope":
        neox = rng.random() < 0.6
        rot = rng.choice([r for r in (32, 64, 96, 128, 256, 512) if r <= D])
        half = rot // 2
        axes = rng.choice([2, 3, 3, 4])
        inter = rng.random() < 0.5
        if inter:
            other = [rng.randint(1, half // axes) for _ in range(axes - 1)]
        else:
            other = [rng.randint(0, half // axes) for _ in range(axes - 1)]
        sections = ",".join(str(x) for x in [half - sum(other)] + other)
        T = _spread(rng, 1, 16384)
        return dict(base, op="rope", T=T, pad=rng.choice([0, 0, min(T, 5)]), rot=rot, neox=neox, sections=sections,
                    inter=inter, max_pos=rng.choice([1000, 4096, 32768]))
    window, sinks = _spread(rng, 1, 8192), _spread(rng, 1, 300)
    base.update(op="attn", kind=op, window=window, sinks=sinks, pad=rng.choice([0, 0, 5]))
    if op == "decode":
        hi = _spread(rng, 1, 32768)
        varlen = rng.random() < 0.5
        return dict(base, S=_spread(rng, 1, 64), M=rng.randint(1, 8), lo=_spread(rng, 1, hi), hi=hi, varlen=varlen,
                    pad=base["pad"] if varlen else 0)
    q_hi = _spread(rng, 1, 8192)
    return dict(base, S=_spread(rng, 1, 16), q_lo=_spread(rng, 1, q_hi), q_hi=q_hi, lo=0, hi=_spread(rng, 1, 8192),
                varlen=True)


def _padded(case):
    """Scores and gathered values that a form with rectangular blocks holds."""
    if case["op"] != "attn":
        return 0
    c, q = _lengths(case)
    longest = max(a + b for a, b in zip(c, q))
    keys = min(case["window"] + 256, longest + case["P"]) + case["sinks"]
    blocks = case["S"] if case["kind"] == "decode" else sum(-(-m // 256) for m in q)
    rows = case["M"] if case["kind"] == "decode" else min(256, case["q_hi"])
    return blocks * keys * max(rows * case["Hq"], case["Hkv"] * case["D"])


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
    """(contexts, query lengths) of the requests: tokens cached before the
    step and new ones.  Decode lengths name the keys with the new tokens."""
    rng = random.Random(case["mix"])
    S = case["S"]
    if case["op"] == "tables" or case["kind"] == "prefill":
        q = [_spread(rng, max(case["q_lo"], 1), case["q_hi"]) for _ in range(S)]
        c = [_spread(rng, case["lo"], case["hi"]) if case["hi"] else 0 for _ in range(S)]
        if case["op"] == "tables" and case["q_lo"] == 0:
            q = [0 if rng.random() < 0.1 else x for x in q]  # waiting requests
        return c, q
    lens = [_spread(rng, case["lo"], case["hi"]) for _ in range(S)]
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
    lo = max(0, n - window)
    return max(0, n) - max(0, lo - min(sinks, lo))


def _union(L, q, window, sinks):
    """Keys that the rows of a request see between them."""
    if L <= 0 or q <= 0:
        return 0
    lo = max(0, min(L, L - q + 1) - window)
    return L - max(0, lo - min(sinks, lo))


def work(case):
    if case["op"] == "tables":
        c, q = _lengths(case)
        P, T = case["P"], sum(q) + case["pad"]
        pages = sum(-(-(a + b) // P) - a // P for a, b in zip(c, q) if b)
        new = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(c, q)) if case["alloc"] else 0
        # lengths (and offsets) in, page ids in and out, maps out
        return {"bytes": (8 + 4 * case["delta"]) * case["S"] + 4 * pages + 4 * new
                + 8 * case["S"] + 4 + 4 * (case["axes"] + 1) * T + 8, "flops": 0}
    if case["op"] == "rope":
        T, live = case["T"], case["T"] - case["pad"]
        D, Hq, Hkv, axes = case["D"], case["Hq"], case["Hkv"], len(case["sections"].split(","))
        return {"bytes": 2 * (2 * T * Hq * D + 4 * live * Hkv * D) + 4 * T * (case["rot"] + axes + 1),
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    c, q = _lengths(case)
    w, k, D = case["window"], case["sinks"], case["D"]
    keys = sum(_union(a + b, b, w, k) for a, b in zip(c, q))
    T = sum(q) + case["pad"]
    seen = sum(_visible(a + i + 1, w, k) for a, b in zip(c, q) for i in range(b))
    return {"bytes": 4 * keys * case["Hkv"] * D + 4 * T * case["Hq"] * D + 4 * keys // case["P"] + 8 * case["S"],
            "flops": 4 * D * case["Hq"] * seen}


# ---------------------------------------------------------------------------
# Inputs.

def _gen(seed, dev, stream):
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + stream * 7919 + 29)
    return g


def _normal(shape, dtype, gen, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)


def _pools(case, pages, seed, dev):
    """K and V pools of seeded values, in the case's layout."""
    P, Hkv, D = case["P"], case["Hkv"], case["D"]
    shape = (pages, P, Hkv, D) if case["layout"] == NHD else (pages, Hkv, P, D)
    dt = DTYPES[case["dtype"]]
    if case["packed"]:
        pool = _normal(shape[:3] + (2 * D,), dt, _gen(seed, dev, 1), dev)
        return pool[..., :D], pool[..., D:]
    return _normal(shape, dt, _gen(seed, dev, 1), dev), _normal(shape, dt, _gen(seed, dev, 2), dev)


def _by_slot(pool, layout):
    """A pool as [page, token, kv head, d]."""
    return pool if layout == NHD else pool.permute(0, 2, 1, 3)


def _attn_inputs(case, seed):
    """Queries, a pool that holds the visible pages alone (those between the
    sinks and the window were given back: -1 in the table), never written
    slots that are NaN, and first keys that draw much of the weight, as the
    first tokens of a trained model do."""
    dev = _device()
    dt = DTYPES[case["dtype"]]
    P, S, D, Hq, Hkv = case["P"], case["S"], case["D"], case["Hq"], case["Hkv"]
    c, q = _lengths(case)
    lens = [max(a + b, 0) for a, b in zip(c, q)]
    W = max(1, max(-(-L // P) for L in lens))
    held = np.zeros((S, W), dtype=bool)
    for s, (L, m) in enumerate(zip(lens, q)):
        if L:
            lo = max(0, L - m + 1 - case["window"])
            held[s, lo // P:-(-L // P)] = True
            held[s, :-(-min(case["sinks"], L) // P)] = True
    pages = max(1, int(held.sum()))
    ids = np.random.RandomState((seed * 7919 + 11) % (1 << 32)).permutation(pages)
    table = np.full((S, W), -1, dtype=np.int32)
    table[held] = ids[:int(held.sum())]
    k, v = _pools(case, pages, seed, dev)
    ks, vs = _by_slot(k, case["layout"]), _by_slot(v, case["layout"])
    start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    T = int(start[-1]) + case["pad"] if case["varlen"] else S * case["M"]
    qs = torch.randn((T, Hkv, Hq // Hkv, D), generator=_gen(seed, dev, 3), device=dev)
    u = torch.randn((Hkv, D), generator=_gen(seed, dev, 4), device=dev) * 0.6
    qs = (qs + u[None, :, None, :]).to(dt).reshape(T, Hq, D)
    # the sinks' keys lean towards the queries
    flat = [(int(table[s, i // P]), i % P) for s, L in enumerate(lens) for i in range(min(case["sinks"], L, 8))]
    if flat:
        at = torch.tensor(flat, device=dev)
        ks[at[:, 0], at[:, 1]] = (ks[at[:, 0], at[:, 1]].float() + u).to(dt)
    stale = [(int(table[s, L // P]), i) for s, L in enumerate(lens) if L % P for i in range(L % P, P)]
    if stale:
        at = torch.tensor(stale, device=dev)
        ks[at[:, 0], at[:, 1]] = float("nan")
        vs[at[:, 0], at[:, 1]] = float("nan")
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    return dict(q=qs, k=k, v=v, table=to(table), lens=to(lens), start=to(start), lens_host=lens,
                start_host=start.tolist(), scale=1.0 / math.sqrt(D))


def _tables_inputs(case, seed):
    """Requests with their pages so far, and a list of free pages."""
    dev = _device()
    c, q = _lengths(case)
    P, S = case["P"], case["S"]
    rs = np.random.RandomState((seed * 7919 + 13) % (1 << 32))
    order = rs.permutation(S)  # other requests for another seed
    c, q = np.array(c)[order], np.array(q)[order]
    have = -(-c // P)
    need = -(-(c + q) // P)
    W = int(need.max()) + 1
    total = int(need.sum())
    pages = total + 64
    ids = rs.permutation(pages).astype(np.int32)
    table = np.full((S, W), -1, dtype=np.int32)
    kept = have if case["alloc"] else need
    table[np.arange(W)[None, :] < kept[:, None]] = ids[:int(kept.sum())]
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    T = int(q.sum()) + case["pad"]
    axes = case["axes"]
    return dict(context=to(c), new=to(q), free=to(ids[int(kept.sum()):]) if case["alloc"] else None,
                cursor=to([0]), table=to(table), start=to(np.zeros(S + 1)), lens=to(np.zeros(S)),
                positions=torch.zeros((axes, T), dtype=torch.int32, device=dev), slots=to(np.zeros(T)),
                next=to([0]), delta=to(rs.randint(-200, 1, S)) if case["delta"] else None, pages=pages)


def _pair_axis(case):
    """The axis of every rotated pair: runs of the sections' lengths, or the
    axes in turn as long as each has pairs left, the rest the first axis."""
    sizes = [int(x) for x in case["sections"].split(",")]
    if not case["inter"]:
        return [a for a, n in enumerate(sizes) for _ in range(n)]
    A = len(sizes)
    return [i % A if i < A * sizes[i % A] else 0 for i in range(sum(sizes))]


def _rope_inputs(case, seed):
    dev = _device()
    dt = DTYPES[case["dtype"]]
    T, D, Hq, Hkv, P, rot = (case[x] for x in ("T", "D", "Hq", "Hkv", "P", "rot"))
    live = T - case["pad"]
    pages = -(-T // P) + 2
    k_cache, v_cache = _pools(case, pages, seed, dev)
    rs = np.random.RandomState((seed * 7919 + 17) % (1 << 32))
    # requests of the batch write runs of neighbouring slots in pages of any order
    ids = rs.permutation(pages)
    at = np.arange(T)
    slots = ids[at // P] * P + at % P
    slots[live:] = -1
    axes = len(case["sections"].split(","))
    # text runs with one position on every axis, images with a grid of them
    pos = np.zeros((axes, T), dtype=np.int64)
    i, p = 0, rs.randint(0, max(1, case["max_pos"] // 4))
    while i < T:
        n = min(T - i, rs.randint(1, 400))
        if rs.rand() < 0.5:
            pos[:, i:i + n] = p + np.arange(n)
            p += n
        else:
            w = rs.randint(1, 40)
            grid = [np.zeros(n, dtype=np.int64), np.arange(n) // w, np.arange(n) % w, np.arange(n) % 3]
            for a in range(axes):
                pos[a, i:i + n] = p + grid[a]
            p += max(1, n // w)
        i += n
        if p >= case["max_pos"] - 500:
            p = rs.randint(0, max(1, case["max_pos"] // 4))
    pos = np.minimum(pos, case["max_pos"] - 1)
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(case["max_pos"], dtype=torch.float64, device=dev)[:, None] * f[None, :]
    q, k, v = (_normal((T, h, D), dt, _gen(seed, dev, 5 + j), dev) for j, h in enumerate((Hq, Hkv, Hkv)))
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    return dict(q=q, k=k, v=v, positions=to(pos), slots=to(slots), live=live, axis=_pair_axis(case),
                table=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(),
                k_cache=k_cache, v_cache=v_cache)


def prepare(case, seed):
    st = {"attn": _attn_inputs, "tables": _tables_inputs, "rope": _rope_inputs}[case["op"]](case, seed)
    st["case"] = case
    if case["op"] == "attn":
        # the work list of a prefill (of the lengths alone, one for all layers
        # of a step): blocks of query rows for the plain form, the plan for
        # the framework's call
        dev = st["q"].device
        B = case["M"] if case["kind"] == "decode" else min(256, max(1, case["q_hi"]))
        qs = st["start_host"]
        items = [(s, i) for s in range(case["S"]) for i in range(0, max(qs[s + 1] - qs[s], 0), B)]
        st["block"] = B
        st["items"] = torch.tensor(items, dtype=torch.int64, device=dev).reshape(-1, 2)
        st["out"] = torch.empty_like(st["q"])
        if own:
            _handles(st)
    if case["op"] == "rope":
        st["q_out"] = torch.empty_like(st["q"])
        st["axis_dev"] = torch.tensor(st["axis"], dtype=torch.int64, device=st["q"].device)
        st["axis"] = bytes(st["axis"])
    return st


def _handles(st):
    """What a program keeps for its calls: scratch and the plan."""
    import paged_split_kv_02_gb300 as pd

    c = st["case"]
    if c["kind"] == "decode":
        st["scratch"] = pd.Scratch(c["S"], c["Hq"], c["Hkv"], c["D"], c["M"], max_splits=64)
        return
    items, st["info"] = pd.paged_prefill_plan_sinks(st["start_host"], st["lens_host"], c["Hq"], c["Hkv"], c["D"],
                                                    c["window"], c["sinks"])
    st["work"] = items.to(st["q"].device)
    st["scratch"] = pd.prefill_scratch(c["Hkv"], c["D"])


# ---------------------------------------------------------------------------
# One pass.

def run(st):
    if own:
        return _run_own(st)
    return {"attn": _plain_attn, "tables": _plain_tables, "rope": _plain_rope}[st["case"]["op"]](st)


def _run_own(st):
    import paged_split_kv_02_gb300 as pd

    c = st["case"]
    if c["op"] == "attn":
        if c["kind"] == "decode":
            pd.paged_decode_attn_sinks(st["q"], st["k"], st["v"], st["table"], st["lens"], st["out"], c["Hq"], c["Hkv"],
                                       c["D"], c["P"], c["M"], c["window"], c["sinks"], st["scale"], c["layout"],
                                       st["scratch"], query_start=st["start"] if c["varlen"] else None)
        else:
            pd.paged_prefill_attn_sinks(st["q"], st["k"], st["v"], st["table"], st["lens"], st["start"], st["work"],
                                        st["info"], st["out"], c["Hq"], c["Hkv"], c["D"], c["P"], c["window"],
                                        c["sinks"], st["scale"], c["layout"], st["scratch"])
        return st["out"]
    if c["op"] == "tables":
        pd.paged_batch_tables(st["context"], st["new"], st["table"], st["start"], st["lens"], st["positions"],
                              st["slots"], c["P"], st["pages"], free_pages=st["free"], cursor=st["cursor"],
                              next_cursor=st["next"], position_delta=st["delta"])
        return [st["table"], st["start"], st["lens"], st["positions"], st["slots"], st["next"]]
    pd.paged_rope_axes_cache_write(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["table"], st["axis"],
                                   st["q_out"], st["k_cache"], st["v_cache"], c["Hq"], c["Hkv"], c["D"], c["rot"],
                                   c["P"], c["layout"], c["neox"])
    return [st["q_out"], st["k_cache"], st["v_cache"]]


def _plain_attn(st):
    """Blocks of B query rows of one request each, the keys of a block (the
    sinks, then the window of its first row up to its last row) gathered
    beside one another, softmax over the masked scores."""
    c = st["case"]
    P, B, Hq, Hkv, D, w, sinks = c["P"], st["block"], c["Hq"], c["Hkv"], c["D"], c["window"], c["sinks"]
    G, T, dev = Hq // Hkv, st["q"].shape[0], st["q"].device
    seq, first = st["items"][:, 0], st["items"][:, 1]
    N = seq.shape[0]
    L, q0 = st["lens"].long()[seq], st["start"].long()[seq]
    qn = st["start"].long()[seq + 1] - q0
    i = first[:, None] + torch.arange(B, device=dev)                   # token of the request [N, B]
    row = torch.where(i < qn[:, None], q0[:, None] + i, T)             # T: no row
    n = (L - qn)[:, None] + i + 1                                      # keys of the row
    lo = (n - w).clamp(min=0)
    far = torch.maximum(lo[:, :1], torch.tensor(sinks, device=dev))    # first gathered key of the window
    K = min(w + B - 1, int(st["table"].shape[1]) * P)
    key = torch.cat([torch.arange(sinks, device=dev).expand(N, -1), far + torch.arange(K, device=dev)], 1)
    there = key < L[:, None]
    page = st["table"].long()[seq[:, None], torch.where(there, key // P, 0)]
    there &= page >= 0
    page = torch.where(there, page, 0)
    kk = torch.where(there[:, :, None, None], _by_slot(st["k"], c["layout"])[page, key % P].float(), 0.0)
    vv = torch.where(there[:, :, None, None], _by_slot(st["v"], c["layout"])[page, key % P].float(), 0.0)
    q = torch.cat([st["q"], st["q"].new_zeros((1, Hq, D))])[row].float()
    q = q.reshape(N, B, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * B, D)
    x = (q @ kk.permute(0, 2, 3, 1)).reshape(N, Hkv, G, B, -1) * st["scale"]
    key, there = key[:, None], there[:, None]
    seen = there & (key < n[..., None]) & ((key >= lo[..., None]) | (key < sinks))
    # a key below the window's first row is a sink, counted once in its own place
    seen = (seen & ((key >= far[..., None]) | (torch.arange(key.shape[-1], device=dev) < sinks)))[:, None, None]
    x = torch.where(seen, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    s = p.sum(-1)
    o = (p.reshape(N, Hkv, G * B, -1) @ vv.permute(0, 2, 1, 3)).reshape(N, Hkv, G, B, D)
    o = torch.where(s[..., None] > 0, o / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    out = st["q"].new_zeros((T + 1, Hq, D))
    out[row.reshape(-1)] = o.permute(0, 3, 1, 2, 4).reshape(N * B, Hq, D).to(out.dtype)
    return out[:T]


def _plain_tables(st):
    c = st["case"]
    P, dev = c["P"], st["new"].device
    T, S = st["slots"].shape[0], c["S"]
    ctx, q = st["context"].long(), st["new"].long()
    end = q.cumsum(0)
    start = torch.cat([end.new_zeros(1), end])
    lens = ctx + q
    t = torch.arange(T, device=dev)
    s = torch.searchsorted(end, t, right=True).clamp(max=S - 1)
    live = t < start[-1]
    pos = ctx[s] + t - start[s]
    page = torch.where(live, pos // P, 0)
    table = st["table"]
    cursor = st["cursor"].long()
    if st["free"] is not None:
        have = (ctx + P - 1) // P
        need = (lens + P - 1) // P - have
        off = cursor + need.cumsum(0) - need
        new = page >= have[s]
        got = st["free"][torch.where(live & new, off[s] + page - have[s], 0)]
        held = torch.where(new, got, table[s, page])
        opens = live & new
        # (rows of other tokens are sent to a column of their own)
        wide = torch.cat([table, table.new_zeros((S, 1))], 1)
        wide[s, torch.where(opens, page, table.shape[1])] = held
        table = wide[:, :-1].contiguous()
        cursor = cursor + need.sum()
    else:
        held = table[s, page]
    slot = torch.where(live, held.long() * P + pos % P, -1)
    if st["delta"] is not None:
        pos = pos + st["delta"].long()[s]
    pos = torch.where(live, pos, 0).expand(c["axes"], T)
    i32 = torch.int32
    return [table, start.to(i32), lens.to(i32), pos.to(i32).contiguous(), slot.to(i32), cursor.to(i32)]


def _rotate(x, cos, sin, rot, neox):
    y = x.float()
    half = rot // 2
    a, b = (y[..., :half], y[..., half:rot]) if neox else (y[..., 0:rot:2], y[..., 1:rot:2])
    c, s = cos[:, None], sin[:, None]
    p, r = a * c - b * s, b * c + a * s
    z = torch.cat([p, r], -1) if neox else torch.stack([p, r], -1).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(st):
    c = st["case"]
    half, live = c["rot"] // 2, st["live"]
    pos = st["positions"].long()[st["axis_dev"]].t()                  # [T, half]
    pair = torch.arange(half, device=pos.device)
    cos, sin = st["table"][pos, pair], st["table"][pos, half + pair]
    q, k = _rotate(st["q"], cos, sin, c["rot"], c["neox"]), _rotate(st["k"], cos, sin, c["rot"], c["neox"])
    slot = st["slots"][:live].long()                                  # padding comes last
    page, tok = slot // c["P"], slot % c["P"]
    _by_slot(st["k_cache"], c["layout"])[page, tok] = k[:live]
    _by_slot(st["v_cache"], c["layout"])[page, tok] = st["v"][:live]
    return [q, st["k_cache"], st["v_cache"]]


# ---------------------------------------------------------------------------
# The definitions in 64 bits.

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    st = _attn_inputs(case, seed)
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
        k_all = torch.arange(L, device=dev)
        for a in range(0, m, 512):
            i = torch.arange(a, min(a + 512, m), device=dev)
            n = L - m + i + 1
            seen = (k_all[None] < n[:, None]) & ((k_all[None] >= n[:, None] - case["window"]) | (k_all[None] < case["sinks"]))
            some = seen.any(0).nonzero()[:, 0]  # keys that a row of the chunk sees
            if not len(some):
                continue
            at = (st["table"][s].long()[some // P], some % P)
            kk, vv = kc[at].double(), vc[at].double()
            seen = seen[:, some]
            for h in range(Hkv):
                q = st["q"][t0 + i, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,kd->gik", q, kk[:, h]) * st["scale"]
                x = x.masked_fill(~seen, float("-inf"))
                p = torch.softmax(x, -1).nan_to_num(0.0)
                out[t0 + i, h * G:(h + 1) * G] = torch.einsum("gik,kd->igd", p, vv[:, h])
    return out


def _exact_rope(case, seed):
    st = _rope_inputs(case, seed)
    half, P = case["rot"] // 2, case["P"]
    i = torch.arange(half, device=st["q"].device)
    first, second = (i, i + half) if case["neox"] else (2 * i, 2 * i + 1)
    table = st["table"].double()
    turned = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        for j in range(half):
            p = st["positions"][st["axis"][j]].long()
            c, s = table[p, j][:, None], table[p, half + j][:, None]
            a, b = x[..., first[j]].double(), x[..., second[j]].double()
            y[..., first[j]], y[..., second[j]] = a * c - b * s, b * c + a * s
        turned.append(y)
    k_pool, v_pool = st["k_cache"].double(), st["v_cache"].double()
    slot = st["slots"].long()
    on = slot >= 0
    at = (slot[on] // P, slot[on] % P)
    _by_slot(k_pool, case["layout"])[at] = turned[1][on]
    _by_slot(v_pool, case["layout"])[at] = st["v"].double()[on]
    return [turned[0], k_pool, v_pool]
