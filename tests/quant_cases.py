"""Caches of codes for the tests of the calls of paged_quant.h."""

from __future__ import annotations

import dataclasses

import numpy as np
import torch

import paged_split_kv_02_gb300 as pd
from oracle import quant_cache as Q
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W

E4M3 = torch.float8_e4m3fn
# half a step of a type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def to_pools(kcodes, vcodes, layout, packed, device="cuda"):
    """(k_cache, v_cache) e4m3 pools of codes [page, token, kv head, d]."""
    t = lambda c: torch.from_numpy(np.ascontiguousarray(  # noqa: E731
        c if layout == W.NHD else c.transpose(0, 2, 1, 3))).to(device)
    k, v = t(kcodes), t(vcodes)
    if packed:
        pool = torch.cat([k, v], -1)
        k, v = pool[..., :k.shape[-1]], pool[..., k.shape[-1]:]
    return k.view(E4M3), v.view(E4M3)


def quantise(x: np.ndarray, factor=None):
    """(codes, scales) of values [page, token, kv head, d]; blocks that hold no
    finite value get a NaN scale; factor: of the scales, [page, blocks, kv head]."""
    pages, P, H, D = x.shape
    b = x.reshape(pages, P // Q.TOKENS, Q.TOKENS, H, D)
    a = np.where(np.isfinite(b), np.abs(b), 0.0).max(axis=(2, 4))
    with np.errstate(divide="ignore"):
        e = np.maximum(np.ceil(np.log2(np.where(a > 0, a, 1.0) / 448.0)), Q.LEAST)
    s = np.where(a > 0, 2.0 ** e, 2.0 ** Q.LEAST)
    if factor is not None:
        s = (s * factor).astype(np.float32).astype(np.float64)
    codes = Q.encode(b / s[:, :, None, :, None]).reshape(x.shape)
    empty = ~np.isfinite(b).any(axis=(2, 4))
    return codes, np.where(empty, np.nan, s).astype(np.float32)


@dataclasses.dataclass
class QuantCase:
    """A decode case whose cache is held in codes; ``exact``: the case with the
    values that they stand for."""
    case: W.DecodeCase
    exact: W.DecodeCase
    k: torch.Tensor
    v: torch.Tensor
    ks: torch.Tensor
    vs: torch.Tensor


def quant_case(case: W.DecodeCase, factors=(None, None), packed=False, device="cuda") -> QuantCase:
    by = (lambda c: c) if case.layout == W.NHD else (lambda c: c.permute(0, 2, 1, 3))
    got = [quantise(by(c).double().numpy(), f) for c, f in zip((case.k_cache, case.v_cache), factors)]
    k, v = to_pools(got[0][0], got[1][0], case.layout, packed, device)
    back = [torch.from_numpy(Q.dequantised(c, s)) for c, s in got]
    back = [b if case.layout == W.NHD else b.permute(0, 2, 1, 3) for b in back]
    return QuantCase(case, dataclasses.replace(case, k_cache=back[0], v_cache=back[1], packed=False), k, v,
                     *(torch.from_numpy(s).to(device) for _, s in got))


def run(qc: QuantCase, sinks=0, scratch=None, out=None, stream=None, check=True):
    c = qc.case
    dev = qc.k.device
    out = torch.empty_like(c.q, device=dev) if out is None else out
    qs = None if c.query_start is None else c.query_start.to(dev)
    rc = pd.paged_decode_attn_quant(c.q.to(dev), qc.k, qc.v, qc.ks, qc.vs, c.block_table.to(dev),
                                    c.seq_lens.to(dev), out, c.num_q_heads, c.num_kv_heads,
                                    c.head_size, c.page_size, c.max_query_len, c.window, sinks,
                                    c.scale, c.layout, scratch, query_start=qs, stream=stream,
                                    check=check)
    return out if check else rc


def near(qc: QuantCase, out: torch.Tensor, sinks=0, rows=None):
    """The outputs against the definition.  Each weight p is rounded to 11 bits,
    half a step of which is 2^-11 of it, so a row's sum is off by at most 2^-11 of
    A = sum p |v| / sum p; a quarter of that is left for the fp32 arithmetic: a
    score is a sum of D products in fp32, D / 16 + 4 roundings of 2^-23 of
    sum |q k| scale (below 30 here: 36 x 2^-23 x 30 < 2^-13 at D = 512), and the
    sums of p and p v round in fp32, 2^-24 a step for as many steps as a warp has
    (below 512: 2^-15).  The result is rounded once to the type."""
    ref = O.attention(qc.exact, sinks, rows)
    mags = dataclasses.replace(qc.exact, v_cache=qc.exact.v_cache.abs())
    A = O.attention(mags, sinks, rows)
    got = out.double().cpu().numpy()
    if rows is not None:
        got = np.stack([got[t, h] for t, h in rows])
    assert np.isfinite(got).all(), "non-finite output"
    h = HALF_STEP[qc.case.dtype]
    off = 1.25 * 2.0 ** -11 * A
    bad = np.abs(got - ref) > h * (np.abs(ref) + off) + off + 2.0 ** -25
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref).max()), float((off).max()))
    return ref
