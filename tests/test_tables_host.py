"""paged_batch_tables on the CPU: refusals (checked on the host before any
launch) and its oracle's pins."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import batch_tables as O
from step_cases import batch

PASSES = -8  # a call that passes every check reaches the missing device


@pytest.fixture(scope="module", autouse=True)
def _built():
    if torch.cuda.is_available():
        pytest.skip("host tensors: for machines without a GPU")
    pd.build()


def test_header_constants():
    text = open(pd.STEP_HEADER).read()
    assert f"#define PD_MAX_AXES {pd.MAX_AXES}" in text
    assert f"#define PD_DEV_NO_PAGE 0x{pd.DEV_NO_PAGE:x}u" in text
    assert "paged_batch_tables" in pd.declared_symbols(pd.STEP_HEADER)


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def _tables(**kw):
    a = dict(c=_i(3), q=_i(3), table=_i(3, 5), start=_i(4), lens=_i(3), pos=_i(2, 9), slots=_i(9), P=16,
             pages=40, free=_i(6), cursor=_i(1), next=_i(1), delta=None)
    a.update(kw)
    return pd.paged_batch_tables(a["c"], a["q"], a["table"], a["start"], a["lens"], a["pos"], a["slots"],
                                 a["P"], a["pages"], free_pages=a["free"], cursor=a["cursor"],
                                 next_cursor=a["next"], position_delta=a["delta"], check=False)


def test_tables_refusals():
    i, shared = _i, _i(64)
    for kw in [dict(), dict(pos=i(9)), dict(delta=i(3)), dict(free=None),
               dict(free=None, cursor=None, next=None), dict(table=i(3, 9)[:, 2:7]),
               dict(pos=i(8, 12)[:, :9]), dict(free=i(0)),
               dict(c=i(0), q=i(0), table=i(0, 5), start=i(1), lens=i(0)), dict(slots=i(0), pos=i(1, 0)),
               dict(c=shared[:3], lens=shared[3:6])]:
        assert _tables(**kw) == PASSES, kw
    for kw, rc in [
            (dict(q=i(2)), -1), (dict(start=i(3)), -1), (dict(lens=i(4)), -1), (dict(table=i(2, 5)), -1),
            (dict(table=i(3, 0)), -1), (dict(pos=i(2, 8)), -1), (dict(pos=i(9, 9)), -1),
            (dict(pos=i(0, 9)), -1), (dict(pos=i(1, 1, 9)), -1), (dict(cursor=None), -1),
            (dict(next=None), -1), (dict(cursor=i(2)), -1), (dict(P=0), -1), (dict(P=-16), -1),
            (dict(pages=0), -1), (dict(pages=2 ** 27, P=16), -1), (dict(table=i(3, 5), P=2 ** 30), -1),
            (dict(delta=i(2)), -1), (dict(c=torch.zeros(3)), -2), (dict(q=i(3).long()), -2),
            (dict(table=torch.zeros(3, 5)), -2), (dict(pos=torch.zeros(2, 9)), -2),
            (dict(slots=i(9).long()), -2), (dict(free=torch.zeros(6)), -2), (dict(delta=torch.zeros(3)), -2),
            (dict(c=i(6)[::2]), -5), (dict(slots=i(18)[::2]), -5), (dict(table=i(3, 10)[:, ::2]), -5),
            (dict(pos=i(2, 18)[:, ::2]), -5),
            # rows that share their entries, axes that share theirs
            (dict(table=i(5).expand(3, 5)), -1), (dict(pos=i(9).expand(2, 9)), -1),
            # an output over an input, or over another output
            (dict(c=shared[:3], lens=shared[:3]), -1), (dict(c=shared[:3], lens=shared[2:5]), -1),
            (dict(cursor=shared[:1], next=shared[:1]), -1), (dict(free=shared[:6], slots=shared[5:14]), -1),
            (dict(start=shared[:4], lens=shared[3:6]), -1),
            (dict(q=shared[:3], table=shared[2:17].view(3, 5)), -1)]:
        assert _tables(**kw) == rc, kw
    with pytest.raises(pd.PagedDecodeError):
        pd.paged_batch_tables(i(3), i(2), i(3, 5), i(4), i(3), i(9), i(9), 16, 40)


def test_oracle_closed_form():
    table, start, lens, pos, slots, cursor = O.batch_tables(
        [0, 15, 16], [2, 2, 0], np.array([[-1, -1], [4, -1], [6, -1]]), 16, 5, 2, [9, 8, 7], 0, [0, 10, 0])
    assert table.tolist() == [[9, -1], [4, 8], [6, -1]] and cursor == 2
    assert start.tolist() == [0, 2, 4, 4] and lens.tolist() == [2, 17, 16]
    assert pos.tolist() == [[0, 1, 25, 26, 0]] * 2
    assert slots.tolist() == [144, 145, 4 * 16 + 15, 8 * 16, -1]


def test_batches_of_the_tests_fit():
    for S in (1, 31, 300):
        c, q, table, free, pages = batch(S, 16, S)
        got = O.batch_tables(c, q, table, 16, int(q.sum()), 1, free, 0)
        assert got[5] <= len(free) and len(set(got[4].tolist())) == int(q.sum())
