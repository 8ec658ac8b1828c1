"""paged_batch_tables against its oracle, through the C ABI: whole numbers, so
equal."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import batch_tables as O
from step_cases import batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _i32(a, dev="cuda"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def _tables(c, q, table, P, pages, T, axes=1, free=None, cursor=0, delta=None, stride=0):
    S = len(c)
    t = dict(table=_i32(table), start=_i32(np.full(S + 1, 7)), lens=_i32(np.full(S, 7)),
             pos=torch.full((axes, T + stride), 7, dtype=torch.int32, device="cuda")[:, :T],
             slots=torch.full((T,), 7, dtype=torch.int32, device="cuda"), next=_i32([7]))
    pd.paged_batch_tables(_i32(c), _i32(q), t["table"], t["start"], t["lens"], t["pos"], t["slots"],
                          P, pages, free_pages=_i32(free) if free is not None else None,
                          cursor=_i32([cursor]), next_cursor=t["next"],
                          position_delta=_i32(delta) if delta is not None else None)
    torch.cuda.synchronize()
    return [t[k].cpu().numpy() for k in ("table", "start", "lens", "pos", "slots", "next")]


def _same(got, want):
    for name, a, b in zip(("table", "start", "lens", "positions", "slots", "next"), got, want):
        assert np.array_equal(a, np.atleast_1d(b) if name == "next" else b), name


@pytest.mark.parametrize("S,P,q_hi,pad,axes", [
    (1, 16, 1, 0, 1), (1, 16, 5000, 3, 3), (7, 48, 9, 0, 1), (31, 16, 1, 1, 4), (256, 16, 4, 40, 1),
    (1023, 32, 3, 0, 1), (1024, 1, 2, 5, 2), (1025, 16, 40, 0, 8), (3000, 784, 7, 100, 3),
    (70, 1056, 3000, 0, 1), (5000, 16, 1, 0, 1), (20000, 16, 3, 0, 1)])
def test_tables_match_the_oracle(S, P, q_hi, pad, axes):
    c, q, table, free, pages = batch(S, P, seed=S + q_hi, q_hi=q_hi, c_hi=900)
    T = int(q.sum()) + pad
    delta = np.random.default_rng(S).integers(-50, 50, S)
    want = O.batch_tables(c, q, table, P, T, axes, free, 0, delta)
    _same(_tables(c, q, table, P, pages, T, axes, free, 0, delta, stride=5), want)


@pytest.mark.parametrize("empty", [0.9, 1.0])
def test_tables_mostly_empty_requests(empty):
    c, q, table, free, pages = batch(4000, 16, seed=9, q_hi=700, empty=empty)
    T = int(q.sum()) + 1
    _same(_tables(c, q, table, 16, pages, T, 1, free), O.batch_tables(c, q, table, 16, T, 1, free))


def test_tables_without_a_free_list_read_the_pages_given():
    c, q, table, free, pages = batch(20, 16, seed=2, q_hi=60)
    T = int(q.sum()) + 2
    full = O.batch_tables(c, q, table, 16, T, 1, free, 0)[0]
    want = O.batch_tables(c, q, full, 16, T)
    got = _tables(c, q, full, 16, pages, T)
    _same(got[:5], want[:5])
    assert got[5][0] == 0  # the cursor as it was


def test_tables_of_a_wider_table_and_without_cursors():
    """Rows inside a wider table (its other entries kept), positions as a
    vector, no cursors."""
    c, q, table, free, pages = batch(6, 16, seed=3, q_hi=30)
    T = int(q.sum())
    full = O.batch_tables(c, q, table, 16, T, 1, free, 0)[0]
    wide = torch.full((6, full.shape[1] + 9), 77, dtype=torch.int32, device="cuda")
    view = wide[:, 4:4 + full.shape[1]]
    view.copy_(_i32(full))
    before = wide.clone()
    start, lens, pos, slots = _i32(np.zeros(7)), _i32(np.zeros(6)), _i32(np.zeros(T)), _i32(np.zeros(T))
    pd.paged_batch_tables(_i32(c), _i32(q), view, start, lens, pos, slots, 16, pages)
    torch.cuda.synchronize()
    want = O.batch_tables(c, q, full, 16, T)
    assert torch.equal(wide, before)
    assert np.array_equal(pos.cpu().numpy(), want[3][0]) and np.array_equal(slots.cpu().numpy(), want[4])


def test_tables_empty_batches():
    got = _tables([], [], np.zeros((0, 3)), 16, 4, 5, free=[1, 2], cursor=1)
    _same(got, (np.zeros((0, 3)), [0], [], np.zeros((1, 5)), np.full(5, -1), 1))
    got = _tables([5, 0], [0, 0], np.array([[3, -1], [-1, -1]]), 16, 4, 0, free=[1, 2], cursor=2)
    _same(got, ([[3, -1], [-1, -1]], [0, 0, 0], [5, 0], np.zeros((1, 0)), [], 2))
    got = _tables([5, 0], [0, 0], np.array([[3, -1], [-1, -1]]), 16, 4, 2, free=[], cursor=0)
    _same(got, ([[3, -1], [-1, -1]], [0, 0, 0], [5, 0], np.zeros((1, 2)), [-1, -1], 0))


def test_tables_step_by_step_in_a_graph():
    """A captured step, replayed: its lengths become the next contexts, its
    cursor the next one."""
    S, P, W_, pages = 9, 16, 12, 120
    g = np.random.default_rng(4)
    q = g.integers(0, 20, S)
    T = int(q.sum()) + 4
    ctx, qd = _i32(np.zeros(S)), _i32(q)
    free = _i32(g.permutation(pages))
    cur, nxt = _i32([0]), _i32([0])
    table = _i32(np.full((S, W_), -1))
    start, lens, pos, slots = _i32(np.zeros(S + 1)), _i32(np.zeros(S)), _i32(np.zeros(T)), _i32(np.zeros(T))

    def step():
        pd.paged_batch_tables(ctx, qd, table, start, lens, pos, slots, P, pages, free_pages=free,
                              cursor=cur, next_cursor=nxt)
        ctx.copy_(lens)
        cur.copy_(nxt)

    step()
    ctx.zero_()
    cur.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    table.fill_(-1)
    want_t, c, cursor = np.full((S, W_), -1), np.zeros(S, dtype=int), 0
    for _ in range(9):
        graph.replay()
        want = O.batch_tables(c, q, want_t, P, T, 1, free.cpu().numpy(), cursor)
        torch.cuda.synchronize()
        _same([table.cpu().numpy(), start.cpu().numpy(), lens.cpu().numpy(), pos.cpu().numpy()[None],
               slots.cpu().numpy(), nxt.cpu().numpy()], want)
        want_t, c, cursor = want[0], want[2], want[5]


def _status():
    torch.cuda.synchronize()
    return pd.paged_decode_device_status(reset=True)


def test_tables_report_a_list_that_is_used_up():
    # request 0 needs 2 pages, request 1 needs 2; the list has 3 left
    got = _tables([0, 4], [20, 40], np.array([[-1] * 4, [9, -1, -1, -1]]), 16, 10, 60,
                  free=[8, 7, 6, 5], cursor=1)
    assert _status() == pd.DEV_NO_PAGE
    assert got[0].tolist() == [[7, 6, -1, -1], [9, 5, -1, -1]] and got[5][0] == 5
    slots = got[4]
    assert slots[:20].tolist() == [7 * 16 + i for i in range(16)] + [6 * 16 + i for i in range(4)]
    assert slots[20:32].tolist() == [9 * 16 + i for i in range(4, 16)]
    assert slots[32:48].tolist() == [5 * 16 + i for i in range(16)]
    assert (slots[48:] == -1).all() and got[2].tolist() == [20, 44]
    # a cursor before the list
    got = _tables([0], [3], np.array([[-1]]), 16, 10, 3, free=[4], cursor=-1)
    assert _status() == pd.DEV_NO_PAGE and got[4].tolist() == [-1, -1, -1] and got[0][0, 0] == -1


def test_tables_report_pages_outside_the_pool():
    got = _tables([0, 4, 17], [20, 1, 1], np.array([[-1, -1], [10, -1], [3, -7]]), 16, 10, 22,
                  free=[10, 2], cursor=0)
    assert _status() == pd.DEV_BAD_PAGE
    assert got[0].tolist() == [[-1, 2], [10, -1], [3, -7]]
    assert got[4].tolist() == [-1] * 16 + [32, 33, 34, 35] + [-1, -1]


def test_tables_report_bad_lengths():
    # past the table's row (2 pages of 16): cut off there
    got = _tables([30, 40], [5, 1], np.array([[1, 2], [3, 4]]), 16, 10, 6, free=[5, 6], cursor=0)
    assert _status() == pd.DEV_BAD_SEQLEN
    assert got[2].tolist() == [32, 32] and got[1].tolist() == [0, 5, 6] and got[5][0] == 0
    assert got[4].tolist() == [2 * 16 + 14, 2 * 16 + 15, -1, -1, -1, -1]
    # negative ones count as 0
    got = _tables([-3, 2], [2, -9], np.array([[1, 2], [3, 4]]), 16, 10, 2, free=[5, 6], cursor=0)
    assert _status() == pd.DEV_BAD_SEQLEN
    assert got[0].tolist() == [[5, 2], [3, 4]] and got[2].tolist() == [2, 2]
    assert got[1].tolist() == [0, 2, 2] and got[4].tolist() == [80, 81]
    # more tokens than rows: cut off, the requests behind get none
    got = _tables([0, 0, 0], [3, 30, 4], np.full((3, 3), -1), 16, 10, 22, free=list(range(9)), cursor=0)
    assert _status() == pd.DEV_BAD_QSTART
    assert got[1].tolist() == [0, 3, 22, 22] and got[2].tolist() == [3, 19, 0] and got[5][0] == 3
    assert got[0].tolist() == [[0, -1, -1], [1, 2, -1], [-1, -1, -1]]
    big = 2 ** 31 - 1
    got = _tables([0, 0, big], [big, big, big], np.full((3, 1), -1), 16, 10, 2, free=[3], cursor=0)
    assert _status() == pd.DEV_BAD_QSTART | pd.DEV_BAD_SEQLEN
    assert got[1].tolist() == [0, 2, 2, 2] and got[4].tolist() == [48, 49] and got[5][0] == 1
