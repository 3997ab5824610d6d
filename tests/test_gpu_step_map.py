"""GPU parity of idx_step_map against the oracle's loops: every output equal, for single
and many requests, requests without a row, pages entered in the middle of a step, a free list
that runs out, tables that are too narrow, padding and dropped rows, both column forms, and
captured into a graph."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
from oracle import step_map as omap
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


def _case(seed, B, longest, most_new, spare=3, cols=None, list_short=0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, B).astype(np.int32)
    new = np.minimum(lens, rng.integers(0, most_new + 1, B)).astype(np.int32)
    new[rng.random(B) < 0.2] = 0
    held, need = -(-(lens - new) // 64), -(-lens // 64)
    cols = (max(1, int(need.max()) if B else 1) + 1) if cols is None else cols
    table = rng.integers(0, 1 << 20, (B, cols)).astype(np.int32)
    table[rng.random((B, cols)) < 0.02] = -1
    entered = int((need - held).sum())
    free = rng.permutation(1 << 20)[:max(entered + 4 - list_short, 0)].astype(np.int32)
    return lens, new, table, free, int(new.sum()) + spare


def _check(lens, new, table, rows, free=None, start=0, columns="sequence", wide=False):
    want, after = omap.step_map(lens, new, table, rows, free, start, gathered=columns == "gathered")
    if wide:                        # a table that is part of a wider one: a row stride of its own
        whole = np.full((table.shape[0], table.shape[1] + 5), -7, np.int32)
        whole[:, :table.shape[1]] = table
        whole = dev(whole)
        bt = whole[:, :table.shape[1]]
    else:
        bt = dev(table)
    kw = {} if free is None else dict(free_pages=dev(free), free_start=dev(np.array([start], np.int64)))
    for _ in range(2):              # a call that is made again writes the same
        got = mx.step_map(dev(lens), dev(new), bt, rows, columns=columns, **kw)
        torch.cuda.synchronize()
        for name, w in want.items():
            g = host(getattr(got, name))
            assert g.dtype == w.dtype and np.array_equal(g, w), (name, np.argwhere(g != w)[:4].tolist())
        assert np.array_equal(host(bt), after)
    if wide:
        assert (host(whole)[:, table.shape[1]:] == -7).all()


@pytest.mark.parametrize("B,longest,most_new", [
    (1, 1, 1), (1, 300, 300), (2, 64, 64), (7, 200, 5), (63, 1000, 70), (64, 500, 3), (257, 700, 2),
    (300, 2000, 900), (1025, 90, 1)])
@pytest.mark.parametrize("columns", ["sequence", "gathered"])
def test_step_map(B, longest, most_new, columns):
    lens, new, table, free, rows = _case(B + longest, B, longest, most_new)
    _check(lens, new, table, rows, free, 2, columns, wide=B % 2 == 1)


def test_no_list_reads_the_table():
    lens, new, table, _, rows = _case(5, 40, 900, 200)
    _check(lens, new, table, rows)


def test_list_runs_out_and_empty_list():
    lens, new, table, free, rows = _case(6, 30, 900, 300, list_short=20)
    _check(lens, new, table, rows, free)
    _check(lens, new, table, rows, free[:0])
    _check(lens, new, table, rows, free, start=len(free) + 3)
    _check(lens, new, table, rows, free, start=-2)


def test_narrow_table_dropped_rows_and_no_rows():
    lens, new, table, free, rows = _case(7, 25, 900, 300, cols=4)
    _check(lens, new, table, rows, free, wide=True)
    # rows behind num_rows are dropped: their pages are entered in the count, not in the table
    lens, new, table, free, _ = _case(8, 25, 900, 300)
    n = int(new.sum()) // 2
    want, _ = omap.step_map(lens, new, table, n, free, 0)
    got = mx.step_map(dev(lens), dev(new), dev(table), n, dev(free), dev(np.zeros(1, np.int64)))
    torch.cuda.synchronize()
    for name, w in want.items():
        assert np.array_equal(host(getattr(got, name)), w), name
    _check(lens, new, table, 0)
    zero = np.zeros_like(new)
    _check(lens, zero, table, 300, free)


def test_no_requests():
    _check(np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 4), np.int32), 7)
    _check(np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 4), np.int32), 0,
           np.array([3], np.int32), 1)


def test_many_requests():
    rng = np.random.default_rng(9)
    B = 65535
    lens = rng.integers(1, 200, B).astype(np.int32)
    new = np.minimum(lens, rng.integers(0, 3, B)).astype(np.int32)
    table = rng.integers(0, 1 << 20, (B, 4)).astype(np.int32)
    _check(lens, new, table, int(new.sum()) + 50, rng.integers(0, 1 << 20, B).astype(np.int32), 0, "gathered")


@pytest.mark.parametrize("B,longest,most_new", [(3, 300000, 250000), (900, 1500, 1400), (2500, 700, 500)])
def test_many_rows(B, longest, most_new):
    # more rows than the workgroups take at once
    lens, new, table, free, _ = _case(B, B, longest, most_new)
    new[0], lens[0] = most_new, longest
    held, need = -(-(lens[0] - new[0]) // 64), -(-lens[0] // 64)
    table = np.pad(table, ((0, 0), (0, max(0, int(need) - table.shape[1]))))
    free = np.concatenate([free, np.arange(need - held, dtype=np.int32)])
    rows = int(new.sum()) + 300
    assert rows > 1024 * 256
    _check(lens, new, table, rows, free, 1, "gathered")


def test_negative_lengths_count_as_zero():
    lens = np.array([100, -5, 70, 30], np.int32)
    new = np.array([2, 3, -1, 30], np.int32)
    want, _ = omap.step_map([100, 0, 70, 30], [2, 0, 0, 30], np.zeros((4, 3), np.int32), 40)
    got = mx.step_map(dev(lens), dev(new), dev(np.zeros((4, 3), np.int32)), 40)
    torch.cuda.synchronize()
    assert np.array_equal(host(got.cu_seq_offsets), want["cu_seq_offsets"])
    # request 1 has new tokens that its length does not hold: they have rows, but no slot
    assert host(got.row_seq)[:36].tolist() == [0] * 2 + [1] * 3 + [3] * 30 + [-1]
    assert (host(got.slot_mapping)[2:5] == -1).all()
    assert np.array_equal(host(got.slot_mapping)[5:35], want["slot_mapping"][2:32])


def test_graph_replays_follow_the_lengths():
    B, cols, rows = 20, 12, 64
    rng = np.random.default_rng(10)
    lens = torch.empty(B, dtype=torch.int32, device="cuda")
    new = torch.empty(B, dtype=torch.int32, device="cuda")
    table = dev(rng.integers(0, 500, (B, cols)).astype(np.int32))
    free = dev(rng.permutation(500).astype(np.int32))
    start = torch.zeros(1, dtype=torch.int64, device="cuda")
    first = host(table).copy()

    def draw():
        n = rng.integers(0, 700, B).astype(np.int32)
        return n, np.minimum(n, rng.integers(0, 4, B)).astype(np.int32)

    a, b = draw()
    lens.copy_(dev(a)), new.copy_(dev(b))
    out = mx.step_map(lens, new, table, rows, free, start)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.step_map(lens, new, table, rows, free, start, **out._asdict())
    for rep in range(4):
        a, b = draw()
        lens.copy_(dev(a)), new.copy_(dev(b)), table.copy_(dev(first))
        start.fill_(rep)
        g.replay()
        torch.cuda.synchronize()
        want, after = omap.step_map(a, b, first, rows, host(free), rep)
        for name, w in want.items():
            assert np.array_equal(host(getattr(out, name)), w), (rep, name)
        assert np.array_equal(host(table), after), rep


def test_refusals_of_the_wrapper():
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, table = torch.ones(3, **i32), torch.zeros((3, 2), **i32)
    free, start = torch.zeros(4, **i32), torch.zeros(1, dtype=torch.int64, device="cuda")
    ok = dict(seq_lens=lens, query_lens=lens, block_table=table, num_rows=3, free_pages=free, free_start=start)
    mx.step_map(**ok)
    for change in (dict(query_lens=lens[:2]), dict(query_lens=lens.long()), dict(block_table=table[:2]),
                   dict(block_table=table.t()), dict(num_rows=-1), dict(free_start=None),
                   dict(free_pages=None), dict(free_next=start), dict(columns="rows"),
                   dict(ke=torch.zeros(4, **i32)), dict(slot_mapping=torch.zeros(3, **i32)),
                   dict(seq_lens=lens.cpu())):
        with pytest.raises(mx.MxidxError):
            mx.step_map(**{**ok, **change})
