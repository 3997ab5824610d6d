"""Refusals of the step's calls, on the CPU: every argument that the host can check is
rejected before a device is touched, empty work is a no-op, and a valid call fails
closed without a device."""

import ctypes
import os

import pytest

import mxfp4_paged_cache_quant_amd as mx

OK, ERR_ARG, ERR_NO_DEVICE = 0, 1, 2
A, MIS = 0x10000, 0x10004       # aligned; aligned to 4 bytes only
ODD = 0x10002


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.lib_path):
        from mxfp4_paged_cache_quant_amd import build
        build.build()
    return mx.lib()


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def _args(base, **change):
    d = dict(base)
    for k in change:
        assert k in d, k
    d.update(change)
    return list(d.values())


MAP = dict(seq_lens=A, query_lens=A, B=4, table=A, stride=8, pages=8, free=A, num_free=16, start=A,
           next=A + 64, page=64, columns=0, rows=10, slots=A, pos=A, seq=A, ks=A, ke=A, cu=A, stream=None)


@pytest.mark.parametrize("change", [
    dict(page=32), dict(B=-1), dict(B=65536), dict(rows=-1), dict(rows=1 << 31), dict(num_free=-1),
    dict(pages=-1), dict(stride=7), dict(columns=2), dict(columns=-1), dict(seq_lens=None),
    dict(query_lens=None), dict(seq_lens=ODD), dict(query_lens=ODD), dict(table=None),
    dict(table=ODD), dict(free=ODD), dict(start=None), dict(start=MIS), dict(next=A),
    dict(next=MIS), dict(slots=MIS), dict(pos=MIS), dict(seq=ODD), dict(ks=ODD), dict(ke=ODD),
    dict(cu=MIS), dict(free=None)])
def test_step_map_refuses(L, change):
    assert L.idx_step_map(*_args(MAP, **change)) == ERR_ARG


def test_step_map_empty_and_no_device(L):
    assert L.idx_step_map(*_args(MAP, rows=0, next=None, cu=None)) == OK
    if _no_gpu():
        assert L.idx_step_map(*_args(MAP)) == ERR_NO_DEVICE
        assert L.idx_step_map(*_args(MAP, B=0, seq_lens=None, query_lens=None)) == ERR_NO_DEVICE
        assert L.idx_step_map(*_args(MAP, free=None, num_free=0, start=None)) == ERR_NO_DEVICE


def _heads(**change):
    d = dict(x=A, out=A, row_stride=256, head_stride=128, out_row_stride=256, out_head_stride=128,
             heads=2, norm=1, weight=A, bias=None, eps=1e-6)
    d.update(change)
    return mx._Heads(*d.values())


def _rope(**change):
    d = dict(cos=A, sin=A, rows=64, positions=A, dim=64, mode=0)
    d.update(change)
    return mx._Rope(*d.values())


def _norm(L, q=None, k=None, dtype=0, T=4, rope=None):
    rope = _rope() if rope is None else rope
    return L.idx_norm_rope(None if q is None else ctypes.addressof(q),
                           None if k is None else ctypes.addressof(k), dtype, T,
                           ctypes.addressof(rope) if rope else None, None)


@pytest.mark.parametrize("change", [
    dict(heads=-1), dict(norm=3), dict(norm=-1), dict(x=None), dict(x=MIS), dict(out=None),
    dict(out=MIS), dict(row_stride=127), dict(row_stride=132), dict(head_stride=64),
    dict(out_row_stride=100), dict(out_head_stride=130), dict(weight=MIS), dict(bias=MIS),
    dict(eps=-1.0), dict(eps=float("nan")), dict(heads=1 << 21)])
def test_norm_rope_refuses_rows(L, change):
    assert _norm(L, q=_heads(**change)) == ERR_ARG
    assert _norm(L, k=_heads(**change)) == ERR_ARG


def test_norm_rope_refuses(L):
    h = _heads()
    assert _norm(L, q=h, dtype=2) == ERR_ARG
    assert _norm(L, q=h, T=-1) == ERR_ARG
    assert L.idx_norm_rope(ctypes.addressof(h), None, 0, 4, None, None) == ERR_ARG   # no rope block
    for change in (dict(dim=8), dict(dim=144), dict(dim=-16), dict(mode=2), dict(rows=-1),
                   dict(cos=None), dict(sin=MIS), dict(positions=MIS),
                   dict(positions=None, rows=3)):
        assert _norm(L, q=h, rope=_rope(**change)) == ERR_ARG, change
    assert _norm(L, q=_heads(row_stride=130), dtype=1) == ERR_ARG     # fp32: a multiple of 4
    assert _norm(L, q=h, T=0) == OK
    assert _norm(L) == OK
    assert _norm(L, q=_heads(heads=0), k=_heads(heads=0, x=None)) == OK
    if _no_gpu():
        assert _norm(L, q=h, k=_heads(weight=None, norm=2)) == ERR_NO_DEVICE
        # one row: its strides are not used
        assert _norm(L, q=_heads(heads=1, row_stride=1, head_stride=1, out_row_stride=1,
                                 out_head_stride=1), T=1) == ERR_NO_DEVICE


LATENT = dict(kv=A, dtype=0, T=4, stride=640, latent=512, norm=1, weight=A, eps=1e-6, rope=None,
              slots=A, cache=A, pages=8, page=64, q_pe=A, H=2, qs=256, qh=128, q_out=2 * A, os=1152,
              oh=576, stream=None)


def _latent(L, rope=None, **change):
    rope = _rope() if rope is None else rope
    return L.idx_latent_insert(*_args(LATENT, rope=ctypes.addressof(rope), **change))


@pytest.mark.parametrize("change", [
    dict(kv=None), dict(kv=MIS), dict(dtype=2), dict(T=-1), dict(T=1 << 40), dict(stride=575),
    dict(stride=580), dict(latent=64), dict(latent=384), dict(norm=2), dict(norm=-1),
    dict(weight=MIS), dict(eps=-1.0), dict(slots=None), dict(slots=MIS), dict(cache=None),
    dict(cache=A + 8), dict(pages=-1), dict(page=16), dict(q_pe=MIS), dict(H=-1), dict(qs=63),
    dict(qh=60), dict(qs=260), dict(q_out=None), dict(q_out=MIS), dict(os=63), dict(oh=68),
    dict(T=1 << 25, H=128)])
def test_latent_insert_refuses(L, change):
    assert _latent(L, **change) == ERR_ARG


@pytest.mark.parametrize("rows,heads", [(1 << 26, 2), ((1 << 20) + 1, 127), (1 << 7, 1 << 20)])
def test_norm_rope_refuses_more_lanes_than_a_launch_has(L, rows, heads):
    # rows * (heads + 1) rows of 16 lanes each: past 2^31 lanes
    assert _norm(L, q=_heads(heads=heads), k=_heads(heads=1), T=rows) == ERR_ARG


def test_latent_insert_and_attn_refuse_more_lanes_than_a_launch_has(L):
    assert _latent(L, T=(1 << 24) + 1, q_pe=None, H=0) == ERR_ARG
    assert _latent(L, T=1 << 24, H=17) == ERR_ARG
    assert L.idx_attn_paged(*_args(ATTN, rows=(1 << 22) + 1)) == ERR_ARG
    if _no_gpu():
        assert _latent(L, T=1 << 24, H=16, qs=1024, qh=64) == ERR_NO_DEVICE
        assert L.idx_attn_paged(*_args(ATTN, rows=1 << 22)) == ERR_NO_DEVICE
        assert _norm(L, q=_heads(), k=_heads(heads=1), T=(1 << 27) // 3) == ERR_NO_DEVICE


def test_in_place_needs_the_same_strides(L):
    for change in (dict(out_row_stride=512), dict(out_head_stride=256)):
        assert _norm(L, q=_heads(**change)) == ERR_ARG
        assert _norm(L, k=_heads(**change)) == ERR_ARG
    same = dict(q_out=A, os=256, oh=128)
    for change in (dict(os=512), dict(oh=64), dict(dtype=1)):
        assert _latent(L, **{**same, **change}) == ERR_ARG
    if _no_gpu():
        assert _norm(L, q=_heads(out_row_stride=512, out=2 * A)) == ERR_NO_DEVICE
        assert _norm(L, q=_heads(out_row_stride=512), T=1) == ERR_NO_DEVICE
        assert _latent(L, **same) == ERR_NO_DEVICE


@pytest.mark.parametrize("k", [(1 << 31) - 1, (1 << 31) - 64, 0x7ffffe01])
def test_attn_refuses_places_past_32_bits(L, k):
    # tiles behind the last place are counted in 32 bits too
    assert L.idx_attn_paged(*_args(ATTN, k=k, idx_stride=k, ws=None, wb=0)) == ERR_ARG
    assert L.idx_attn_paged(*_args(ATTN, most=k, idx=None, bt=1 << 26, ws=None, wb=0)) == ERR_ARG
    assert L.idx_attn_workspace_bytes(4, 2, 512, k) == 0


def test_latent_insert_rope_and_empty(L):
    for change in (dict(dim=0), dict(dim=128), dict(mode=5), dict(cos=None), dict(positions=MIS),
                   dict(positions=None, rows=3)):
        assert _latent(L, rope=_rope(**change)) == ERR_ARG, change
    assert _latent(L, T=0) == OK
    if _no_gpu():
        assert _latent(L) == ERR_NO_DEVICE
        assert _latent(L, q_pe=None, H=0, q_out=None) == ERR_NO_DEVICE
        assert _latent(L, norm=0, weight=MIS) == ERR_NO_DEVICE      # not read
        assert _latent(L, pages=0, cache=None) == ERR_NO_DEVICE     # every slot is outside


ATTN = dict(q=A, qs=2 * 576, qh=576, rows=4, H=2, latent=512, cache=A, pages=8, page=64, table=A,
            bt=16, B=2, seq=A, ks=A, ke=A, idx=A, idx_stride=32, k=32, most=1000, scale=0.1, out=A,
            os=1024, oh=512, lse=A, ws=0x20000, wb=1 << 40, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=MIS), dict(qs=575), dict(qh=570), dict(qh=580), dict(rows=-1), dict(rows=1 << 26),
    dict(H=0), dict(H=129), dict(latent=64), dict(latent=576), dict(cache=None), dict(cache=A + 8),
    dict(pages=-1), dict(page=32), dict(table=None), dict(table=ODD), dict(bt=15), dict(B=-1),
    dict(seq=ODD), dict(seq=None, rows=3), dict(ks=ODD), dict(ke=None), dict(ke=ODD), dict(idx=ODD),
    dict(idx_stride=31), dict(k=-1), dict(most=-1), dict(most=1 << 31), dict(out=None),
    dict(out=A + 4), dict(os=511), dict(oh=510), dict(oh=514), dict(lse=ODD)])
def test_attn_refuses(L, change):
    assert L.idx_attn_paged(*_args(ATTN, **change)) == ERR_ARG


def test_attn_workspace(L):
    for bad in ((-1, 8, 512, 100), (4, 0, 512, 100), (4, 129, 512, 100), (4, 8, 500, 100),
                (4, 8, 512, -1)):
        assert L.idx_attn_workspace_bytes(*bad) == 0
    need = L.idx_attn_workspace_bytes(4, 2, 512, 32)
    if need:
        for change in (dict(ws=None), dict(ws=0x20010), dict(wb=need - 1)):
            assert L.idx_attn_paged(*_args(ATTN, **change)) == ERR_ARG
    assert L.idx_attn_paged(*_args(ATTN, rows=0, q=None)) == OK
    assert L.idx_attn_paged(*_args(ATTN, B=0)) == OK
    if _no_gpu():
        assert L.idx_attn_paged(*_args(ATTN)) == ERR_NO_DEVICE
        assert L.idx_attn_paged(*_args(ATTN, seq=None, ks=None, idx=None, lse=None)) == ERR_NO_DEVICE
        assert L.idx_attn_paged(*_args(ATTN, most=0, table=None, pages=0, cache=None)) == ERR_NO_DEVICE


# sizes whose rows are split over the tokens: the partial sums need the workspace
SPLIT = [dict(k=2048, idx_stride=2048), dict(idx=None, most=1000), dict(k=2048, idx_stride=2048, H=64, qs=64 * 576, os=64 * 512)]


@pytest.mark.parametrize("sizes", SPLIT)
def test_attn_refuses_a_workspace_that_does_not_hold_the_partial_sums(L, sizes):
    call = {**ATTN, **sizes}
    need = L.idx_attn_workspace_bytes(call["rows"], call["H"], call["latent"],
                                      call["k"] if call["idx"] else call["most"])
    assert need > 0
    for change in (dict(ws=None), dict(ws=0x20010), dict(ws=0x20080), dict(wb=need - 1), dict(wb=0)):
        assert L.idx_attn_paged(*_args(call, **change)) == ERR_ARG, change
    if _no_gpu():
        assert L.idx_attn_paged(*_args(call, wb=need)) == ERR_NO_DEVICE


@pytest.mark.parametrize("latent", [128, 256, 512])
def test_attn_workspace_of_the_largest_call_holds_the_smaller_ones(L, latent):
    rows = [1, 2, 3, 7, 16, 33, 64, 128, 129, 200, 256, 257, 512, 1024, 5000]
    heads = [1, 8, 16, 17, 32, 33, 64, 65, 96, 128]
    entries = [0, 1, 64, 65, 128, 129, 192, 256, 257, 1000, 2048, 8192, 40000, 131072, 1 << 30]
    most, size = L.idx_attn_workspace_max_bytes, {}
    for r in rows:
        for h in heads:
            for e in entries:
                size[r, h, e] = L.idx_attn_workspace_bytes(r, h, latent, e)
                assert size[r, h, e] <= most(r, h, latent, e), (r, h, e)
    for r in rows:                       # and it grows with each of them
        for h in heads:
            for e0, e1 in zip(entries, entries[1:]):
                assert most(r, h, latent, e0) <= most(r, h, latent, e1)
    for r0, r1 in zip(rows, rows[1:]):
        assert all(most(r0, h, latent, e) <= most(r1, h, latent, e) for h in heads for e in entries)
    for h0, h1 in zip(heads, heads[1:]):
        assert all(most(r, h0, latent, e) <= most(r, h1, latent, e) for r in rows for e in entries)
    assert max(most(r, h, latent, e) for r in rows for h in heads for e in entries) < 34 << 20
    # what a program keeps for its largest batch serves every batch
    kept = mx.attn_workspace(256, 64, latent, 2048, device="cpu").numel()
    assert kept >= max(size[r, h, e] for r, h, e in size if r <= 256 and h <= 64 and e <= 2048)
    for bad in ((-1, 8, latent, 100), (4, 0, latent, 100), (4, 8, 500, 100), (4, 8, latent, -1)):
        assert most(*bad) == 0


def test_wrappers_refuse_host_tensors():
    import torch
    z = torch.zeros
    with pytest.raises(mx.MxidxError):
        mx.step_map(z(2, dtype=torch.int32), z(2, dtype=torch.int32), z((2, 2), dtype=torch.int32), 4)
    with pytest.raises(mx.MxidxError):
        mx.norm_rope(z((2, 2, 128)), None, z((4, 32)), z((4, 32)), 64)
    with pytest.raises(mx.MxidxError):
        mx.norm_rope(None, None, z((4, 32)), z((4, 32)), 64)
    with pytest.raises(mx.MxidxError):
        mx.latent_insert(z((2, 576)), z(2, dtype=torch.int64), z((1, 64, 576), dtype=torch.bfloat16),
                         z((4, 32)), z((4, 32)))
    with pytest.raises(mx.MxidxError):
        mx.attn_paged(z((2, 2, 576), dtype=torch.bfloat16), z((1, 64, 576), dtype=torch.bfloat16),
                      z((2, 1), dtype=torch.int32), z(2, dtype=torch.int32), 0.1)
