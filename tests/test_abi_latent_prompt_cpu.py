"""Refusals of the 4-bit latent cache's and the prompts' calls, on the CPU: every argument that the
host can check is rejected before a device is touched, empty work is a no-op, a valid call fails
closed without a device, and one workspace holds every call."""

import ctypes
import os

import pytest
import torch

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


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


def _args(base, **change):
    d = dict(base)
    for k in change:
        assert k in d, k
    d.update(change)
    return list(d.values())


def _rope(**change):
    d = dict(cos=A, sin=A, rows=64, positions=A, dim=64, mode=0)
    d.update(change)
    return mx._Rope(*d.values())


INSERT = dict(kv=A, dtype=0, T=4, stride=640, latent=512, norm=1, weight=A, eps=1e-6, rope=None, slots=A,
              cache=A, pages=8, page=64, q_pe=A, H=2, qs=256, qh=128, q_out=2 * A, os=1152, oh=576, stream=None)


def _insert(L, rope=None, **change):
    rope = _rope() if rope is None else rope
    return L.idx_latent_insert_mxfp4(*_args(INSERT, rope=ctypes.addressof(rope), **change))


@pytest.mark.parametrize("change", [
    dict(kv=None), dict(kv=MIS), dict(dtype=2), dict(T=-1), dict(T=(1 << 24) + 1), dict(stride=575), dict(stride=580),
    dict(latent=64), dict(latent=384), dict(norm=2), dict(norm=-1), dict(weight=MIS), dict(eps=-1.0),
    dict(eps=float("nan")), dict(slots=None), dict(slots=MIS), dict(cache=None), dict(cache=A + 8), dict(pages=-1),
    dict(page=16), dict(q_pe=MIS), dict(H=-1), dict(qs=63), dict(qh=60), dict(q_out=None), dict(q_out=MIS), dict(os=63),
    dict(oh=68), dict(T=1 << 24, H=17), dict(q_out=A)])
def test_insert_refuses(L, change):
    assert _insert(L, **change) == ERR_ARG


def test_insert_rope_and_empty(L):
    for change in (dict(dim=0), dict(dim=128), dict(mode=5), dict(cos=None), dict(positions=MIS), dict(positions=None, rows=3)):
        assert _insert(L, rope=_rope(**change)) == ERR_ARG, change
    assert _insert(L, T=0) == OK


@no_gpu
def test_insert_without_a_device(L):
    assert _insert(L) == ERR_NO_DEVICE
    assert _insert(L, eps=0.0, norm=0, weight=MIS) == ERR_NO_DEVICE        # the weight is not read
    assert _insert(L, pages=0, cache=None, q_pe=None, H=0, q_out=None) == ERR_NO_DEVICE


GATHER = dict(cache=A, pages=8, page=64, latent=256, table=A, bt=4, lens=A, cu=A, batch=3, most=256, total=100, out=A,
              stride=320, stream=None)


@pytest.mark.parametrize("change", [
    dict(cache=None), dict(cache=A + 8), dict(pages=-1), dict(page=32), dict(latent=100), dict(table=None), dict(table=ODD),
    dict(bt=3), dict(lens=None), dict(lens=ODD), dict(cu=None), dict(cu=MIS), dict(batch=-1), dict(batch=65536),
    dict(most=-1), dict(most=(1 << 29) + 1, bt=1 << 30), dict(total=-1), dict(out=None), dict(out=A + 8), dict(stride=319),
    dict(stride=324)])
def test_gather_refuses(L, change):
    assert L.idx_latent_gather_mxfp4(*_args(GATHER, **change)) == ERR_ARG


def test_gather_empty(L):
    for change in (dict(batch=0), dict(most=0), dict(total=0), dict(pages=0)):
        assert L.idx_latent_gather_mxfp4(*_args(GATHER, **change, out=None)) == OK


@no_gpu
def test_gather_without_a_device(L):
    assert L.idx_latent_gather_mxfp4(*_args(GATHER)) == ERR_NO_DEVICE
    assert L.idx_latent_gather_mxfp4(*_args(GATHER, total=1, stride=0)) == ERR_NO_DEVICE


ATTN = dict(q=A, qs=2 * 576, qh=576, rows=4, H=2, latent=512, cache=A, pages=8, page=64, table=A, bt=16, B=2, seq=A,
            ks=A, ke=A, idx=A, idx_stride=32, k=32, most=1000, scale=0.1, out=A, os=1024, oh=512, lse=A, ws=0x20000,
            wb=1 << 40, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=MIS), dict(qs=575), dict(qh=580), dict(rows=-1), dict(rows=(1 << 22) + 1), dict(H=0), dict(H=129),
    dict(latent=64), dict(cache=None), dict(cache=A + 8), dict(pages=-1), dict(pages=1 << 26), dict(page=32),
    dict(table=None), dict(bt=15), dict(B=-1), dict(seq=ODD), dict(seq=None, rows=3), dict(ks=ODD), dict(ke=None),
    dict(idx=ODD), dict(idx_stride=31), dict(k=-1), dict(most=-1), dict(most=1 << 31), dict(out=None), dict(out=A + 4),
    dict(os=511), dict(oh=514), dict(lse=ODD)])
def test_attn_refuses(L, change):
    assert L.idx_attn_paged_mxfp4(*_args(ATTN, **change)) == ERR_ARG


@pytest.mark.parametrize("sizes", [dict(k=2048, idx_stride=2048), dict(idx=None, most=1000)])
def test_attn_refuses_a_workspace_that_does_not_hold_the_partial_sums(L, sizes):
    call = {**ATTN, **sizes}
    need = L.idx_attn_workspace_bytes(call["rows"], call["H"], call["latent"], call["k"] if call["idx"] else call["most"])
    assert need > 0
    for change in (dict(ws=None), dict(ws=0x20010), dict(wb=need - 1), dict(wb=0)):
        assert L.idx_attn_paged_mxfp4(*_args(call, **change)) == ERR_ARG, change


def test_attn_empty(L):
    assert L.idx_attn_paged_mxfp4(*_args(ATTN, rows=0, q=None)) == OK
    assert L.idx_attn_paged_mxfp4(*_args(ATTN, B=0)) == OK


@no_gpu
def test_attn_without_a_device(L):
    assert L.idx_attn_paged_mxfp4(*_args(ATTN)) == ERR_NO_DEVICE
    assert L.idx_attn_paged_mxfp4(*_args(ATTN, most=0, table=None, pages=0, cache=None)) == ERR_NO_DEVICE


PROMPT = dict(q=A, qs=512, qh=128, T=10, Hq=4, k=A, ks=256, kh=128, v=A, vs=256, vh=128, S=300, Hk=2, dk=128, dv=128,
              seq=A, new=A, B=3, most=300, causal=1, scale=0.1, out=A, os=512, oh=128, lse=A, ws=0x20000, wb=1 << 40,
              stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=MIS), dict(qs=127), dict(qs=516), dict(qh=127), dict(qh=132), dict(T=-1), dict(T=(1 << 22) + 1),
    dict(Hq=0), dict(Hq=129), dict(Hq=5), dict(Hk=0), dict(Hk=-1), dict(k=None), dict(k=MIS), dict(ks=127), dict(ks=260),
    dict(kh=64), dict(ks=(1 << 23) + 8), dict(v=None), dict(v=MIS), dict(vs=127), dict(vs=260), dict(vh=64),
    dict(vs=(1 << 23) + 8), dict(S=-1), dict(dk=64), dict(dv=64), dict(dk=192, dv=192), dict(dk=96, dv=96), dict(seq=None),
    dict(seq=ODD), dict(new=None), dict(new=ODD), dict(B=-1), dict(B=65536), dict(most=-1), dict(most=1 << 31),
    dict(out=None), dict(out=A + 4), dict(os=127), dict(os=514), dict(oh=126), dict(lse=ODD)])
def test_prompt_refuses(L, change):
    assert L.idx_attn_prompt(*_args(PROMPT, **change)) == ERR_ARG


def test_prompt_workspace(L):
    need = L.idx_attn_prompt_workspace_bytes(10, 4, 2, 128, 128, 3, 300)
    assert need > 0
    for change in (dict(ws=None), dict(ws=0x20010), dict(wb=need - 1), dict(wb=0)):
        assert L.idx_attn_prompt(*_args(PROMPT, **change)) == ERR_ARG, change
    for bad in ((-1, 4, 2, 128, 128, 3, 300), (10, 5, 2, 128, 128, 3, 300), (10, 4, 2, 128, 64, 3, 300),
                (10, 4, 2, 128, 128, -1, 300), (10, 4, 2, 128, 128, 3, -1)):
        assert L.idx_attn_prompt_workspace_bytes(*bad) == 0
    # one buffer for every call, and none where the rows alone fill the card
    most = 0
    for T in (1, 2, 3, 7, 16, 61, 64, 244, 500, 1000, 4096, 16384, 100000, 1 << 22):
        for Hq, Hk in ((1, 1), (8, 1), (16, 2), (16, 16), (5, 1), (96, 4), (128, 1), (128, 128), (128, 2)):
            for B in (1, 2, 16, 64, 1000, 65535):
                for n in (1, 256, 257, 1000, 65536, 0x7ffffe00):
                    for dk, dv in mx.PROMPT_DIMS:
                        most = max(most, L.idx_attn_prompt_workspace_bytes(T, Hq, Hk, dk, dv, B, n))
    assert 0 < most <= mx.PROMPT_MAX_WORKSPACE
    assert L.idx_attn_prompt_workspace_bytes(16384, 16, 16, 192, 128, 1, 16384) == 0
    assert mx.attn_prompt_workspace("cpu").numel() == mx.PROMPT_MAX_WORKSPACE


def test_prompt_empty(L):
    assert L.idx_attn_prompt(*_args(PROMPT, T=0, q=None)) == OK
    assert L.idx_attn_prompt(*_args(PROMPT, B=0, seq=None, new=None)) == OK


@no_gpu
def test_prompt_without_a_device(L):
    assert L.idx_attn_prompt(*_args(PROMPT)) == ERR_NO_DEVICE
    assert L.idx_attn_prompt(*_args(PROMPT, S=0, k=None, v=None, causal=0, lse=None)) == ERR_NO_DEVICE
    assert L.idx_attn_prompt(*_args(PROMPT, T=1, qs=0, os=0, S=1, ks=0, vs=0)) == ERR_NO_DEVICE
    assert L.idx_attn_prompt(*_args(PROMPT, T=1 << 22, Hq=128, Hk=128, qs=1 << 14, os=1 << 14, ks=1 << 14, vs=1 << 14)) \
        == ERR_NO_DEVICE


def test_wrappers_refuse_host_tensors():
    z = torch.zeros
    bf = dict(dtype=torch.bfloat16)
    cache = z((1, 64 * mx.latent_mxfp4_row_bytes(512)), dtype=torch.uint8)
    with pytest.raises(mx.MxidxError):
        mx.latent_insert_mxfp4(z((2, 576)), z(2, dtype=torch.int64), cache, z((4, 32)), z((4, 32)))
    with pytest.raises(mx.MxidxError):
        mx.latent_gather_mxfp4(cache, z((2, 1), dtype=torch.int32), z(2, dtype=torch.int32), z(2, dtype=torch.int64), 64, 2)
    with pytest.raises(mx.MxidxError):
        mx.attn_paged_mxfp4(z((2, 2, 576), **bf), cache, z((2, 1), dtype=torch.int32), z(2, dtype=torch.int32), 0.1)
    with pytest.raises(mx.MxidxError):
        mx.attn_prompt(z((2, 2, 128), **bf), z((2, 2, 128), **bf), z((2, 2, 128), **bf), z(1, dtype=torch.int32),
                       z(1, dtype=torch.int32), 0.1)


def test_prompt_refuses_more_requests_than_a_workgroup_looks_through(L):
    assert L.idx_attn_prompt(*_args(PROMPT, B=1025)) == ERR_ARG
    assert L.idx_attn_prompt_workspace_bytes(10, 4, 2, 128, 128, 1025, 300) == 0
    assert L.idx_attn_prompt(*_args(PROMPT, B=1024, T=0)) == OK
