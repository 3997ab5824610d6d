"""idx_call on the CPU: the calls of a serving step by number, with their arguments in 8-byte words, answer
as the calls themselves; other counts, numbers and integers that do not fit are refused."""

import ctypes
import os
import struct

import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx

OK, ERR_ARG = 0, 1
A = 0x10000
CALLS = ["idx_step_map", "idx_norm_rope", "idx_latent_insert", "idx_latent_insert_mxfp4", "idx_latent_gather_mxfp4",
         "idx_attn_paged", "idx_attn_paged_mxfp4", "idx_attn_prompt"]


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.lib_path):
        from mxfp4_paged_cache_quant_amd import build
        build.build()
    return mx.lib()


GATHER = dict(cache=A, pages=8, page=64, latent=256, table=A, bt=4, lens=A, cu=A, batch=0, most=256, total=100, out=A,
              stride=320, stream=0)
PROMPT = dict(q=A, qs=512, qh=128, T=0, Hq=4, k=A, ks=256, kh=128, v=A, vs=256, vh=128, S=300, Hk=2, dk=128, dv=128,
              seq=A, new=A, B=3, most=300, causal=1, scale=0.1, out=A, os=512, oh=128, lse=A, ws=0x20000, wb=1 << 40, stream=0)


def _invoke(L, name, args):
    words = struct.pack("=" + "".join("d" if isinstance(a, float) else "q" for a in args), *args)
    return L.idx_call(L.idx_entry(name.encode()), words, len(args))


def test_entries(L):
    assert sorted(L.idx_entry(n.encode()) for n in CALLS) == list(range(len(CALLS)))
    assert L.idx_entry(b"idx_topk") == -1 and L.idx_entry(b"") == -1 and L.idx_entry(None) == -1
    for entry in (-1, len(CALLS), 1 << 20):
        assert L.idx_call(entry, bytes(8 * 14), 14) == ERR_ARG
    n = L.idx_entry(b"idx_latent_gather_mxfp4")
    assert L.idx_call(n, None, 14) == ERR_ARG
    for count in (0, 13, 15, -1):
        assert L.idx_call(n, bytes(8 * 15), count) == ERR_ARG
    for name in CALLS:
        assert L.idx_call(L.idx_entry(name.encode()), bytes(8 * 64), len(mx.EXPORTS[name][1])) in (OK, ERR_ARG)


@pytest.mark.parametrize("name,base", [("idx_latent_gather_mxfp4", GATHER), ("idx_attn_prompt", PROMPT)])
def test_answers_as_the_call(L, name, base):
    call = getattr(L, name)
    assert _invoke(L, name, list(base.values())) == call(*base.values()) == OK
    for key, value in base.items():
        for other in (-1, 7, 1 << 24):
            # device work, or what idx_call itself refuses
            if key in ("stream", "scale", "B", "batch") or (key, other) in (("T", 7), ("wb", -1)):
                continue
            args = list({**base, key: other}.values())
            assert _invoke(L, name, args) == call(*args), (key, other)


def test_integers_that_do_not_fit(L):
    # they would be taken modulo 2^32 (or as a size of their own) by the call
    for change in (dict(Hq=(1 << 32) + 4), dict(B=-(1 << 32)), dict(causal=1 << 31), dict(wb=-1)):
        assert _invoke(L, "idx_attn_prompt", list({**PROMPT, **change}.values())) == ERR_ARG, change


def test_wrapper_refuses_what_is_no_number(monkeypatch):
    device = torch.device("cpu", 0)
    monkeypatch.setattr(mx._torch()._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    for args in ([None] + list(GATHER.values())[1:-1], list(GATHER.values())[:-2] + [1.5], list(GATHER.values())[:-2],
                 list(GATHER.values())[:-2] + [1 << 64]):
        with pytest.raises(mx.MxidxError):
            mx._call("idx_latent_gather_mxfp4", device, None, *args)
