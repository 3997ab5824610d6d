"""idx_attn_prompt takes up to 256 query heads (16 key heads of groups of 16), on the CPU: sizes beyond are
refused, and one workspace holds every call."""

import os

import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
from tests.test_abi_latent_prompt_cpu import ERR_ARG, ERR_NO_DEVICE, PROMPT, _args

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.lib_path):
        from mxfp4_paged_cache_quant_amd import build
        build.build()
    return mx.lib()


@no_gpu
@pytest.mark.parametrize("Hq,Hk", [(129, 1), (144, 16), (256, 1), (256, 16), (256, 128), (256, 256)])
def test_heads_that_are_taken(L, Hq, Hk):
    wide = dict(Hq=Hq, Hk=Hk, qs=Hq * 128, os=Hq * 128, ks=Hk * 128, vs=Hk * 128)
    assert L.idx_attn_prompt(*_args(PROMPT, **wide)) == ERR_NO_DEVICE
    assert L.idx_attn_prompt(*_args(PROMPT, **wide, T=16384, S=16384, most=16384, B=4)) == ERR_NO_DEVICE


def test_heads_that_are_not(L):
    for Hq, Hk in ((257, 1), (512, 2), (256, 15), (256, 512), (0, 1), (-256, 16)):
        assert L.idx_attn_prompt(*_args(PROMPT, Hq=Hq, Hk=Hk, qs=1 << 17, os=1 << 17, ks=1 << 17, vs=1 << 17)) == ERR_ARG
        assert L.idx_attn_prompt_workspace_bytes(10, Hq, Hk, 128, 128, 3, 300) == 0


def test_one_workspace_holds_every_call(L):
    most = 0
    for T in (1, 2, 5, 16, 64, 244, 1000, 4096, 1 << 20):
        for Hq, Hk in ((129, 1), (160, 20), (200, 8), (256, 1), (256, 2), (256, 16), (256, 128), (256, 256)):
            for B in (1, 2, 16, 1024):
                for n in (1, 257, 65536, 0x7ffffe00):
                    for dk, dv in mx.PROMPT_DIMS:
                        most = max(most, L.idx_attn_prompt_workspace_bytes(T, Hq, Hk, dk, dv, B, n))
    assert 0 < most <= mx.PROMPT_MAX_WORKSPACE
