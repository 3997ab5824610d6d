"""Workspace sizes of the attention over the MXFP4 latent cache, on the CPU: none where its rows are not
split, else those of the attention over the bf16 cache, and the call asks for no more."""

import itertools
import os

import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
from tests.test_abi_latent_prompt_cpu import ATTN, ERR_ARG, ERR_NO_DEVICE, _args

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")

WHOLE = {128: 5, 256: 4, 512: 3}            # tiles of 64 tokens up to which a row is not split


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.lib_path):
        from mxfp4_paged_cache_quant_amd import build
        build.build()
    return mx.lib()


def test_sizes(L):
    for latent, rows, H in itertools.product((128, 256, 512), (0, 1, 3, 16, 100, 1024), (1, 8, 32, 64, 128)):
        for n in (0, 1, 64, 65, 192, 193, 256, 257, 320, 321, 2048, 131072):
            got, bf16 = mx.attn_workspace_bytes(rows, H, latent, n, mxfp4=True), mx.attn_workspace_bytes(rows, H, latent, n)
            assert got == (0 if n <= 64 * WHOLE[latent] else bf16), (latent, rows, H, n)
    assert mx.attn_workspace_bytes(1, 8, 512, 192) > 0
    for bad in ((-1, 2, 512, 32), (4, 0, 512, 32), (4, 129, 512, 32), (4, 2, 100, 32), (4, 2, 512, -1)):
        assert L.idx_attn_workspace_bytes_mxfp4(*bad) == 0


@no_gpu
@pytest.mark.parametrize("latent", [128, 256, 512])
def test_short_windows_need_no_workspace(L, latent):
    n = 64 * WHOLE[latent]
    base = dict(ATTN, latent=latent, qs=2 * 576, qh=576, ws=None, wb=0, bt=n // 64 + 1)
    for sizes in (dict(idx=None, most=n), dict(k=n, idx_stride=n, most=n), dict(idx=None, most=n, ws=0x20010)):
        assert L.idx_attn_paged_mxfp4(*_args(base, **sizes)) == ERR_NO_DEVICE, sizes
        assert L.idx_attn_paged(*_args(base, **sizes)) == ERR_ARG, sizes
    for sizes in (dict(idx=None, most=n + 1), dict(k=n + 1, idx_stride=n + 1, most=n)):
        assert L.idx_attn_paged_mxfp4(*_args(base, **sizes)) == ERR_ARG, sizes
