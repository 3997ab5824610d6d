"""Every size that perf/more_operators.py lists or draws is one that the calls take, on the CPU: with
addresses that hold them the calls fail for want of a device, not for an argument."""

import ctypes
import importlib.util
import os
import random

import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx

A, ERR_NO_DEVICE = 0x10000, 2
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.lib_path):
        from mxfp4_paged_cache_quant_amd import build
        build.build()
    return mx.lib()


@pytest.fixture(scope="module")
def cases():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _status(L, m, c):
    lens, latent = m._lengths(c), c.get("latent")
    if c["op"] == "prompt":
        lens, new = m._prompt_lengths(c)
        Hq, Hk, dk, dv = c["q_heads"], c["kv_heads"], c["dk"], c["dv"]
        row = Hk * (dk + dv)
        return L.idx_attn_prompt(A, Hq * dk, dk, sum(new) + c["spare"], Hq, A, row, dk + dv, A, row, dk + dv, sum(lens), Hk,
                                 dk, dv, A, A, len(lens), max(lens), int(c["causal"]), 0.1, A, Hq * dv, dv, A, A,
                                 mx.PROMPT_MAX_WORKSPACE, None)
    if c["op"] == "attn":
        rows, H, k, most = len(lens) * c["rows"], c["heads"], c["k"], max(lens)
        size = mx.attn_workspace_max_bytes(rows, H, latent, k or most)
        return L.idx_attn_paged_mxfp4(A, H * (latent + 64), latent + 64, rows, H, latent, A, 1 << 20, 64, A, (most + 63) // 64,
                                      len(lens), A, A, A, A if k else None, k, k, most, 0.1, A, H * latent, latent, A,
                                      A if size else None, size, None)
    if c["op"] == "write":
        T, H = sum(lens) + c["padded"], c["heads"]
        rope = mx._Rope(A, A, 1 << 30, A, 64, 0)
        return L.idx_latent_insert_mxfp4(A, 0 if c["dtype"] == "bf16" else 1, T, latent + 64, latent, 1, A, 1e-6,
                                         ctypes.addressof(rope), A, A, 1 << 20, 64, A if H else None, H, H * 64, 64,
                                         2 * A if H else None, H * (latent + 64), latent + 64, None)
    return L.idx_latent_gather_mxfp4(A, 1 << 20, 64, latent, A, (max(lens) + 63) // 64, A, A, len(lens), max(lens), sum(lens),
                                     A, latent + 64, None)


def test_listed_and_drawn_sizes_are_taken(L, cases):
    for c in cases.listed() + [cases.draw(random.Random(seed)) for seed in range(2000)]:
        assert _status(L, cases, c) == ERR_NO_DEVICE, c
