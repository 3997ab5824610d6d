"""GPU parity of idx_attn_paged in each of its forms (heads a workgroup, tile, split or whole,
32-bit places or row numbers) against the float64 oracle: what the forms must have in
common.  Tolerances: oracle/latent_attn.py."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
from oracle import latent_attn as oattn
from tests.gpu_helpers import dev
from tests.test_gpu_attn_paged import _bf16, _case, _close, _to_dev

pytestmark = pytest.mark.gpu

# A weight's rounding to bf16 leaves at most 2^-8 of it, and rounding that leaves 2^-8 of what is left.
TWO_PARTS = 2.0 ** -16


def _rows_close(got, c, next_n, pick, what=""):
    """Rows `pick` of a call against the oracle, the weights' rounding taken as that of two parts."""
    part = dict(c, q=c["q"][pick], ke=c["ke"][pick], row_seq=(pick // next_n).astype(np.int32))
    for name in ("indices", "ks"):
        part[name] = None if c[name] is None else c[name][pick]
    _close((got[0][dev(pick)], got[1][dev(pick)]),
           oattn.attn(part["q"], part["cache"], part["bt"], part["ke"], part["scale"], part["indices"], part["ks"],
                      part["row_seq"], weight_rounding=TWO_PARTS), what)


# 64 heads a workgroup: 32-token tiles, 64-token tiles, and those with the tokens split
@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("rows,H,n", [(520, 64, 300), (260, 128, 500), (300, 64, 200), (60, 128, 1400)])
@pytest.mark.parametrize("k", [0, 600])
def test_weights_of_many_rows_in_two_parts(latent, rows, H, n, k):
    next_n = rows // 5 if rows % 5 == 0 else rows // 2
    c = _case(rows + n, [n] * (rows // next_n), next_n=next_n, H=H, latent=latent, k=k, q_scale=0.5)
    got = mx.attn_paged(**_to_dev(c, float("nan")))
    torch.cuda.synchronize()
    _rows_close(got, c, next_n, np.arange(0, rows, 17))


@pytest.mark.parametrize("rows,H", [(3, 16), (3, 32), (140, 128), (520, 64)])
@pytest.mark.parametrize("lift", [3.3, 5.1, 7.9])
def test_one_late_token_outweighs_the_others(rows, H, lift):
    # the last token, in a later tile than the first, is about 2^lift times as heavy as each other,
    # which is no power of two and does not raise the reference: its weight must not round the output
    latent, n = 128, 100
    c = _case(rows, [n], next_n=rows, H=H, latent=latent, q_scale=0.05)
    c["ke"][:] = n
    c["q"][:, :, latent] = 8.0
    c["cache"][..., latent] = 0.0
    c["cache"][c["bt"][0, (n - 1) // 64], (n - 1) % 64, latent] = lift * np.log(2.0) / (8.0 * c["scale"])
    c["cache"] = _bf16(c["cache"])
    got = mx.attn_paged(**_to_dev(c, float("nan")))
    torch.cuda.synchronize()
    _rows_close(got, c, rows, np.unique(np.linspace(0, rows - 1, 7).astype(np.int64)))


# rows of one sequence x heads -> 16, 32 and 64 heads a workgroup, the last with 64- and 32-token tiles and
# with the tokens split
FORMS = [(3, 12), (200, 16), (3, 32), (200, 30), (130, 128), (520, 64), (60, 128)]


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("over", [0, 1])
@pytest.mark.parametrize("rows,H", FORMS)
@pytest.mark.parametrize("k", [0, 600])
def test_rows_on_both_sides_of_2_and_4_gib(latent, over, rows, H, k):
    # the largest cache whose rows 32-bit offsets reach, and one page more: pages around byte 2^31
    # (one of whose rows begins 128 bytes below it), the last ones and others; NaN in all the rest
    page_bytes = 64 * (latent + 64) * 2
    pages = 0xfffe0000 // page_bytes + over
    middle = (1 << 31) // page_bytes
    used = np.array([pages - 1, 0, middle, middle + 1, middle - 1, pages - 2, 1, pages // 3], np.int32)
    n = 500 if rows > 60 else 1400
    used = np.concatenate([used, np.arange(10, 10 + 22 - len(used), dtype=np.int32)])[:(n + 63) // 64]
    c = _case(rows + H, [n], next_n=rows, H=H, latent=latent, k=k, q_scale=0.5)
    d = _to_dev(c)
    d["cache"] = torch.full((pages, 64, latent + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    vals = torch.from_numpy(c["cache"][c["bt"][0]]).to(torch.bfloat16).cuda()
    d["cache"][torch.from_numpy(used.astype(np.int64)).cuda()] = vals
    d["block_table"] = dev(used[None])
    got = mx.attn_paged(**d)
    torch.cuda.synchronize()
    _rows_close(got, c, rows, np.unique(np.linspace(0, rows - 1, 9).astype(np.int64)))


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("H", [5, 16, 17, 32])
@pytest.mark.parametrize("n,k", [(1100, 0), (1100, 700), (70, 0), (2100, 2048)])
def test_prefill_of_few_heads(latent, H, n, k):
    # whole rows of up to 33 tiles in groups of 16 and 32 heads: more rows than workgroups that rows are split for
    c = _case(H + n, [n, n - 3], next_n=260, H=H, latent=latent, k=k, q_scale=0.5, gathered=True)
    assert mx.attn_workspace_bytes(520, H, latent, k or c["bt"].shape[1] * 64) == 0
    got = mx.attn_paged(**_to_dev(c, float("nan")))
    torch.cuda.synchronize()
    _rows_close(got, c, 260, np.array([0, 1, 129, 254, 259, 260, 300, 519]))
