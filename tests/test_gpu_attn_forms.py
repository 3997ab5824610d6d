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
