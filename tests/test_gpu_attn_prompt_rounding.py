"""idx_attn_prompt where the weights' rounding to bf16 does not average out: one token of the largest score
and thousands of equal lower ones, whose weight lies just beside the middle of two bf16 values, so that all
of them round the same way.  The output stays within the oracle's bound (the weights' rounding and the
output's own), and the statistics, which take the weights unrounded, within theirs."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
from oracle import prompt_attn as opa
from tests.gpu_helpers import host
from tests.test_gpu_attn_prompt import _args, _case, _close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("n,new,Hq,Hk", [(3000, 3, 4, 2), (3000, 200, 2, 2), (700, 700, 2, 1)])
@pytest.mark.parametrize("weight", [0.5 * (1 + 0.99 * 2.0 ** -8), 0.5 * (1 + 1.01 * 2.0 ** -8), 0.25 * (1 + 0.9 * 2.0 ** -8)])
def test_equal_weights_that_are_no_bf16(dims, n, new, Hq, Hk, weight):
    c = _case(n + new, [n], [new], Hq, Hk, dims)
    c["q"], c["k"] = np.zeros_like(c["q"]), np.zeros_like(c["k"])
    c["q"][..., 5], c["k"][3, :, 5] = 2.0, 1.0               # scores: 2 * scale for token 3, 0 for the others
    c["scale"] = float(np.float32(-0.5 * np.log(weight)))
    c["v"] = np.abs(c["v"])
    out, lse = mx.attn_prompt(**_args(c))
    torch.cuda.synchronize()
    _close((out, lse), opa.attn(c["q"], c["k"], c["v"], [n], [new], c["scale"]))
    # equal values come out off by the weights' half step and the output's own at most
    a = _args(dict(c, v=np.full_like(c["v"], 1.5)))
    got = host(mx.attn_prompt(**a)[0].float()).astype(np.float64)
    assert (np.abs(got - 1.5) <= 1.5 * (2 * 2.0 ** -8 + 2.0 ** -14)).all()
