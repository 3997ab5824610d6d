"""GPU parity of idx_attn_prompt with more than 128 query heads, in one and more blocks of a group's heads,
whole and split, against the float64 oracle.  Tolerances: oracle/prompt_attn.py."""

import pytest

import mxfp4_paged_cache_quant_amd as mx
from tests.test_gpu_attn_prompt import DIMS, _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("Hq,Hk", [(129, 1), (200, 8), (160, 20), (256, 1), (256, 2), (256, 16), (256, 256)])
def test_whole_prompts_and_ends(dims, Hq, Hk):
    _check(_case(Hq, [7, 70, 1, 40], [7, 5, 1, 40], Hq, Hk, dims, spare=2))
    _check(_case(Hk, [65, 9], [1, 1], Hq, Hk, dims, causal=False))


@pytest.mark.parametrize("lens,new,Hq,Hk", [([900], [1], 256, 16), ([700, 300], [3, 2], 256, 1), ([1100], [1], 192, 192)])
def test_split_rows(lens, new, Hq, Hk):
    assert mx.attn_prompt_workspace_bytes(sum(new), Hq, Hk, 128, 128, len(lens), max(lens)) > 0
    _check(_case(len(lens), lens, new, Hq, Hk, (128, 128)), max_seq_len=max(lens), workspace=mx.attn_prompt_workspace())
