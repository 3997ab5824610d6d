"""CPU pins of the packed prompts' oracle: hand-worked rows."""

import math

import numpy as np

from oracle import prompt_attn


def test_hand_worked():
    # two requests of 2 and 1 tokens; dk = dv = 1; two query heads share the key head
    q = np.array([[[1.0], [0.0]], [[1.0], [2.0]], [[3.0], [1.0]], [[9.0], [9.0]]])
    k, v = np.array([[[0.0]], [[math.log(3.0)]], [[5.0]]]), np.array([[[2.0]], [[6.0]], [[-1.0]]])
    out, lse, ob, lb = prompt_attn.attn(q, k, v, [2, 1], [2, 1], 1.0)
    assert out[0, :, 0].tolist() == [2.0, 2.0] and lse[0].tolist() == [0.0, 0.0]
    assert np.allclose(out[1, :, 0], [(2 + 18) / 4, (2 + 54) / 10]) and np.allclose(lse[1], [math.log(4), math.log(10)])
    assert out[2, :, 0].tolist() == [-1.0, -1.0] and lse[2].tolist() == [15.0, 5.0]
    assert np.isnan(out[3]).all() and np.isnan(lse[3]).all()                       # behind the last request
    assert (ob[:3] > 0).all() and (lb[:3] > 0).all()


def test_windows():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 1, 2)), rng.standard_normal((4, 1, 2)), rng.standard_normal((4, 1, 2))
    # all tokens, no mask: every row the same window
    out = prompt_attn.attn(q, k, v, [4], [4], 0.0, causal=False)[0]
    assert np.allclose(out[:4, 0], v[:, 0].mean(0))
    # the last two of four tokens are the rows; with a scale of 0 row i averages 3 + i tokens
    out = prompt_attn.attn(q, k, v, [4], [2], 0.0)[0]
    assert np.allclose(out[0, 0], v[:3, 0].mean(0)) and np.allclose(out[1, 0], v[:, 0].mean(0)) and np.isnan(out[2:]).all()
    # more rows than tokens: the first ones see none; an empty request; tokens past the bound and past S
    out, lse, _, _ = prompt_attn.attn(q, k, v, [1, 0, 9], [2, 1, 2], 0.0, max_seq_len=2)
    assert (out[[0, 2]] == 0).all() and np.isneginf(lse[[0, 2]]).all() and np.allclose(out[1, 0], v[0, 0])
    assert np.allclose(out[3:, 0], v[1:3, 0].mean(0))
