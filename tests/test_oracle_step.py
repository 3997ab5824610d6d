"""CPU pins of the oracles of the step around the indexer: hand-worked request maps,
norms, rotations and attention rows."""

import math

import numpy as np
import pytest

from oracle import latent_attn, norm_rope, rope, step_map


def test_step_map_hand_worked():
    # request 0: 130 tokens, 3 new (positions 127..129: page 1's last place, then page 2, entered);
    # request 1: 64 tokens, none new; request 2: 65 tokens, all new (enters pages 0 and 1)
    table = np.array([[7, 3, 0], [5, 0, 0], [0, 0, 0]], np.int32)
    free = np.array([9, 11, 13, 15], np.int32)
    out, after = step_map.step_map([130, 64, 65], [3, 0, 65], table, 70, free, 1, gathered=True)
    assert after.tolist() == [[7, 3, 11], [5, 0, 0], [13, 15, 0]]
    assert out["free_next"].tolist() == [4]
    assert out["cu_seq_offsets"].tolist() == [0, 130, 194, 259]
    assert out["slot_mapping"][:4].tolist() == [3 * 64 + 63, 11 * 64, 11 * 64 + 1, 13 * 64]
    assert out["slot_mapping"][66:].tolist() == [13 * 64 + 63, 15 * 64, -1, -1][0:4]
    assert out["positions"][:5].tolist() == [127, 128, 129, 0, 1]
    assert out["row_seq"].tolist() == [0] * 3 + [2] * 65 + [-1] * 2
    assert out["ks"][[0, 3, 69]].tolist() == [0, 194, 0]
    assert out["ke"][[0, 2, 3, 67, 69]].tolist() == [128, 130, 195, 259, 0]


def test_step_map_list_runs_out():
    out, after = step_map.step_map([1, 129], [1, 129], np.zeros((2, 3), np.int32), 130,
                                   np.array([4, 6], np.int32), 0)
    assert after.tolist() == [[4, 0, 0], [6, -1, -1]]
    assert out["free_next"].tolist() == [4]
    assert out["slot_mapping"][:2].tolist() == [4 * 64, 6 * 64]
    assert (out["slot_mapping"][65:] == -1).all()
    assert out["ke"][129] == 129


def test_norm_hand_worked():
    x = np.array([3.0, -1.0, 1.0, 1.0])
    y, _ = norm_rope.norm(x, "rms", eps=1.0)           # mean square 3, r = 1/2
    assert np.allclose(y, x / 2)
    y, _ = norm_rope.norm(x, "layer", weight=[1, 2, 1, 1], bias=[0, 0, 0, 5], eps=2.0)
    assert np.allclose(y, [1.0, -2.0, 0.0, 5.0])       # mean 1, variance 2, r = 1/2
    y, _ = norm_rope.norm(x, "none")
    assert np.array_equal(y, x)


@pytest.mark.parametrize("mode", ["neox", "interleaved"])
def test_rope_agrees_with_the_query_encoders_rotation(mode):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 128)).astype(np.float32)
    ang = rng.standard_normal((9, 32))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = np.array([0, 8, 9, -1, 3])                   # rows 2 and 3: outside the table
    y, scale = norm_rope.rope(x.astype(np.float64), np.abs(x).astype(np.float64), cos, sin, 64, mode, pos)
    want = rope.apply_rope(x, cos, sin, 64, mode, pos)
    assert (np.abs(y - want) <= 3 * 2.0 ** -24 * scale).all()
    assert np.array_equal(y[2:4], x[2:4])


def test_attn_hand_worked():
    # two tokens with scores 0 and log 3: weights 1/4 and 3/4; latent 128, one head
    cache = np.zeros((2, 64, 192))
    cache[1, 0, 0], cache[1, 1, 1] = 4.0, 8.0
    cache[1, 1, 191] = 1.0
    q = np.zeros((3, 1, 192))
    q[:, 0, 191] = 2 * math.log(3.0)
    table = np.array([[1]], np.int32)
    out, lse, _, _ = latent_attn.attn(q, cache, table, np.array([2, 0, 2]), 0.5,
                                      indices=np.array([[0, 1, -1], [0, 1, 2], [1, 1, 2]]))
    assert np.allclose(out[0, 0, :2], [1.0, 6.0]) and np.allclose(lse[0, 0], math.log(4.0))
    assert (out[1] == 0).all() and lse[1, 0] == -np.inf
    assert np.allclose(out[2, 0, :2], [0.0, 8.0])       # an entry twice counts twice
    assert np.allclose(lse[2, 0], math.log(6.0))


def test_attn_columns_and_pages():
    rng = np.random.default_rng(0)
    cache = rng.standard_normal((3, 64, 192))
    q = rng.standard_normal((2, 2, 192))
    table = np.array([[2, 5], [1, 0]], np.int32)       # page 5 is not in the cache
    ks = np.array([0, 100])
    a, la, _, _ = latent_attn.attn(q, cache, table, np.array([70, 170]), 0.1, ks=ks, row_seq=[0, 1])
    b, lb, _, _ = latent_attn.attn(q, cache, table, np.array([64, 170]), 0.1, ks=ks, row_seq=[0, 1],
                                   indices=np.arange(200)[None, :].repeat(2, 0))
    assert np.allclose(a, b) and np.allclose(la, lb)
    c, _, _, _ = latent_attn.attn(q, cache, table, np.array([70, 170]), 0.1, row_seq=[-1, 2])
    assert np.isnan(c).all()
