"""CPU pins of the MXFP4 latent cache's oracle: a hand-worked row, the page layout and its way back."""

import numpy as np

from oracle import latent_mxfp4 as olm

COS, SIN = np.ones((1, 32), np.float32), np.zeros((1, 32), np.float32)


def test_row_hand_worked():
    # block 0: largest 3 -> scale 2^-1 (byte 126), 3 = 6 * 2^-1 (code 7), -0.75 = -1.5 * 2^-1 (code 3, sign)
    kv = np.zeros((1, 128 + 64))
    kv[0, 0], kv[0, 1], kv[0, 32], kv[0, 128], kv[0, 191] = 3.0, -0.75, 7.0, 1.0, -2.0
    codes, scales, pos = olm.encode(kv, 128, "none", None, COS, SIN, "neox")
    assert codes.shape == (1, 64) and scales.shape == (1, 4) and pos.shape == (1, 64)
    assert codes[0, 0] == 7 | (11 << 4) and scales[0].tolist() == [126, 128, 0, 0]
    assert pos[0, 0] == 0x3F80 and pos[0, 63] == 0xC000 and not pos[0, 1:63].any()


def test_tie_goes_to_the_even_code():
    kv = np.zeros((1, 192))
    kv[0, 0] = 7.0                                         # scale 2: 3.5, between 3 (code 5) and 4 (code 6)
    codes, scales, _ = olm.encode(kv, 128, "none", None, COS, SIN, "neox")
    assert scales[0, 0] == 128 and codes[0, 0] == 6


def test_norm_hand_worked():
    x = np.array([[2.0] * 64 + [-2.0] * 64])
    assert olm.normed(x, 128, "rms", np.full(128, 0.5), 0.0).tolist() == [[0.5] * 64 + [-0.5] * 64]
    assert olm.normed(x * 0, 128, "rms", None, 0.0).tolist() == [[0.0] * 128]


def test_pages_and_back():
    rng = np.random.default_rng(0)
    for latent in (128, 256, 512):
        assert olm.row_bytes(latent) == {128: 196, 256: 264, 512: 400}[latent]
        cache = np.full((3, 64 * olm.row_bytes(latent)), 0xA5, np.uint8)
        kv = rng.standard_normal((4, latent + 64)).astype(np.float32).astype(np.float64)
        enc = olm.encode(kv, latent, "none", None, COS, SIN, "neox", np.full(4, 9))     # not rotated
        slots = [130, 5, -1, 3 * 64]
        new = olm.insert(cache, latent, *enc, slots)
        rows = olm.values(new, latent)
        assert np.abs(rows[130, :latent] - kv[0, :latent]).max() < np.abs(kv[0, :latent]).max() / 5
        assert np.abs(rows[5, latent:] / kv[1, latent:] - 1).max() <= 2.0 ** -8
        changed = (new != cache).sum()
        assert 0 < changed <= 2 * olm.row_bytes(latent)
        assert new[0, 5 * latent // 2] == enc[0][1, 0]
        out = olm.gather(new, latent, np.array([[2, 1]]), [70], [1], 67, np.full((66, latent + 64), 7.0))
        assert (out[0] == 7).all() and (out[1] == rows[128]).all() and (out[3] == rows[130]).all()
        assert (out[65] == rows[64]).all()
