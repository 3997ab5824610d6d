"""Row norms and rotations of the indexer's and the latent cache's rows (oracle, float64).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

  rms:    y = x / sqrt(mean(x^2) + eps) * weight + bias
  layer:  the same of x - mean(x)
  rope:   the pairs (j, j + d/2) (neox) or (2j, 2j + 1) (interleaved) of the d rotated
          dims turned by the angle of index j; rows whose table row is outside the
          table stay as they are.

``scale_of`` returns, with the row, the magnitude that fp32 arithmetic's error is relative
to: |w| r (|x| + mean|x|) + |b| for the norm, summed over a rotated pair.
"""

import numpy as np

from .rope import rope_pairs

# fp32 roundings (units of 2^-24) between an input row and its result: a sum over up
# to 512 values is 8 adds in a lane and 6 over lanes, with the products 15; the norm
# takes half of that through the square root, plus mean, eps, root, quotient,
# weight and bias (6), the mean subtracted before squaring adds 15 of mean|x|; the
# rotation two products and a sum (3).  15/2 + 6 + 15 + 3 < 32.
FP32_STEPS = 32


def norm(x, kind, weight=None, bias=None, eps=1e-6):
    """(y, scale) of rows x [..., n] (float64)."""
    x = np.asarray(x, np.float64)
    if kind == "none":
        return x.copy(), np.abs(x)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(x.shape[-1]) if bias is None else np.asarray(bias, np.float64)
    m = x.mean(-1, keepdims=True) if kind == "layer" else 0.0
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    scale = np.abs(w) * r * (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) + np.abs(b)
    return (x - m) * r * w + b, scale


def rope(y, scale, cos, sin, rope_dim, mode, positions=None):
    """Rotate the first rope_dim dims of y [T, H, n] (and carry scale)."""
    y, scale = y.copy(), scale.copy()
    T = y.shape[0]
    if rope_dim == 0 or T == 0:
        return y, scale
    pos = np.arange(T) if positions is None else np.asarray(positions, np.int64)
    inside = (pos >= 0) & (pos < cos.shape[0])
    row = np.where(inside, pos, 0)
    c = np.where(inside[:, None], np.asarray(cos, np.float64)[row], 1.0)[:, None, :]
    s = np.where(inside[:, None], np.asarray(sin, np.float64)[row], 0.0)[:, None, :]
    ia, ib, _ = rope_pairs(rope_dim, mode)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    both = scale[..., ia] + scale[..., ib]
    scale[..., ia] = scale[..., ib] = both
    return y, scale


def bound(ref, scale, half_step):
    """How far a result may be off: fp32 arithmetic, then one rounding (half a step) to its type."""
    fp32 = FP32_STEPS * 2.0 ** -24 * scale
    return fp32 + half_step * (np.abs(ref) + fp32) + 2.0 ** -126
