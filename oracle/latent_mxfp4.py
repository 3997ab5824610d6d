"""MXFP4 latent cache: rows in, pages, rows out (oracle, float64 and integers).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A token's row: `latent` values in the MXFP4 row format of ``oracle/mxfp4.py`` (latent / 2 code bytes,
latent / 32 scale bytes) and 64 rotated values in bf16.  A page: 64 code rows, 64 scale rows,
64 positional rows.
"""

import numpy as np

from . import mxfp4, rope

PAGE, ROPE = 64, 64


def row_bytes(latent):
    return latent // 2 + latent // 32 + 2 * ROPE


def normed(x, latent, norm, weight=None, eps=1e-6):
    """fp32 rows of the latent part: the norm in float64, rounded once."""
    x = np.asarray(x, np.float64)[:, :latent]
    if norm == "none":
        return x.astype(np.float32)
    mean = np.square(x).mean(-1, keepdims=True) + eps
    inv = 1.0 / np.sqrt(np.where(mean == 0, 1.0, mean))
    return (x * inv * (1.0 if weight is None else np.asarray(weight, np.float64))).astype(np.float32)


def encode(kv, latent, norm, weight, cos, sin, mode, positions=None, eps=1e-6):
    """(codes [T, latent/2], scales [T, latent/32], positional bf16 bits [T, 64]) of rows kv."""
    kv = np.asarray(kv, np.float64)
    codes, scales = mxfp4.quantize_rows(normed(kv, latent, norm, weight, eps).astype(np.float64))
    pe = rope.apply_rope(kv[:, None, latent:], cos, sin, ROPE, mode, positions)[:, 0]
    bits = pe.view(np.uint32).astype(np.uint64)
    bits = ((bits + 0x7FFF + ((bits >> 16) & 1)) >> 16).astype(np.uint16)
    T = kv.shape[0]
    return codes.reshape(T, -1), scales.reshape(T, -1), bits


def parts(cache, latent):
    """Views of the code, scale and positional rows [pages, 64, bytes] of a cache [pages, page bytes]."""
    a, b = PAGE * latent // 2, PAGE * latent // 32
    n = cache.shape[0]
    return (cache[:, :a].reshape(n, PAGE, -1), cache[:, a:a + b].reshape(n, PAGE, -1),
            cache[:, a + b:].reshape(n, PAGE, -1))


def insert(cache, latent, codes, scales, pos_bits, slots):
    """A copy of the cache with the rows at their slots; slots outside it write nothing."""
    out = cache.copy()
    a, b = PAGE * latent // 2, PAGE * latent // 32
    for t, s in enumerate(np.asarray(slots, np.int64).tolist()):
        if not 0 <= s < cache.shape[0] * PAGE:
            continue
        page, off = out[s // PAGE], s % PAGE
        page[off * latent // 2:(off + 1) * latent // 2] = codes[t]
        page[a + off * latent // 32:a + (off + 1) * latent // 32] = scales[t]
        page[a + b + off * 128:a + b + (off + 1) * 128] = pos_bits[t].view(np.uint8)
    return out


def values(cache, latent):
    """float64 rows [pages * 64, latent + 64] of every slot (a value past bf16's range is infinite)."""
    codes, scales, pos = (np.ascontiguousarray(p) for p in parts(cache, latent))
    n = cache.shape[0] * PAGE
    x = mxfp4.dequantize_rows(codes, scales).reshape(n, latent)
    x = np.where(np.abs(x) >= 2.0 ** 128, np.copysign(np.inf, x), x)
    return np.concatenate([x, mxfp4.bf16_bits_to_f64(pos.reshape(n, 128).view(np.uint16))], 1)


def gather(cache, latent, block_table, seq_lens, offsets, max_seq_len, out):
    """`out` (float64 [total, latent + 64]) with the tokens' rows written."""
    rows, out = values(cache, latent), out.copy()
    for b, n in enumerate(seq_lens):
        for j in range(max(0, min(int(n), max_seq_len))):
            page, to = int(block_table[b, j // PAGE]), int(offsets[b]) + j
            if 0 <= page < cache.shape[0] and 0 <= to < len(out):
                out[to] = rows[page * PAGE + j % PAGE]
    return out
