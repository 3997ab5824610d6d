"""Attention over the paged latent cache (oracle, float64).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

For query row r and head h over the row's visible tokens j (cached rows c_j of
latent + 64 values):  s_j = scale * q . c_j,  out = sum_j softmax_j(s) c_j[:latent],
lse = log sum_j exp(s_j).  No visible token: out = 0, lse = -inf.
"""

import numpy as np

PAGE = 64


def visible_rows(r, block_table, num_pages, seq, ks, ke, indices, max_tokens):
    """Cache rows (page * 64 + offset) of the row's visible tokens, one per list entry."""
    window = min(max(int(ke) - int(ks), 0), max_tokens)
    tok = np.arange(window) if indices is None else indices.astype(np.int64) - int(ks)
    tok = tok[(tok >= 0) & (tok < window)]
    if len(tok) == 0:
        return np.zeros(0, np.int64)
    page = block_table[seq, tok // PAGE].astype(np.int64)
    ok = (page >= 0) & (page < num_pages)
    return page[ok] * PAGE + tok[ok] % PAGE


def attn(q, cache, block_table, ke, scale, indices=None, ks=None, row_seq=None, max_tokens=None,
         weight_rounding=2.0 ** -16):
    """(out, lse, out_bound, lse_bound) as float64; rows of no sequence are NaN.

    The bounds follow the definition's error in the arithmetic it is computed in.
    u = 2^-24 (fp32), h = 2^-8 (half a bf16 step), d = latent + 64 products per score:
      |ds_j|  <= d u scale sum|q c_j| + 4 u |s_j|           (fp32 sum; scaling, base change, exp)
      |dlse|  <= max|ds| + (2n + 32) u + 4 u |lse|          (n positive terms, each added with
                                                             a rescaling: two roundings)
      |dout|  <= (w + 2 max|ds| + (4n + 64) u) sum_j p_j |c_j| + h |out|
    (the weights' rounding w = weight_rounding: two bf16 parts, h^2; score and sum errors in weight
    and total; the output's rounding)."""
    q, rows = np.asarray(q, np.float64), np.asarray(cache, np.float64).reshape(-1, cache.shape[-1])
    R, H, d = q.shape
    L = d - 64
    B = block_table.shape[0]
    max_tokens = block_table.shape[1] * PAGE if max_tokens is None else max_tokens
    u, h = 2.0 ** -24, 2.0 ** -8
    out, lse = np.full((R, H, L), np.nan), np.full((R, H), np.nan)
    out_b, lse_b = np.zeros((R, H, L)), np.zeros((R, H))
    for r in range(R):
        seq = r // (R // B) if row_seq is None else int(row_seq[r])
        if not 0 <= seq < B:
            continue
        at = visible_rows(r, block_table, cache.shape[0], seq, 0 if ks is None else ks[r], ke[r],
                          None if indices is None else indices[r], max_tokens)
        n = len(at)
        if n == 0:
            out[r], lse[r] = 0.0, -np.inf
            continue
        c = rows[at]
        s = q[r] @ c.T * scale
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(-1, keepdims=True)
        p /= total
        out[r], lse[r] = p @ c[:, :L], (top + np.log(total))[:, 0]
        ds = (d * u * abs(scale) * (np.abs(q[r]) @ np.abs(c).T) + 4 * u * np.abs(s)).max(-1)
        lse_b[r] = ds + (2 * n + 32) * u + 4 * u * np.abs(lse[r])
        out_b[r] = (weight_rounding + 2 * ds + (4 * n + 64) * u)[:, None] * (p @ np.abs(c[:, :L])) + h * np.abs(out[r])
    return out, lse, out_b, lse_b
