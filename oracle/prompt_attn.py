"""Attention of packed requests over contiguous keys and values (oracle, float64).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Request b has seq_lens[b] tokens, in order behind the requests' before it in k [S, Hk, dk] and
v [S, Hk, dv]; its last query_lens[b] are rows of q [T, Hq, dk], in order behind the requests'
before it.  Row i sees (causal) the tokens up to its position seq_lens[b] - query_lens[b] + i.
Query head h reads key / value head h // (Hq / Hk).  No visible token: out = 0, lse = -inf.
"""

import numpy as np


def attn(q, k, v, seq_lens, query_lens, scale, causal=True, max_seq_len=None):
    """(out, lse, out_bound, lse_bound) as float64; rows of no request are NaN.

    The bounds follow the definition's error in the arithmetic it is computed in.
    u = 2^-24 (fp32), h = 2^-8 (half a bf16 step), d products per score:
      |ds_j|  <= d u |scale| sum|q k_j| + 4 u |s_j|         (fp32 sum; scaling, base change, exp)
      |dlse|  <= max|ds| + (2n + 32) u + 4 u |lse|          (n positive terms, each added with
                                                             a rescaling: two roundings)
      |dout|  <= (h + 2 max|ds| + (4n + 64) u) sum_j p_j |v_j| + h |out|
    (the weights' rounding to bf16; score and sum errors in weight and total; the output's rounding)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, Hq, dk = q.shape
    S, Hk, dv = v.shape
    u, h = 2.0 ** -24, 2.0 ** -8
    out, lse = np.full((T, Hq, dv), np.nan), np.full((T, Hq), np.nan)
    out_b, lse_b = np.zeros((T, Hq, dv)), np.zeros((T, Hq))
    row = key = 0
    for n, new in zip(seq_lens, query_lens):
        n, new = max(int(n), 0), max(int(new), 0)
        there = max(min(n, S - key, n if max_seq_len is None else max_seq_len), 0)
        for i in range(min(new, T - row)):
            sees = there if not causal else max(min(there, n - new + i + 1), 0)
            t = row + i
            if sees == 0:
                out[t], lse[t] = 0.0, -np.inf
                continue
            for head in range(Hq):
                kk, vv = k[key:key + sees, head // (Hq // Hk)], v[key:key + sees, head // (Hq // Hk)]
                s = kk @ q[t, head] * scale
                p = np.exp(s - s.max())
                lse[t, head] = s.max() + np.log(p.sum())
                p /= p.sum()
                out[t, head] = p @ vv
                ds = (dk * u * abs(scale) * (np.abs(kk) @ np.abs(q[t, head])) + 4 * u * np.abs(s)).max()
                lse_b[t, head] = ds + (2 * sees + 32) * u + 4 * u * abs(lse[t, head])
                out_b[t, head] = (h + 2 * ds + (4 * sees + 64) * u) * (p @ np.abs(vv)) + h * np.abs(out[t, head])
        row, key = row + new, key + n
    return out, lse, out_b, lse_b
