"""The serving-step operators around the indexer, as cases that can be timed and compared.

Four operators take a step from request lengths to the attention's output:

* ``map``     request lengths -> block-table entries, slots, positions, windows (``step_map``);
* ``norm``    per-head norm and rotation of the indexer's query and key rows (``norm_rope``);
* ``latent``  norm, rotation and paged insert of the main cache's latent rows, with the
              rotation of the query's positional part (``latent_insert``);
* ``attn``    attention of the step's query rows over the paged latent cache, over every
              token of the window or over a top-k list (``attn_paged``).

``own`` chooses between the plain torch form and the package's kernels.
"""

import math

import numpy as np
import torch

own = False

PAGE = 64
DIM = 128           # indexer head dim
ROPE = 64           # rotated part of a latent row


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode token for each of 16 requests: the call is launch latency
        dict(name="map_decode", op="map", seqs=16, lo=8000, hi=8192, new_lo=1, new_hi=1,
             spare_rows=0, gathered=False),
        # a mixed step: many decoding requests and some long prompts, rows of padding behind
        # them, columns of a gathered prefill
        dict(name="map_mixed", op="map", seqs=515, lo=1, hi=16384, new_lo=0, new_hi=8192,
             spare_rows=77, gathered=True),
        # a decode step's indexer rows: layer norm on the key, rotation of both
        dict(name="norm_decode", op="norm", tokens=16, q_heads=32, k_heads=1, dtype="bf16",
             q_norm="none", k_norm="layer", rope=64, mode="neox"),
        # fp32 rows, odd count, both normed, interleaved pairs over the whole head
        dict(name="norm_f32_odd", op="norm", tokens=1021, q_heads=20, k_heads=3, dtype="f32",
             q_norm="rms", k_norm="rms", rope=128, mode="interleaved"),
        # a prefill chunk's indexer rows
        dict(name="norm_chunk", op="norm", tokens=8192, q_heads=64, k_heads=1, dtype="bf16",
             q_norm="rms", k_norm="layer", rope=64, mode="neox"),
        # a decode step's latent rows
        dict(name="latent_decode", op="latent", tokens=16, padded=0, heads=64, latent=512,
             dtype="bf16", mode="interleaved"),
        # a prefill chunk's latent rows, the last rows padding
        dict(name="latent_chunk", op="latent", tokens=16384, padded=100, heads=32, latent=512,
             dtype="bf16", mode="neox"),
        # one request, few heads, a short context: latency
        dict(name="attn_one", op="attn", seqs=1, rows=1, lo=257, hi=257, heads=8, latent=256,
             k=0, gathered=False),
        # the decode batch after its top-2048
        dict(name="attn_topk_decode", op="attn", seqs=16, rows=1, lo=8192, hi=8192, heads=64,
             latent=512, k=2048, gathered=False),
        # contexts read whole, ragged, two query tokens for each request
        dict(name="attn_dense_decode", op="attn", seqs=16, rows=2, lo=5001, hi=8191, heads=128,
             latent=512, k=0, gathered=False),
        # the long-context batch after its top-2048: tokens scattered over a cache of gigabytes
        dict(name="attn_topk_long", op="attn", seqs=64, rows=1, lo=32768, hi=131072, heads=128,
             latent=512, k=2048, gathered=False),
        # a prefill chunk, every row with a list of its own
        dict(name="attn_topk_chunk", op="attn", seqs=2, rows=512, lo=9000, hi=16384, heads=64,
             latent=512, k=2048, gathered=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "norm", "latent", "attn", "attn"])
    if op == "map":
        seqs = _log(rng, 1, 4096)
        hi = _log(rng, 64, 16384)
        return dict(op=op, seqs=seqs, lo=_log(rng, 1, hi), hi=hi, new_lo=rng.choice([0, 1]),
                    new_hi=_log(rng, 1, max(1, min(hi, (1 << 21) // seqs))),
                    spare_rows=rng.randrange(0, 256), gathered=rng.random() < 0.5)
    if op == "norm":
        q_heads = rng.choice([0, 8, 16, 20, 32, 64])
        return dict(op=op, tokens=_log(rng, 1, 8192), q_heads=q_heads,
                    k_heads=rng.choice([1, 2, 3, 8]) if q_heads else 1,
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    q_norm=rng.choice(["none", "rms", "layer"]),
                    k_norm=rng.choice(["rms", "layer"]), rope=rng.choice([0, 32, 64, 96, 128]),
                    mode=rng.choice(["neox", "interleaved"]))
    if op == "latent":
        tokens = _log(rng, 1, 16384)
        return dict(op=op, tokens=tokens, padded=rng.randrange(0, 1 + tokens // 4),
                    heads=rng.choice([0, 8, 20, 32, 64]) if tokens > 8192
                    else rng.choice([0, 8, 20, 32, 64, 128]),
                    latent=rng.choice([128, 256, 512, 512]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    mode=rng.choice(["neox", "interleaved"]))
    heads = rng.choice([1, 5, 8, 12, 32, 40, 64, 96, 128])
    latent = rng.choice([128, 256, 512, 512, 512])
    form = rng.choice(["dense", "dense", "topk", "topk", "chunk"])
    if form == "chunk":
        hi = _log(rng, 300, 16384)
        return dict(op=op, seqs=rng.choice([1, 2, 3]), rows=_log(rng, 8, min(hi, 320)), hi=hi,
                    lo=_log(rng, max(300, hi // 4), hi), heads=min(heads, 64), latent=latent,
                    k=_log(rng, 16, 2048), gathered=True)
    seqs = _log(rng, 1, 64)
    hi = _log(rng, 2, 131072 if form == "topk" else max(64, min(131072, 300000 // seqs)))
    return dict(op=op, seqs=seqs, rows=rng.choice([1, 1, 2, 3]), lo=_log(rng, max(1, hi // 5), hi),
                hi=hi, heads=heads, latent=latent, k=_log(rng, 16, 2048) if form == "topk" else 0,
                gathered=False)


def _lengths(case):
    """Context lengths: spread evenly over [lo, hi]."""
    n = case["seqs"]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, n - 1) for i in range(n)] \
        if n > 1 else [case["hi"]]


def _new_tokens(case):
    """New tokens of each request of a mixed step: mostly new_lo .. 4, every 37th request long."""
    out = []
    for i, n in enumerate(_lengths(case)):
        q = case["new_hi"] if i % 37 == 0 else case["new_lo"] + i % 4
        out.append(min(n, case["new_hi"], q))
    return out


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _torch_type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _tables(rows, dims):
    """cos / sin of pos * 10000^(-2j/dims), fp32, from 64-bit angles."""
    half = dims // 2
    inv = 10000.0 ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / max(dims, 1))
    ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
    return ang.cos().float().contiguous(), ang.sin().float().contiguous()


def _prepare_map(case, seed):
    rs = np.random.RandomState(seed)
    order = rs.permutation(case["seqs"])
    lens = np.asarray(_lengths(case), np.int64)[order]
    new = np.asarray(_new_tokens(case), np.int64)[order]
    held = (lens - new + PAGE - 1) // PAGE
    need = (lens + PAGE - 1) // PAGE
    cols = int(need.max()) + 1
    start = 5
    pages = int(need.sum()) + start + 3
    perm = rs.permutation(pages).astype(np.int32)
    table = np.zeros((case["seqs"], cols), np.int32)
    used = int(held.sum())
    col = np.arange(cols)
    off = np.cumsum(held) - held
    mine = col[None, :] < held[:, None]
    table[mine] = perm[(off[:, None] + col[None, :])[mine]]
    rows = int(new.sum()) + case["spare_rows"]
    rows = max(1, rows)
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    s = dict(rows=rows, gathered=case["gathered"], seq_lens=dev(lens, np.int32),
             query_lens=dev(new, np.int32), table=dev(table, np.int32),
             free=dev(perm[used:], np.int32), start=dev([start], np.int64),
             next=torch.zeros(1, dtype=torch.int64, device="cuda"))
    i64, i32 = torch.int64, torch.int32
    s["out"] = {n: torch.empty(rows, dtype=t, device="cuda") for n, t in (
        ("slot_mapping", i64), ("positions", i64), ("row_seq", i32), ("ks", i32), ("ke", i32))}
    s["out"]["cu_seq_offsets"] = torch.empty(case["seqs"] + 1, dtype=i64, device="cuda")
    return s


def _prepare_norm(case, seed):
    g, t = _gen(seed), _torch_type(case["dtype"])
    T, Hq, Hk = case["tokens"], case["q_heads"], case["k_heads"]
    s = dict(rope=case["rope"], mode=case["mode"], q_norm=case["q_norm"], k_norm=case["k_norm"])
    # rows as a projection leaves them: q and k side by side in one buffer, wide-ranging scales
    x = _randn(g, (T, Hq + Hk, DIM), t) * torch.exp(_randn(g, (T, Hq + Hk, 1), torch.float32)).to(t)
    x += 0.25
    s["q"], s["k"] = (x[:, :Hq] if Hq else None), x[:, Hq:]
    s["cos"], s["sin"] = _tables(8192, case["rope"])
    s["positions"] = torch.randint(0, 8192, (T,), generator=g, device="cuda")
    for n in ("q", "k"):
        s[n + "_weight"] = 1 + 0.2 * _randn(g, (DIM,), torch.float32)
        s[n + "_bias"] = 0.1 * _randn(g, (DIM,), torch.float32) if case[n + "_norm"] == "layer" else None
    s["q_out"] = torch.empty((T, Hq, DIM), dtype=t, device="cuda") if Hq else None
    s["k_out"] = torch.empty((T, Hk, DIM), dtype=t, device="cuda")
    return s


def _prepare_latent(case, seed):
    g, t = _gen(seed), _torch_type(case["dtype"])
    T, H, L, live = case["tokens"], case["heads"], case["latent"], case["tokens"] - case["padded"]
    pages = -(-live // PAGE) + 2
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    # the requests' pages lie anywhere in the cache, their tokens in order within each
    page = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(live, device="cuda")
    slots[:live] = page[at // PAGE] * PAGE + at % PAGE
    s = dict(live=live, latent=L, mode=case["mode"], slots=slots, weight=1 + 0.2 * _randn(g, (L,), torch.float32))
    # kv and the other outputs of one projection share a buffer: the row stride is wider than a row
    s["kv"] = (_randn(g, (T, L + ROPE + 32), t) * 2)[:, :L + ROPE]
    s["cos"], s["sin"] = _tables(8192, ROPE)
    s["positions"] = torch.randint(0, 8192, (T,), generator=g, device="cuda")
    s["cache"] = torch.zeros((pages, PAGE, L + ROPE), dtype=torch.bfloat16, device="cuda")
    # the query's positional part is the tail of each head of its projection, and goes to the
    # tail of each head of the attention's query
    s["q_pe"] = _randn(g, (T, H, DIM + ROPE), t)[:, :, DIM:] if H else None
    s["q"] = torch.zeros((T, H, L + ROPE), dtype=torch.bfloat16, device="cuda") if H else None
    return s


def _prepare_attn(case, seed):
    g, rs = _gen(seed), np.random.RandomState(seed)
    B, n, H, L = case["seqs"], case["rows"], case["heads"], case["latent"]
    lens = rs.permutation(np.asarray(_lengths(case), np.int64))
    need = (lens + PAGE - 1) // PAGE
    cols, pages = int(need.max()), int(need.sum()) + 3
    perm = rs.permutation(pages).astype(np.int32)
    table = np.zeros((B, cols), np.int32)
    off = np.cumsum(need) - need
    col = np.arange(cols)
    mine = col[None, :] < need[:, None]
    table[mine] = perm[(off[:, None] + col[None, :])[mine]]
    base = (np.cumsum(lens) - lens) if case["gathered"] else np.zeros(B, np.int64)
    ks = np.repeat(base, n)
    ke = ks + np.maximum(np.repeat(lens, n) - n + np.tile(np.arange(n), B) + 1, 0)
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    s = dict(latent=L, longest=int(lens.max()), scale=(L + ROPE) ** -0.5,
             cache=_randn(g, (pages, PAGE, L + ROPE), torch.bfloat16),
             q=_randn(g, (B * n, H, L + ROPE), torch.bfloat16) * 2,
             table=dev(table, np.int32), row_seq=dev(np.repeat(np.arange(B), n), np.int32),
             ks=dev(ks, np.int32) if case["gathered"] else None, ke=dev(ke, np.int32), indices=None)
    if case["k"]:
        # distinct tokens of each row's window, recent ones likelier, as idx_topk returns them:
        # column numbers, -1 behind the last
        k = min(case["k"], s["longest"])
        count = dev(ke - ks, np.int64)
        parts = []
        for a in range(0, B * n, 128):   # keys of 128 rows at a time
            c = torch.arange(s["longest"], device="cuda")
            key = torch.rand((min(128, B * n - a), s["longest"]), generator=g, device="cuda")
            key += c / s["longest"]
            key.masked_fill_(c[None, :] >= count[a:a + 128, None], -1.0)
            top = key.topk(k, dim=1)
            parts.append(torch.where(top.values >= 0, top.indices, -1))
        idx = torch.cat(parts)
        idx = torch.where(idx >= 0, idx + dev(ks, np.int64)[:, None], -1).to(torch.int32)
        s["indices"] = torch.full((B * n, case["k"]), -1, dtype=torch.int32, device="cuda")
        s["indices"][:, :k] = idx
    s["out"] = torch.empty((B * n, H, L), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((B * n, H), dtype=torch.float32, device="cuda")
    if own:
        import mxfp4_paged_cache_quant_amd as mx
        s["workspace"] = mx.attn_workspace(B * n, H, L, case["k"] or s["longest"])
    return s


def prepare(case, seed):
    return {"op": case["op"], **{"map": _prepare_map, "norm": _prepare_norm, "latent": _prepare_latent,
                                 "attn": _prepare_attn}[case["op"]](case, seed)}


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _run_map(s):
    if own:
        import mxfp4_paged_cache_quant_amd as mx
        mx.step_map(s["seq_lens"], s["query_lens"], s["table"], s["rows"], free_pages=s["free"],
                    free_start=s["start"], free_next=s["next"],
                    columns="gathered" if s["gathered"] else "sequence", **s["out"])
        return {"table": s["table"], "free_next": s["next"], **s["out"]}
    lens, new, table = s["seq_lens"].long(), s["query_lens"].long(), s["table"].long()
    held = (lens - new + PAGE - 1) // PAGE
    grown = (lens + PAGE - 1) // PAGE - held
    taken = torch.cumsum(grown, 0)
    col = torch.arange(table.shape[1], device=table.device)
    fresh = s["start"] + (taken - grown)[:, None] + col - held[:, None]
    is_new = (col >= held[:, None]) & (col < (held + grown)[:, None])
    table = torch.where(is_new, s["free"].long()[fresh.clamp(0, s["free"].numel() - 1)], table)
    ends = torch.cumsum(new, 0)
    n = torch.arange(s["rows"], device=table.device)
    b = torch.searchsorted(ends, n, right=True)
    live = b < lens.numel()
    b = b.clamp(max=lens.numel() - 1)
    pos = torch.where(live, lens[b] - ends[b] + n, 0)
    offsets = torch.cumsum(lens, 0) - lens
    ks = torch.where(live, offsets[b], 0) if s["gathered"] else torch.zeros_like(pos)
    i32 = torch.int32
    return {"table": table.to(i32), "free_next": s["start"] + taken[-1:],
            "slot_mapping": torch.where(live, table[b, pos // PAGE] * PAGE + pos % PAGE, -1),
            "positions": pos, "row_seq": torch.where(live, b, -1).to(i32), "ks": ks.to(i32),
            "ke": torch.where(live, ks + pos + 1, 0).to(i32),
            "cu_seq_offsets": torch.cat([offsets, (offsets + lens)[-1:]])}


def _normed(x, kind, weight, bias, eps=1e-6):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    return y if bias is None else y + bias


def _rotated(x, cos, sin, mode):
    """The rows [T, H, d] rotated by the angles [T, d/2]."""
    d = x.shape[-1]
    a, b = (x[..., :d // 2], x[..., d // 2:]) if mode == "neox" else (x[..., 0::2], x[..., 1::2])
    c, s = cos[:, None, :], sin[:, None, :]
    a, b = a * c - b * s, b * c + a * s
    return torch.cat([a, b], -1) if mode == "neox" else torch.stack([a, b], -1).flatten(-2)


def _run_norm(s):
    if own:
        import mxfp4_paged_cache_quant_amd as mx
        q, k = mx.norm_rope(s["q"], s["k"], s["cos"], s["sin"], s["rope"], s["mode"],
                            positions=s["positions"], q_norm=s["q_norm"], q_weight=s["q_weight"],
                            q_bias=s["q_bias"], k_norm=s["k_norm"], k_weight=s["k_weight"],
                            k_bias=s["k_bias"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    cos, sin, r = s["cos"][s["positions"]], s["sin"][s["positions"]], s["rope"]
    out = {}
    for n in ("q", "k"):
        if s[n] is None:
            out[n] = None
            continue
        y = _normed(s[n].float(), s[n + "_norm"], s[n + "_weight"], s[n + "_bias"])
        y = torch.cat([_rotated(y[..., :r], cos, sin, s["mode"]), y[..., r:]], -1)
        out[n] = y.to(s[n].dtype)
    return out


def _run_latent(s):
    L = s["latent"]
    if own:
        import mxfp4_paged_cache_quant_amd as mx
        mx.latent_insert(s["kv"], s["slots"], s["cache"], s["cos"], s["sin"], s["mode"],
                         positions=s["positions"], weight=s["weight"], q_pe=s["q_pe"],
                         q_out=None if s["q"] is None else s["q"][:, :, L:])
        return {"cache": s["cache"], "q": s["q"]}
    cos, sin = s["cos"][s["positions"]], s["sin"][s["positions"]]
    kv = s["kv"].float()
    pe = _rotated(kv[:, None, L:], cos, sin, s["mode"])[:, 0]
    row = torch.cat([_normed(kv[:, :L], "rms", s["weight"], None), pe], -1).to(torch.bfloat16)
    s["cache"].view(-1, L + ROPE)[s["slots"][:s["live"]]] = row[:s["live"]]
    if s["q"] is not None:
        s["q"][:, :, L:] = _rotated(s["q_pe"].float(), cos, sin, s["mode"]).to(torch.bfloat16)
    return {"cache": s["cache"], "q": s["q"]}


def _run_attn(s):
    if own:
        import mxfp4_paged_cache_quant_amd as mx
        out, lse = mx.attn_paged(s["q"], s["cache"], s["table"], s["ke"], s["scale"],
                                 indices=s["indices"], ks=s["ks"], row_seq=s["row_seq"],
                                 max_tokens=s["longest"], out=s["out"], lse=s["lse"],
                                 workspace=s["workspace"])
        return {"out": out, "lse": lse}
    ks = torch.zeros_like(s["ke"]) if s["ks"] is None else s["ks"]
    count = (s["ke"] - ks).long()[:, None]
    if s["indices"] is None:
        tok = torch.arange(s["longest"], device=ks.device)[None, :]
        valid = tok < count
    else:
        tok = s["indices"].long() - ks.long()[:, None]
        valid = (s["indices"] >= 0) & (tok >= 0) & (tok < count)
    tok = torch.where(valid, tok, 0)
    page = s["table"][s["row_seq"].long()[:, None], tok // PAGE].long()
    rows = s["cache"].view(-1, s["cache"].shape[-1])[page * PAGE + tok % PAGE].float()
    score = torch.bmm(s["q"].float(), rows.transpose(1, 2).contiguous()) * s["scale"]
    score.masked_fill_(~valid[:, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p, rows[..., :s["latent"]].contiguous()) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": out.to(torch.bfloat16), "lse": (top + torch.log(total))[..., 0]}


def run(state):
    return {"map": _run_map, "norm": _run_norm, "latent": _run_latent, "attn": _run_attn}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "map":
        new = _new_tokens(case)
        rows = sum(new) + case["spare_rows"]
        pages = sum(-(-n // PAGE) + 1 for n in new)
        return {"bytes": 28 * rows + 8 * pages + (4 + 4 + 8) * case["seqs"], "flops": 0}
    size = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] == "norm":
        rows = case["tokens"] * (case["q_heads"] + case["k_heads"])
        return {"bytes": rows * DIM * size * 2 + case["tokens"] * (8 + 4 * case["rope"]),
                "flops": rows * DIM * 8}
    if case["op"] == "latent":
        T, live, w = case["tokens"], case["tokens"] - case["padded"], case["latent"] + ROPE
        return {"bytes": live * w * (size + 2) + T * (16 + 4 * ROPE) + T * case["heads"] * ROPE * (size + 2),
                "flops": live * w * 6 + T * case["heads"] * ROPE * 3}
    H, L, n = case["heads"], case["latent"], case["rows"]
    read = tokens = 0
    for length in _lengths(case):
        seen = [max(0, length - n + i + 1) for i in range(n)]
        if case["k"]:
            seen = [min(case["k"], v) for v in seen]
        read += min(length, sum(seen)) if case["k"] else max(seen)
        tokens += sum(seen)
    io = case["seqs"] * n * (H * (2 * (L + ROPE) + 2 * L + 4) + 4 * case["k"] + 8)
    return {"bytes": read * 2 * (L + ROPE) + io, "flops": tokens * H * 2 * (2 * L + ROPE)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(x, norm, weight, bias, cos, sin, rope, mode, start=0):
    """Rows [T, H, d] in 64 bits: norm over the row, then the pairs from dim `start` on rotated."""
    x = x.double()
    if norm != "none":
        mu = x.sum(-1, keepdim=True) / x.shape[-1] if norm == "layer" else 0.0
        var = ((x - mu) ** 2).sum(-1, keepdim=True) / x.shape[-1]
        x = (x - mu) / torch.sqrt(var + 1e-6) * weight.double()
        if bias is not None:
            x = x + bias.double()
    if rope == 0:
        return x
    out = x.clone()
    j = torch.arange(rope // 2, device=x.device)
    a, b = (start + j, start + j + rope // 2) if mode == "neox" else (start + 2 * j, start + 2 * j + 1)
    turn = torch.complex(cos.double(), sin.double())[:, None, :]
    z = torch.complex(x[..., a], x[..., b]) * turn
    out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_attn(case, s):
    outs, lses = [], []
    ke, table, seq = s["ke"].tolist(), s["table"].long(), s["row_seq"].tolist()
    ks = [0] * len(ke) if s["ks"] is None else s["ks"].tolist()
    L = s["latent"]
    for r in range(len(ke)):
        n = max(0, ke[r] - ks[r])
        if s["indices"] is None:
            tok = torch.arange(n, device="cuda")
        else:
            tok = s["indices"][r].long()
            tok = tok[tok >= 0] - ks[r]
        rows = s["cache"][table[seq[r]][tok // PAGE], tok % PAGE].double()
        sc = torch.mm(s["q"][r].double(), rows.t().contiguous()) * s["scale"]
        lse = torch.logsumexp(sc, -1) if tok.numel() else torch.full((sc.shape[0],), -math.inf,
                                                                     device="cuda", dtype=torch.float64)
        w = torch.exp(sc - lse[:, None]) if tok.numel() else sc
        outs.append(torch.mm(w, rows[:, :L].contiguous()))
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def exact(case, seed):
    if case["op"] == "map":
        return None     # whole numbers alone
    s = prepare(case, seed)
    if case["op"] == "norm":
        cos, sin = s["cos"][s["positions"]], s["sin"][s["positions"]]
        return {n: None if s[n] is None else
                _exact_rows(s[n], s[n + "_norm"], s[n + "_weight"], s[n + "_bias"], cos, sin,
                            s["rope"], s["mode"]) for n in ("q", "k")}
    if case["op"] == "latent":
        cos, sin = s["cos"][s["positions"]], s["sin"][s["positions"]]
        L, live = s["latent"], s["live"]
        kv = s["kv"][:live, None]
        row = torch.cat([_exact_rows(kv[..., :L], "rms", s["weight"], None, cos[:live], sin[:live], 0, "neox"),
                         _exact_rows(kv[..., L:], "none", None, None, cos[:live], sin[:live], ROPE,
                                     s["mode"])], -1)[:, 0]
        cache = s["cache"].double()
        cache.view(-1, L + ROPE)[s["slots"][:live]] = row
        q = None
        if s["q"] is not None:
            q = s["q"].double()
            q[:, :, L:] = _exact_rows(s["q_pe"], "none", None, None, cos, sin, ROPE, s["mode"])
        return {"cache": cache, "q": q}
    return _exact_attn(case, s)
