"""The operators of a serving step together, as a server calls them: a prefill of two prompts,
then decode steps that cross page borders, from request lengths to the attention's output --
step_map -> norm_rope -> latent_insert and the indexer's insert / logits / top-k ->
attn_paged.  Each stage is held to its oracle on the stage's own inputs, the caches to what the
oracles' slots say, and a captured decode step to the eager one."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import latent_attn as oattn, mxfp4 as omx, norm_rope as onr, paged_cache as opc, step_map as omap, \
    topk as otk
from tests.gpu_helpers import dev, host, rope_tables

pytestmark = pytest.mark.gpu

H, LATENT, HI, TOPK, PAGES = 20, 256, 32, 96, 40


class Server:
    """A toy server's state: caches, block tables, a free list, and drawn projections."""

    def __init__(self, seed, B):
        self.rng = np.random.default_rng(seed)
        self.B, self.cols = B, 8
        self.table = torch.zeros((B, self.cols), dtype=torch.int32, device="cuda")
        self.free = dev(self.rng.permutation(PAGES).astype(np.int32))
        self.start = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.next = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.index_cache = torch.zeros((PAGES, 64 * 68), dtype=torch.uint8, device="cuda")
        self.cache = torch.zeros((PAGES, 64, LATENT + 64), dtype=torch.bfloat16, device="cuda")
        self.cos, self.sin = (dev(t) for t in rope_tables(512, 64))
        self.w_k = dev(self.rng.standard_normal(128).astype(np.float32))
        self.b_k = dev(self.rng.standard_normal(128).astype(np.float32))
        self.w_l = dev(self.rng.standard_normal(LATENT).astype(np.float32))

    def projections(self, rows):
        """What the model hands over for a step's rows, bf16."""
        bf = lambda *s: dev(workloads.bf16_bits(self.rng.standard_normal(s).astype(np.float32)))  # noqa: E731
        q = bf(rows, H, LATENT + 64)
        return dict(kv=bf(rows, LATENT + 64), q=q, q_pe=bf(rows, H, 64), k_index=bf(rows, 128),
                    q_index=bf(rows, HI, 128),
                    w=dev(self.rng.random((rows, HI)).astype(np.float32)))

    def rows_in(self, m, p, k_index):
        """The step's rows into both caches: the indexer's key (not yet encoded) and the latent rows."""
        _, k = mx.norm_rope(None, p["k_index"], self.cos, self.sin, 64, "neox", positions=m.positions,
                            k_norm="layer", k_weight=self.w_k, k_bias=self.b_k, k_out=k_index)
        mx.latent_insert(p["kv"], m.slot_mapping, self.cache, self.cos, self.sin, "interleaved",
                         positions=m.positions, weight=self.w_l, q_pe=p["q_pe"], q_out=p["q"][..., LATENT:])
        return k


def _check_rows(s, m, p, k, before, rows):
    """norm_rope's and latent_insert's outputs against the oracle, at the oracle's slots."""
    pos, slots = host(m.positions), host(m.slot_mapping)
    cos, sin = host(s.cos), host(s.sin)
    exact = lambda t: host(t.float()).astype(np.float64)  # noqa: E731
    y, sc = onr.norm(exact(p["k_index"])[:, None], "layer", host(s.w_k), host(s.b_k))
    y, sc = onr.rope(y, sc, cos, sin, 64, "neox", pos)
    assert (np.abs(exact(k)[:, None] - y) <= onr.bound(y, sc, 2.0 ** -8)).all()
    kv = exact(p["kv"])
    y, sc = onr.norm(kv[:, :LATENT], "rms", host(s.w_l))
    r, rs = onr.rope(kv[:, None, LATENT:], np.abs(kv[:, None, LATENT:]), cos, sin, 64, "interleaved", pos)
    y, sc = np.concatenate([y, r[:, 0]], 1), np.concatenate([sc, rs[:, 0]], 1)
    live = slots >= 0
    flat = exact(s.cache).reshape(-1, LATENT + 64)
    assert (np.abs(flat[slots[live]] - y[live]) <= onr.bound(y[live], sc[live], 2.0 ** -8)).all()
    rest = np.ones(len(flat), bool)
    rest[slots[live]] = False
    assert np.array_equal(flat[rest], before[rest])          # other tokens' rows as they were
    q = exact(p["q_pe"])
    y, sc = onr.rope(q, np.abs(q), cos, sin, 64, "interleaved", pos)
    assert (np.abs(exact(p["q"][..., LATENT:]) - y) <= onr.bound(y, sc, 2.0 ** -8)).all()


def _check_attn(s, p, got, m, idx, ks, ke):
    out, lse = (host(t.float()).astype(np.float64) for t in got)
    ro, rl, bo, bl = oattn.attn(host(p["q"].float()).astype(np.float64), host(s.cache.float()).astype(np.float64),
                                host(s.table), host(ke), (LATENT + 64) ** -0.5, host(idx),
                                None if ks is None else host(ks), host(m.row_seq))
    live = ~np.isnan(rl[:, 0])
    assert (np.abs(out - ro)[live] <= bo[live]).all() and (np.abs(lse - rl)[live] <= bl[live]).all()
    return live


def _prefill(s, lens, padding=5):
    new = np.asarray(lens, np.int32)
    rows = int(new.sum()) + padding
    want, table = omap.step_map(new, new, host(s.table), rows, host(s.free), int(host(s.start)[0]), gathered=True)
    m = mx.step_map(dev(new), dev(new), s.table, rows, s.free, s.start, s.next, columns="gathered")
    for name, w in want.items():
        assert np.array_equal(host(getattr(m, name)), w), name
    assert np.array_equal(host(s.table), table)
    s.start.copy_(s.next)
    p = s.projections(rows)
    before = host(s.cache.float()).astype(np.float64).reshape(-1, LATENT + 64)
    k = s.rows_in(m, p, None)
    mx.insert(k, m.slot_mapping, s.index_cache)
    _check_rows(s, m, p, k, before, rows)
    ref = opc.insert(np.zeros((PAGES, 64 * 68), np.uint8), host(k.float()).astype(np.float64), want["slot_mapping"])
    assert np.array_equal(host(s.index_cache), ref)
    total = int(new.sum())
    kv, ksc = mx.gather(s.index_cache, s.table, dev(new), m.cu_seq_offsets[:-1].contiguous(), int(new.max()), total)
    qv, qs = mx.quantize_rope(p["q_index"], s.cos, s.sin, 64, "neox", positions=m.positions)
    logits = mx.logits_prefill(qv, qs, kv, ksc, p["w"], m.ks, m.ke)
    idx = mx.topk(logits, m.ks, m.ke, TOPK)
    sets = otk.top_k_per_row(host(logits), host(m.ks), host(m.ke), TOPK)
    g = host(idx)
    assert all(sorted(g[r].tolist()) == sorted(sets[r].tolist()) for r in range(rows))
    got = mx.attn_paged(p["q"], s.cache, s.table, m.ke, (LATENT + 64) ** -0.5, indices=idx, ks=m.ks,
                        row_seq=m.row_seq, out=torch.full((rows, H, LATENT), 3.0, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    live = _check_attn(s, p, got, m, idx, m.ks, m.ke)
    assert live.tolist() == [True] * total + [False] * padding
    assert (got[0][total:] == 3.0).all()                     # rows behind the last token, as they were


def _decode(s, lens, p, b, check=True):
    """One decode step in the buffers b (all of a captured step's)."""
    m = mx.step_map(lens, b["new"], s.table, s.B, s.free, s.start, s.next, **b["map"])
    k = s.rows_in(m, p, b["k"])
    logits = mx.logits_paged_insert_rope(p["q_index"], k, p["w"], s.index_cache, s.table, lens, 1, s.cols * 64,
                                         s.cos, s.sin, 64, "neox", logits=b["logits"], clean=True)
    mx.topk(logits, None, m.ke, TOPK, out=b["idx"])
    got = mx.attn_paged(p["q"], s.cache, s.table, m.ke, (LATENT + 64) ** -0.5, indices=b["idx"],
                        row_seq=m.row_seq, out=b["out"], lse=b["lse"], workspace=b["ws"])
    s.start.copy_(s.next)
    return m, k, got


def _buffers(s):
    e = lambda *shape, t=torch.float32: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
    i64, i32, B = torch.int64, torch.int32, s.B
    return dict(new=torch.ones(B, dtype=i32, device="cuda"), k=e(B, 128, t=torch.bfloat16),
                logits=e(B, s.cols * 64), idx=e(B, TOPK, t=i32), out=e(B, H, LATENT, t=torch.bfloat16),
                lse=e(B, H), ws=mx.attn_workspace(B, H, LATENT, TOPK),
                map=dict(slot_mapping=e(B, t=i64), positions=e(B, t=i64), row_seq=e(B, t=i32), ks=e(B, t=i32),
                         ke=e(B, t=i32), cu_seq_offsets=e(B + 1, t=i64)))


def test_prefill_then_decode():
    s = Server(1, 3)
    lens = np.array([62, 130, 255], np.int32)
    _prefill(s, lens)
    b = _buffers(s)
    for step in range(4):                                    # requests 0 and 2 enter a page on the way
        lens = lens + 1
        want, table = omap.step_map(lens, np.ones(3, np.int32), host(s.table), 3, host(s.free),
                                    int(host(s.start)[0]))
        p = s.projections(3)
        before = host(s.cache.float()).astype(np.float64).reshape(-1, LATENT + 64)
        index_before = host(s.index_cache).copy()
        m, k, got = _decode(s, dev(lens), p, b)
        torch.cuda.synchronize()
        for name, w in want.items():
            assert np.array_equal(host(getattr(m, name)), w), (step, name)
        assert np.array_equal(host(s.table), table)
        _check_rows(s, m, p, k, before, 3)
        ref = opc.insert(index_before, host(k.float()).astype(np.float64), want["slot_mapping"])
        assert np.array_equal(host(s.index_cache), ref)
        g, sets = host(b["idx"]), otk.top_k_per_row(host(b["logits"]), np.zeros(3, np.int32), want["ke"], TOPK)
        assert all(sorted(g[r].tolist()) == sorted(sets[r].tolist()) for r in range(3))
        _check_attn(s, p, got, m, b["idx"], None, m.ke)
    assert int(host(s.start)[0]) == 1 + 3 + 4 + 1 + 1        # pages of the prompts, then two entered


def test_captured_decode_steps_match_eager():
    def run(captured):
        s = Server(2, 5)
        _prefill(s, np.array([60, 1, 127, 64, 200], np.int32), padding=0)
        b = _buffers(s)
        lens = dev(np.array([60, 1, 127, 64, 200], np.int32))
        p = s.projections(5)
        saved = [t.clone() for t in (s.table, s.start, s.index_cache, s.cache, lens, p["q"])]
        if captured:
            lens.add_(1)
            _decode(s, lens, p, b)                           # loads what the first calls load
            for t, o in zip((s.table, s.start, s.index_cache, s.cache, lens, p["q"]), saved):
                t.copy_(o)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                lens.add_(1)
                _decode(s, lens, p, b)
            for t, o in zip((s.table, s.start, s.index_cache, s.cache, lens, p["q"]), saved):
                t.copy_(o)
        out = []
        for step in range(6):
            new = s.projections(5)
            for name in p:
                p[name].copy_(new[name])
            if captured:
                g.replay()
                torch.cuda.synchronize()
                _ = torch.randn(1000, device="cuda").sum().item()
            else:
                lens.add_(1)
                _decode(s, lens, p, b)
                torch.cuda.synchronize()
            # (which tokens, not in which order: that is the attention's sum)
            out.append([t.clone() for t in (b["out"], b["lse"], b["idx"], s.table, s.start, s.index_cache, s.cache)])
        return out

    for step, (x, y) in enumerate(zip(run(False), run(True))):
        for i, (u, v) in enumerate(zip(x, y)):
            assert torch.equal(u, v), (step, i)
