"""The 4-bit latent cache's calls as a server runs them together: a prefill in two steps (step map, rows
written, cached contexts read back, prompts attended) and decode steps (rows written, windows
attended in the cache), eager and captured, every stage held to its oracle."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import latent_attn as oattn, latent_mxfp4 as olm, mxfp4 as omx, prompt_attn as opa
from tests.gpu_helpers import dev, host, rope_tables

pytestmark = pytest.mark.gpu

LATENT, H, B, PAGES, COLS, ROWS = 256, 16, 3, 24, 8, 300
SCALE = 192 ** -0.5


def _bits(rng, shape, scale=1.0):
    return workloads.bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


class Server:
    """The buffers that a program keeps, and its oracle's copy of the cache."""

    def __init__(self, seed):
        self.rng = np.random.default_rng(seed)
        i32, bf = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        self.lens, self.new = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.table = torch.zeros((B, COLS), **i32)
        self.free = dev(self.rng.permutation(PAGES).astype(np.int32))
        self.start, self.next = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
        self.cache = torch.full((PAGES, 64 * olm.row_bytes(LATENT)), 0xFF, dtype=torch.uint8, device="cuda")
        self.kv, self.pe = torch.zeros((ROWS, LATENT + 64), **bf), torch.zeros((ROWS, H, 64), **bf)
        self.q, self.qp = torch.zeros((ROWS, H, LATENT + 64), **bf), torch.zeros((ROWS, H, 192), **bf)
        self.rows = torch.zeros((B * COLS * 64, LATENT + 64), **bf)
        self.out, self.lse = torch.zeros((ROWS, H, 128), **bf), torch.zeros((ROWS, H), device="cuda")
        self.dec, self.dec_lse = torch.zeros((ROWS, H, LATENT), **bf), torch.zeros((ROWS, H), device="cuda")
        self.w = dev((1 + 0.2 * self.rng.standard_normal(LATENT)).astype(np.float32))
        self.tables = rope_tables(COLS * 64, 64)
        self.cos, self.sin = (dev(t) for t in self.tables)
        self.ws, self.pws = mx.attn_workspace(ROWS, H, LATENT, COLS * 64), mx.attn_prompt_workspace()
        self.mirror = host(self.cache).copy()
        self.held = np.zeros(B, np.int64)

    def step(self, prefill):
        m = mx.step_map(self.lens, self.new, self.table, ROWS, self.free, self.start, self.next)
        mx.latent_insert_mxfp4(self.kv, m.slot_mapping, self.cache, self.cos, self.sin, positions=m.positions,
                               weight=self.w, q_pe=self.pe, q_out=self.q[..., LATENT:])
        if prefill:
            # one key and value head: the row's end and the row's beginning stand for its projections
            mx.latent_gather_mxfp4(self.cache, self.table, self.lens, m.cu_seq_offsets, COLS * 64, len(self.rows),
                                   out=self.rows)
            mx.attn_prompt(self.qp, self.rows[:, None, LATENT - 128:], self.rows[:, None, :128], self.lens, self.new,
                           SCALE, max_seq_len=COLS * 64, out=self.out, lse=self.lse, workspace=self.pws)
        else:
            mx.attn_paged_mxfp4(self.q, self.cache, self.table, m.ke, SCALE, row_seq=m.row_seq, out=self.dec,
                                lse=self.dec_lse, workspace=self.ws)
        self.map = m

    def feed(self, new):
        """The next step's requests and projections."""
        self.start.copy_(self.next)
        self.held = self.held + new
        self.lens.copy_(dev(self.held.astype(np.int32)))
        self.new.copy_(dev(np.asarray(new, np.int32)))
        self.bits = [_bits(self.rng, s, 2.0) for s in ((ROWS, LATENT + 64), (ROWS, H, 64), (ROWS, H, 192), (ROWS, H, LATENT))]
        self.kv.copy_(dev(self.bits[0])), self.pe.copy_(dev(self.bits[1])), self.qp.copy_(dev(self.bits[2]))
        self.q[..., :LATENT] = dev(self.bits[3])
        self.counts = np.asarray(new)

    def check(self, prefill, what):
        n = int(self.counts.sum())
        slots, pos = host(self.map.slot_mapping), host(self.map.positions)
        assert (slots[:n] >= 0).all() and (slots[n:] == -1).all(), what
        enc = olm.encode(omx.bf16_bits_to_f64(self.bits[0]), LATENT, "rms", host(self.w), *self.tables, "neox", pos)
        self.mirror = olm.insert(self.mirror, LATENT, *enc, slots)
        assert np.array_equal(host(self.cache), self.mirror), what
        table, lens = host(self.table), host(self.lens)
        if prefill:
            total = int(lens.sum())
            off = np.cumsum(lens) - lens
            want = olm.gather(self.mirror, LATENT, table, lens, off, COLS * 64, np.zeros((total, LATENT + 64)))
            assert np.array_equal(host(self.rows[:total].float()).astype(np.float64), want), what
            ro, rl, bo, bl = opa.attn(omx.bf16_bits_to_f64(self.bits[2]), want[:, None, LATENT - 128:], want[:, None, :128],
                                      lens, self.counts, SCALE)
            got, lse = host(self.out.float()), host(self.lse)
        else:
            q = host(self.q.float()).astype(np.float64)
            ro, rl, bo, bl = oattn.attn(q, olm.values(self.mirror, LATENT).reshape(PAGES, 64, -1), table, host(self.map.ke),
                                        SCALE, None, None, host(self.map.row_seq))
            got, lse = host(self.dec.float()), host(self.dec_lse)
        assert (np.abs(got - ro) - bo)[:n].max() <= 0 and (np.abs(lse - rl) - bl)[:n].max() <= 0, what


STEPS = [(True, [90, 3, 0]), (True, [70, 61, 130]), (False, [1, 1, 1]), (False, [1, 0, 1]), (True, [5, 200, 2]), (False, [2, 2, 2])]


@pytest.mark.parametrize("captured", [False, True])
def test_prefill_in_steps_then_decode(captured):
    s = Server(1)
    graphs = {}
    if captured:
        for prefill in (True, False):                     # warm and capture over requests without tokens
            s.step(prefill)
            torch.cuda.synchronize()
            graphs[prefill] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[prefill]):
                s.step(prefill)
            graphs[prefill] = (graphs[prefill], s.map)
    for i, (prefill, new) in enumerate(STEPS):
        s.feed(new)
        if captured:
            graphs[prefill][0].replay()
            s.map = graphs[prefill][1]
        else:
            s.step(prefill)
        torch.cuda.synchronize()
        s.check(prefill, (i, captured))
