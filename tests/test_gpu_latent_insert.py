"""GPU parity of idx_latent_insert against the float64 oracle: cache rows and rotated query
parts, both types, every latent size, both pairings, with and without the norm, slots that
write nothing (and leave their rows as they were), strided inputs and outputs, a cache beyond
4 GiB, and captured into a graph.  Tolerances: oracle/norm_rope.py."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import mxfp4 as omx, norm_rope as onr
from tests.gpu_helpers import dev, host, rope_tables

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


def _draw(rng, shape, dtype):
    x = workloads.draw_values(rng, shape, "normal") * 3
    return workloads.bf16_bits(x) if dtype == "bf16" else x


def _exact(x, dtype):
    return omx.bf16_bits_to_f64(x) if dtype == "bf16" else x.astype(np.float64)


def _want(kv, latent, norm, w, cos, sin, mode, pos):
    y, sc = onr.norm(kv[:, :latent], norm, w)
    p, ps = onr.rope(kv[:, None, latent:], np.abs(kv[:, None, latent:]), cos, sin, 64, mode, pos)
    return np.concatenate([y, p[:, 0]], 1), np.concatenate([sc, ps[:, 0]], 1)


def _close(got, ref, scale, what):
    off = np.abs(got - ref) - onr.bound(ref, scale, HALF)
    assert (off <= 0).all(), (what, np.argwhere(off > 0)[:4].tolist(), float(off.max()))


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["neox", "interleaved"])
@pytest.mark.parametrize("T,H,norm", [(1, 1, "rms"), (7, 0, "rms"), (66, 5, "none"), (300, 40, "rms")])
def test_latent_insert(latent, dtype, mode, T, H, norm):
    rng = np.random.default_rng(T + latent)
    pages = -(-T // 64) + 2
    kv = _draw(rng, (T, latent + 64), dtype)
    q_pe = _draw(rng, (T, H, 64), dtype)
    w = rng.standard_normal(latent).astype(np.float32) if H != 5 else None
    cos, sin = rope_tables(700, 64)
    pos = rng.integers(0, 700, T).astype(np.int64)
    slots = rng.permutation(pages * 64)[:T].astype(np.int64)
    if T > 5:
        pos[3] = 700                                          # outside the table: not rotated
        slots[[1, 4, 5]] = [-1, pages * 64, 1 << 40]          # write nothing
    cache = torch.full((pages, 64, latent + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    got = mx.latent_insert(dev(kv), dev(slots), cache, dev(cos), dev(sin), mode, positions=dev(pos), norm=norm,
                           weight=None if w is None else dev(w), q_pe=dev(q_pe) if H else None)
    torch.cuda.synchronize()
    ref, scale = _want(_exact(kv, dtype), latent, norm, w, cos, sin, mode, pos)
    rows = host(cache.float()).astype(np.float64).reshape(-1, latent + 64)
    live = (slots >= 0) & (slots < pages * 64)
    _close(rows[slots[live]], ref[live], scale[live], "cache")
    untouched = np.ones(len(rows), bool)
    untouched[slots[live]] = False
    assert (rows[untouched] == 5.0).all()
    if H:
        q = _exact(q_pe, dtype)
        y, sc = onr.rope(q, np.abs(q), cos, sin, 64, mode, pos)
        _close(host(got[1].float()), y, sc, "q")


def test_strided_views():
    # kv and the query's positional part inside wider projections, the query's tail as the output
    rng = np.random.default_rng(8)
    T, H, latent = 50, 6, 256
    proj = _draw(rng, (T, latent + 64 + 40), "bf16")
    qproj = _draw(rng, (T, H, 192), "bf16")
    cos, sin = rope_tables(T, 64)
    cache = torch.zeros((1, 64, latent + 64), dtype=torch.bfloat16, device="cuda")
    q = torch.full((T, H, latent + 64), 2.0, dtype=torch.bfloat16, device="cuda")
    slots = np.arange(T, dtype=np.int64)
    _, qo = mx.latent_insert(dev(proj)[:, 8:8 + latent + 64], dev(slots), cache, dev(cos), dev(sin),
                             q_pe=dev(qproj)[..., 128:], q_out=q[..., latent:])
    torch.cuda.synchronize()
    ref, scale = _want(_exact(proj, "bf16")[:, 8:8 + latent + 64], latent, "rms", None, cos, sin, "neox", None)
    _close(host(cache[0, :T].float()), ref, scale, "cache")
    qe = _exact(qproj, "bf16")[..., 128:]
    y, sc = onr.rope(qe, np.abs(qe), cos, sin, 64, "neox", None)
    _close(host(q[..., latent:].float()), y, sc, "q")
    assert (q[..., :latent] == 2.0).all() and qo.data_ptr() == q[..., latent:].data_ptr()


@pytest.mark.parametrize("T,H", [(1, 1), (50, 6), (8200, 33)])
def test_query_in_place(T, H):
    # the query's tail rotated where it lies, one row a run and several
    gen = torch.Generator("cuda").manual_seed(T)
    q = torch.randn((T, H, 192), device="cuda", generator=gen, dtype=torch.float32).bfloat16()
    kv = torch.randn((T, 192), device="cuda", generator=gen, dtype=torch.float32).bfloat16()
    cos, sin = rope_tables(T, 64)
    cache = torch.zeros((-(-T // 64), 64, 192), dtype=torch.bfloat16, device="cuda")
    args = dict(slot_mapping=torch.arange(T, device="cuda"), cache=cache, cos=dev(cos), sin=dev(sin))
    before = q.clone()
    _, want = mx.latent_insert(kv, q_pe=before[..., 128:], **args)
    mx.latent_insert(kv, q_pe=q[..., 128:], q_out=q[..., 128:], **args)
    assert torch.equal(q[..., 128:], want) and torch.equal(q[..., :128], before[..., :128])


@pytest.mark.parametrize("latent,dtype,T,H", [(512, "bf16", 16401, 0), (128, "f32", 16385, 17), (256, "bf16", 8200, 33)])
def test_many_tokens(latent, dtype, T, H):
    # two tokens a wave and several heads a run, on every 97th token
    rng = np.random.default_rng(T)
    kv, q_pe = _draw(rng, (T, latent + 64), dtype), _draw(rng, (T, H, 64), dtype)
    w = rng.standard_normal(latent).astype(np.float32)
    cos, sin = rope_tables(500, 64)
    pos = rng.integers(0, 501, T).astype(np.int64)            # 500: outside the table
    pages = -(-T // 64) + 1
    slots = rng.permutation(pages * 64)[:T].astype(np.int64)
    slots[7::61] = -1
    cache = torch.full((pages, 64, latent + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    got = mx.latent_insert(dev(kv), dev(slots), cache, dev(cos), dev(sin), "interleaved", positions=dev(pos),
                           weight=dev(w), q_pe=dev(q_pe) if H else None)
    torch.cuda.synchronize()
    rows = host(cache.float()).astype(np.float64).reshape(-1, latent + 64)
    pick = np.union1d(np.arange(0, T, 97), [T - 2, T - 1])
    ref, scale = _want(_exact(kv[pick], dtype), latent, "rms", w, cos, sin, "interleaved", pos[pick])
    live = slots[pick] >= 0
    _close(rows[slots[pick][live]], ref[live], scale[live], "cache")
    rest = np.ones(len(rows), bool)
    rest[slots[slots >= 0]] = False
    assert (rows[rest] == 5.0).all() and not (rows[~rest] == 5.0).all(1).any()
    if H:
        q = _exact(q_pe[pick], dtype)
        y, sc = onr.rope(q, np.abs(q), cos, sin, 64, "interleaved", pos[pick])
        _close(host(got[1][dev(pick)].float()), y, sc, "q")


def test_cache_beyond_4_gib():
    latent, pages = 512, 60000                                # 4.4 GB
    cache = torch.zeros((pages, 64, latent + 64), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(9)
    kv = _draw(rng, (4, latent + 64), "f32")
    slots = np.array([pages * 64 - 1, 0, pages * 64 - 700, (1 << 31) // 1152 + 3], np.int64)
    cos, sin = rope_tables(4, 64)
    mx.latent_insert(dev(kv), dev(slots), cache, dev(cos), dev(sin), "interleaved")
    torch.cuda.synchronize()
    ref, scale = _want(kv.astype(np.float64), latent, "rms", None, cos, sin, "interleaved", None)
    flat = cache.view(-1, latent + 64)
    _close(host(flat[dev(slots)].float()), ref, scale, "cache")
    assert int((flat.abs().amax(1) != 0).sum()) == 4


def test_graph_replays_match_eager():
    rng = np.random.default_rng(10)
    T, H, latent = 16, 8, 512
    kv, q_pe = dev(_draw(rng, (T, latent + 64), "bf16")), dev(_draw(rng, (T, H, 64), "bf16"))
    cos, sin = (dev(t) for t in rope_tables(100, 64))
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    cache = torch.zeros((4, 64, latent + 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((T, H, latent + 64), dtype=torch.bfloat16, device="cuda")
    args = dict(positions=pos, q_pe=q_pe, q_out=q[..., latent:])
    mx.latent_insert(kv, slots.copy_(torch.arange(T)), cache, cos, sin, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.latent_insert(kv, slots, cache, cos, sin, **args)
    for rep in range(3):
        kv.copy_(dev(_draw(rng, (T, latent + 64), "bf16")))
        pos.copy_(dev(rng.integers(0, 100, T).astype(np.int64)))
        slots.copy_(dev(rng.permutation(256)[:T].astype(np.int64)))
        cache.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = cache.clone(), q.clone()
        cache.zero_(), q.zero_()
        mx.latent_insert(kv, slots, cache, cos, sin, **args)
        torch.cuda.synchronize()
        assert torch.equal(got[0], cache) and torch.equal(got[1], q), rep


def test_refusals_of_the_wrapper():
    cos, sin = (dev(t) for t in rope_tables(8, 64))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kv, cache = torch.zeros((4, 320), **bf), torch.zeros((1, 64, 320), **bf)
    q, slots = torch.zeros((4, 2, 64), **bf), torch.arange(4, device="cuda")
    ok = dict(kv=kv, slot_mapping=slots, cache=cache, cos=cos, sin=sin, q_pe=q)
    mx.latent_insert(**ok)
    for change in (dict(kv=kv.half()), dict(kv=kv[:, :256]), dict(kv=kv.float()), dict(cache=cache.float()),
                   dict(cache=cache[:, :32]), dict(cache=torch.zeros((1, 64, 300), **bf)),
                   dict(slot_mapping=slots[:3]), dict(slot_mapping=slots.int()), dict(cos=cos[:, :16]),
                   dict(norm="layer"), dict(weight=torch.ones(320, device="cuda")), dict(q_pe=q[:3]),
                   dict(q_out=q.float()), dict(q_out=q[:, :1]), dict(q_pe=None, q_out=q), dict(mode="x"),
                   dict(kv=kv.t().contiguous().t()), dict(cache=cache.cpu())):
        with pytest.raises(mx.MxidxError):
            mx.latent_insert(**{**ok, **change})
