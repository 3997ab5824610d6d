"""GPU parity of the MXFP4 latent cache's writer and reader against the oracle, bit for bit: codes,
scales and positional bytes of every latent size, type and pairing, values at the codes' borders, tiny,
huge and zero rows, every code under every scale read back, slots, pages, lengths and offsets
outside their ranges, strided rows, caches beyond 4 GiB, other streams and graphs."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import latent_mxfp4 as olm, mxfp4 as omx, norm_rope as onr
from tests.gpu_helpers import dev, host, rope_tables

pytestmark = pytest.mark.gpu

CANARY = 0xA5


def _draw(rng, shape, dtype, scale=3.0):
    x = (workloads.draw_values(rng, shape, "normal") * scale).astype(np.float32)
    return workloads.bf16_bits(x) if dtype == "bf16" else x


def _exact(x, dtype):
    return omx.bf16_bits_to_f64(x) if dtype == "bf16" else x.astype(np.float64)


def _cache(pages, latent, fill=CANARY):
    return torch.full((pages, 64 * olm.row_bytes(latent)), fill, dtype=torch.uint8, device="cuda")


def _insert_and_check(kv, dtype, latent, slots, pages, mode="neox", norm="rms", weight=None, eps=1e-6, pos=None,
                      tables=None, q_pe=None):
    cos, sin = rope_tables(len(slots), 64) if tables is None else tables
    cache = _cache(pages, latent)
    got = mx.latent_insert_mxfp4(dev(kv), dev(slots), cache, dev(cos), dev(sin), mode, norm=norm, eps=eps,
                                 positions=None if pos is None else dev(pos),
                                 weight=None if weight is None else dev(weight),
                                 q_pe=None if q_pe is None else dev(q_pe))
    torch.cuda.synchronize()
    want = olm.insert(np.full(cache.shape, CANARY, np.uint8), latent,
                      *olm.encode(_exact(kv, dtype), latent, norm, weight, cos, sin, mode, pos, eps), slots)
    got_parts, want_parts = olm.parts(host(cache), latent), olm.parts(want, latent)
    for name, g, w in zip(("codes", "scales", "positional"), got_parts, want_parts):
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:4].tolist(), int((g != w).sum()))
    return got


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["neox", "interleaved"])
@pytest.mark.parametrize("T,H,norm", [(1, 1, "rms"), (7, 0, "rms"), (66, 5, "none"), (300, 40, "rms")])
def test_insert_bytes(latent, dtype, mode, T, H, norm):
    rng = np.random.default_rng(T + latent)
    pages = -(-T // 64) + 2
    kv, q_pe = _draw(rng, (T, latent + 64), dtype), _draw(rng, (T, H, 64), dtype)
    w = rng.standard_normal(latent).astype(np.float32) if H != 5 else None
    cos, sin = rope_tables(700, 64)
    pos = rng.integers(0, 700, T).astype(np.int64)
    slots = rng.permutation(pages * 64)[:T].astype(np.int64)
    if T > 5:
        pos[3] = 700                                          # outside the table: not rotated
        slots[[1, 4, 5]] = [-1, pages * 64, 1 << 40]          # write nothing
    got = _insert_and_check(kv, dtype, latent, slots, pages, mode, norm, w, pos=pos, tables=(cos, sin),
                            q_pe=q_pe if H else None)
    if H:
        q = _exact(q_pe, dtype)
        y, sc = onr.rope(q, np.abs(q), cos, sin, 64, mode, pos)
        assert (np.abs(host(got[1].float()) - y) <= onr.bound(y, sc, 2.0 ** -8)).all()


@pytest.mark.parametrize("latent,T,dtype", [(512, 16500, "bf16"), (256, 16384, "f32"), (128, 33000, "bf16")])
def test_insert_bytes_of_many_rows(latent, T, dtype):
    # millions of normed values, some within an fp32 rounding of a code's border; two tokens a wave
    rng = np.random.default_rng(T)
    pages = -(-T // 64)
    slots = rng.permutation(pages * 64)[:T].astype(np.int64)
    kv = _draw(rng, (T, latent + 64), dtype)
    _insert_and_check(kv, dtype, latent, slots, pages, weight=(1 + 0.2 * rng.standard_normal(latent)).astype(np.float32))


@pytest.mark.parametrize("latent", [128, 512])
def test_insert_values_at_the_codes_borders(latent):
    # blocks of a largest value 6 * 2^e, or the neighbours of that, and values at each border and its neighbours
    T = 96
    kv = np.zeros((T, latent + 64), np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(9)), np.nextafter(mids, np.float32(0))])
    tops = np.array([6.0, np.nextafter(np.float32(6), np.float32(9)), np.nextafter(np.float32(6), np.float32(0)), 3.0])
    for t in range(T):
        for b in range(latent // 32):
            block = np.concatenate([[tops[(t + b) % 4]], near, -near[:10]]).astype(np.float32)
            kv[t, 32 * b:32 * b + 32] = np.ldexp(np.roll(block, t), (t - 48) * 2 + b % 3)
    _insert_and_check(kv, "f32", latent, np.arange(T, dtype=np.int64), 2, norm="none")


def test_insert_tiny_huge_and_zero_rows():
    latent, rng = 256, np.random.default_rng(2)
    x = rng.standard_normal((12, latent + 64)).astype(np.float32)
    scale = [1.0, 0.0, 2.0 ** -126, 2.0 ** -140, 2.0 ** 100, 2.0 ** 125, 1e-20, 1e20, 0.0, 2.0 ** -149, 1.0, 3.0]
    kv = (x.astype(np.float64) * np.array(scale)[:, None]).astype(np.float32)
    kv[10, :latent] = 0
    kv[10, 77] = -1e30                                        # one value alone
    kv[11, 5:9] = -0.0
    slots = np.arange(12, dtype=np.int64) * 5
    for norm, eps in (("none", 1e-6), ("rms", 1e-6), ("rms", 0.0), ("rms", 1e-300)):
        _insert_and_check(kv, "f32", latent, slots, 1, norm=norm, eps=eps)


def test_insert_strided_views():
    rng = np.random.default_rng(8)
    T, H, latent = 50, 6, 256
    proj, qproj = _draw(rng, (T, latent + 64 + 40), "bf16"), _draw(rng, (T, H, 192), "bf16")
    cos, sin = rope_tables(T, 64)
    a, b = _cache(1, latent, 0), _cache(1, latent, 0)
    q = torch.zeros((T, H, latent + 64), dtype=torch.bfloat16, device="cuda")
    slots = dev(np.arange(T, dtype=np.int64))
    mx.latent_insert_mxfp4(dev(proj)[:, :latent + 64], slots, a, dev(cos), dev(sin), q_pe=dev(qproj)[:, :, 128:],
                           q_out=q[:, :, latent:])
    _, plain = mx.latent_insert_mxfp4(dev(np.ascontiguousarray(proj[:, :latent + 64])), slots, b, dev(cos), dev(sin),
                                      q_pe=dev(np.ascontiguousarray(qproj[:, :, 128:])))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(q[:, :, latent:], plain) and not q[:, :, :latent].any()


@pytest.mark.parametrize("latent", [128, 256, 512])
def test_gather_every_code_under_every_scale(latent):
    # page p: the token's codes and scales run over all bytes (255, no number, apart)
    pages = 40
    cache = np.zeros((pages, 64 * olm.row_bytes(latent)), np.uint8)
    codes, scales, pos = olm.parts(cache, latent)
    n = pages * 64
    codes[:] = (np.arange(n)[:, None] * 7 + np.arange(latent // 2)[None, :]).reshape(codes.shape) % 256
    scales[:] = ((np.arange(n)[:, None] * (latent // 32) + np.arange(latent // 32)[None, :]) % 255).reshape(scales.shape)
    cache = np.concatenate([p.reshape(pages, -1) for p in (codes, scales, pos)], 1)
    bits = np.random.default_rng(1).integers(0, 0x7F80, (pages, 64, 64)).astype(np.uint16)
    cache[:, -64 * 128:] = bits.reshape(pages, -1).view(np.uint8)
    bt = np.arange(pages, dtype=np.int32)[None]
    got = mx.latent_gather_mxfp4(dev(cache), dev(bt), dev(np.array([n], np.int32)), dev(np.zeros(1, np.int64)), n, n)
    torch.cuda.synchronize()
    got = omx.bf16_bits_to_f64(host(got.view(torch.int16)).view(np.uint16))
    want = olm.values(cache, latent)
    assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()
    assert np.array_equal(np.signbit(got), np.signbit(want))


def _filled(rng, pages, latent):
    cache = rng.integers(0, 256, (pages, 64 * olm.row_bytes(latent))).astype(np.uint8)
    a, b = 64 * latent // 2, 64 * latent // 32
    cache[:, a:a + b] = rng.integers(120, 132, (pages, b))
    cache[:, a + b:] = workloads.bf16_bits(rng.standard_normal((pages, 64 * 64)).astype(np.float32)).view(np.uint8)
    return cache


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("lens,max_len", [([1], 1), ([64, 0, 65, 1, 130], 130), ([300, 7], 129), ([63, -5, 200], 200)])
def test_gather(latent, lens, max_len):
    rng = np.random.default_rng(sum(lens) + latent)
    bt, _, pages = workloads.allocate_pages(rng, np.maximum(lens, 0), spare_pages=1, min_cols=-(-max_len // 64))
    cache, total = _filled(rng, pages, latent), sum(max(n, 0) for n in lens)
    off = np.cumsum(np.maximum(lens, 0)) - np.maximum(lens, 0)
    if len(lens) == 5:
        bt[2, 1], bt[4, 0] = pages, -1                      # outside the cache: skipped
        off = off + 3                                         # the last rows fall behind the output
    buf = torch.full((total, latent + 64 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :latent + 64]
    got = mx.latent_gather_mxfp4(dev(cache), dev(bt), dev(np.array(lens, np.int32)), dev(off.astype(np.int64)), max_len,
                                 total, out=out)
    torch.cuda.synchronize()
    assert got is out and (buf[:, latent + 64:] == 7).all()
    want = olm.gather(cache, latent, bt, lens, off, max_len, np.full((total, latent + 64), 7.0))
    assert np.array_equal(host(out.float()).astype(np.float64), want)


def test_gather_makes_zeros_and_takes_longer_offsets():
    rng = np.random.default_rng(4)
    cache = dev(_filled(rng, 2, 128))
    lens, off = torch.tensor([3, 0], dtype=torch.int32).cuda(), torch.tensor([1, 4, 4]).cuda()
    bt = torch.tensor([[1], [0]], dtype=torch.int32).cuda()
    out = mx.latent_gather_mxfp4(cache, bt, lens, off, 64, 6)
    torch.cuda.synchronize()
    rows = olm.values(host(cache), 128)
    assert np.array_equal(host(out.float())[1:4], rows[64:67]) and not out[[0, 4, 5]].any()


def test_cache_beyond_4_gib_and_another_stream():
    latent, pages = 512, 180000                               # 4.6 GB
    cache = torch.zeros((pages, 64 * olm.row_bytes(latent)), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(9)
    kv = _draw(rng, (4, latent + 64), "f32")
    at = np.array([pages - 1, 0, pages - 700, (1 << 32) // cache.shape[1] + 1])
    slots = (at * 64 + [63, 0, 5, 9]).astype(np.int64)
    cos, sin = rope_tables(4, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = [dev(a) for a in (kv, slots, cos, sin)]
    torch.cuda.synchronize()
    mx.latent_insert_mxfp4(args[0], args[1], cache, args[2], args[3], "interleaved", stream=s)
    out = mx.latent_gather_mxfp4(cache, dev(at.astype(np.int32)[:, None]), dev(np.full(4, 64, np.int32)),
                                 dev(np.arange(4, dtype=np.int64) * 64), 64, 256, stream=s)
    s.synchronize()
    small = np.zeros((4, cache.shape[1]), np.uint8)
    want = olm.values(olm.insert(small, latent, *olm.encode(kv, latent, "rms", None, cos, sin, "interleaved"),
                                 np.arange(4) * 64 + slots % 64), latent)
    assert np.array_equal(host(out.float()).astype(np.float64), want)
    assert int((cache.view(torch.int64).amax(1) != 0).sum()) <= 4


def test_graph_replays_match_eager():
    rng = np.random.default_rng(10)
    T, H, latent = 16, 8, 512
    kv, q_pe = dev(_draw(rng, (T, latent + 64), "bf16")), dev(_draw(rng, (T, H, 64), "bf16"))
    cos, sin = (dev(t) for t in rope_tables(100, 64))
    pos, slots = (torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2))
    cache, q = _cache(4, latent, 0), torch.zeros((T, H, latent + 64), dtype=torch.bfloat16, device="cuda")
    bt, lens = dev(np.array([[2, 0], [1, 3]], np.int32)), dev(np.array([100, 128], np.int32))
    off, rows = dev(np.array([0, 100], np.int64)), torch.zeros((228, latent + 64), dtype=torch.bfloat16, device="cuda")

    def step():
        mx.latent_insert_mxfp4(kv, slots, cache, cos, sin, positions=pos, q_pe=q_pe, q_out=q[..., latent:])
        mx.latent_gather_mxfp4(cache, bt, lens, off, 128, 228, out=rows)

    slots.copy_(torch.arange(T))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(3):
        kv.copy_(dev(_draw(rng, (T, latent + 64), "bf16")))
        pos.copy_(dev(rng.integers(0, 100, T).astype(np.int64)))
        slots.copy_(dev(rng.permutation(256)[:T].astype(np.int64)))
        cache.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = cache.clone(), q.clone(), rows.clone()
        cache.zero_(), q.zero_(), rows.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (cache, q, rows))) and rows.any(), rep


def test_refusals_of_the_wrappers():
    cos, sin = (dev(t) for t in rope_tables(8, 64))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kv, cache = torch.zeros((4, 320), **bf), _cache(1, 256)
    q, slots = torch.zeros((4, 2, 64), **bf), torch.arange(4, device="cuda")
    ok = dict(kv=kv, slot_mapping=slots, cache=cache, cos=cos, sin=sin, q_pe=q)
    mx.latent_insert_mxfp4(**ok)
    for change in (dict(kv=kv.half()), dict(kv=kv[:, :256]), dict(kv=kv.float()), dict(cache=cache.char()),
                   dict(cache=cache[:, :-64]), dict(cache=_cache(1, 128)), dict(cache=cache.view(1, 64, -1)),
                   dict(cache=cache.view(-1)), dict(slot_mapping=slots[:3]), dict(slot_mapping=slots.int()),
                   dict(norm="layer"), dict(weight=torch.ones(320, device="cuda")), dict(q_pe=None, q_out=q),
                   dict(cache=cache.cpu())):
        with pytest.raises(mx.MxidxError):
            mx.latent_insert_mxfp4(**{**ok, **change})
    i32 = dict(dtype=torch.int32, device="cuda")
    ok = dict(cache=cache, block_table=torch.zeros((2, 1), **i32), seq_lens=torch.ones(2, **i32),
              cu_seq_offsets=torch.arange(2, device="cuda"), max_seq_len=64, total_tokens=2)
    mx.latent_gather_mxfp4(**ok)
    for change in (dict(cache=cache.char()), dict(block_table=torch.zeros((2, 1), device="cuda")),
                   dict(max_seq_len=65), dict(seq_lens=torch.ones(3, **i32)), dict(total_tokens=-1),
                   dict(cu_seq_offsets=torch.arange(1, device="cuda")), dict(cu_seq_offsets=torch.zeros(2, **i32)),
                   dict(out=torch.zeros((2, 192), **bf)), dict(out=torch.zeros((1, 320), **bf)),
                   dict(out=torch.zeros((2, 320), device="cuda")), dict(out=torch.zeros((320, 2), **bf).t()),
                   dict(max_seq_len=-1)):
        with pytest.raises(mx.MxidxError):
            mx.latent_gather_mxfp4(**{**ok, **change})
