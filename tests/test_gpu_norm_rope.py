"""GPU parity of idx_norm_rope against the float64 oracle: both types, every norm, both
pairings, parts of the head and all of it, one and many heads, strided rows, in place, rows
outside the table, zero rows; and its place in the framework: without a norm, quantize of its
output gives quantize_rope's bytes.  Tolerances: oracle/norm_rope.py."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import mxfp4 as omx, norm_rope as onr
from tests.gpu_helpers import dev, host, rope_tables

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _rows(rng, shape, dtype, dist="lognormal"):
    x = workloads.draw_values(rng, shape, dist) + np.float32(0.3)
    return workloads.bf16_bits(x) if dtype == "bf16" else x.astype(np.float32)


def _exact(x, dtype):
    return omx.bf16_bits_to_f64(x) if dtype == "bf16" else x.astype(np.float64)


def _check(got, x, dtype, kind, w, b, eps, cos, sin, rope_dim, mode, pos, what=""):
    y, scale = onr.norm(_exact(x, dtype).reshape(x.shape[0], -1, 128), kind, w, b, eps)
    y, scale = onr.rope(y, scale, cos, sin, rope_dim, mode, pos)
    g = host(got.float()).astype(np.float64).reshape(y.shape)
    off = np.abs(g - y) - onr.bound(y, scale, HALF[dtype])
    assert (off <= 0).all(), (what, np.argwhere(off > 0)[:4].tolist(), float(off.max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["neox", "interleaved"])
@pytest.mark.parametrize("rope_dim", [0, 16, 64, 96, 128])
@pytest.mark.parametrize("q_norm,k_norm", [("none", "layer"), ("rms", "rms"), ("layer", "none")])
def test_norm_rope(dtype, mode, rope_dim, q_norm, k_norm):
    rng = np.random.default_rng(rope_dim + 7 * (mode == "neox"))
    T, Hq, Hk = 37, 5, 2
    q, k = _rows(rng, (T, Hq, 128), dtype), _rows(rng, (T, Hk, 128), dtype)
    w = [rng.standard_normal(128).astype(np.float32) for _ in range(2)]
    b = [rng.standard_normal(128).astype(np.float32), None]
    cos, sin = rope_tables(900, rope_dim)
    pos = rng.integers(0, 900, T).astype(np.int64)
    pos[[2, 9]] = [-1, 900]
    qo, ko = mx.norm_rope(dev(q), dev(k), dev(cos), dev(sin), rope_dim, mode, positions=dev(pos),
                          q_norm=q_norm, q_weight=dev(w[0]), q_bias=dev(b[0]), k_norm=k_norm,
                          k_weight=dev(w[1]), eps=1e-5)
    torch.cuda.synchronize()
    _check(qo, q, dtype, q_norm, w[0], b[0], 1e-5, cos, sin, rope_dim, mode, pos, "q")
    _check(ko, k, dtype, k_norm, w[1], None, 1e-5, cos, sin, rope_dim, mode, pos, "k")


@pytest.mark.parametrize("T,Hq,Hk", [(1, 0, 1), (1, 1, 0), (1, 32, 1), (3, 0, 7), (16, 64, 1), (511, 1, 1),
                                     (4097, 3, 1), (1000, 65, 1)])
def test_sizes_and_strides(T, Hq, Hk):
    rng = np.random.default_rng(T + Hq)
    cos, sin = rope_tables(T, 64)
    # q and k side by side in one buffer, as one projection leaves them, with a gap behind
    x = _rows(rng, (T, (Hq + Hk) * 128 + 24), "bf16", "normal")
    d = dev(x)
    q = d[:, :Hq * 128].unflatten(1, (Hq, 128)) if Hq else None
    k = d[:, Hq * 128:(Hq + Hk) * 128].unflatten(1, (Hk, 128)) if Hk else None
    before = d.clone()
    out = torch.full_like(d, 3.0)
    qo = out[:, :Hq * 128].unflatten(1, (Hq, 128)) if Hq else None
    ko = out[:, Hq * 128:(Hq + Hk) * 128].unflatten(1, (Hk, 128)) if Hk else None
    w = rng.standard_normal(128).astype(np.float32)
    gq, gk = mx.norm_rope(q, k, dev(cos), dev(sin), 64, "interleaved", q_norm="rms", q_weight=dev(w),
                          k_norm="layer", q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert torch.equal(d, before) and (out[:, (Hq + Hk) * 128:] == 3.0).all()
    xr = x[:, :(Hq + Hk) * 128].reshape(T, Hq + Hk, 128)
    if Hq:
        _check(gq, xr[:, :Hq], "bf16", "rms", w, None, 1e-6, cos, sin, 64, "interleaved", None, "q")
    if Hk:
        _check(gk, xr[:, Hq:], "bf16", "layer", None, None, 1e-6, cos, sin, 64, "interleaved", None, "k")
    # in place: the same values
    iq, ik = mx.norm_rope(q, k, dev(cos), dev(sin), 64, "interleaved", q_norm="rms", q_weight=dev(w),
                          k_norm="layer", q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(d[:, :(Hq + Hk) * 128], out[:, :(Hq + Hk) * 128])


@pytest.mark.parametrize("T,Hq,Hk,dtype", [(2100, 64, 1, "bf16"), (8200, 63, 2, "bf16"), (8200, 41, 0, "f32")])
def test_runs_of_heads(T, Hq, Hk, dtype):
    # enough rows for runs of four and more heads, some of them cut short, on every 101st token
    gen = torch.Generator("cuda").manual_seed(T + Hq)
    draw = lambda h: torch.randn((T, h, 128), device="cuda", generator=gen).to(  # noqa: E731
        torch.bfloat16 if dtype == "bf16" else torch.float32)
    q, k = draw(Hq), draw(Hk) if Hk else None
    rng = np.random.default_rng(T)
    w = [rng.standard_normal(128).astype(np.float32) for _ in range(2)]
    cos, sin = rope_tables(300, 96)
    pos = rng.integers(-1, 301, T).astype(np.int64)
    qo, ko = mx.norm_rope(q, k, dev(cos), dev(sin), 96, "neox", positions=dev(pos), q_norm="rms", q_weight=dev(w[0]),
                          k_norm="layer", k_weight=dev(w[1]))
    torch.cuda.synchronize()
    pick = np.union1d(np.arange(0, T, 101), [T - 1])
    for name, x, y, kind, weight in (("q", q, qo, "rms", w[0]), ("k", k, ko, "layer", w[1])):
        if x is not None:
            part = host(x[dev(pick)].view(torch.int16)).view(np.uint16) if dtype == "bf16" else host(x[dev(pick)])
            _check(y[dev(pick)], part, dtype, kind, weight, None, 1e-6, cos, sin, 96,
                   "neox", pos[pick], name)


def test_heads_in_front_of_tokens():
    # [H, T, 128] seen as [T, H, 128]: a head stride larger than the row stride
    rng = np.random.default_rng(4)
    x = _rows(rng, (6, 50, 128), "f32")
    cos, sin = rope_tables(50, 128)
    qo, _ = mx.norm_rope(dev(x).transpose(0, 1), None, dev(cos), dev(sin), 128, "neox", q_norm="rms",
                         q_out=torch.empty((6, 50, 128), device="cuda").transpose(0, 1))
    torch.cuda.synchronize()
    _check(qo.contiguous(), x.transpose(1, 0, 2), "f32", "rms", None, None, 1e-6, cos, sin, 128, "neox", None)


def test_means_that_are_large_beside_the_spread():
    # layer norm of values 1000 + N(0, 1): the mean is subtracted before squaring
    rng = np.random.default_rng(5)
    x = (1000 + rng.standard_normal((64, 128))).astype(np.float32)
    e = torch.empty((0, 0), device="cuda")
    _, ko = mx.norm_rope(None, dev(x), e, e, 0, k_norm="layer")
    torch.cuda.synchronize()
    _check(ko, x, "f32", "layer", None, None, 1e-6, np.zeros((0, 0)), np.zeros((0, 0)), 0, "neox", None)


def test_zero_rows_and_far_values():
    x = np.zeros((4, 128), np.float32)
    x[1], x[2], x[3, ::2] = 1e-18, 3e15, -2.0
    e = torch.empty((0, 0), device="cuda")
    for kind in ("rms", "layer"):
        _, ko = mx.norm_rope(None, dev(x), e, e, 0, k_norm=kind)
        torch.cuda.synchronize()
        _check(ko, x, "f32", kind, None, None, 1e-6, np.zeros((0, 0)), np.zeros((0, 0)), 0, "neox", None, kind)
        assert (host(ko)[0] == 0).all()


@pytest.mark.parametrize("mode", ["neox", "interleaved"])
def test_without_a_norm_it_is_the_query_encoders_rotation(mode):
    rng = np.random.default_rng(6)
    q = dev(_rows(rng, (20, 16, 128), "f32"))
    cos, sin = (dev(t) for t in rope_tables(20, 64))
    qo, _ = mx.norm_rope(q, None, cos, sin, 64, mode)
    v, s = mx.quantize(qo)
    v2, s2 = mx.quantize_rope(q, cos, sin, 64, mode)
    torch.cuda.synchronize()
    assert torch.equal(v, v2) and torch.equal(s, s2)


def test_no_rows():
    e = torch.empty((0, 3, 128), device="cuda")
    cos, sin = (dev(t) for t in rope_tables(4, 64))
    qo, ko = mx.norm_rope(e, e[:, 0], cos, sin, 64)
    assert qo.shape == e.shape and ko.shape == (0, 128)


def test_other_stream_and_graph():
    rng = np.random.default_rng(7)
    x = _rows(rng, (33, 4, 128), "bf16", "normal")
    cos, sin = rope_tables(33, 64)
    q, c, s = dev(x), dev(cos), dev(sin)
    ref, _ = mx.norm_rope(q, None, c, s, 64, q_norm="rms")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = mx.norm_rope(q, None, c, s, 64, q_norm="rms", stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.norm_rope(q, None, c, s, 64, q_norm="rms", q_out=out)
    for rep in range(3):
        q.copy_(dev(_rows(rng, x.shape, "bf16", "normal")))
        g.replay()
        torch.cuda.synchronize()
        want, _ = mx.norm_rope(q, None, c, s, 64, q_norm="rms")
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


def test_refusals_of_the_wrapper():
    cos, sin = (dev(t) for t in rope_tables(8, 64))
    x = torch.zeros((4, 2, 128), device="cuda")
    ok = dict(q=x, k=x, cos=cos, sin=sin, rope_dim=64)
    mx.norm_rope(**ok)
    for change in (dict(q=x.half()), dict(k=x.bfloat16()), dict(k=x[:3]), dict(q=x[..., :64]),
                   dict(q=x.transpose(1, 2)), dict(cos=cos[:4]), dict(cos=cos[:, :16]), dict(rope_dim=40),
                   dict(rope_dim=32), dict(mode="half"), dict(q_norm="batch"), dict(q_out=x[:, :1]),
                   dict(q_out=x.bfloat16()), dict(q_norm="rms", q_weight=torch.zeros(64, device="cuda")),
                   dict(positions=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(eps=-1.0, q_norm="rms"),
                   dict(q=x.cpu()), dict(cos=cos[:3].contiguous(), sin=sin[:3].contiguous())):
        with pytest.raises(mx.MxidxError):
            mx.norm_rope(**{**ok, **change})
