"""GPU parity of idx_attn_prompt against the float64 oracle: every pair of head sizes, groups of 1 to
128 heads, requests of one token to thousands and of none, whole prompts, their ends and single rows,
causal and not, split and unsplit, requests longer than the keys or the rows that there are,
neighbours' and padding rows poisoned with NaN, strided rows, rows behind the last request, other
streams, concurrent calls and graphs.  Tolerances: oracle/prompt_attn.py."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import mxfp4 as omx, prompt_attn as opa
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (128, 128), (192, 128)]


def _bf16(x):
    return omx.bf16_bits_to_f64(workloads.bf16_bits(np.asarray(x, np.float32)))


def _case(seed, lens, new, Hq=4, Hk=2, dims=(128, 128), spare=0, scale=None, causal=True, q_scale=2.0):
    rng = np.random.default_rng(seed)
    S, T = sum(max(n, 0) for n in lens), sum(max(n, 0) for n in new) + spare
    dk, dv = dims
    return dict(q=_bf16(rng.standard_normal((T, Hq, dk)) * q_scale), k=_bf16(rng.standard_normal((S, Hk, dk))),
                v=_bf16(rng.standard_normal((S, Hk, dv)) + 0.25), lens=lens, new=new,
                scale=dk ** -0.5 if scale is None else scale, causal=causal)


def _t(x):
    return torch.from_numpy(x).to(torch.bfloat16).cuda()


def _args(c):
    return dict(q=_t(c["q"]), k=_t(c["k"]), v=_t(c["v"]), seq_lens=dev(np.array(c["lens"], np.int32)),
                query_lens=dev(np.array(c["new"], np.int32)), scale=c["scale"], causal=c["causal"])


def _close(got, want, what=""):
    out, lse = (host(t.float()).astype(np.float64) for t in got)
    ro, rl, bo, bl = want
    live = ~np.isnan(rl)
    assert not np.isnan(out[live]).any() and not np.isnan(lse[live]).any(), what
    empty = live & np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse) & live, empty) and (out[empty] == 0).all(), what
    some = live & ~empty
    off = np.abs(out - ro)[some] - bo[some]
    assert not (off > 0).any(), (what, np.argwhere((np.abs(out - ro) - bo > 0) & some[..., None])[:4].tolist(), float(off.max()))
    off = np.abs(lse[some] - rl[some]) - bl[some]
    assert not (off > 0).any(), (what, "lse", float(off.max()))


def _oracle(c, max_seq_len=None):
    return opa.attn(c["q"], c["k"], c["v"], c["lens"], c["new"], c["scale"], c["causal"], max_seq_len)


def _check(c, **kw):
    got = mx.attn_prompt(**_args(c), **kw)
    torch.cuda.synchronize()
    _close(got, _oracle(c, kw.get("max_seq_len")))
    return got


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 2), (8, 1), (6, 2), (5, 1), (12, 4), (33, 1), (64, 2), (128, 1), (48, 16)])
def test_heads(dims, Hq, Hk):
    _check(_case(Hq, [7, 70, 1], [7, 5, 1], Hq, Hk, dims))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193, 300])
def test_whole_prompts(dims, n):
    _check(_case(n, [n], [n], 2, 1, dims))
    _check(_case(n, [n, 3], [n, 3], 3, 3, dims, causal=False))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("Hq,Hk", [(4, 4), (8, 2), (16, 1)])
@pytest.mark.parametrize("new", [1, 2, 3, 8, 17, 64, 130])
def test_ends_of_prompts(dims, Hq, Hk, new):
    _check(_case(new, [200, 131, 64 + new, new], [new] * 4, Hq, Hk, dims, spare=3))


@pytest.mark.parametrize("causal", [True, False])
def test_packed_requests_of_every_kind(causal):
    # none, without rows, without tokens, more rows than tokens, negative lengths
    lens = [0, 33, 5, -4, 64, 0, 1, 150, 10]
    new = [0, 0, 5, 2, 64, 3, 1, 20, -3]
    _check(_case(1, lens, new, 6, 3, spare=5, causal=causal))
    _check(_case(2, [3, 200], [9, 260], 2, 1, (64, 64), causal=causal))


@pytest.mark.parametrize("B", [63, 64, 65, 200, 1000])
def test_many_requests(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 9, B).tolist()
    new = [int(rng.integers(0, n + 1)) for n in lens]
    _check(_case(B, lens, new, 2, 1, (64, 64), spare=2))


def test_search_past_16_bit_lengths():
    # keys' offsets beyond 2^16, in and across the chunks of requests
    lens = [70000] + [3] * 70 + [66000, 5]
    new = [1] + [1] * 70 + [2, 5]
    c = _case(3, lens, new, 2, 2, (64, 64))
    _check(c)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("lens,new,Hq,Hk", [([3000], [1], 8, 1), ([2500, 900], [40, 40], 4, 2), ([5000], [5], 16, 16),
                                            ([700] * 3, [1] * 3, 2, 1), ([1100], [128], 1, 1)])
def test_split_rows(dims, lens, new, Hq, Hk):
    c = _case(len(lens), lens, new, Hq, Hk, dims, spare=1)
    T, B = c["q"].shape[0], len(lens)
    assert mx.attn_prompt_workspace_bytes(T, Hq, Hk, *dims, B, max(lens)) > 0
    _check(c, max_seq_len=max(lens), workspace=mx.attn_prompt_workspace())
    # a bound much above the lengths: splits without a token
    _check(c, max_seq_len=100000)


def test_neighbours_and_padding_do_not_leak():
    # a request whose rows are none: its tokens are NaN; NaN behind the last token and in unused rows
    c = _case(4, [70, 90, 65], [70, 0, 10], 4, 1, (192, 128))
    a = _args(c)
    a["k"][70:160], a["v"][70:160] = float("nan"), float("inf")
    k = torch.full((300, 1, 192), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full((300, 1, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    k[:225], v[:225] = a["k"], a["v"]
    q = torch.full((120, 4, 192), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:80] = a["q"]
    for kk, vv in ((k[:225], v[:225]), (k, v)):
        out, lse = mx.attn_prompt(**dict(a, q=q, k=kk, v=vv))
        torch.cuda.synchronize()
        _close((out[:80], lse[:80]), _oracle(c))
        assert not out[80:].any() and torch.isneginf(lse[80:]).all()


@pytest.mark.parametrize("new", [5, 40])
def test_rows_and_keys_that_there_are(new):
    # the requests' rows pass T, their tokens pass S, and max_seq_len bounds them
    c = _case(5, [150, 140], [new, new], 4, 2, (128, 128))
    a, T = _args(c), 2 * new - 3
    got = mx.attn_prompt(**dict(a, q=a["q"][:T].contiguous(), k=a["k"][:230].contiguous(), v=a["v"][:230].contiguous()))
    torch.cuda.synchronize()
    cut = dict(c, q=c["q"][:T], k=c["k"][:230], v=c["v"][:230])
    _close(got, _oracle(cut))
    _check(c, max_seq_len=100)
    none = mx.attn_prompt(**dict(a, k=a["k"][:0], v=a["v"][:0]))
    torch.cuda.synchronize()
    assert not none[0].any() and torch.isneginf(none[1]).all()


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 4.0])
def test_scales(scale):
    _check(_case(6, [100, 20], [50, 20], 4, 2, (64, 64), scale=scale))


def test_large_scores_and_a_dominating_token():
    c = _case(7, [260], [260], 2, 1, (128, 128), q_scale=60.0)
    _check(c)
    c["k"] = c["k"].copy()
    c["k"][[3, 100, 200]] *= 8                                # the maximum rises late
    _check(c)


def test_strides():
    c = _case(8, [90, 70], [30, 70], 6, 3, (192, 128), spare=2)
    a = _args(c)
    q = torch.zeros((102, 8, 224), dtype=torch.bfloat16, device="cuda")
    q[:, 1:7, 16:208] = a["q"]
    kv = torch.zeros((3, 160, 336), dtype=torch.bfloat16, device="cuda")          # heads first
    kv[:, :, :192], kv[:, :, 200:328] = a["k"].transpose(0, 1), a["v"].transpose(0, 1)
    buf = torch.full((102, 9, 140), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 2:8, 4:132]
    lse = torch.full((102, 6), 3.0, device="cuda")
    got = mx.attn_prompt(**dict(a, q=q[:, 1:7, 16:208], k=kv[:, :, :192].transpose(0, 1),
                                v=kv[:, :, 200:328].transpose(0, 1)), out=out, lse=lse)
    torch.cuda.synchronize()
    _close(got, _oracle(c))
    assert (out[100:] == 3).all() and (lse[100:] == 3).all()   # behind the last request
    out[:] = 3.0
    assert (buf == 3).all()


def test_keys_beyond_4_gib():
    # one key head of a wide row: the request's keys begin at 4.6 GB
    rows, stride = 1150, 2_000_000
    buf = torch.zeros((rows * stride,), dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((rows, 1, 128), (stride, 128, 1))
    v = buf[256:].as_strided((rows, 1, 128), (stride, 128, 1))
    c = _case(9, [150], [9], 2, 1)
    k[1000:], v[1000:] = _t(c["k"]), _t(c["v"])
    a = _args(c)
    out, lse = mx.attn_prompt(**dict(a, k=k, v=v, seq_lens=dev(np.array([1000, 150], np.int32)),
                                     query_lens=dev(np.array([0, 9], np.int32))))
    torch.cuda.synchronize()
    _close((out, lse), _oracle(c))


def test_two_streams_at_once():
    cs = [_case(20 + i, [1500, 300], [3, 200], 4, 2) for i in range(2)]
    args, streams = [_args(c) for c in cs], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i] = mx.attn_prompt(**args[i], stream=s)
    torch.cuda.synchronize()
    for g, c in zip(got, cs):
        _close(g, _oracle(c))


@pytest.mark.parametrize("lens,new", [([2000, 70], [2, 1]), ([300, 300], [200, 150])])
def test_graph_replays_match_eager(lens, new):
    c = _case(10, lens, new, 8, 2, (192, 128), spare=4)
    a, ws = _args(c), mx.attn_prompt_workspace()
    T = c["q"].shape[0]
    out, lse = torch.zeros((T, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, 8), device="cuda")
    call = lambda: mx.attn_prompt(**a, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        a["q"].copy_(torch.randn_like(a["q"]))
        a["seq_lens"].copy_(dev(np.array([lens[0] - 9 * rep, lens[1] - rep], np.int32)))
        a["query_lens"].copy_(dev(np.array([new[0], max(new[1] - rep, 0)], np.int32)))
        out.zero_(), lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        out.zero_(), lse.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse) and out.any(), rep
        want = dict(c, q=host(a["q"].float()).astype(np.float64), lens=host(a["seq_lens"]).tolist(),
                    new=host(a["query_lens"]).tolist())
        _close((out, lse), _oracle(want))


def test_no_rows_and_no_requests():
    a = _args(_case(11, [10], [10]))
    out, lse = mx.attn_prompt(**dict(a, q=a["q"][:0]))
    assert out.shape == (0, 4, 128)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, lse = mx.attn_prompt(**dict(a, seq_lens=none, query_lens=none))
    torch.cuda.synchronize()
    assert not out.any() and torch.isneginf(lse).all()


def test_refusals_of_the_wrapper():
    a = _args(_case(12, [300], [3], 4, 2))
    mx.attn_prompt(**a)
    q, k, v = a["q"], a["k"], a["v"]
    for change in (dict(q=q.float()), dict(k=k.float()), dict(q=q[..., :64]), dict(v=v[..., :64]), dict(k=k[:10]),
                   dict(k=k[:, :1]), dict(q=q[:, :3]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                   dict(seq_lens=a["seq_lens"].long()), dict(query_lens=a["query_lens"].repeat(2)),
                   dict(out=torch.zeros((3, 4, 128), device="cuda")), dict(lse=torch.zeros((3, 3), device="cuda")),
                   dict(max_seq_len=-1), dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                   dict(workspace=torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 26)),
                   dict(q=q[..., 1:65]), dict(k=k.cpu())):
        with pytest.raises(mx.MxidxError):
            mx.attn_prompt(**{**a, **change})


def test_two_graphs_share_a_workspace():
    cs = [_case(30, [900, 40], [2, 5], 8, 2), _case(31, [300, 700, 5], [40, 1, 5], 4, 2, (192, 128))]
    ws, graphs = mx.attn_prompt_workspace(), []
    for c in cs:
        a = _args(c)
        mx.attn_prompt(**a, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = mx.attn_prompt(**a, workspace=ws)
        graphs.append((g, got, a))
    ws.fill_(0xFF)
    for rep in range(3):
        for (g, got, _), c in zip(graphs, cs):
            g.replay()
            torch.cuda.synchronize()
            _close(got, _oracle(c), rep)
