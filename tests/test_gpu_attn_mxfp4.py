"""GPU parity of idx_attn_paged_mxfp4 against the float64 oracle over the rows that the cache's bytes
stand for: every latent size and grouping of heads, windows and lists from no token to thousands,
unsplit and split, places that hold no visible token poisoned (scale bytes of no number, NaN in the
positional part), pages outside the cache, blocks of very different scales, a cache beyond 4 GiB,
another stream and graphs; and what the writer wrote, read by the attention.  Tolerances:
oracle/latent_attn.py."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import latent_attn as oattn, latent_mxfp4 as olm, mxfp4 as omx
from tests.gpu_helpers import dev, host, rope_tables

pytestmark = pytest.mark.gpu


def _bf16(x):
    return omx.bf16_bits_to_f64(workloads.bf16_bits(np.asarray(x, np.float32)))


def _filled(rng, pages, latent, lo=124, hi=128):
    cache = rng.integers(0, 256, (pages, 64 * olm.row_bytes(latent))).astype(np.uint8)
    a, b = 64 * latent // 2, 64 * latent // 32
    cache[:, a:a + b] = rng.integers(lo, hi, (pages, b))
    cache[:, a + b:] = workloads.bf16_bits(rng.standard_normal((pages, 64 * 64)).astype(np.float32)).view(np.uint8)
    return cache


def _case(seed, lens, next_n=1, H=8, latent=512, k=0, gathered=False, lo=124, hi=128):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int64)
    B = len(lens)
    bt, _, pages = workloads.allocate_pages(rng, lens, spare_pages=2)
    c = dict(lens=lens, bt=bt, pages=pages, latent=latent, scale=(latent + 64) ** -0.5,
             q=_bf16(rng.standard_normal((B * next_n, H, latent + 64)) * 2), cache=_filled(rng, pages, latent, lo, hi),
             indices=None, row_seq=None)
    base = np.cumsum(lens) - lens if gathered else np.zeros(B, np.int64)
    ks = np.repeat(base, next_n)
    n = np.maximum(np.repeat(lens, next_n) - next_n + np.tile(np.arange(next_n), B) + 1, 0)
    c["ks"], c["ke"] = (ks.astype(np.int32) if gathered else None), (ks + n).astype(np.int32)
    if k:
        idx = np.full((B * next_n, k), -1, np.int32)
        for r in range(B * next_n):
            take = rng.permutation(int(n[r]))[:k]
            idx[r, np.sort(rng.permutation(k)[:len(take)])] = take + ks[r]
            idx[r, rng.random(k) > 0.9] = -1
        c["indices"] = idx
    return c


def _poisoned(c):
    """The cache with every place that no visible token of any row holds made unusable."""
    seen = np.zeros(c["pages"] * 64, bool)
    R = len(c["ke"])
    for r in range(R):
        seq = r // (R // len(c["lens"])) if c["row_seq"] is None else int(c["row_seq"][r])
        if 0 <= seq < len(c["lens"]):
            seen[oattn.visible_rows(r, c["bt"], c["pages"], seq, 0 if c["ks"] is None else c["ks"][r], c["ke"][r],
                                    None if c["indices"] is None else c["indices"][r], c["bt"].shape[1] * 64)] = True
    parts = [p.copy().reshape(c["pages"] * 64, -1) for p in olm.parts(c["cache"], c["latent"])]
    for p in parts:
        p[~seen] = 0xFF                       # codes -6, scales of no number, NaN
    return np.concatenate([p.reshape(c["pages"], -1) for p in parts], 1)


def _args(c, poison=True):
    opt = lambda n: None if c[n] is None else dev(c[n])  # noqa: E731
    return dict(q=torch.from_numpy(c["q"]).to(torch.bfloat16).cuda(), cache=dev(_poisoned(c) if poison else c["cache"]),
                block_table=dev(c["bt"]), ke=dev(c["ke"]), scale=c["scale"], indices=opt("indices"), ks=opt("ks"),
                row_seq=opt("row_seq"))


def _oracle(c, max_tokens=None):
    rows = olm.values(c["cache"], c["latent"]).reshape(c["pages"], 64, -1)
    return oattn.attn(c["q"], rows, c["bt"], c["ke"], c["scale"], c["indices"], c["ks"], c["row_seq"], max_tokens)


def _close(got, want, what=""):
    out, lse = (host(t.float()).astype(np.float64) for t in got)
    ro, rl, bo, bl = want
    live = ~np.isnan(rl)
    assert not np.isnan(out[live[:, 0]]).any() and not np.isnan(lse[live]).any(), what
    empty = live & np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse) & live, empty) and (out[empty] == 0).all(), what
    off = np.abs(out - ro) - bo
    assert not (off[live] > 0).any(), (what, np.argwhere((off > 0) & live[..., None])[:4].tolist(), float(off[live].max()))
    some = live & ~empty
    off = np.abs(lse - rl)[some] - bl[some]
    assert not (off > 0).any(), (what, "lse", float(off.max()))


def _check(c, what="", **kw):
    got = mx.attn_paged_mxfp4(**_args(c), **kw)
    torch.cuda.synchronize()
    _close(got, _oracle(c, kw.get("max_tokens")), what)


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("H", [1, 5, 16, 17, 32, 40, 64, 65, 128])
def test_heads(latent, H):
    _check(_case(H, [130, 1, 64, 257], H=H, latent=latent))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 1000])
@pytest.mark.parametrize("H,latent", [(8, 512), (64, 256), (128, 512), (128, 128)])
def test_lengths(n, H, latent):
    _check(_case(n, [n], H=H, latent=latent))


@pytest.mark.parametrize("H,latent", [(8, 512), (32, 512), (64, 512), (40, 256), (64, 128), (128, 512)])
@pytest.mark.parametrize("k", [1, 16, 63, 64, 200, 777])
def test_lists(H, latent, k):
    _check(_case(k, [300, 700, 40], next_n=2, H=H, latent=latent, k=k, gathered=True))


@pytest.mark.parametrize("H,rows", [(64, 600), (16, 600), (128, 300), (32, 550)])
def test_many_rows(H, rows):
    # the groupings of heads and tiles that few rows do not take
    _check(_case(rows, [150] * (rows // 50), next_n=50, H=H, latent=512, k=70))
    _check(_case(rows, [70] * (rows // 50), next_n=50, H=H, latent=256))


@pytest.mark.parametrize("H,latent,n", [(1, 512, 9000), (64, 128, 20000), (128, 256, 5000), (32, 512, 2500), (64, 512, 2100)])
def test_split_rows(H, latent, n):
    _check(_case(n, [n, n // 3], H=H, latent=latent))


def test_scales_far_apart():
    # values of one block up to 2^40 times another's, and blocks of the smallest scale
    c = _case(3, [200, 33], H=20, latent=256, lo=105, hi=146)
    rng = np.random.default_rng(0)
    c["cache"][:, 64 * 128:64 * 136][rng.random((c["pages"], 64 * 8)) < 0.2] = 0
    c["q"] = _bf16(c["q"] * 2.0 ** -19)
    _check(c)


def test_no_token_no_page_and_rows_of_no_sequence():
    c = _case(5, [100, 80, 7], next_n=2, H=6, latent=256, k=40)
    c["bt"][0, 1], c["bt"][1, 0] = -1, c["pages"]            # pages outside the cache: tokens skipped
    c["ke"][2] = 0
    c["indices"][4] = -1
    c["row_seq"] = np.array([0, 1, 2, -1, 1, 3], np.int32)
    args = _args(c)
    out = torch.full((6, 6, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 6), 7.0, device="cuda")
    got = mx.attn_paged_mxfp4(**args, out=out, lse=lse)
    torch.cuda.synchronize()
    _close(got, _oracle(c))
    assert (out[[3, 5]] == 7).all() and (lse[[3, 5]] == 7).all()
    # no pages at all: every row is empty, nothing is read
    none = dict(args, cache=args["cache"][:0])
    out, lse = mx.attn_paged_mxfp4(**none)
    torch.cuda.synchronize()
    assert not out[[0, 1, 2, 4]].any() and torch.isneginf(lse[[0, 1, 2, 4]]).all()


def test_max_tokens_and_strides():
    c = _case(6, [260, 130], next_n=3, H=10, latent=128)
    q = torch.zeros((6, 12, 128 + 64 + 32), dtype=torch.bfloat16, device="cuda")
    args = _args(c)
    q[:, :10, :192] = args["q"]
    buf = torch.full((6, 14, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    got = mx.attn_paged_mxfp4(**dict(args, q=q[:, :10, :192]), max_tokens=100, out=buf[:, 2:12, 16:144])
    torch.cuda.synchronize()
    _close(got, _oracle(c, 100))
    buf[:, 2:12, 16:144] = 3.0
    assert (buf == 3).all()


def test_cache_beyond_4_gib_on_another_stream():
    latent, pages = 512, 180000                               # 4.6 GB
    small = _case(8, [700, 64], H=64, latent=latent)
    cache = torch.zeros((pages, 64 * olm.row_bytes(latent)), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    at = rng.permutation(pages)[:small["pages"]]
    at[0], at[1] = pages - 1, (1 << 32) // cache.shape[1]
    args = _args(small)
    cache[dev(at.astype(np.int64))] = args["cache"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mx.attn_paged_mxfp4(**dict(args, cache=cache, block_table=dev(at[small["bt"]].astype(np.int32))), stream=s)
    s.synchronize()
    _close(got, _oracle(small))


def test_what_the_writer_wrote():
    rng = np.random.default_rng(11)
    latent, H, lens = 512, 16, np.array([90, 200])
    bt, slots, pages = workloads.allocate_pages(rng, lens, spare_pages=1)
    kv = workloads.bf16_bits(rng.standard_normal((lens.sum(), latent + 64)).astype(np.float32) * 2)
    cos, sin = rope_tables(lens.sum(), 64)
    cache = torch.full((pages, 64 * olm.row_bytes(latent)), 0xFF, dtype=torch.uint8, device="cuda")
    mx.latent_insert_mxfp4(dev(kv), dev(slots), cache, dev(cos), dev(sin))
    c = _case(11, lens, H=H, latent=latent)
    want = olm.insert(np.full(cache.shape, 0xFF, np.uint8), latent,
                      *olm.encode(omx.bf16_bits_to_f64(kv), latent, "rms", None, cos, sin, "neox"), slots)
    c.update(bt=bt, pages=pages, cache=want)
    got = mx.attn_paged_mxfp4(**dict(_args(c), cache=cache))
    torch.cuda.synchronize()
    _close(got, _oracle(c))


@pytest.mark.parametrize("H,n", [(8, 200), (64, 3000)])
def test_graph_replays_match_eager(H, n):
    c = _case(12, [n, n // 2], H=H, latent=512, k=128 if H == 8 else 0)
    args = _args(c, poison=False)
    ws = mx.attn_workspace(2, H, 512, args["block_table"].shape[1] * 64)
    out = torch.zeros((2, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, H), device="cuda")
    call = lambda: mx.attn_paged_mxfp4(**args, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        args["q"].copy_(torch.randn_like(args["q"]))
        args["ke"].sub_(rep * 7)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        out.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse) and out.any(), rep


def test_refusals_of_the_wrapper():
    args = _args(_case(13, [100], H=4, latent=256), poison=False)
    mx.attn_paged_mxfp4(**args)
    for change in (dict(cache=args["cache"].char()), dict(cache=args["cache"][:, :-64]), dict(q=args["q"][..., :256]),
                   dict(cache=torch.zeros((3, 64, 320), dtype=torch.bfloat16, device="cuda")),
                   dict(max_tokens=129), dict(ke=args["ke"].long())):
        with pytest.raises(mx.MxidxError):
            mx.attn_paged_mxfp4(**{**args, **change})


def test_two_graphs_share_a_workspace():
    cs, ws, graphs = [_case(30, [900, 40], H=40, latent=256), _case(31, [700], H=64, latent=512, k=600)], None, []
    ws = mx.attn_workspace(2, 64, 512, 1024)
    ws = torch.full((max(ws.numel(), mx.attn_workspace_max_bytes(2, 64, 256, 1024)),), 0xFF, dtype=torch.uint8, device="cuda")
    for c in cs:
        a = _args(c)
        mx.attn_paged_mxfp4(**a, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = mx.attn_paged_mxfp4(**a, workspace=ws)
        graphs.append((g, got, a))
    for rep in range(3):
        for (g, got, _), c in zip(graphs, cs):
            ws.fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            _close(got, _oracle(c), rep)


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("H", [8, 32, 128])
def test_short_windows_split_and_whole(latent, H):
    # both sides of the sizes up to which a row is not split, for one row and for three
    for n in (65, 128, 129, 192, 193, 256, 257, 320, 321):
        _check(_case(n, [n], H=H, latent=latent))
    _check(_case(7, [321, 64, 200], H=H, latent=latent, k=190))
