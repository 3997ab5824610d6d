"""GPU parity of idx_attn_paged against the float64 oracle: windows from no token to
thousands, lists with gaps, duplicates and foreign columns, every latent size, head counts from
one to 128, several rows for a sequence, masked places that hold NaN and infinities, pages
outside the cache, strided queries and outputs, a cache beyond 4 GiB, other streams,
concurrent calls and graphs.  Tolerances: oracle/latent_attn.py."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
import workloads
from oracle import latent_attn as oattn, mxfp4 as omx
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


def _bf16(x):
    return omx.bf16_bits_to_f64(workloads.bf16_bits(np.asarray(x, np.float32)))


def _case(seed, lens, next_n=1, H=8, latent=512, k=0, q_scale=2.0, gathered=False, keep=0.9):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int64)
    B = len(lens)
    bt, _, pages = workloads.allocate_pages(rng, lens, spare_pages=2)
    c = dict(lens=lens, bt=bt, pages=pages, H=H, latent=latent, scale=(latent + 64) ** -0.5,
             q=_bf16(rng.standard_normal((B * next_n, H, latent + 64)) * q_scale),
             cache=_bf16(rng.standard_normal((pages, 64, latent + 64))), indices=None, row_seq=None)
    base = np.cumsum(lens) - lens if gathered else np.zeros(B, np.int64)
    ks = np.repeat(base, next_n)
    n = np.maximum(np.repeat(lens, next_n) - next_n + np.tile(np.arange(next_n), B) + 1, 0)
    c["ks"], c["ke"] = (ks.astype(np.int32) if gathered else None), (ks + n).astype(np.int32)
    if k:
        idx = np.full((B * next_n, k), -1, np.int32)
        for r in range(B * next_n):
            take = rng.permutation(int(n[r]))[:k]
            at = np.sort(rng.permutation(k)[:len(take)])
            idx[r, at] = take + ks[r]
            idx[r, rng.random(k) > keep] = -1
        c["indices"] = idx
    return c


def _to_dev(c, poison=None):
    cache = torch.from_numpy(c["cache"]).to(torch.bfloat16).cuda()
    if poison is not None:
        # every place that no visible token of any row holds
        seen = np.zeros(c["pages"] * 64, bool)
        R = len(c["ke"])
        for r in range(R):
            seq = r // (R // len(c["lens"])) if c["row_seq"] is None else int(c["row_seq"][r])
            if 0 <= seq < len(c["lens"]):
                seen[oattn.visible_rows(r, c["bt"], c["pages"], seq, 0 if c["ks"] is None else c["ks"][r],
                                        c["ke"][r], None if c["indices"] is None else c["indices"][r],
                                        c["bt"].shape[1] * 64)] = True
        cache.view(-1, cache.shape[-1])[dev(~seen)] = poison
    opt = lambda n: None if c[n] is None else dev(c[n])  # noqa: E731
    return dict(q=torch.from_numpy(c["q"]).to(torch.bfloat16).cuda(), cache=cache, block_table=dev(c["bt"]),
                ke=dev(c["ke"]), scale=c["scale"], indices=opt("indices"), ks=opt("ks"), row_seq=opt("row_seq"))


def _oracle(c, max_tokens=None):
    return oattn.attn(c["q"], c["cache"], c["bt"], c["ke"], c["scale"], c["indices"], c["ks"], c["row_seq"],
                      max_tokens)


def _close(got, want, what=""):
    out, lse = (host(t.float()).astype(np.float64) for t in got)
    ro, rl, bo, bl = want
    live = ~np.isnan(rl)
    assert not np.isnan(out[live[:, 0]]).any() and not np.isnan(lse[live]).any(), what
    empty = live & np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse) & live, empty), what
    assert (out[empty] == 0).all(), what
    off = np.abs(out - ro) - bo
    assert not (off[live] > 0).any(), (what, np.argwhere((off > 0) & live[..., None])[:4].tolist(),
                                       float(off[live].max()))
    some = live & ~empty
    off = np.abs(lse - rl)[some] - bl[some]
    assert not (off > 0).any(), (what, "lse", float(off.max()))


def _check(c, poison=float("nan"), what="", **kw):
    got = mx.attn_paged(**_to_dev(c, poison), **kw)
    torch.cuda.synchronize()
    _close(got, _oracle(c, kw.get("max_tokens")), what)


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("H", [1, 5, 8, 16, 17, 32, 40, 64, 65, 96, 128])
def test_heads(latent, H):
    _check(_case(H, [130, 1, 64, 257], H=H, latent=latent))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 500, 513, 1000])
@pytest.mark.parametrize("H,latent", [(8, 512), (64, 256), (128, 512)])
def test_lengths(n, H, latent):
    _check(_case(n, [n], H=H, latent=latent))


@pytest.mark.parametrize("k", [1, 3, 16, 33, 64, 100, 250, 2048])
@pytest.mark.parametrize("H,latent", [(8, 128), (64, 512), (128, 256)])
def test_lists(k, H, latent):
    _check(_case(k, [1500, 40, 3, 700], H=H, latent=latent, k=k))


@pytest.mark.parametrize("next_n", [2, 3])
@pytest.mark.parametrize("k", [0, 70])
def test_rows_of_one_sequence(next_n, k):
    # sequences shorter than their rows: the first rows see nothing
    _check(_case(next_n, [300, 1, 2, 95, 64], next_n=next_n, H=16, latent=256, k=k))


@pytest.mark.parametrize("k", [0, 50])
def test_gathered_columns_and_row_order(k):
    c = _case(11, [100, 260, 30, 64], H=12, latent=128, k=k, gathered=True)
    # rows in another order than the sequences, two of them of no sequence
    order = np.array([2, 0, 3, 1, 0, 2])
    for name in ("q", "ks", "ke", "indices"):
        c[name] = None if c[name] is None else c[name][order]
    c["row_seq"] = np.where(np.arange(6) == 4, -1, np.where(np.arange(6) == 5, 4, order)).astype(np.int32)
    d = _to_dev(c, float("nan"))
    out = torch.full((6, 12, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 12), 7.0, device="cuda")
    got = mx.attn_paged(**d, out=out, lse=lse)
    torch.cuda.synchronize()
    _close(got, _oracle(c))
    assert (out[4:] == 7).all() and (lse[4:] == 7).all()


def test_lists_with_foreign_and_double_entries():
    c = _case(12, [200, 90], H=8, latent=128, k=40)
    c["indices"][0, :10] = [5, 5, 200, 10000, -1, -2147483648, 2147483647, 5, 199, 0]
    c["indices"][1, :] = -1
    _check(c)
    c["indices"] = c["indices"][:, :0]
    _check(c)


@pytest.mark.parametrize("k", [0, 64])
def test_rows_that_see_nothing(k):
    c = _case(13, [90, 70, 128], H=20, latent=256, k=k)
    c["ke"][:] = [0, 70, -5]
    _check(c)
    c["ke"][:] = 0
    _check(c)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("k", [0, 90])
def test_masked_places_hold_anything(poison, k):
    _check(_case(14, [70, 129, 1, 300], H=64, latent=512, k=k), poison)


@pytest.mark.parametrize("k", [0, 150])
def test_pages_outside_the_cache(k):
    c = _case(15, [400, 200, 64], H=16, latent=128, k=k)
    c["bt"][0, [0, 3]] = [-1, c["pages"]]
    c["bt"][1, :] = 1 << 30
    _check(c)


def test_max_tokens_bounds_the_window():
    c = _case(16, [400, 200, 64], H=16, latent=128)
    _check(c, None, max_tokens=150)
    _check(c, None, max_tokens=0)
    _check(_case(16, [400, 200, 64], H=16, latent=128, k=90), None, max_tokens=150)


@pytest.mark.parametrize("q_scale,lift", [(40.0, 0.0), (2.0, 300.0), (2.0, -300.0), (0.0, 0.0)])
def test_peaked_flat_and_far_scores(q_scale, lift):
    # weights that are one-hot, scores far from zero on one side (never seen together with 0),
    # and equal scores
    c = _case(17, [300, 65], H=16, latent=256, q_scale=q_scale)
    c["q"][:, :, 256] += lift / c["scale"]
    c["q"] = _bf16(c["q"])
    c["cache"][..., 256] = 1.0
    _check(c)


@pytest.mark.parametrize("H,latent", [(1, 512), (16, 128), (20, 512), (32, 256), (64, 512)])
@pytest.mark.parametrize("k", [0, 120])
def test_weights_of_few_rows_in_two_parts(H, latent, k):
    # a weight's rounding leaves 2^-8 of it at most, and rounding that 2^-8 of what is left
    c = _case(H, [300, 65, 1000], H=H, latent=latent, k=k)
    got = mx.attn_paged(**_to_dev(c, float("nan")))
    torch.cuda.synchronize()
    _close(got, oattn.attn(c["q"], c["cache"], c["bt"], c["ke"], c["scale"], c["indices"], c["ks"], c["row_seq"],
                           weight_rounding=2.0 ** -16))


def test_growing_maximum():
    # each token scores above all before it: every step rescales what was summed
    c = _case(18, [500], H=32, latent=128, q_scale=0.5)
    c["q"][:, :, 128] = 8.0
    c["cache"].reshape(-1, 192)[:, 128] = 0.0
    for j in range(500):
        c["cache"][c["bt"][0, j // 64], j % 64, 128] = j / 16
    c["cache"] = _bf16(c["cache"])
    _check(c)


def test_strided_query_and_output():
    c = _case(19, [100, 300], H=24, latent=256)
    d = _to_dev(c, float("nan"))
    wide = torch.zeros((2, 30, 256 + 64 + 16), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:27, 8:328] = d["q"]
    d["q"] = wide[:, 3:27, 8:328]
    big = torch.full((24, 2, 300), 9.0, dtype=torch.bfloat16, device="cuda")
    table = torch.full((2, d["block_table"].shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    table[:, :-3] = d["block_table"]
    d["block_table"] = table[:, :-3]
    got = mx.attn_paged(**d, out=big.transpose(0, 1)[..., 20:276])
    torch.cuda.synchronize()
    _close((got[0].contiguous(), got[1]), _oracle(c))
    assert (big[..., :20] == 9).all() and (big[..., 276:] == 9).all()


@pytest.mark.parametrize("k", [0, 500])
def test_cache_beyond_4_gib(k):
    latent, pages, H = 512, 60000, 64                          # 4.4 GB
    rng = np.random.default_rng(20)
    cache = torch.zeros((pages, 64, latent + 64), dtype=torch.bfloat16, device="cuda")
    used = np.array([59999, 0, 58255, 29128, 59000, 3, 40000, 59998], np.int32)
    vals = _bf16(rng.standard_normal((len(used), 64, latent + 64)))
    cache[torch.from_numpy(used.astype(np.int64)).cuda()] = torch.from_numpy(vals).to(torch.bfloat16).cuda()
    c = _case(21, [500], H=H, latent=latent, k=k)
    small = dict(c, cache=vals, bt=np.arange(8, dtype=np.int32)[None])
    d = _to_dev(c)
    d["cache"], d["block_table"] = cache, dev(used[None])
    got = mx.attn_paged(**d)
    torch.cuda.synchronize()
    _close(got, _oracle(small))


@pytest.mark.parametrize("rows,H", [(3, 8), (3, 20), (200, 64), (600, 40)])
@pytest.mark.parametrize("k", [0, 130])
def test_many_and_few_rows_of_a_cache_beyond_4_gib(rows, H, k):
    # every grouping of heads and tile, with rows' numbers instead of their places
    latent, pages = 512, 60000
    used = np.array([59999, 0, 58255, 29128, 59000, 3, 40000, 59998, 5, 30000, 44444], np.int32)
    c = _case(rows, [650], next_n=rows, H=H, latent=latent, k=k)
    vals = c["cache"][c["bt"][0]]
    d = _to_dev(c)
    d["cache"] = torch.zeros((pages, 64, latent + 64), dtype=torch.bfloat16, device="cuda")
    d["cache"][torch.from_numpy(used.astype(np.int64)).cuda()] = torch.from_numpy(vals).to(torch.bfloat16).cuda()
    d["block_table"] = dev(used[None])
    got = mx.attn_paged(**d)
    torch.cuda.synchronize()
    pick = np.unique(np.array([0, 1, rows // 2, rows - 2, rows - 1]))
    part = dict(c, q=c["q"][pick], ke=c["ke"][pick], indices=None if k == 0 else c["indices"][pick],
                row_seq=np.zeros(len(pick), np.int32))
    _close((got[0][dev(pick)], got[1][dev(pick)]), _oracle(part))


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("rows,H,n", [(520, 64, 97), (300, 100, 33), (150, 64, 700), (70, 128, 1400)])
@pytest.mark.parametrize("k", [0, 70])
def test_many_rows(latent, rows, H, n, k):
    # two workgroups a CU, one, and one whose tokens are split; NaN in all places that no row sees
    c = _case(rows, [n, 64, 1, n - 1, n], next_n=rows // 5, H=H, latent=latent, k=k)
    got = mx.attn_paged(**_to_dev(c, float("nan")))
    torch.cuda.synchronize()
    pick = np.arange(0, rows, 9)
    part = dict(c, q=c["q"][pick], ke=c["ke"][pick], indices=None if k == 0 else c["indices"][pick],
                row_seq=(pick // (rows // 5)).astype(np.int32))
    _close((got[0][dev(pick)], got[1][dev(pick)]), _oracle(part))


@pytest.mark.parametrize("k", [0, 2048])
def test_decode_batch(k):
    # the decode workload's batch of 16 x 8192, on two of its rows
    lens = np.full(16, 8192)
    c = _case(22, lens, H=64, latent=512, k=k, keep=1.0)
    d = _to_dev(c)
    got = mx.attn_paged(**d)
    torch.cuda.synchronize()
    pick = np.array([0, 13])
    part = dict(c, q=c["q"][pick], ke=c["ke"][pick], indices=None if k == 0 else c["indices"][pick],
                row_seq=pick.astype(np.int32))
    _close((got[0][dev(pick)], got[1][dev(pick)]), _oracle(part))


def test_long_windows_of_mixed_lengths():
    c = _case(23, [9000, 3, 700, 0, 2048], H=8, latent=128)
    _check(c)


@pytest.mark.parametrize("lens,H,latent,k", [([33000], 40, 128, 0), ([17000, 0, 100], 8, 512, 0), ([20000, 19000], 64, 256, 0),
                                             ([5000], 3, 128, 4999), ([3000, 40], 20, 512, 1500)])
def test_many_splits(lens, H, latent, k):
    # up to 128 splits of a row, joined by several groups of lanes; splits that see nothing among them
    _check(_case(H, lens, H=H, latent=latent, k=k))


def test_same_call_gives_the_same_bits():
    c = _case(24, [3000, 900, 5000, 64], H=40, latent=512)
    d = _to_dev(c)
    ws = mx.attn_workspace(4, 40, 512, d["block_table"].shape[1] * 64)
    first = mx.attn_paged(**d, workspace=ws)
    torch.cuda.synchronize()
    for _ in range(3):
        ws.fill_(255)
        again = mx.attn_paged(**d, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_two_streams_at_once():
    # calls that run at the same time, each with a workspace of its own (allocated by the call)
    cs = [_case(25 + i, [2000 + 100 * i, 70], H=32, latent=256) for i in range(2)]
    ds = [_to_dev(c) for c in cs]
    refs = [mx.attn_paged(**d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        got += [mx.attn_paged(**d, stream=s) for d, s in zip(ds, streams)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], refs[i % 2][0]) and torch.equal(g[1], refs[i % 2][1]), i


@pytest.mark.parametrize("k", [0, 300])
def test_graph_replays_match_eager(k):
    c = _case(27, [1200, 300, 64, 2500], H=64, latent=512, k=k)
    d = _to_dev(c)
    rng = np.random.default_rng(28)
    most = d["block_table"].shape[1] * 64
    ws = mx.attn_workspace(4, 64, 512, k or most)
    out, lse = mx.attn_paged(**d, workspace=ws)
    torch.cuda.synchronize()
    # two graphs that share the workspace, replayed in turn
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    half = {n: (v[:2] if isinstance(v, torch.Tensor) and n in ("q", "ke", "indices") else v) for n, v in d.items()}
    half["row_seq"] = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    out2, lse2 = torch.empty_like(out[:2]), torch.empty_like(lse[:2])
    with torch.cuda.graph(g):
        mx.attn_paged(**d, out=out, lse=lse, workspace=ws)
    with torch.cuda.graph(g2):
        mx.attn_paged(**half, out=out2, lse=lse2, workspace=ws)
    for rep in range(4):
        d["q"].copy_(torch.from_numpy(rng.standard_normal(c["q"].shape)))
        d["ke"].copy_(dev(rng.integers(0, 65, 4).astype(np.int32)) if rep == 2 else dev(c["ke"]))
        g.replay(), g2.replay(), g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, lse, out2, lse2)]
        _ = torch.randn(1000, device="cuda").sum().item()
        want = mx.attn_paged(**d) + mx.attn_paged(**half)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep


def test_no_rows_and_refusals():
    bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    q, cache = torch.zeros((4, 2, 320), **bf), torch.zeros((3, 64, 320), **bf)
    bt, ke = torch.zeros((2, 3), **i32), torch.ones(4, **i32)
    ok = dict(q=q, cache=cache, block_table=bt, ke=ke, scale=0.1)
    mx.attn_paged(**ok)
    out, lse = mx.attn_paged(q[:0], cache, bt, ke[:0], 0.1)
    assert out.shape == (0, 2, 256) and lse.shape == (0, 2)
    out, lse = mx.attn_paged(q, cache[:0], bt, ke, 0.1)       # no page: nothing is visible
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()
    for change in (dict(q=q.float()), dict(q=q[..., :256]), dict(q=q.transpose(1, 2)), dict(cache=cache.float()),
                   dict(cache=cache[..., :300]), dict(cache=cache[:, :32]), dict(block_table=bt.long()),
                   dict(block_table=bt.t()), dict(ke=ke[:3]), dict(ke=ke.long()), dict(ks=ke[:3]),
                   dict(row_seq=ke[:3]), dict(indices=bt), dict(indices=torch.zeros((4, 3), device="cuda")),
                   dict(max_tokens=193), dict(max_tokens=-1), dict(out=q), dict(lse=ke.float()),
                   dict(q=torch.zeros((4, 129, 320), **bf)), dict(q=q[:, :0]),
                   dict(q=q[:3], ke=ke[:3]), dict(ke=ke.cpu())):
        with pytest.raises(mx.MxidxError):
            mx.attn_paged(**{**ok, **change})
    need = mx.attn_workspace_bytes(4, 2, 256, 192)
    if need:
        with pytest.raises(mx.MxidxError):
            mx.attn_paged(**ok, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
