"""GPU parity of idx_attn_paged_mxfp4 on both sides of the size up to which 32-bit offsets reach the
cache, against the float64 oracle: every latent size in every grouping of heads and tile, split and
whole, windows and lists with holes, pages outside the cache; page 0 and every place that no row
sees hold scale bytes of no number and NaN.  Tolerances: oracle/latent_attn.py."""

import numpy as np
import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx
from oracle import latent_attn as oattn, latent_mxfp4 as olm
from tests.gpu_helpers import dev
from tests.test_gpu_attn_mxfp4 import _case, _close, _poisoned

pytestmark = pytest.mark.gpu

REACH = 0xfffe0000                          # of the 32-bit offsets

# rows of one sequence x heads -> 16, 32 and 64 heads a workgroup, the last with 64- and 32-token tiles and
# with the tokens split
FORMS = [(3, 12), (200, 16), (3, 32), (200, 30), (130, 128), (520, 64), (60, 128)]


def _rows_close(got, c, pick, what=""):
    """Rows `pick` of a call over one sequence against the oracle."""
    cut = lambda n: None if c[n] is None else c[n][pick]  # noqa: E731
    rows = olm.values(c["cache"], c["latent"]).reshape(c["pages"], 64, -1)
    want = oattn.attn(c["q"][pick], rows, c["bt"], c["ke"][pick], c["scale"], cut("indices"), cut("ks"),
                      np.zeros(len(pick), np.int32))
    _close((got[0][dev(pick)], got[1][dev(pick)]), want, what)


def _placed(c, pages, used):
    """The case's call over a cache of `pages` pages whose pages `used` hold the sequence's tokens."""
    cache = torch.full((pages, 64 * olm.row_bytes(c["latent"])), 0xFF, dtype=torch.uint8, device="cuda")
    table = c["bt"].copy()
    for i, p in enumerate(c["bt"][0]):
        if 0 <= p < c["pages"]:
            cache[int(used[i])] = dev(_poisoned(c)[p])
            table[0, i] = used[i]
        else:
            table[0, i] = -1 if p < 0 else pages
    opt = lambda n: None if c[n] is None else dev(c[n])  # noqa: E731
    return dict(q=torch.from_numpy(c["q"]).to(torch.bfloat16).cuda(), cache=cache, block_table=dev(table),
                ke=dev(c["ke"]), scale=c["scale"], indices=opt("indices"), ks=opt("ks"))


def _used(pages, page_bytes, n):
    """Page numbers for a sequence of n tokens: the last ones, those around byte 2^31, and others; not page 0."""
    middle = (1 << 31) // page_bytes
    used = [pages - 1, middle, middle + 1, pages - 2, 1, middle - 1, pages // 3]
    return np.array((used + list(range(10, 40)))[:(n + 63) // 64])


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("over", [0, 1])
@pytest.mark.parametrize("rows,H", FORMS)
@pytest.mark.parametrize("k", [0, 600])
def test_rows_on_both_sides_of_4_gib(latent, over, rows, H, k):
    # the largest cache that 32-bit offsets reach, and one page more
    page_bytes = 64 * olm.row_bytes(latent)
    pages = REACH // page_bytes + over
    n = 500 if rows > 60 else 1400
    c = _case(rows + H, [n], next_n=rows, H=H, latent=latent, k=k)
    got = mx.attn_paged_mxfp4(**_placed(c, pages, _used(pages, page_bytes, n)))
    torch.cuda.synchronize()
    _rows_close(got, c, np.unique(np.linspace(0, rows - 1, 9).astype(np.int64)))


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("rows,H", FORMS)
def test_places_without_a_row_beyond_4_gib(latent, rows, H):
    # a page of the table outside the cache on either side, windows that end inside every tile, empty lists
    page_bytes = 64 * olm.row_bytes(latent)
    pages, n = REACH // page_bytes + 1, 333
    for k in (0, 150):
        c = _case(rows + H + k, [n], next_n=rows, H=H, latent=latent, k=k)
        c["bt"][0, 1], c["bt"][0, 3] = -1, c["pages"]
        c["ke"][::4] = np.arange(len(c["ke"][::4])) % 130
        if k:
            c["indices"][1::4] = -1
        got = mx.attn_paged_mxfp4(**_placed(c, pages, _used(pages, page_bytes, n)))
        torch.cuda.synchronize()
        _rows_close(got, c, np.unique(np.concatenate([np.arange(3), np.linspace(0, rows - 1, 9).astype(np.int64)])), k)
