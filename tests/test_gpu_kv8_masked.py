"""kv8_attention where NaN or infinity stands at positions or in pages that some queries of a call do not see: drafts that
come before it, and windows that begin after it.  They change nothing there; a query that sees a NaN value has NaN in that
element alone."""
import math

import pytest
import torch

from kv8_reference import Cache, attention
from test_gpu_kv8_attention import E4, I8, queries, run

pytestmark = pytest.mark.gpu


def check(got, cache, lens, q, scale, window):
    """As the finite calls' check, with NaN where the formulas have NaN."""
    out, lse = (t.cpu().double() for t in got)
    ref, mag, ref_lse, size = attention(cache, lens, q, scale, window)
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    weight = 2.0 ** -11 + 2.0 ** -20 + size[..., None] * 2.0 ** -17
    top = torch.nan_to_num(mag).amax(-1, keepdim=True)
    tol = 2.0 ** -8 * ref.abs() + weight * mag * 1.01 + max(lens) * 2.0 ** -31 * top * 8 + 1e-38
    ok = ~torch.isnan(ref)
    assert ((out - ref).abs()[ok] <= tol[ok]).all()
    tol = 2.0 ** -18 + (max(lens) / 8) * 2.0 ** -24 + 2.0 ** -22 * ref_lse.abs() + size * 2.0 ** -17
    assert ((lse - ref_lse).abs() <= tol).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,m", [(1, 5), (4, 4), (3, 8), (8, 8)])
@pytest.mark.parametrize("window", [0, 20])
def test_nan_values_of_drafts(cuda, d, hq, m, window):
    lens = [37, 66, 9]
    cache = Cache(3, 5, 1, d, 16, E4).fill(lens)
    for b, back in ((0, 2), (1, 1), (1, 4), (2, 3)):
        pos = lens[b] - back
        for dim in (3 * b, 3 * b + 1, d - 1 - back):
            cache.v.view(torch.uint8)[cache.table[b, pos // 16], 0, pos % 16, dim] = 0x7F if dim % 2 else 0xFF
    q = queries(3, m, hq, d)
    got = run(cuda, cache, lens, q, window=window)
    assert torch.isnan(got[0]).any() and not torch.isnan(got[0][:, 0]).all()
    check(got, cache, lens, q, d ** -0.5, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m", [1, 3])
def test_nan_values_before_the_window(cuda, d, m):
    lens, window = [40, 500], 10
    cache = Cache(2, 32, 2, d, 16, E4).fill(lens)
    for b in range(2):
        for pos in range(lens[b] - 24, lens[b] - m - window + 1):
            cache.v.view(torch.uint8)[cache.table[b, pos // 16], :, pos % 16] = 0x7F
    q = queries(2, m, 4, d)
    got = run(cuda, cache, lens, q, window=window)
    assert torch.isfinite(got[0]).all()
    check(got, cache, lens, q, d ** -0.5, window)


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("page", [1, 3])      # seen by the first query alone, by the last alone
@pytest.mark.parametrize("which", ["k", "v"])
def test_scales_of_pages_that_one_query_sees(cuda, dtype, value, page, which):
    lens, window, m = [49], 16, 3             # queries at 46, 47, 48
    cache = Cache(1, 4, 1, 64, 16, dtype).fill(lens)
    q = queries(1, m, 4, 64)
    want = run(cuda, cache, lens, q, window=window)
    (cache.ks if which == "k" else cache.vs)[cache.table[0, page]] = value
    got = run(cuda, cache, lens, q, window=window)
    sees = 0 if page == 1 else 2
    others = [i for i in range(m) if i != sees]
    if which == "v" or math.isnan(value):         # (a score of -inf has weight 0)
        assert not torch.isfinite(got[0][0, sees]).any()
    assert torch.isfinite(got[0][0, others]).all()
    # the reference of the running sum may differ, so not bit for bit: two roundings to bf16 and to 11 bits
    assert (got[0][0, others].float() - want[0][0, others].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()
    rows = range(m) if which == "v" else others   # the log-sum-exp is the keys' alone
    for i in rows:
        assert ((got[1][0, i] - want[1][0, i]).abs() <= 1e-5).all()
