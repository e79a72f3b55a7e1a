"""kv8_append where a new row holds NaN or infinity.  e4m3 has a code for what is not a finite number: the element gets it and
has no part in the scale.  int8 has none: the scale of the page and head becomes NaN, so that all of it reads as NaN."""
import math

import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q
from kv8_reference import Cache
from test_gpu_kv8_append import E4, I8, emulate, prefix, rows, same

pytestmark = pytest.mark.gpu
BAD = [math.nan, math.inf, -math.inf]


def append(cuda, dev, k, v, lens, counts, one):
    w4q.kv8_append(k.to(cuda), v.to(cuda), *dev, torch.tensor(lens, dtype=torch.int32, device=cuda),
                   cu_tokens=None if one else prefix(counts, cuda))


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("counts", [None, [1, 1, 1], [40, 3, 9], [300, 0, 2]])
def test_e4m3_keeps_them_as_nan_codes(cuda, bad, d, counts):
    before, one = [5, 16, 0], counts is None
    counts = counts or [1, 1, 1]
    lens, n = [a + c for a, c in zip(before, counts)], sum(counts)
    cache = Cache(3, 32, 2, d, 16, E4).fill(before)
    dev = cache.to(cuda)
    k, v = rows(n, 2, d, 1), rows(n, 2, d, 2)
    last = n - 1
    # the formulas' codes with the elements left out (0 has no part in a maximum), then their own code
    emulate(cache, "k", k.float().index_put((torch.tensor(0), torch.tensor(1), torch.tensor(3)), torch.tensor(0.0)), lens, counts)
    wrote = emulate(cache, "v", v.float().index_put((torch.tensor(last), torch.tensor(0), torch.tensor(d - 1)), torch.tensor(0.0)),
                    lens, counts)
    for blk, slot, token in wrote:
        if token == 0:
            cache.k.view(torch.uint8)[blk, 1, slot, 3] = 0x7F
        if token == last:
            cache.v.view(torch.uint8)[blk, 0, slot, d - 1] = 0x7F
    k[0, 1, 3], v[last, 0, d - 1] = bad, bad
    append(cuda, dev, k, v, lens, counts, one)
    same(cache, dev[:4])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("one", [True, False])
def test_e4m3_row_of_nothing_else(cuda, bad, one):
    """No finite element but zeros: the scale is 0 and the codes still tell."""
    cache = Cache(1, 1, 1, 64, 16, E4)
    dev = cache.to(cuda)
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    k[0, 0, 10] = bad
    append(cuda, dev, k, k, [1], [1], one)
    kr, vr = w4q.kv8_read(*dev, torch.tensor([1], dtype=torch.int32, device=cuda))
    for t in (kr, vr):
        assert torch.isnan(t[0, 0, 10]) and (t[0, 0, torch.arange(64, device=cuda) != 10] == 0).all()


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("one", [True, False])
def test_int8_marks_the_page(cuda, bad, d, page, one):
    """The page of the bad element reads as NaN, now and after further tokens; other pages, heads and sequences do not."""
    before = [3, page - 1, 0]
    cache = Cache(3, 4, 2, d, page, I8).fill(before)
    dev = cache.to(cuda)
    lens = list(before)
    for step in range(3):
        counts = [1, 1, 1] if one else [2, 3, page + 1]
        lens = [a + c for a, c in zip(lens, counts)]
        n = sum(counts)
        k, v = rows(n, 2, d, 10 + step), rows(n, 2, d, 20 + step)
        kk = k.clone()
        if step == 0:
            k[0, 1, 3] = bad
        emulate(cache, "k", kk.float(), lens, counts)
        emulate(cache, "v", v.float(), lens, counts)
        append(cuda, dev, k, v, lens, counts, one)
    kr, _ = w4q.kv8_read(*dev, torch.tensor(lens, dtype=torch.int32, device=cuda), cu_tokens=prefix(lens, cuda), tokens=sum(lens))
    ks = dev[2].cpu()
    marked = int(cache.table[0, 0])
    assert torch.isnan(ks[marked, 1])
    cache.ks[marked, 1] = math.nan
    cache.k[marked, 1] = dev[0][marked, 1].cpu()   # codes without a scale
    same(cache, dev[:4])
    first = kr[:min(lens[0], page)].cpu()
    assert torch.isnan(first[:, 1]).all() and torch.isfinite(first[:, 0]).all() and torch.isfinite(kr[page:].cpu()).all()


def test_int8_marked_page_begins_anew(cuda):
    cache = Cache(1, 1, 1, 64, 16, I8)
    dev = cache.to(cuda)
    k = rows(1, 1, 64, 1)
    append(cuda, dev, k * math.nan, k, [1], [1], True)
    assert torch.isnan(dev[2].cpu()[cache.table[0, 0], 0])
    append(cuda, dev, k, k, [1], [1], True)
    emulate(cache, "k", k.float(), [1], [1])
    emulate(cache, "v", k.float(), [1], [1])
    same(cache, dev[:4])
