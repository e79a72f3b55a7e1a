"""kv8_attention at the ends of the ranges of scores and scales."""
import pytest
import torch

from kv8_reference import Cache, attention
from test_gpu_kv8_attention import E4, I8, check, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e30, -1e30, 1e33, -1e33])
def test_scores_of_any_finite_size_are_seen(cuda, d, size):
    """One position: its weight is 1, whatever its score is."""
    lens = [1, 1]
    cache = Cache(2, 1, 1, d, 16, I8).fill(lens)
    cache.k[:] = 1
    cache.ks[:] = 1.0
    q = torch.full((2, 1, 3, d), size / d, dtype=torch.bfloat16)
    out, lse = (t.cpu().double() for t in run(cuda, cache, lens, q, scale=1.0))
    score = q.double().sum(-1)
    assert ((lse - score).abs() <= 2.0 ** -20 * score.abs()).all()
    for b in range(2):
        blk = int(cache.table[b, 0])
        v = (cache.v[blk, 0, 0].double() * cache.vs[blk, 0].double()).expand(3, d)
        assert ((out[b, 0] - v).abs() <= 2.0 ** -8 * v.abs() + 2.0 ** -11 * v.abs()).all()


def small(dtype, lens, e):
    """A cache whose scales of values are spread by a factor of 12 from 2^e up."""
    cache = Cache(len(lens), -(-max(lens) // 16), 2, 64, 16, dtype).fill(lens)
    g = torch.Generator().manual_seed(9)
    there = ~torch.isnan(cache.vs)
    cache.vs[there] = (2.0 ** e * (1 + 11 * torch.rand(cache.vs.shape, generator=g)))[there]
    return cache


@pytest.mark.parametrize("e", [-80, -70, 70])
@pytest.mark.parametrize("dtype", [I8, E4])
def test_value_scales_far_from_one(cuda, e, dtype):
    lens = [1000, 130, 1]
    cache, q = small(dtype, lens, e), queries(3, 1, 4, 64)
    out, lse = run(cuda, cache, lens, q)
    check(out, lse, cache, lens, q, 0.125, 0)
    assert (out.float().abs().amax(-1) > 0).all()


@pytest.mark.parametrize("dtype", [I8, E4])
def test_value_scales_of_2_to_the_minus_100_keep_fewer_bits(cuda, dtype):
    """The largest weight is then at least 2^(84 - 100 + 7) in f16, whose step there is 2^-24: every position is off by at
    most 2^-16 of the largest term, whose value's elements are within a factor of 4.5 (448 / 100) of any other's."""
    lens = [1, 16, 130]
    cache, q = small(dtype, lens, -100), queries(3, 1, 4, 64)
    out, _ = run(cuda, cache, lens, q)
    ref, mag, _, size = attention(cache, lens, q, 0.125, 0)
    weight = 2.0 ** -11 + 2.0 ** -20 + size[..., None] * 2.0 ** -17
    n = torch.tensor(lens).view(3, 1, 1, 1)
    tol = 2.0 ** -8 * ref.abs() + weight * mag * 1.01 + n * 4.5 * 2.0 ** -16 * mag.amax(-1, keepdim=True)
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    assert (out.float().abs().amax(-1) > 0).all()
