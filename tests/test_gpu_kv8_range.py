"""kv8_attention at the ends of the ranges of scores and scales."""
import pytest
import torch

from kv8_reference import Cache
from test_gpu_kv8_attention import I8, run

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
