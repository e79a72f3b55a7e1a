"""kv8_attention's log-sum-exp where a score is NaN: NaN, as the output is, and not the -inf of a query that sees nothing."""
import math

import pytest
import torch

from kv8_reference import Cache
from test_gpu_kv8_attention import E4, I8, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("length", [40, 20000])   # one CTA; parts that CTAs join
def test_nan_scores_give_nan(cuda, dtype, length):
    lens = [length, 17, 0]
    cache = Cache(3, -(-length // 64), 2, 64, 64, dtype).fill(lens)
    if dtype == E4:
        cache.k.view(torch.uint8)[cache.table[0, 0], 1, 5, 9] = 0x7F
    else:
        cache.ks[cache.table[0, 0], 1] = math.nan
    q = queries(3, 1, 4, 64)
    out, lse = (t.cpu() for t in run(cuda, cache, lens, q))
    assert torch.isnan(out[0, 0, 2:]).all() and torch.isnan(lse[0, 0, 2:]).all()
    assert torch.isfinite(out[0, 0, :2]).all() and torch.isfinite(lse[0, 0, :2]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


def test_nan_query_gives_nan_for_its_head_alone(cuda):
    lens = [100]
    cache = Cache(1, 2, 1, 64, 64, I8).fill(lens)
    q = queries(1, 1, 4, 64)
    q[0, 0, 2, 7] = math.nan
    out, lse = (t.cpu() for t in run(cuda, cache, lens, q))
    bad = torch.tensor([False, False, True, False])
    assert torch.equal(torch.isnan(lse[0, 0]), bad) and torch.equal(torch.isnan(out[0, 0]).all(1), bad)
    assert torch.isfinite(out[0, 0, ~bad]).all()
