"""kv8_attention for every number of query rows that a kv head can have: each padded tile shape, and several tiles."""
import pytest

from test_gpu_kv8_attention import E4, I8, check, queries, run
from kv8_reference import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,m", [(7, 1), (9, 1), (3, 5), (17, 1), (5, 4), (24, 1), (5, 5), (31, 1), (8, 5), (7, 7), (16, 4), (1, 64)])
def test_rows(cuda, d, hq, m):
    lens = [1, 63, 70, 500, 0]
    cache = Cache(len(lens), 8, 1, d, 64, E4 if d == 64 else I8).fill(lens)
    q = queries(len(lens), m, hq, d)
    check(*run(cuda, cache, lens, q), cache, lens, q, d ** -0.5, 0)
    check(*run(cuda, cache, lens, q, window=33), cache, lens, q, d ** -0.5, 33)


@pytest.mark.parametrize("d,hq,m", [(64, 5, 4), (64, 8, 5), (128, 8, 6)])
def test_rows_of_a_long_sequence(cuda, d, hq, m):
    lens = [12345, 700]
    cache = Cache(2, 97, 2, d, 128, I8).fill(lens)
    q = queries(2, m, 2 * hq, d)
    check(*run(cuda, cache, lens, q), cache, lens, q, d ** -0.5, 0)
