"""Lengths that pass the block table: positions beyond it are nowhere.  The writer drops them, the reader gives zeros, and the
attention goes up to the table's last position."""
import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q
from kv8_reference import Cache
from test_gpu_kv8_append import E4, I8, emulate, prefix, rows, same
from test_gpu_kv8_attention import check, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [I8, E4])
def test_positions_beyond_the_table(cuda, dtype):
    lens, counts, room = [40, 32, 70], [10, 3, 6], 32    # the last sequence lies beyond its table with all its new tokens
    cache = Cache(3, 2, 2, 64, 16, dtype).fill([30, 29, 32])
    dev = cache.to(cuda)
    n = sum(counts)
    k, v = rows(n, 2, 64, 1), rows(n, 2, 64, 2)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=cuda)
    w4q.kv8_append(k.to(cuda), v.to(cuda), *dev, lens_d, cu_tokens=prefix(counts, cuda))
    inside = [0, 1, 10, 11, 12]                          # positions 30, 31 and 29, 30, 31
    emulate(cache, "k", k[inside].float(), [room, room, room], [2, 3, 0])
    emulate(cache, "v", v[inside].float(), [room, room, room], [2, 3, 0])
    same(cache, dev[:4])
    kr, vr = w4q.kv8_read(*dev, lens_d, cu_tokens=prefix(counts, cuda), tokens=n)
    outside = torch.tensor([i for i in range(n) if i not in inside], device=cuda)
    assert (kr[outside] == 0).all() and (vr[outside] == 0).all()
    want, _ = w4q.kv8_read(*dev, torch.full((3,), room, dtype=torch.int32, device=cuda), cu_tokens=prefix([2, 3, 0], cuda), tokens=5)
    assert torch.equal(kr[inside], want) and (want != 0).any()
    q = queries(3, 1, 4, 64)
    out, lse = run(cuda, cache, lens, q)
    check(out, lse, cache, [room] * 3, q, 0.125, 0)
