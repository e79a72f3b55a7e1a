"""kv8_attention against the formulas in fp64.

Tolerances, from the arithmetic that w4q.h promises.  The output is rounded once to bf16 (2^-8 relative).  A softmax
weight is off by its f16 rounding (2^-11) and by the error of its exponent: a score is an fp32 sum of at most 256
exact products, off by less than 2^-18 of sum |q| |k| scale = size, twice (the weight and the largest), plus
2^-20 for the exponential itself; each acts on sum w |v| = mag.  What f16 cannot hold is below 2^-31 of the largest
term of a sum for each of its positions.  lse: the same exponent's error, and n / 8 fp32 additions in a row."""
import math

import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q
from kv8_reference import Cache, attention

I8, E4 = torch.int8, torch.float8_e4m3fn
pytestmark = pytest.mark.gpu


def check(out, lse, cache, lens, q, scale, window):
    ref, mag, ref_lse, size = attention(cache, lens, q, scale, window)
    out, lse = out.cpu().double(), lse.cpu().double()
    longest = max(max(lens), 1)
    weight = 2.0 ** -11 + 2.0 ** -20 + size[..., None] * 2.0 ** -17
    tol = 2.0 ** -8 * ref.abs() + weight * mag * 1.01 + longest * 2.0 ** -31 * mag.amax(-1, keepdim=True) * 8 + 1e-38
    assert torch.isfinite(out).all()
    bad = (out - ref).abs() - tol
    assert (bad <= 0).all(), "off by %g over the tolerance" % bad.max()
    empty = torch.isinf(ref_lse)
    assert torch.equal(empty, torch.isinf(lse)) and (lse[empty] < 0).all()
    assert (out[empty] == 0).all()
    tol = (2.0 ** -18 + (longest / 8) * 2.0 ** -24 + 2.0 ** -22 * ref_lse.abs() + size * 2.0 ** -17)[~empty]
    assert ((lse - ref_lse)[~empty].abs() <= tol).all()


def run(cuda, cache, lens, q, scale=None, window=0, workspace=None):
    kc, vc, ks, vs, table = cache.to(cuda)
    n, m, hq, d = q.shape
    lse = torch.full((n, m, hq), math.nan, device=cuda)
    out = torch.full((n, m, hq, d), math.nan, dtype=torch.bfloat16, device=cuda)
    w4q.kv8_attention(q.to(cuda), kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device=cuda),
                      scale=scale, window=window, out=out, lse=lse, workspace=workspace)
    return out, lse


def queries(n, m, hq, d, seed=5, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, m, hq, d, generator=g) * size).to(torch.bfloat16)


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,m", [(1, 1, 1), (8, 1, 1), (6, 2, 1), (10, 2, 3), (16, 1, 4)])
def test_against_fp64(cuda, dtype, d, page, hq, hkv, m):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 300]
    cache = Cache(len(lens), -(-300 // page), hkv, d, page, dtype).fill(lens)
    q = queries(len(lens), m, hq, d)
    check(*run(cuda, cache, lens, q), cache, lens, q, d ** -0.5, 0)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1 << 40])
@pytest.mark.parametrize("dtype,d,m", [(I8, 64, 1), (E4, 128, 5)])
def test_windows(cuda, window, dtype, d, m):
    lens = [3, 16, 40, 99, 260, 1, 0]
    cache = Cache(len(lens), 17, 2, d, 16, dtype).fill(lens)
    q = queries(len(lens), m, 4, d)
    check(*run(cuda, cache, lens, q, window=window), cache, lens, q, d ** -0.5, min(window, 1 << 20))


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("d,hkv,hq,m,length", [(64, 1, 5, 1, 50001), (128, 2, 8, 2, 30011), (256, 1, 2, 1, 9001)])
def test_one_long_sequence_is_split_and_joined(cuda, dtype, d, hkv, hq, m, length):
    cache = Cache(1, -(-length // 128), hkv, d, 128, dtype).fill([length])
    q = queries(1, m, hq, d)
    check(*run(cuda, cache, [length], q), cache, [length], q, d ** -0.5, 0)


def test_uneven_batch(cuda):
    lens = [7000, 1, 0, 333, 64, 64, 2, 900, 5, 0, 0, 4111]
    cache = Cache(len(lens), 110, 3, 128, 64, I8).fill(lens)
    q = queries(len(lens), 1, 21, 128)
    check(*run(cuda, cache, lens, q), cache, lens, q, 128 ** -0.5, 0)


def test_many_idle_sequences(cuda):
    lens = [0] * 700
    lens[3], lens[650] = 100, 40
    cache = Cache(700, 2, 1, 64, 64, I8).fill(lens)
    q = queries(700, 1, 2, 64)
    check(*run(cuda, cache, lens, q), cache, lens, q, 0.125, 0)


@pytest.mark.parametrize("size,scale", [(2.0 ** -100, None), (2.0 ** -133, 1e6), (2.0 ** 60, 2.0 ** -63), (30.0, None), (0.0, None)])
def test_query_magnitudes(cuda, size, scale):
    lens = [200, 70]
    cache = Cache(2, 4, 2, 128, 64, I8).fill(lens)
    q = queries(2, 1, 8, 128, size=size)
    q[0, 0, 1] = 0
    check(*run(cuda, cache, lens, q, scale=scale), cache, lens, q, 128 ** -0.5 if scale is None else scale, 0)


@pytest.mark.parametrize("spread", [3.0, 20.0, 40.0])
@pytest.mark.parametrize("dtype", [I8, E4])
def test_scales_far_apart(cuda, spread, dtype):
    lens = [1000, 130]
    cache = Cache(2, 63, 2, 64, 16, dtype).fill(lens, spread=spread)
    cache.vs[cache.table[0, 3]] = 0.0
    q = queries(2, 1, 4, 64)
    check(*run(cuda, cache, lens, q), cache, lens, q, 0.125, 0)


def test_all_values_zero(cuda):
    cache = Cache(1, 2, 1, 64, 64, I8).fill([100])
    cache.vs[:] = 0.0
    q = queries(1, 1, 1, 64)
    check(*run(cuda, cache, [100], q), cache, [100], q, 0.125, 0)


@pytest.mark.parametrize("dtype", [I8, E4])
def test_holes_in_the_table_are_left_out(cuda, dtype):
    lens = [200, 64, 300]
    cache = Cache(3, 5, 2, 128, 64, dtype).fill(lens)
    cache.table[0, 1] = -1
    cache.table[1, 0] = -7        # nothing left of this one
    cache.table[2, 4] = cache.blocks
    q = queries(3, 1, 4, 128)
    check(*run(cuda, cache, lens, q), cache, lens, q, 128 ** -0.5, 0)


def test_lengths_beyond_the_table_and_below_zero(cuda):
    cache = Cache(3, 2, 1, 64, 16, I8).fill([32, 32, 32])
    q = queries(3, 1, 2, 64)
    out, lse = run(cuda, cache, [1000, -5, 32], q)
    check(out, lse, cache, [32, 0, 32], q, 0.125, 0)


def test_strided_queries(cuda):
    lens = [77, 140]
    cache = Cache(2, 3, 2, 64, 64, E4).fill(lens)
    wide = queries(2 * 3, 1, 12, 64).view(6, 12 * 64).to(cuda)   # 8 query heads of 12 in a projection's row
    q = wide[:, :512].view(2, 3, 8, 64)
    kc, vc, ks, vs, table = cache.to(cuda)
    lse = torch.empty(2, 3, 8, device=cuda)
    out = w4q.kv8_attention(q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device=cuda), lse=lse)
    check(out, lse, cache, lens, q.cpu(), 0.125, 0)


def test_one_workspace_serves_calls_of_any_size(cuda):
    cases = [(1, 1, 20000, 1, 8, 128), (40, 1, 500, 8, 8, 64), (1, 2, 9000, 2, 16, 64), (3, 1, 3000, 1, 4, 256)]
    need = max(w4q.kv8_workspace_bytes(n, m, hq, hkv, d) for n, m, _, hkv, hq, d in cases)
    ws = torch.zeros(need, dtype=torch.uint8, device=cuda)
    for n, m, length, hkv, hq, d in cases + cases[::-1]:
        lens = [length - i for i in range(n)]
        cache = Cache(n, -(-length // 64), hkv, d, 64, I8).fill(lens)
        q = queries(n, m, hq, d)
        a = run(cuda, cache, lens, q, workspace=ws)
        b = run(cuda, cache, lens, q, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        if n < 40:
            check(*a, cache, lens, q, d ** -0.5, 0)


def test_graph_replay_follows_the_lengths(cuda):
    full = [900, 20, 333]
    cache = Cache(3, 15, 2, 128, 64, I8).fill(full)
    q = queries(3, 1, 8, 128)
    kc, vc, ks, vs, table = cache.to(cuda)
    qd, lens = q.to(cuda), torch.tensor(full, dtype=torch.int32, device=cuda)
    ws = torch.zeros(w4q.kv8_workspace_bytes(3, 1, 8, 2, 128), dtype=torch.uint8, device=cuda)
    out, lse = torch.empty(3, 1, 8, 128, dtype=torch.bfloat16, device=cuda), torch.empty(3, 1, 8, device=cuda)

    def call():
        w4q.kv8_attention(qd, kc, vc, ks, vs, table, lens, out=out, lse=lse, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([900, 20, 333], [1, 0, 64], [640, 19, 200]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, cache, now, q, 128 ** -0.5, 0)


def test_on_a_stream_of_its_own(cuda):
    lens = [500, 90]
    cache = Cache(2, 8, 2, 64, 64, I8).fill(lens)
    q = queries(2, 1, 8, 64)
    args = [q.to(cuda), *cache.to(cuda), torch.tensor(lens, dtype=torch.int32, device=cuda)]
    lse = torch.empty(2, 1, 8, device=cuda)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    out = w4q.kv8_attention(*args, lse=lse, stream=stream)
    stream.synchronize()
    check(out, lse, cache, lens, q, 0.125, 0)


def test_offsets_beyond_32_bits(cuda):
    hkv, page, d = 8, 64, 128
    blocks = (1 << 32) // (hkv * page * d) + 40
    small = Cache(2, 4, hkv, d, page, I8).fill([200, 256])
    kc, vc = (torch.empty(blocks, hkv, page, d, dtype=I8, device=cuda) for _ in range(2))
    ks, vs = (torch.empty(blocks, hkv, device=cuda) for _ in range(2))
    at = torch.arange(blocks - small.blocks, blocks, device=cuda)
    kc[at], vc[at], ks[at], vs[at] = (t.to(cuda) for t in (small.k, small.v, small.ks, small.vs))
    table = (small.table + (blocks - small.blocks)).to(cuda)
    q = queries(2, 1, 16, d)
    lse = torch.empty(2, 1, 16, device=cuda)
    out = w4q.kv8_attention(q.to(cuda), kc, vc, ks, vs, table, torch.tensor([200, 256], dtype=torch.int32, device=cuda), lse=lse)
    check(out, lse, small, [200, 256], q, d ** -0.5, 0)
