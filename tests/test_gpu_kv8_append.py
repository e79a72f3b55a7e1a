"""qk_norm_rope, kv8_append and kv8_read.

A row without norm and rotation is quantized bit for bit as the fp32 formulas say.  With them a normed element is off by
at most 2^-20 of its row's largest (a sum of head_dim squares, a square root, five roundings), so a scale is off by
2^-20 relative and a code goes to a neighbour only where its quotient lies within 2^-12 of a rounding's edge."""
import math

import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q
from kv8_reference import TOP, Cache, encode, norm_rope, rope_table

I8, E4 = torch.int8, torch.float8_e4m3fn
pytestmark = pytest.mark.gpu


def rows(n, heads, d, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, d, generator=g) * size).to(torch.bfloat16)


def near(out, ref):
    """bf16 of fp64 rows, whose elements were off by 2^-20 of the row's largest."""
    ref, out = ref.double(), out.cpu().double()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -19 * ref.abs().amax(-1, keepdim=True)
    assert ((out - ref).abs() <= tol).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 0), (3, 5, 2), (64, 32, 8), (1500, 9, 3)])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, True), (32, False), (64, True), (64, False)])
@pytest.mark.parametrize("weights", ["qk", "q", ""])
def test_norm_rope(cuda, d, tokens, hq, hk, rot, interleaved, weights):
    q, k = rows(tokens, hq, d, 1), rows(tokens, max(hk, 1), d, 2)
    qw, kw = rows(1, 1, d, 3)[0, 0], rows(1, 1, d, 4)[0, 0]
    table = rope_table(999, rot) if rot else None
    pos = torch.randint(0, 999, (tokens,), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    dev = lambda t: None if t is None else t.to(cuda)  # noqa: E731
    qo, ko = w4q.qk_norm_rope(dev(q), dev(k) if hk else None, dev(qw) if "q" in weights else None,
                              dev(kw) if "k" in weights else None, dev(table), dev(pos), eps=1e-5, interleaved=interleaved)
    near(qo, norm_rope(q, qw if "q" in weights else None, table, pos, 1e-5, interleaved))
    if hk:
        near(ko, norm_rope(k, kw if "k" in weights else None, table, pos, 1e-5, interleaved))
    else:
        assert ko is None


def test_norm_rope_whole_head_strided_and_by_token_number(cuda):
    d, hq, hk, n = 128, 6, 2, 50
    qkv = rows(n, hq + 2 * hk + 1, d, 9).view(n, -1).to(cuda)
    q, k = qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    table = rope_table(n, d)
    qo, ko = w4q.qk_norm_rope(q, k, None, None, table.to(cuda))
    near(qo, norm_rope(q.cpu(), None, table, torch.arange(n), 0, False))
    near(ko, norm_rope(k.cpu(), None, table, torch.arange(n), 0, False))


def test_norm_rope_of_zero_and_tiny_and_huge_rows(cuda):
    q = rows(4, 1, 64, 1)
    q[0] = 0
    q[1] *= 2.0 ** -60
    q[2] *= 2.0 ** 50
    w = rows(1, 1, 64, 2)[0, 0]
    out, _ = w4q.qk_norm_rope(q.to(cuda), None, w.to(cuda), eps=1e-6)
    near(out, norm_rope(q, w, None, None, 1e-6, False))
    assert (out[0] == 0).all()


def test_positions_outside_the_table_use_its_ends(cuda):
    q, table = rows(3, 2, 64, 1), rope_table(10, 64)
    out, _ = w4q.qk_norm_rope(q.to(cuda), None, cos_sin=table.to(cuda),
                              positions=torch.tensor([-3, 10, 1 << 30], dtype=torch.int32, device=cuda))
    near(out, norm_rope(q, None, table, torch.tensor([0, 9, 9]), 0, False))


def emulate(cache, which, x, lens, counts):
    """The writer's rule on fp32 rows x [tokens, heads, d]; returns [(page, head, slot, x row)] of the new tokens."""
    c, s = (cache.k, cache.ks) if which == "k" else (cache.v, cache.vs)
    top, page, at, wrote = torch.tensor(TOP[cache.dtype]), cache.page, 0, []
    for b, n in enumerate(counts):
        before = lens[b] - n
        for i in range(before // page, -(-lens[b] // page) if n else 0):
            lo, hi = max(before, i * page), min(lens[b], (i + 1) * page)
            blk = int(cache.table[b, i])
            if lo < hi and 0 <= blk < cache.blocks:
                y = x[at + lo - before:at + hi - before]                     # [new, heads, d]
                held = max(0, before - i * page)
                old = s[blk].clone() if held else torch.zeros(x.shape[1])
                new = torch.maximum(y.abs().amax((0, 2)) / top, old)
                r = torch.where(new > old, old / new, torch.ones(()))
                if held:
                    codes = encode(c[blk, :, :held].float() * r[:, None, None], torch.ones(()), cache.dtype)
                    grew = (new > old)[:, None, None]
                    c[blk, :, :held] = torch.where(grew, codes, c[blk, :, :held].float()).to(cache.dtype)
                s[blk] = new
                codes = encode(y.transpose(0, 1), new[:, None, None], cache.dtype).to(cache.dtype)
                c[blk, :, lo - i * page:hi - i * page] = codes
                wrote += [(blk, lo - i * page + j, at + lo - before + j) for j in range(hi - lo)]
        at += n
    return wrote


def prefix(counts, cuda):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(cuda)


def same(cache, device_tensors):
    kc, vc, ks, vs = (t.cpu() for t in device_tensors)
    for mine, theirs in ((cache.k, kc), (cache.v, vc)):
        assert torch.equal(mine.view(torch.uint8), theirs.view(torch.uint8))
    for mine, theirs in ((cache.ks, ks), (cache.vs, vs)):
        assert torch.equal(torch.nan_to_num(mine, -1.0), torch.nan_to_num(theirs, -1.0))


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128), (256, 64), (256, 128)])
@pytest.mark.parametrize("one", [True, False])
def test_codes_bit_for_bit_over_several_steps(cuda, dtype, d, page, one):
    hkv = 3
    plan = [[1] * 5] * 4 if one else [[0, 1, 37, 200, 5], [3, 0, 1, 129, 64], [1, 1, 1, 0, 300]]
    lens = [0, 1, page - 1, 2 * page - 2, 30]
    width = -(-1000 // page)
    cache = Cache(5, width, hkv, d, page, dtype).fill(lens)
    dev = cache.to(cuda)
    for step, counts in enumerate(plan):
        lens = [a + n for a, n in zip(lens, counts)]
        n = sum(counts)
        k, v = rows(n, hkv, d, 10 + step, 1.0 + step), rows(n, hkv, d, 50 + step, 3.0 - step)
        k[n // 2] = 0
        emulate(cache, "k", k.float(), lens, counts)
        emulate(cache, "v", v.float(), lens, counts)
        w4q.kv8_append(k.to(cuda), v.to(cuda), *dev, torch.tensor(lens, dtype=torch.int32, device=cuda),
                       cu_tokens=None if one else prefix(counts, cuda))
        same(cache, dev[:4])


@pytest.mark.parametrize("dtype", [I8, E4])
def test_a_page_of_zeros_then_values_then_growth(cuda, dtype):
    cache = Cache(1, 1, 1, 64, 16, dtype)
    dev = cache.to(cuda)
    for i, size in enumerate([0.0, 1.0, 0.25, 64.0, 2.0 ** -130, 2.0 ** 100]):
        k, v = rows(1, 1, 64, i, size), rows(1, 1, 64, 99 + i, size)
        emulate(cache, "k", k.float(), [i + 1], [1])
        emulate(cache, "v", v.float(), [i + 1], [1])
        w4q.kv8_append(k.to(cuda), v.to(cuda), *dev, torch.tensor([i + 1], dtype=torch.int32, device=cuda))
        same(cache, dev[:4])


@pytest.mark.parametrize("one", [True, False])
def test_idle_sequences_holes_and_full_tables_write_nothing(cuda, one):
    cache = Cache(4, 2, 2, 64, 16, I8).fill([0, 0, 0, 8])
    cache.table[2, 0] = -1
    dev = cache.to(cuda)
    lens, counts = [0, 33, 5, 9], [1, 1, 1, 1]                # idle; past its table; a hole; ordinary
    k, v = rows(4, 2, 64, 1), rows(4, 2, 64, 2)
    quiet = [0, 0, 0, 9]
    at = [0, 0, 0, 1]
    emulate(cache, "k", k[3:].float(), quiet, at)
    emulate(cache, "v", v[3:].float(), quiet, at)
    w4q.kv8_append(k.to(cuda), v.to(cuda), *dev, torch.tensor(lens, dtype=torch.int32, device=cuda),
                   cu_tokens=None if one else prefix(counts, cuda))
    same(cache, dev[:4])


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("d,rot,interleaved,norm", [(64, 64, False, True), (128, 64, True, True), (256, 256, False, False)])
@pytest.mark.parametrize("counts", [None, [0, 70, 1, 0, 20]])
def test_fused_norm_and_rotation(cuda, dtype, d, rot, interleaved, norm, counts):
    hq, hkv, page, before = 6, 2, 32, [0, 3, 31, 32, 100]
    one = counts is None
    counts = counts or [1] * 5
    lens = [a + n for a, n in zip(before, counts)]
    n = sum(counts)
    cache = Cache(5, 8, hkv, d, page, dtype).fill(before)
    dev = cache.to(cuda)
    qkv = rows(n, hq + 2 * hkv, d, 3, 1.5).view(n, -1).to(cuda)
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split((hq * d, hkv * d, hkv * d), 1))
    qw, kw = (rows(1, 1, d, i)[0, 0] for i in (5, 6))
    if not norm:
        qw = kw = None
    table = rope_table(300, rot)
    pos = torch.tensor([p for a, e in zip(before, lens) for p in range(a, e)])
    lens_d = torch.tensor(lens, dtype=torch.int32, device=cuda)
    qo = w4q.kv8_append(k, v, *dev, lens_d, cu_tokens=None if one else prefix(counts, cuda), q=q,
                        q_weight=None if qw is None else qw.to(cuda), k_weight=None if kw is None else kw.to(cuda),
                        cos_sin=table.to(cuda), eps=1e-5, interleaved=interleaved)
    near(qo, norm_rope(q.cpu(), qw, table, pos, 1e-5, interleaved))
    turned = norm_rope(k.cpu(), kw, table, pos, 1e-5, interleaved)
    wrote = emulate(cache, "k", turned.float(), lens, counts)
    emulate(cache, "v", v.cpu().float(), lens, counts)
    kc, vc, ks, vs = (t.cpu() for t in dev[:4])
    assert torch.equal(vc.view(torch.uint8), cache.v.view(torch.uint8))
    assert torch.equal(torch.nan_to_num(vs, -1.0), torch.nan_to_num(cache.vs, -1.0))
    assert torch.equal(torch.isnan(ks), torch.isnan(cache.ks))
    ok = ~torch.isnan(cache.ks)
    assert ((ks[ok] - cache.ks[ok]).abs() <= 2.0 ** -19 * cache.ks[ok]).all()
    for blk, slot, token in wrote:
        exact = turned[token] / ks[blk].double()[:, None]                    # the quotient, in codes
        got = kc[blk, :, slot].double()
        if dtype == I8:
            assert ((got - exact).abs() <= 0.5 + 127 * 2.0 ** -18).all()
        else:
            step = torch.exp2(exact.abs().clamp_min(2.0 ** -6).log2().floor() - 3)
            assert ((got - exact).abs() <= step / 2 + 448 * 2.0 ** -18).all()


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("d,hkv", [(64, 5), (128, 2), (256, 1)])
def test_read_returns_the_values(cuda, dtype, d, hkv):
    lens, counts = [40, 0, 16, 7, 90], [13, 0, 16, 1, 90]
    cache = Cache(5, 6, hkv, d, 16, dtype).fill(lens)
    cache.table[4, 2] = -1
    dev = cache.to(cuda)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=cuda)
    k, v = w4q.kv8_read(*dev, lens_d, cu_tokens=prefix(counts, cuda), tokens=sum(counts))
    at = 0
    for b, n in enumerate(counts):
        for pos in range(lens[b] - n, lens[b]):
            blk = int(cache.table[b, pos // 16])
            for out, c, s in ((k, cache.k, cache.ks), (v, cache.v, cache.vs)):
                ref = torch.zeros(hkv, d) if blk < 0 else c[blk, :, pos % 16].float() * s[blk][:, None]
                assert torch.equal(out[at].cpu(), ref.to(torch.bfloat16))
            at += 1
    k1, _ = w4q.kv8_read(*dev, lens_d)
    assert (k1[1] == 0).all() and torch.equal(k1[0], k[12])


def test_no_tokens(cuda):
    cache = Cache(2, 2, 2, 64, 16, I8)
    dev = cache.to(cuda)
    lens, cu = torch.zeros(2, dtype=torch.int32, device=cuda), torch.zeros(3, dtype=torch.int32, device=cuda)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=cuda)
    q = w4q.kv8_append(none, none, *dev, lens, cu_tokens=cu, q=none)
    k, v = w4q.kv8_read(*dev, lens, cu_tokens=cu, tokens=0)
    qo, ko = w4q.qk_norm_rope(none, none)
    assert q.shape == k.shape == v.shape == qo.shape == ko.shape == (0, 2, 64)
    same(cache, dev[:4])


def test_offsets_beyond_32_bits(cuda):
    hkv, page, d = 8, 64, 128
    blocks = (1 << 32) // (hkv * page * d) + 9
    kc, vc = (torch.empty(blocks, hkv, page, d, dtype=I8, device=cuda) for _ in range(2))
    ks, vs = (torch.empty(blocks, hkv, device=cuda) for _ in range(2))
    table = torch.tensor([[blocks - 1], [blocks - 2]], dtype=torch.int32, device=cuda)
    lens = torch.tensor([10, 64], dtype=torch.int32, device=cuda)
    k, v = rows(74, hkv, d, 1).to(cuda), rows(74, hkv, d, 2).to(cuda)
    w4q.kv8_append(k, v, kc, vc, ks, vs, table, lens, cu_tokens=prefix([10, 64], cuda))
    k2, v2 = w4q.kv8_read(kc, vc, ks, vs, table, lens, cu_tokens=prefix([10, 64], cuda), tokens=74)
    for a, b in ((k, k2), (v, v2)):
        assert (a.float() - b.float()).abs().max() <= a.abs().max().float() / 127 * 0.51 + a.abs().max().float() * 2.0 ** -8


def test_graph_of_append_and_attention(cuda):
    """Two steps of a decode loop by one graph: the lengths advance on the device."""
    hq, hkv, d, page, n = 8, 2, 64, 16, 3
    cache = Cache(n, 4, hkv, d, page, I8).fill([14, 15, 1])
    kc, vc, ks, vs, table = dev = cache.to(cuda)
    lens = torch.tensor([14, 15, 1], dtype=torch.int32, device=cuda)
    qkv = rows(n, hq + 2 * hkv, d, 3).view(n, -1).to(cuda)
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split((hq * d, hkv * d, hkv * d), 1))
    ws = torch.zeros(w4q.kv8_workspace_bytes(n, 1, hq, hkv, d), dtype=torch.uint8, device=cuda)
    qo, out = torch.empty(n, hq, d, dtype=torch.bfloat16, device=cuda), torch.empty(n, 1, hq, d, dtype=torch.bfloat16, device=cuda)

    def step():
        lens.add_(1)
        w4q.kv8_append(k, v, *dev, lens, q=q, q_out=qo)
        w4q.kv8_attention(qo.view(n, 1, hq, d), *dev, lens, out=out, workspace=ws)

    saved = [t.clone() for t in (kc, vc, ks, vs, lens)]
    step()
    step()
    want = [t.clone() for t in (out, ks, vs)] + [kc.clone(), vc.clone()]
    for t, s in zip((kc, vc, ks, vs, lens), saved):
        t.copy_(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (out, ks, vs, kc, vc)):
        assert torch.equal(torch.nan_to_num(a.float(), -1.0), torch.nan_to_num(b.float(), -1.0))
    assert not math.isnan(float(out.float().sum()))
