"""The decode-step operators around the quantized linear layer, as they are timed and checked:

  rotate   norms of the query and key heads and their position rotation, in one pass
  append   the same, with the new keys and values quantized into a cache held in 8 bits
  attend   attention of a few query tokens of each sequence over that cache
  moe      a mixture-of-experts layer of 1 to 64 tokens, experts in the packed 4-bit format

Each has its plain form here, in elementary torch operations and 32 bits.  With `own` set, `run`
makes the calls that a program makes of gemv_w4a16_gemm_gb300.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # 64 sequences in decode, one token each: the launch and a little memory traffic
        dict(name="rotate 64 tokens", kind="rotate", tokens=64, hq=32, hkv=8, d=128, rot=128, pairs=False, norm=True),
        # a long prompt of a model with 52 query heads (6656 / 128), half of each head rotated, in adjacent pairs
        dict(name="rotate 8191 tokens", kind="rotate", tokens=8191, hq=52, hkv=4, d=128, rot=64, pairs=True, norm=True),
        # the decode step's write: one token of each of 64 sequences
        dict(name="append 64 x 1", kind="append", seqs=64, new=1, ctx=4096, hq=32, hkv=8, d=128, page=64, fp8=False, rot=128, norm=True),
        # prompts of uneven lengths, into a cache whose pages are small
        dict(name="append 5 x 2000", kind="append", seqs=5, new=2000, ctx=777, hq=32, hkv=8, d=128, page=16, fp8=True, rot=128, norm=False),
        # a single short conversation: latency
        dict(name="attend 1 x 130", kind="attend", seqs=1, queries=1, length=130, even=True, hq=32, hkv=8, d=128, page=16, fp8=False, window=0),
        # a batch of uneven sequences
        dict(name="attend 32 x 4000", kind="attend", seqs=32, queries=1, length=4000, even=False, hq=32, hkv=8, d=128, page=64, fp8=True, window=0),
        # drafts of five tokens checked at once, attention limited to a window
        dict(name="attend 48 x 8000 drafts", kind="attend", seqs=48, queries=5, length=8000, even=False, hq=32, hkv=8, d=64, page=32, fp8=False, window=1024),
        # one long document: the whole card on one sequence
        dict(name="attend 1 x 131071", kind="attend", seqs=1, queries=1, length=131071, even=True, hq=32, hkv=4, d=128, page=64, fp8=False, window=0),
        # a full batch of long sequences: the cache's bandwidth
        dict(name="attend 64 x 16000", kind="attend", seqs=64, queries=1, length=16000, even=True, hq=64, hkv=8, d=128, page=64, fp8=False, window=0),
        # one token through 8 of 128 small experts: latency
        dict(name="moe 1 of 128", kind="moe", tokens=1, hidden=2048, inter=768, experts=128, topk=8, sigmoid=False),
        # a batch that touches nearly every expert with a few tokens each
        dict(name="moe 32 of 128", kind="moe", tokens=32, hidden=2048, inter=768, experts=128, topk=8, sigmoid=True),
        # the largest batch through a few wide experts
        dict(name="moe 64 of 16", kind="moe", tokens=64, hidden=6656, inter=4096, experts=16, topk=2, sigmoid=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rotate", "append", "attend", "attend", "moe"))
    if kind == "moe":
        hidden, inter = 256 * rng.choice((1, 2, 3, 4, 5, 7, 8, 11, 16, 20)), 256 * rng.choice((1, 2, 3, 4, 5, 8))
        experts = min(_log(rng, 4, 256), max(4, 16 * 6656 * 4096 // (hidden * inter)))
        return dict(kind=kind, tokens=_log(rng, 1, 64), hidden=hidden, inter=inter, experts=experts,
                    topk=rng.randint(1, min(8, experts)), sigmoid=rng.random() < 0.5)
    d = rng.choice((64, 128, 128, 256))
    hq, hkv = rng.choice(((1, 1), (7, 7), (8, 1), (4, 2), (10, 2), (8, 4), (28, 4), (20, 4), (40, 8), (64, 8)))
    if kind == "rotate":
        return dict(kind=kind, tokens=_log(rng, 1, 8000), hq=hq, hkv=hkv, d=d, rot=rng.choice((d, d // 2)),
                    pairs=rng.random() < 0.5, norm=rng.random() < 0.7)
    if kind == "append":
        seqs = _log(rng, 1, 128)
        return dict(kind=kind, seqs=seqs, new=1 if rng.random() < 0.5 else _log(rng, 2, 10000 // seqs), ctx=_log(rng, 1, 4000),
                    hq=hq, hkv=hkv, d=d, page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5, rot=rng.choice((d, d // 2)),
                    norm=rng.random() < 0.5)
    seqs, queries = _log(rng, 1, 128), rng.choice((1, 1, 1, 2, 4, 8))
    length = _log(rng, queries, min(131071, 900_000_000 // (seqs * hkv * d)))
    return dict(kind=kind, seqs=seqs, queries=queries, length=length, even=rng.random() < 0.3, hq=hq, hkv=hkv, d=d,
                page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5, window=rng.choice((0, 0, 0, _log(rng, 16, 4096))))


# ------------------------------------------------------------------ inputs

def _table(positions, rot, base=10000.0):
    """fp32 [positions, rot]: the cosines of the rot / 2 angles of each position, then the sines."""
    inv = base ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def _lengths(case, g):
    n, top = case["seqs"], case.get("length") or case["ctx"]
    if case.get("even"):
        return torch.full((n,), top, dtype=torch.int32, device=DEV)
    return torch.randint(max(case.get("queries", 1), top // 8), top + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _pages(seqs, most, page, g):
    """A block table in which every sequence owns pages scattered over the pool, and the pool's size."""
    per = -(-most // page)
    order = torch.randperm(seqs * per + 1, generator=g, device=DEV)[:seqs * per]
    return order.to(torch.int32).view(seqs, per), seqs * per + 1


def _pool(blocks, hkv, page, d, fp8, g):
    """Quantized pages of gaussian values whose size differs from page to page and head to head."""
    cache = torch.empty(blocks, hkv, page, d, dtype=torch.float8_e4m3fn if fp8 else torch.int8, device=DEV)
    scale = torch.empty(blocks, hkv, dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (hkv * page * d))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn(n, hkv, page, d, generator=g, device=DEV)
        x *= 0.5 + torch.rand(n, hkv, 1, 1, generator=g, device=DEV)
        s = x.abs().amax((2, 3)) / (448.0 if fp8 else 127.0)
        x /= s[:, :, None, None]
        cache[i:i + n] = x.to(torch.float8_e4m3fn) if fp8 else x.round().clamp(-127, 127).to(torch.int8)
        scale[i:i + n] = s
    return cache, scale


def _codes(rows, K, g):
    """The 4-bit codes, bf16 scales and zero points of a gaussian weight (groups of 32, asymmetric min-max), and its packed
    bytes in the layout that include/w4q.h describes."""
    w = torch.randn(rows, K // 32, 32, generator=g, device=DEV) * K ** -0.5
    lo, hi = w.amin(2), w.amax(2)
    s = ((hi - lo) / 15).to(torch.bfloat16)
    sf = s.float()[:, :, None]
    z = (-lo[:, :, None] / sf).round().clamp(0, 15)
    q = ((w / sf).round() + z).clamp(0, 15).to(torch.uint8)
    return q.view(rows, K), s, z[:, :, 0].to(torch.uint8)


def _pack(rows, K, g):
    B = K // 256
    out = torch.zeros(-(-rows // 128), B, 8, 2432, dtype=torch.uint8, device=DEV)
    step = 16 * max(8, (1 << 25) // (16 * K) // 8 * 8)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q, s, z = _codes(n, K, g)
        t = n // 16
        # rows: (tile, a, r); columns: (super-block, sub-block, word, e, lane column, h)
        q = q.view(t, 2, 8, B, 4, 4, 2, 4, 2).permute(3, 0, 4, 2, 7, 5, 8, 1, 6)  # b t sb r c j h a e
        q = (q[..., 0] | (q[..., 1] << 4)).reshape(B, t, 2048)
        sb = s.view(torch.int16).view(t, 2, 8, B, 2, 4).permute(3, 0, 4, 2, 5, 1).reshape(B, t, 128).view(torch.uint8)
        zb = z.view(t, 2, 8, B, 8).permute(3, 0, 2, 4, 1).reshape(B, t, 128)
        tiles = torch.cat((q, sb, zb), 2)
        pad = -t % 8
        if pad:
            tiles = torch.cat((tiles, tiles.new_zeros(B, pad, 2432)), 1)
        out[r // 128:r // 128 + (t + pad) // 8] = tiles.view(B, -1, 8, 2432).transpose(0, 1)
    return out.view(-1)


def _unpack(packed, rows, K):
    """The weight that the packed bytes stand for, fp32 [rows, K]."""
    T, B = rows // 16, K // 256
    t = packed.reshape(-1, B, 8, 2432).transpose(0, 1).reshape(B, -1, 2432)[:, :T]
    q = t[..., :2048].reshape(B, T, 4, 8, 4, 4, 2, 2)  # b t sb r c j h a
    q = torch.stack((q & 15, q >> 4), -1)
    q = q.permute(1, 7, 3, 0, 2, 5, 8, 4, 6).reshape(rows, K // 32, 32)
    s = t[..., 2048:2304].contiguous().view(torch.bfloat16).view(B, T, 2, 8, 4, 2).permute(1, 5, 3, 0, 2, 4)
    z = t[..., 2304:].reshape(B, T, 8, 8, 2).permute(1, 4, 2, 0, 3)
    w = (q.float() - z.reshape(rows, -1, 1).float()) * s.reshape(rows, -1, 1).float()
    return w.view(rows, K)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kind, bf = case["kind"], torch.bfloat16
    st = dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    if kind == "moe":
        h, i, e = case["hidden"], case["inter"], case["experts"]
        st["x"] = randn(case["tokens"], h).to(bf)
        st["router"] = (randn(e, h) * (2.0 * h ** -0.5)).to(bf)
        st["bias"] = randn(e) * 0.1 if case["sigmoid"] else None
        # each expert's gate rows, then its up rows; the experts one after the other
        st["w13"] = _pack(e * 2 * i, h, g)
        st["w2"] = _pack(e * h, i, g)
        if own:
            from gemv_w4a16_gemm_gb300 import w4q
            st["workspace"] = torch.empty(max(16, w4q.moe_workspace_bytes(case["tokens"], h, i, e, case["topk"])),
                                          dtype=torch.uint8, device=DEV)
        return st
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if kind == "attend":
        lens = _lengths(case, g)
        st["table"], blocks = _pages(case["seqs"], case["length"], case["page"], g)
        st["lens"] = lens
        st["q"] = randn(case["seqs"], case["queries"], hq, d).to(bf)
        st["kc"], st["ks"] = _pool(blocks, hkv, case["page"], d, case["fp8"], g)
        st["vc"], st["vs"] = _pool(blocks, hkv, case["page"], d, case["fp8"], g)
        if own:
            from gemv_w4a16_gemm_gb300 import w4q
            # its counters have to be zero before the first call; every call leaves them so
            st["workspace"] = torch.zeros(max(16, w4q.kv8_workspace_bytes(case["seqs"], case["queries"], hq, hkv, d)),
                                          dtype=torch.uint8, device=DEV)
        return st
    # the rows of a fused projection: query heads, key heads, value heads
    if kind == "rotate":
        tokens = case["tokens"]
        st["pos"] = torch.randint(0, 4096 + tokens, (tokens,), generator=g, device=DEV, dtype=torch.int32)
        most = 4096 + tokens
    else:
        seqs, new = case["seqs"], case["new"]
        # the lengths go by the case alone, so that every seed reads back as many tokens
        gl = torch.Generator(device=DEV).manual_seed(seqs * 1000003 + new * 1009 + case["ctx"])
        before = torch.randint(0, case["ctx"] + 1, (seqs,), generator=gl, device=DEV, dtype=torch.int32)
        # now and then a sequence has no token in this step
        counts = torch.full_like(before, 1) if new == 1 else torch.randint(0, new + 1, (seqs,), generator=gl, device=DEV, dtype=torch.int32)
        if new > 1:
            counts[0] = new
        st["cu"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
        tokens = int(st["cu"][-1])
        st["lens"] = before + counts
        most, page = case["ctx"] + new, case["page"]
        st["table"], blocks = _pages(seqs, most, page, g)
        st["kc"], st["ks"] = _pool(blocks, hkv, page, d, case["fp8"], g)
        st["vc"], st["vs"] = _pool(blocks, hkv, page, d, case["fp8"], g)
        # what is read back: the new tokens and, before them, the rest of the page that the first of them falls into
        back = counts + torch.where(counts > 0, before % page, 0)
        st["back"] = torch.cat((back.new_zeros(1), back.cumsum(0))).to(torch.int32)
        st["nback"] = int(st["back"][-1])
    st["tokens"] = tokens
    qkv = (randn(tokens, (hq + 2 * hkv) * d) * 1.5).to(bf)
    st["q"], st["k"], st["v"] = (t.unflatten(1, (-1, d)) for t in qkv.split((hq * d, hkv * d, hkv * d), 1))
    st["qw"] = (1 + 0.1 * randn(d)).to(bf) if case["norm"] else None
    st["kw"] = (1 + 0.1 * randn(d)).to(bf) if case["norm"] else None
    st["cs"] = _table(most, case["rot"])
    return st


# ------------------------------------------------------------- plain forms

def _turned(x, w, cs, pos, pairs):
    """x [tokens, heads, d]: each head divided by its root mean square and weighted (if w is given), then rotated."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    rot = cs.shape[1]
    c, s = cs[pos.long()][:, None].chunk(2, -1)
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _owners(cu, tokens):
    """The sequence of each of the tokens that cu's prefix sums lay out one after the other."""
    return torch.searchsorted(cu[1:], torch.arange(tokens, device=DEV, dtype=torch.int32), right=True)


def _places(lens, cu, tokens, table, page):
    """Position, page and slot of each token: the last cu[b + 1] - cu[b] positions of sequence b."""
    b = _owners(cu, tokens)
    pos = lens[b] - cu[b + 1] + torch.arange(tokens, device=DEV, dtype=torch.int32)
    return pos, table[b, pos // page].long(), (pos % page).long()


def _stored(x, cache, scale, table, lens, cu, places, page):
    """Writes the tokens x [tokens, heads, d] into the pages; a page's scale grows with what it has to hold."""
    fp8 = cache.dtype == torch.float8_e4m3fn
    top = 448.0 if fp8 else 127.0

    def codes(v):
        return v.to(torch.float8_e4m3fn) if fp8 else v.round().clamp(-top, top).to(torch.int8)

    _, blk, slot = places
    counts = cu[1:] - cu[:-1]
    before = lens - counts
    # pages that held tokens before: their old scale stands, as the least that the new one may be
    part = ((counts > 0) & (before % page != 0)).nonzero()[:, 0]
    pblk = table[part, before[part] // page].long()
    old = scale[pblk]
    grown = torch.zeros_like(scale)
    grown.index_reduce_(0, blk, x.abs().amax(-1), "amax")
    grown /= top
    grown[pblk] = torch.maximum(grown[pblk], old)
    scale[blk] = grown[blk]
    held = cache[pblk].float()
    r = torch.where(grown[pblk] > old, old / grown[pblk], 1.0)
    cache[pblk] = codes(held * r[:, :, None, None])
    s = grown[blk][..., None]
    cache[blk, :, slot] = codes(torch.where(s > 0, x / s, 0.0))


def _held(cache, scale, places):
    _, blk, slot = places
    return (cache[blk, :, slot].float() * scale[blk][..., None]).to(torch.bfloat16)


def _append_plain(st):
    page, cu, lens, table = st["page"], st["cu"], st["lens"], st["table"]
    places = _places(lens, cu, st["tokens"], table, page)
    q = _turned(st["q"], st["qw"], st["cs"], places[0], False).to(torch.bfloat16)
    k = _turned(st["k"], st["kw"], st["cs"], places[0], False)
    _stored(k, st["kc"], st["ks"], table, lens, cu, places, page)
    _stored(st["v"].float(), st["vc"], st["vs"], table, lens, cu, places, page)
    back = _places(lens, st["back"], st["nback"], table, page)
    return q, _held(st["kc"], st["ks"], back), _held(st["vc"], st["vs"], back)


def _seen(lens, queries, length, window):
    """[seqs, queries, length]: whether a query sees a position."""
    at = torch.arange(length, device=DEV, dtype=torch.int32)
    last = lens[:, None] - queries + torch.arange(queries, device=DEV, dtype=torch.int32)  # each query's own position
    seen = at <= last[..., None]
    if window:
        seen &= at > last[..., None] - window
    return seen


def _attend_plain(st):
    q, table, lens, hkv, d = st["q"].float(), st["table"].long(), st["lens"], st["hkv"], st["d"]
    n, m, hq, _ = q.shape
    seen = _seen(lens, m, table.shape[1] * st["page"], st["window"])[:, None, None]

    def whole(cache, scale):
        x = cache[table].float()
        x *= scale[table][..., None, None]
        x = x.transpose(1, 2).reshape(n, hkv, -1, d)
        return x.masked_fill_(~seen.any(-2)[:, 0, 0][:, None, :, None], 0.0)  # whatever lies past the end

    q = q.view(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.reshape(n, hkv, -1, d), whole(st["kc"], st["ks"]).transpose(2, 3)).view(n, hkv, hq // hkv, m, -1)
    s = (s * d ** -0.5).masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    s = (s - top).exp_()
    total = s.sum(-1, keepdim=True)
    s = torch.where(total > 0, s / total, 0.0)
    o = torch.matmul(s.view(n, hkv, -1, s.shape[-1]), whole(st["vc"], st["vs"])).view(n, hkv, hq // hkv, m, d)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(n, m, hq)
    return o.permute(0, 3, 1, 2, 4).reshape(n, m, hq, d).to(torch.bfloat16), lse


def _chosen(logits, bias, topk):
    """Each token's experts and their weights, which sum to one: the largest scores (with the bias, where there is one)."""
    score = logits.softmax(-1) if bias is None else torch.sigmoid(logits)
    ids = torch.argsort(score if bias is None else score + bias, dim=-1, descending=True, stable=True)[:, :topk]
    w = score.gather(1, ids)
    return ids, w / w.sum(-1, keepdim=True)


def _moe_plain(st):
    x, h, i, e = st["x"].float(), st["hidden"], st["inter"], st["experts"]
    ids, w = _chosen(x @ st["router"].float().T, st["bias"], st["topk"])
    w13, w2 = st["w13"].view(e, -1), st["w2"].view(e, -1)  # whole 128-row groups of the layout belong to one expert
    if st["tokens"] * st["topk"] <= e:  # few tokens: the chosen experts' weights alone are multiplied
        w13 = _unpack(w13[ids.view(-1)], ids.numel() * 2 * i, h).view(*ids.shape, 2 * i, h)
        w2 = _unpack(w2[ids.view(-1)], ids.numel() * h, i).view(*ids.shape, h, i)
        gate, up = torch.einsum("mh,mkih->mki", x, w13).chunk(2, -1)
        y = torch.einsum("mki,mkhi->mkh", gate * torch.sigmoid(gate) * up, w2)
        return torch.einsum("mkh,mk->mh", y, w).to(torch.bfloat16)
    gate, up = torch.matmul(x, _unpack(w13, e * 2 * i, h).view(e, 2 * i, h).transpose(1, 2)).chunk(2, -1)  # [e, tokens, i]
    y = torch.matmul(gate * torch.sigmoid(gate) * up, _unpack(w2, e * h, i).view(e, h, i).transpose(1, 2))
    full = torch.zeros(len(x), e, device=DEV).scatter_(1, ids, w)
    return torch.einsum("emh,me->mh", y, full).to(torch.bfloat16)


def run(st):
    kind = st["kind"]
    if own:
        return _run_own(st)
    if kind == "rotate":
        return [_turned(st[n], st[n + "w"], st["cs"], st["pos"], st["pairs"]).to(torch.bfloat16) for n in ("q", "k")]
    if kind == "append":
        q, k, v = _append_plain(st)
        return {"q": q, "k": k, "v": v, "k_scale": st["ks"], "v_scale": st["vs"]}
    if kind == "attend":
        out, lse = _attend_plain(st)
        return {"out": out, "lse": lse}
    return _moe_plain(st)


def _run_own(st):
    from gemv_w4a16_gemm_gb300 import w4q
    kind = st["kind"]
    if kind == "rotate":
        return list(w4q.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["cs"], st["pos"], eps=1e-6, interleaved=st["pairs"]))
    if kind == "moe":
        return w4q.moe_w4a16(st["x"], st["router"], st["w13"], st["w2"], inter=st["inter"], topk=st["topk"], bias=st["bias"],
                             sigmoid=st["sigmoid"], renormalize=True, workspace=st["workspace"])
    cache = (st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["lens"])
    if kind == "append":
        q = w4q.kv8_append(st["k"], st["v"], *cache, cu_tokens=st["cu"], q=st["q"], q_weight=st["qw"], k_weight=st["kw"],
                           cos_sin=st["cs"], eps=1e-6)
        # the cache's new contents as values; a program goes straight on to the attention
        k, v = w4q.kv8_read(*cache, cu_tokens=st["back"], tokens=st["nback"])
        return {"q": q, "k": k, "v": v, "k_scale": st["ks"], "v_scale": st["vs"]}
    lse = torch.empty(st["q"].shape[:3], dtype=torch.float32, device=DEV)
    out = w4q.kv8_attention(st["q"], *cache, window=st["window"], lse=lse, workspace=st["workspace"])
    return {"out": out, "lse": lse}


# -------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    if kind == "moe":
        m, h, i, e, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
        touched = e * (1 - (1 - k / e) ** m)  # experts that m tokens choose, on average
        return {"bytes": touched * 3 * h * i * 19 / 32 + 2 * e * h + 4 * m * h, "flops": 2.0 * m * (e * h + k * 3 * h * i)}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if kind == "rotate":
        t = case["tokens"]
        return {"bytes": t * ((hq + hkv) * d * 4 + case["rot"] * 4), "flops": 8.0 * t * (hq + hkv) * d}
    if kind == "append":
        n = case["seqs"] * (1 if case["new"] == 1 else (case["new"] + 1) / 2)
        # q, k, v read; q written; k, v written, and read back as values
        return {"bytes": n * d * (hq * 4 + hkv * 2 * (2 + 1 + 1 + 2)) + 4 * n * case["rot"], "flops": 10.0 * n * (hq + 2 * hkv) * d}
    length = case["length"] if case["even"] else case["length"] * 9 / 16
    if case["window"]:
        length = min(length, case["window"] + case["queries"] - 1)
    n, m = case["seqs"], case["queries"]
    return {"bytes": n * (2 * length * hkv * d + 4 * m * hq * d + 4 * m * hq + length * hkv * 8 / case["page"]),
            "flops": 4.0 * n * m * length * hq * d}


# ------------------------------------------------------------------- exact

def _exact_turn(x, w, cs, pos, pairs):
    x, cs = x.double(), cs.double()[pos.long()]
    if w is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
    half = cs.shape[1] // 2
    first = torch.arange(half, device=DEV) * 2 if pairs else torch.arange(half, device=DEV)
    second = first + (1 if pairs else half)
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(cs[:, :half], cs[:, half:])[:, None]
    x = x.clone()
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_weight(packed, row, rows, K):
    """Rows row .. row + rows of the packed weight, one element at a time from the layout's description."""
    n = torch.arange(row, row + rows, device=DEV)[:, None]
    k = torch.arange(K, device=DEV)[None]
    t, b = n // 16, k // 256
    base = ((t // 8 * (K // 256) + b) * 8 + t % 8) * 2432
    a, r, kk = n % 16 // 8, n % 8, k % 256
    c = kk % 16
    byte = 512 * (kk // 64) + 16 * (4 * r + c % 8 // 2) + 4 * (kk % 64 // 16) + a + 2 * (c % 2)
    q = (packed[base + byte] >> (4 * (c // 8)).to(torch.uint8)) & 15
    grp = kk // 32
    s = packed.view(torch.bfloat16)[(base + 2048 + 128 * (grp // 4) + 16 * r + 4 * (grp % 4) + 2 * a) // 2]
    z = packed[base + 2304 + 16 * r + 2 * grp + a]
    return (q.double() - z.double()) * s.double()


def exact(case, seed):
    st, kind = prepare(case, seed), case["kind"]
    if kind == "rotate":
        return [_exact_turn(st[n], st[n + "w"], st["cs"], st["pos"], case["pairs"]) for n in ("q", "k")]
    if kind == "append":
        cu, lens = st["cu"].tolist(), st["lens"].tolist()
        pos = torch.cat([torch.arange(e - (cu[b + 1] - cu[b]), e) for b, e in enumerate(lens)]).to(DEV)
        # a stored code goes to one side or the other of a rounding: it has no value in 64 bits
        return {"q": _exact_turn(st["q"], st["qw"], st["cs"], pos, False), "k": None, "v": None, "k_scale": None, "v_scale": None}
    if kind == "attend":
        hkv, d, page, m, win = case["hkv"], case["d"], case["page"], case["queries"], case["window"]
        grp, out, lse = case["hq"] // hkv, [], []
        for b, n in enumerate(st["lens"].tolist()):
            o = torch.zeros(m, case["hq"], d, dtype=torch.float64, device=DEV)
            z = torch.full((m, case["hq"]), -math.inf, dtype=torch.float64, device=DEV)
            blk = st["table"][b, :-(-n // page)].long()
            for h in range(hkv):
                k, v = ((st[c + "c"][blk, h].double() * st[c + "s"][blk, h].double()[:, None, None]).view(-1, d)[:n] for c in "kv")
                for i in range(m):
                    end = n - m + i + 1
                    lo = max(0, end - win) if win else 0
                    if end <= lo:
                        continue
                    s = st["q"][b, i, h * grp:(h + 1) * grp].double() @ k[lo:end].T / math.sqrt(d)
                    z[i, h * grp:(h + 1) * grp] = torch.logsumexp(s, -1)
                    o[i, h * grp:(h + 1) * grp] = torch.softmax(s, -1) @ v[lo:end]
            out.append(o)
            lse.append(z)
        return {"out": torch.stack(out), "lse": torch.stack(lse)}
    x, h, i, k = st["x"].double(), case["hidden"], case["inter"], case["topk"]
    out = torch.zeros_like(x)
    score = x @ st["router"].double().T
    score = torch.sigmoid(score) if case["sigmoid"] else score.exp() / score.exp().sum(-1, keepdim=True)
    rank = score + st["bias"].double() if case["sigmoid"] else score
    picked = torch.zeros_like(score, dtype=torch.bool)
    for _ in range(k):
        picked.scatter_(1, rank.masked_fill(picked, -math.inf).argmax(-1, keepdim=True), True)
    score = torch.where(picked, score, 0.0)
    score = score / score.sum(-1, keepdim=True)
    for e in range(case["experts"]):
        rows = picked[:, e].nonzero()[:, 0]
        if not len(rows):
            continue
        w = _exact_weight(st["w13"], e * 2 * i, 2 * i, h)
        gate, up = x[rows] @ w[:i].T, x[rows] @ w[i:].T
        y = (gate / (1 + (-gate).exp()) * up) @ _exact_weight(st["w2"], e * h, h, i).T
        out[rows] += score[rows, e, None] * y
    return out
