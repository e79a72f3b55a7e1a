"""The 8-bit cache and what lies around it, from the formulas, in plain torch on the CPU: fp64, but for the quantizer,
which is defined in fp32."""
import math

import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def rope_table(positions, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def norm_rope(x, weight, table, pos, eps, interleaved):
    """fp64 [tokens, heads, head_dim]."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    if table is None:
        return x
    rot = table.shape[1]
    c, s = table[pos.long()].double()[:, None].chunk(2, -1)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def encode(y, scale, dtype):
    """Codes of fp32 rows under an fp32 scale, as codes' values (fp32)."""
    q = torch.where(scale > 0, y / scale, torch.zeros(()))
    if dtype == torch.int8:
        return q.round().clamp(-127, 127)
    return q.clamp(-448, 448).to(dtype).float()


class Cache:
    """A cache of `seqs` sequences with scattered pages; whatever is not written is filled with what could hurt."""

    def __init__(self, seqs, width, kv_heads, head_dim, page, dtype, seed=0, spare=3, blocks=None):
        g = torch.Generator().manual_seed(seed)
        self.page, self.dtype = page, dtype
        self.blocks = blocks or seqs * width + spare
        order = torch.randperm(self.blocks, generator=g)[:seqs * width]
        self.table = order.to(torch.int32).view(seqs, width)
        shape = (self.blocks, kv_heads, page, head_dim)
        # 0x7f: NaN in e4m3, the largest code in int8
        self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8).view(dtype) for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:2], math.nan) for _ in range(2))

    def fill(self, lens, seed=1, spread=0.0):
        """Gaussian codes below the lengths, scales 2^(+-spread) apart."""
        g = torch.Generator().manual_seed(seed)
        kv_heads, d = self.k.shape[1], self.k.shape[3]
        for b, n in enumerate(lens):
            for i in range(-(-n // self.page)):
                blk, m = int(self.table[b, i]), min(self.page, n - i * self.page)
                if blk < 0 or blk >= self.blocks:
                    continue
                for c, s in ((self.k, self.ks), (self.v, self.vs)):
                    x = torch.randn(kv_heads, m, d, generator=g)
                    x = (x * 40).round().clamp(-127, 127) if self.dtype == torch.int8 else x * 40
                    c[blk, :, :m] = x.to(self.dtype)
                    e = spread if c is self.v else 0.0
                    s[blk] = (0.5 + torch.rand(kv_heads, generator=g)) / 40 * torch.exp2(
                        (torch.rand(kv_heads, generator=g) * 2 - 1) * e)
        return self

    def to(self, device):
        return [t.to(device) for t in (self.k, self.v, self.ks, self.vs, self.table)]


def attention(cache, lens, q, scale, window):
    """(out, sum of weight * |v|, lse, bound on the scores' sizes) in fp64 for q [seqs, queries, heads, head_dim]."""
    n, m, hq, d = q.shape
    kv = cache.k.shape[1]
    grp = hq // kv
    out, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full((n, m, hq), -math.inf, dtype=torch.float64)
    size = torch.zeros(n, m, hq, dtype=torch.float64)
    for b, length in enumerate(lens):
        if length <= 0:
            continue
        pages = cache.table[b, :-(-length // cache.page)].long()
        real = (pages >= 0) & (pages < cache.blocks)
        there = real.repeat_interleave(cache.page)[:length]
        idx = torch.where(real, pages, 0)
        for h in range(kv):
            k, v = ((c.view(torch.uint8)[idx, h].view(c.dtype).double() * s[idx, h].double()[:, None, None]).reshape(-1, d)[:length]
                    for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)))
            k, v = (torch.where(there[:, None], x, torch.zeros((), dtype=torch.float64)) for x in (k, v))
            for i in range(m):
                own = length - m + i
                at = torch.arange(length)
                see = (at <= own) & there
                if window > 0:
                    see &= at > own - window
                if not bool(see.any()):
                    continue
                qq = q[b, i, h * grp:(h + 1) * grp].double()
                s = (qq @ k[see].T) * scale
                w = torch.softmax(s, -1)
                hs = slice(h * grp, (h + 1) * grp)
                out[b, i, hs] = w @ v[see]
                mag[b, i, hs] = w @ v[see].abs()
                lse[b, i, hs] = torch.logsumexp(s, -1)
                size[b, i, hs] = (abs(scale) * (qq.abs() @ k[see].abs().T)).amax(-1)
    return out, mag, lse, size
