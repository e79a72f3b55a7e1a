"""The example layer over several decode steps against a plain one in fp64 that keeps its keys and values unrounded.

What separates them: bf16 roundings of qkv, q, the attention, h, the experts' output and x (2^-8 each, independent), and the
cache's codes (half a step of 127 under a page's largest value, or 4 bits in e4m3) on keys and values.  Over a whole
output that stays below 2% of its norm (int8) or 4% (e4m3)."""
import pytest
import torch

from examples.decoder_layer import DecoderLayer
from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


def dense(packed, n, k):
    q, s, z = w4q.w4_unpack_weights(packed, n, k)
    return ((q.view(n, k // 32, 32).double() - z.double()[..., None]) * s.double()[..., None]).view(n, k)


class Plain:
    def __init__(self, layer):
        self.l = layer
        self.qkv, self.o = dense(layer.w_qkv, layer.n_qkv, layer.hidden), dense(layer.w_o, layer.hidden, layer.k_o)
        e, i, h = layer.experts, layer.inter, layer.hidden
        self.w13, self.w2 = dense(layer.w13, e * 2 * i, h).view(e, 2, i, h), dense(layer.w2, e * h, i).view(e, h, i)
        self.keys, self.values = [], []

    @staticmethod
    def norm(x, w):
        return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()

    def turn(self, x, w, pos):
        x = self.norm(x, w)
        c, s = self.l.cos_sin[pos].double().chunk(2)
        a, b = x.chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    def step(self, x, pos, ids):
        l, x = self.l, x.double()
        m, d = x.shape[0], l.head_dim
        q, k, v = (self.norm(x, l.attn_norm) @ self.qkv.T).split((l.k_o, l.kv_heads * d, l.kv_heads * d), 1)
        q, k = self.turn(q.view(m, -1, d), l.q_norm, pos), self.turn(k.view(m, -1, d), l.k_norm, pos)
        self.keys.append(k)
        self.values.append(v.view(m, -1, d))
        keys, values = (torch.stack(t, 2).repeat_interleave(l.heads // l.kv_heads, 1) for t in (self.keys, self.values))
        p = torch.softmax((q[:, :, None] @ keys.transpose(2, 3)) * d ** -0.5, -1)
        x = x + (p @ values).reshape(m, -1) @ self.o.T
        h = self.norm(x, l.moe_norm)
        score = torch.softmax(h @ l.router.double().T, -1)
        # the layer's own choice: close scores may go either way after its roundings
        w = score.gather(1, ids)
        top = score.sort(1, descending=True).values[:, :ids.shape[1]]
        assert (w.sum(1) >= 0.9 * top.sum(1)).all()
        w = w / w.sum(1, keepdim=True)
        out = x.clone()
        for r in range(m):
            for j, e in enumerate(ids[r].tolist()):
                gate, up = self.w13[e] @ h[r]
                out[r] += w[r, j] * (self.w2[e] @ (gate / (1 + torch.exp(-gate)) * up))
        return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs", [1, 5, 12])
def test_steps_against_fp64(cuda, seqs, fp8, monkeypatch):
    layer = DecoderLayer(seqs, 64, hidden=512, heads=8, kv_heads=2, head_dim=64, experts=16, inter=256, topk=3, page=16, fp8=fp8)
    plain = Plain(layer)
    chosen = torch.empty(seqs, 3, dtype=torch.int32, device=cuda)
    moe = w4q.moe_w4a16
    monkeypatch.setattr(w4q, "moe_w4a16", lambda *a, **k: moe(*a, ids=chosen, **k))
    for pos in range(20):
        g = torch.Generator(device=cuda).manual_seed(100 + pos)
        x = torch.randn(seqs, 512, generator=g, device=cuda).to(torch.bfloat16)
        y = layer.step(x)
        ref = plain.step(x, pos, chosen.long())
        assert (y.double() - ref).norm() <= (0.04 if fp8 else 0.02) * ref.norm()
    assert layer.lens.tolist() == [20] * seqs


def test_graph_equals_eager(cuda):
    make = lambda: DecoderLayer(3, 64, hidden=512, heads=8, kv_heads=2, head_dim=64, experts=8, inter=256, topk=2, page=16)  # noqa: E731
    eager, captured = make(), make()
    x = torch.randn(3, 512, device=cuda).to(torch.bfloat16)
    want = [eager.step(x) for _ in range(5)]
    captured.step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = captured.step(x)
    captured.lens.fill_(1)      # the capture ran nothing
    for i in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
