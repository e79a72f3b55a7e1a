"""One decoder layer in decode, from the library's calls alone but for two root-mean-square norms and two additions:

    qkv = W4A16(norm(x));  q, k, v into the 8-bit cache, normed per head and rotated;  attention over the cache;
    x += W4A16(attention);  x += experts(norm(x)), the experts in W4

for 1 to 64 sequences with one new token each, captured in a CUDA graph.  `python examples/decoder_layer.py` runs a few
steps on random weights and prints the time of one.
"""
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gemv_w4a16_gemm_gb300 import w4q  # noqa: E402


def rms_norm(x, weight, eps=1e-6):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()).to(torch.bfloat16)


class DecoderLayer:
    """Weights, cache and workspaces of one layer for `seqs` sequences of up to `longest` tokens."""

    def __init__(self, seqs, longest, hidden=2048, heads=32, kv_heads=4, head_dim=128, experts=64, inter=768, topk=8,
                 page=64, fp8=False, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).to(torch.bfloat16)

        def scale(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device=device)).to(torch.bfloat16)

        self.seqs, self.hidden, self.heads, self.kv_heads, self.head_dim = seqs, hidden, heads, kv_heads, head_dim
        self.experts, self.inter, self.topk = experts, inter, topk
        self.n_qkv, self.k_o = (heads + 2 * kv_heads) * head_dim, heads * head_dim
        self.w_qkv = w4q.w4_pack_weights(weight(self.n_qkv, hidden))
        self.w_o = w4q.w4_pack_weights(weight(hidden, self.k_o))
        self.router = weight(experts, hidden)
        self.w13 = w4q.w4_pack_weights(weight(experts * 2 * inter, hidden))
        self.w2 = w4q.w4_pack_weights(weight(experts * hidden, inter))
        self.attn_norm, self.moe_norm = scale(hidden), scale(hidden)
        self.q_norm, self.k_norm = scale(head_dim), scale(head_dim)
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim)
        angle = torch.arange(longest, device=device, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float()

        # sequence b owns pages b * width .. (b + 1) * width - 1
        width = -(-longest // page)
        shape = (seqs * width, kv_heads, page, head_dim)
        kind = torch.float8_e4m3fn if fp8 else torch.int8
        self.cache = [torch.zeros(shape, dtype=kind, device=device), torch.zeros(shape, dtype=kind, device=device),
                      torch.zeros(shape[:2], device=device), torch.zeros(shape[:2], device=device),
                      torch.arange(seqs * width, dtype=torch.int32, device=device).view(seqs, width),
                      torch.zeros(seqs, dtype=torch.int32, device=device)]
        self.lens = self.cache[5]
        # one workspace for the linear layers and the experts; the attention's has to start at zero and stays so
        need = max(w4q.workspace_bytes(seqs, self.n_qkv, hidden), w4q.workspace_bytes(seqs, hidden, self.k_o),
                   w4q.moe_workspace_bytes(seqs, hidden, inter, experts, topk), 16)
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self.attn_workspace = torch.zeros(w4q.kv8_workspace_bytes(seqs, 1, heads, kv_heads, head_dim), dtype=torch.uint8,
                                          device=device)

    def step(self, x):
        """x bf16 [seqs, hidden], one new token of every sequence -> the layer's output; the lengths grow by one."""
        self.lens.add_(1)
        m, d, split = x.shape[0], self.head_dim, (self.k_o, self.kv_heads * self.head_dim, self.kv_heads * self.head_dim)
        qkv = w4q.w4a16_gemm(rms_norm(x, self.attn_norm), self.w_qkv, self.n_qkv, self.hidden, workspace=self.workspace)
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split(split, 1))
        q = w4q.kv8_append(k, v, *self.cache, q=q, q_weight=self.q_norm, k_weight=self.k_norm, cos_sin=self.cos_sin)
        a = w4q.kv8_attention(q.view(m, 1, self.heads, d), *self.cache, workspace=self.attn_workspace)
        x = x + w4q.w4a16_gemm(a.view(m, self.k_o), self.w_o, self.hidden, self.k_o, workspace=self.workspace)
        h = rms_norm(x, self.moe_norm)
        return x + w4q.moe_w4a16(h, self.router, self.w13, self.w2, self.inter, self.topk, workspace=self.workspace)


def main():
    seqs, longest, steps = 16, 4096, 64
    layer = DecoderLayer(seqs, longest)
    layer.lens.fill_(1000)
    x = torch.randn(seqs, layer.hidden, device="cuda").to(torch.bfloat16)
    layer.step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(x)
    graph.replay()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    print("%d sequences at about %d tokens: %.1f us a layer and step, output norm %.3f" % (
        seqs, int(layer.lens[0]), (time.perf_counter() - start) / steps * 1e6, float(y.float().norm())))
    assert w4q.device_error() == 0


if __name__ == "__main__":
    main()
