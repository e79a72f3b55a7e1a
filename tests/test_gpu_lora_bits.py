"""A x keeps fp32's bits on its way into the second product of the adapters, whatever the rank and the number of an adapter's
tokens: sums that are exact in fp32 give exact results."""
import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


def parts(v):
    """fp32 as three bf16 whose sum it is."""
    out = []
    for _ in range(3):
        out.append(v.bfloat16())
        v = v - out[-1].float()
    assert (v == 0).all()
    return out


# one launch and two (rank * K above 2^18, or a rank above 32), both widths of a lane's pieces, 1 to 16 tokens of a tile
@pytest.mark.parametrize("rank,K", [(8, 256), (16, 4096), (16, 32768), (24, 264), (32, 512), (40, 256), (64, 2048), (72, 256), (128, 512), (256, 264)])
def test_the_last_bits_of_h_count(cuda, rank, K):
    """Ranks in pairs hold v and v without its last 8 bits, of 24; B takes their difference, which 8 bits hold."""
    g = torch.Generator(device=cuda).manual_seed(rank + K)
    adapters, N = 6, 70
    bits = torch.randint(1 << 23, 1 << 24, (adapters, rank // 2), generator=g, device=cuda)
    bits |= 1                                             # the last one is set
    v = torch.empty(adapters, rank, device=cuda)
    v[:, ::2], v[:, 1::2] = bits.float(), (bits & ~255).float()
    A = torch.zeros(adapters, rank, K, device=cuda).bfloat16()
    at = torch.randperm(K, generator=g, device=cuda)[:3]
    for column, part in zip(at, parts(v)):
        A[:, :, column] = part
    B = torch.zeros(adapters, N, rank, device=cuda).bfloat16()
    pair = torch.arange(N, device=cuda) % (rank // 2)
    B[:, torch.arange(N, device=cuda), 2 * pair] = 1.0
    B[:, torch.arange(N, device=cuda), 2 * pair + 1] = -1.0
    for counts in ([1], [2], [1, 2, 3, 4, 5], [4, 8, 1, 9], [6, 7, 16], [3, 33, 12]):
        ids = torch.tensor([a for a, c in enumerate(counts) for _ in range(c)], device=cuda)
        ids = ids[torch.randperm(len(ids), generator=g, device=cuda)].int()
        x = torch.zeros(len(ids), K, device=cuda).bfloat16()
        x[:, at] = (2.0 ** (torch.arange(len(ids), device=cuda) % 5 - 2)).bfloat16()[:, None]
        want = (bits & 255).double()[ids.long()][:, pair] * x[:, at[:1]].double()
        out = w4q.lora_add(torch.zeros(len(ids), N, dtype=torch.bfloat16, device=cuda), x, A, B, ids)
        assert torch.equal(out.double(), want), counts
