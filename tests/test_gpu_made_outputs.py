"""Tensors that the calls make themselves are torch's like any others: dispatch modes see them, and the filling of memory
that is not initialised reaches them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


def rotated(cuda):
    """A call with an output that is written in part: queries behind the last sequence's are left as they are."""
    k = torch.randn(6, 2, 64, device=cuda).bfloat16()
    cache = [torch.zeros(4, 2, 16, 64, dtype=torch.int8, device=cuda) for _ in range(2)] + \
            [torch.zeros(4, 2, device=cuda) for _ in range(2)] + \
            [torch.arange(4, dtype=torch.int32, device=cuda).view(2, 2), torch.tensor([3, 1], dtype=torch.int32, device=cuda)]
    q = torch.randn(6, 4, 64, device=cuda).bfloat16()
    return w4q.kv8_append(k, k, *cache, q=q, cu_tokens=torch.tensor([0, 3, 4], dtype=torch.int32, device=cuda))


def test_dispatch_modes_see_new_tensors(cuda):
    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.names = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(str(func))
            return func(*args, **(kwargs or {}))

    x = torch.randn(3, 256, device=cuda).bfloat16()
    want = w4q.add_rms_norm(x, x)
    with Seen() as seen:
        got = w4q.add_rms_norm(x, x)
    assert sum("empty" in n for n in seen.names) == 2     # the norm and the sum
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fill", [True, False])
def test_deterministic_mode_fills_new_tensors(cuda, fill):
    was = torch.are_deterministic_algorithms_enabled(), torch.is_deterministic_algorithms_warn_only_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    want = rotated(cuda)
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = fill
        out = rotated(cuda)
    finally:
        torch.use_deterministic_algorithms(was[0], warn_only=was[1])
        torch.utils.deterministic.fill_uninitialized_memory = was[2]
    assert out.shape == want.shape == (6, 4, 64)
    if fill:
        assert out[4:].isnan().all()


def test_new_tensors_in_inference_mode(cuda):
    x = torch.randn(3, 256, device=cuda).bfloat16()
    want = w4q.add_rms_norm(x, x)
    with torch.inference_mode():
        got = w4q.add_rms_norm(x, x)
        assert got[0].is_inference()
    assert torch.equal(got[0], want[0]) and not want[0].is_inference()
