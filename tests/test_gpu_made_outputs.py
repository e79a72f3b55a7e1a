"""Tensors that the calls make themselves are torch's like any others: dispatch modes see them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


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
def test_results_in_deterministic_mode(cuda, fill):
    """(The filling itself shows in no result: the calls write all of what they make.)"""
    was = torch.are_deterministic_algorithms_enabled(), torch.is_deterministic_algorithms_warn_only_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    x = torch.randn(5, 512, device=cuda).bfloat16()
    want = w4q.add_rms_norm_a8(x, x)
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = fill
        got = w4q.add_rms_norm_a8(x, x)
    finally:
        torch.use_deterministic_algorithms(was[0], warn_only=was[1])
        torch.utils.deterministic.fill_uninitialized_memory = was[2]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_new_tensors_in_inference_mode(cuda):
    x = torch.randn(3, 256, device=cuda).bfloat16()
    want = w4q.add_rms_norm(x, x)
    with torch.inference_mode():
        got = w4q.add_rms_norm(x, x)
        assert got[0].is_inference()
    assert torch.equal(got[0], want[0]) and not want[0].is_inference()
