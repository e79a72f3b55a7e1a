"""The ends of the norm's range: rows and weights up to those that w4q.h names give right values, and a row beyond them
leaves its neighbours alone."""
import pytest
import torch

from ends_reference import BF16_HALF_STEP, norm
from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -16   # a root, two products and sums of at most 1024 squares


def close(out, ref, steps=BF16_HALF_STEP):
    assert torch.isfinite(out).all()
    assert ((out.double() - ref).abs() <= ref.abs() * (steps + 2 * FP32)).all()


# row's power, weight's power: squares that just have room, products of row and weight at both ends of fp32's normal range
@pytest.mark.parametrize("row,weight,eps", [(55, 0, 1e-6), (55, 70, 1e-6), (40, 84, 1e-6), (0, 124, 1e-6), (-50, 0, 0.0), (-50, -70, 0.0),
                                            (-56, 0, 0.0), (-56, 100, 0.0), (0, -120, 1e-6), (-20, -100, 0.0)])
@pytest.mark.parametrize("hidden", [256, 1024])
def test_rows_and_weights_at_the_ends(cuda, row, weight, eps, hidden):
    g = torch.Generator(device=cuda).manual_seed(row + hidden)
    x = ((1 + torch.rand(5, hidden, generator=g, device=cuda, dtype=torch.float64)) * 2.0 ** row).bfloat16()
    w = ((1 + torch.rand(hidden, generator=g, device=cuda, dtype=torch.float64)) * 2.0 ** weight).bfloat16()
    x[::2] *= -1
    want = norm(x, None, w, eps)[1]
    out, _ = w4q.add_rms_norm(x, None, w, eps=eps)
    close(out, want)
    for by_row in (False, True):
        codes, scales, _ = w4q.add_rms_norm_a8(x, None, w, eps=eps, row=by_row)
        top = want.view(5, 1 if by_row else hidden // 32, -1)
        s = scales.double().view(5, -1, 1)
        close(s, top.abs().amax(-1, keepdim=True) / 127, 2.0 ** -23)
        assert ((codes.double().view_as(top) * s - top).abs() <= s * (0.5 + 127 * 3 * FP32)).all()


def test_a_row_beyond_the_ends_stays_by_itself(cuda):
    g = torch.Generator(device=cuda).manual_seed(1)
    x = torch.randn(4, 512, generator=g, device=cuda).bfloat16()
    w = (torch.rand(512, generator=g, device=cuda) + 0.5).bfloat16()
    w[7] = 2.0 ** 100
    want = w4q.add_rms_norm(x, None, w, eps=0.0)[0]
    x[1] = (x[1].double() * 2.0 ** 50).bfloat16()       # its products with the weight overflow
    x[3] = (x[3].double() * 2.0 ** -100).bfloat16()     # its squares are all 0
    out = w4q.add_rms_norm(x, None, w, eps=0.0)[0]
    assert torch.equal(out[[0, 2]], want[[0, 2]])
    assert not out[1, 7].isfinite() and torch.isfinite(out[1, :7]).all()
    assert not out[3].isfinite().any()
