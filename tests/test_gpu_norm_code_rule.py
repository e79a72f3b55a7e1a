"""The norm's codes are those that the activation quantizer gives the same values: rint of the fp32 quotient."""
import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("power", [0, -40, 60, -115])
def test_codes_are_the_quantizers(cuda, row, power):
    """Rows of ones and minus ones have the root 1, so that y is the weight itself, to the bit; every other weight is a power
    of two below its group's (row's) largest, half of which is the middle of two codes."""
    hidden = 4096
    top = torch.arange(128, device=cuda, dtype=torch.float64) / 128 + 1
    g = torch.Generator(device=cuda).manual_seed(3)
    for begin in (range(0, 128, 16) if row else (0,)):
        many = top[begin:begin + 1].expand(128) if row else top
        w = many[:, None] * 2.0 ** -torch.randint(0, 9, (128, 32), generator=g, device=cuda).double()
        w[:, 1::2] *= 1 + torch.randint(0, 64, (128, 16), generator=g, device=cuda).double() / 64
        w = torch.minimum(w, many[:, None])
        w[:, 0] = many
        w[:, 2] = many / 2
        w = (w.reshape(-1) * 2.0 ** power).bfloat16()
        x = torch.where(torch.rand(3, hidden, generator=g, device=cuda) < 0.5, -1.0, 1.0).bfloat16()
        out = torch.empty_like(x)
        codes, scales, _ = w4q.add_rms_norm_a8(x, None, w, eps=0.0, row=row, out=out)
        assert torch.equal(out.float(), x.float() * w.float())
        want, want_scales = (w4q.w4a8_quantize_act_rowscale if row else w4q.w4a8_quantize_act)(out)
        assert torch.equal(scales, want_scales.view_as(scales))
        assert torch.equal(codes, want)
