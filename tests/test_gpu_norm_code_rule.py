"""The norm's codes beside those that the activation quantizer gives the same values: rint of a product with the reciprocal
and rint of the quotient, which are the same but next to the middle of two codes."""
import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("power", [0, -40, 60, -115])
def test_codes_are_the_quantizers_but_next_to_a_middle(cuda, row, power):
    """Rows of ones and minus ones have the root 1, so that y is the weight itself, to the bit.  Every other weight is a power
    of two below its group's (row's) largest, the half of which is the middle of two codes.  The reciprocal and the quotient
    are each off by 2^-24 of 127 at most: the codes may differ within 2^-16 of a middle, by one."""
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
        quotient = out.double().view(3, 1 if row else 128, -1) / scales.double().view(3, -1, 1)
        middle = ((quotient.abs() % 1 - 0.5).abs() <= 2.0 ** -16).view(3, hidden)
        assert torch.equal(codes[~middle], want[~middle])
        assert ((codes.int() - want.int()).abs() <= 1).all()
