"""moe_w4a16, row by row: what a token gets does not depend on the others of its batch."""
import math

import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q
from test_gpu_moe import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts", [8, 200])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_weights_of_a_token_without_finite_scores(cuda, sigmoid, renormalize, experts, value):
    layer = Layer(256, 256, experts)
    x = layer.x(11)
    want_ids, want = torch.empty(11, 2, dtype=torch.int32, device=cuda), torch.empty(11, 2, device=cuda)
    w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2, sigmoid=sigmoid, renormalize=renormalize, ids=want_ids, weights=want)
    x[4, 7] = value
    x[4, 8] = -value          # inf - inf in every logit
    layer.router[:, 7:9] = 1.0
    ids, w = torch.empty(11, 2, dtype=torch.int32, device=cuda), torch.empty(11, 2, device=cuda)
    out = w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2, sigmoid=sigmoid, renormalize=renormalize, ids=ids, weights=w)
    assert torch.isnan(w[4]).all() and torch.isnan(out[4]).all()
    keep = [i for i in range(11) if i != 4]
    assert torch.isfinite(w[keep]).all() and torch.isfinite(out[keep]).all()
    assert (ids >= 0).all() and (ids < experts).all() and (ids[:, 0] != ids[:, 1]).all()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_softmax_with_one_nan_logit_is_nan(cuda, sigmoid):
    """A NaN in one expert's router row: every softmax score is NaN, of the sigmoid scores that expert's alone."""
    layer = Layer(256, 256, 8)
    layer.router[3] = math.nan
    ids, w = torch.empty(5, 2, dtype=torch.int32, device=cuda), torch.empty(5, 2, device=cuda)
    w4q.moe_w4a16(layer.x(5), layer.router, layer.w13, layer.w2, 256, 2, sigmoid=sigmoid, ids=ids, weights=w)
    assert (ids != 3).all()
    assert torch.isfinite(w).all() if sigmoid else torch.isnan(w).all()


@pytest.mark.parametrize("topk,inter", [(1, 256), (3, 256), (4, 1024), (2, 2048)])
@pytest.mark.parametrize("tokens", [1, 5, 8, 9, 12, 16, 17, 33, 64])
def test_a_row_keeps_its_precision_in_any_batch(cuda, topk, inter, tokens):
    """topk * inter up to 4096: h enters the second product with 16 bits, whatever the number of tokens is.  The bound of
    test_gpu_moe without the 2^-8 of a bf16 h."""
    layer = Layer(512, inter, 6)
    x = layer.x(64)[:tokens]
    ids, weights = torch.empty(tokens, topk, dtype=torch.int32, device=cuda), torch.empty(tokens, topk, device=cuda)
    out = w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, inter, topk, ids=ids, weights=weights)
    ref, mag = layer.reference(x, ids.long(), weights)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * mag).all()
