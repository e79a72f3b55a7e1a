"""moe_w4a16 against the formulas in fp64, on the weights that the packed bytes stand for.

Tolerances, from the arithmetic that w4q.h promises: the output is rounded once to bf16 (2^-8 relative), and each h
is (2^-8, acting on mag = sum weight |W2| |h|); silu, the fp32 sums and the choice's weights add less than 2^-14
relative of mag.  Rounding errors are independent, so their 2-norm over a whole output stays below that of two uniform
roundings, sqrt(2 / 3) 2^-8 = 0.0032 of the output's own (0.0035 with the rest)."""
import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


def dequantized(packed, n, k):
    q, s, z = w4q.w4_unpack_weights(packed, n, k)
    w = (q.view(n, k // 32, 32).double() - z.double()[..., None]) * s.double()[..., None]
    return w.view(n, k)


class Layer:
    def __init__(self, hidden, inter, experts, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.hidden, self.inter, self.experts = hidden, inter, experts
        self.router = (r(experts, hidden) * 2 * hidden ** -0.5).to(torch.bfloat16)
        self.w13 = w4q.w4_pack_weights((r(experts * 2 * inter, hidden) * hidden ** -0.5).to(torch.bfloat16))
        self.w2 = w4q.w4_pack_weights((r(experts * hidden, inter) * inter ** -0.5).to(torch.bfloat16))
        self.bias = r(experts) * 0.2

    def x(self, tokens, seed=1, size=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return (torch.randn(tokens, self.hidden, generator=g, device="cuda") * size).to(torch.bfloat16)

    def reference(self, x, ids, weights):
        """(out, mag) in fp64 for the given choice."""
        w13 = dequantized(self.w13, self.experts * 2 * self.inter, self.hidden).view(self.experts, 2, self.inter, self.hidden)
        w2 = dequantized(self.w2, self.experts * self.hidden, self.inter).view(self.experts, self.hidden, self.inter)
        out, mag = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for e in range(self.experts):
            m, k = (ids == e).nonzero(as_tuple=True)
            if len(m):
                gate, up = x[m].double() @ w13[e, 0].T, x[m].double() @ w13[e, 1].T
                h = gate / (1 + torch.exp(-gate)) * up
                w = weights[m, k].double()[:, None]
                out.index_add_(0, m, w * (h @ w2[e].T))
                mag.index_add_(0, m, w.abs() * (h.abs() @ w2[e].abs().T))
        return out, mag


def choose(layer, x, topk, bias, sigmoid, renormalize, scale):
    """ids, weights (fp64) and, per token, how far the choice is from another one, against the logits' error."""
    logits = x.double() @ layer.router.double().T
    # an fp32 sum in at most hidden / 32 dependent steps of an MMA, and the joining of at most 64 parts
    err = (layer.hidden / 32 + 64) * 2.0 ** -23 * (x.double().abs() @ layer.router.double().abs().T).amax(1)
    score = torch.sigmoid(logits) if sigmoid else torch.softmax(logits, 1)
    key = (score + (bias.double() if bias is not None else 0)) if sigmoid else logits
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    ids = order[:, :topk]
    sorted_key = key.gather(1, order)
    gap = (sorted_key[:, :-1] - sorted_key[:, 1:])[:, :topk].amin(1) if layer.experts > 1 else torch.full_like(err, 1.0)
    w = score.gather(1, ids)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    off = err * 0.25 if sigmoid else err   # the sigmoid's slope
    return ids, w * scale, gap > 4 * off + 2.0 ** -20, err


def check(layer, x, topk, bias=None, sigmoid=False, renormalize=True, scale=1.0, workspace=None):
    m = x.shape[0]
    ids = torch.full((m, topk), -1, dtype=torch.int32, device="cuda")
    weights = torch.full((m, topk), float("nan"), device="cuda")
    out = torch.full_like(x, float("nan"))
    w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, layer.inter, topk, bias=bias, sigmoid=sigmoid, renormalize=renormalize,
                  scale=scale, out=out, ids=ids, weights=weights, workspace=workspace)
    want, w, clear, err = choose(layer, x, topk, bias, sigmoid, renormalize, scale)
    assert clear.any() or m < 8
    assert torch.equal(ids[clear].long(), want[clear])
    assert ((weights.double() - w)[clear].abs() <= w[clear].abs() * (2 * err[clear, None] + 2.0 ** -18)).all()
    srt = ids.long().sort(1).values
    assert (srt[:, 1:] > srt[:, :-1]).all() and (srt >= 0).all() and (srt < layer.experts).all()
    ref, mag = layer.reference(x, ids.long(), weights)
    assert torch.isfinite(out).all()
    diff = (out.double() - ref).abs()
    assert (diff <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13) * mag).all()
    assert diff.norm() <= 0.0035 * ref.norm()
    return out


@pytest.mark.parametrize("hidden,inter,experts,topk", [(256, 256, 1, 1), (256, 256, 4, 4), (512, 256, 8, 2), (1024, 512, 16, 3),
                                                       (2048, 768, 40, 8), (768, 1280, 33, 5), (256, 512, 512, 16)])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 33, 64])
def test_against_fp64(cuda, hidden, inter, experts, topk, tokens):
    layer = Layer(hidden, inter, experts)
    check(layer, layer.x(tokens), topk)
    check(layer, layer.x(tokens, 2), topk, bias=layer.bias, sigmoid=True, scale=2.5)


@pytest.mark.parametrize("tokens", [1, 8, 64])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_weights_without_renormalization(cuda, tokens, sigmoid):
    layer = Layer(512, 256, 24)
    check(layer, layer.x(tokens), 4, sigmoid=sigmoid, renormalize=False, scale=0.5)


@pytest.mark.parametrize("tokens", [3, 20, 64])
def test_every_token_to_one_expert(cuda, tokens):
    """All tokens share their experts: 64 tokens of one expert, several passes over its tiles."""
    layer = Layer(512, 512, 6)
    x = layer.x(1).repeat(tokens, 1)
    out = check(layer, x, 2)
    assert (out == out[0]).all()


@pytest.mark.parametrize("tokens", [1, 10])
def test_equal_scores_go_to_the_lower_number(cuda, tokens):
    layer = Layer(256, 256, 20)
    layer.router[:] = layer.router[3]
    ids = torch.empty(tokens, 5, dtype=torch.int32, device="cuda")
    for sigmoid in (False, True):
        w4q.moe_w4a16(layer.x(tokens), layer.router, layer.w13, layer.w2, 256, 5, sigmoid=sigmoid, ids=ids)
        assert (ids == torch.arange(5, device="cuda")).all()
    w4q.moe_w4a16(layer.x(tokens) * 0, layer.router, layer.w13, layer.w2, 256, 5, ids=ids)
    assert (ids == torch.arange(5, device="cuda")).all()


def test_bias_moves_the_choice_and_not_the_weight(cuda):
    layer = Layer(256, 256, 12)
    bias = torch.zeros(12, device="cuda")
    bias[7], bias[2] = 100.0, -100.0
    x = layer.x(30)
    ids, w = torch.empty(30, 12, dtype=torch.int32, device="cuda"), torch.empty(30, 12, device="cuda")
    w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 12, bias=bias, sigmoid=True, renormalize=False, ids=ids, weights=w)
    assert (ids[:, 0] == 7).all() and (ids[:, 11] == 2).all()
    score = torch.sigmoid(x.double() @ layer.router.double().T)
    assert (w.double() - score.gather(1, ids.long())).abs().max() < 1e-5


@pytest.mark.parametrize("size", [0.0, 2.0 ** -40, 2.0 ** 20])
def test_magnitudes(cuda, size):
    layer = Layer(512, 256, 8)
    x = layer.x(5) * size
    ids, w = torch.empty(5, 2, dtype=torch.int32, device="cuda"), torch.empty(5, 2, device="cuda")
    out = w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2, ids=ids, weights=w)
    ref, mag = layer.reference(x, ids.long(), w)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7.9 * mag + 2.0 ** -100).all()


def test_tokens_with_nan_or_infinity_leave_the_others_alone(cuda):
    layer = Layer(512, 256, 8)
    x = layer.x(12)
    want = w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2)
    y = x.clone()
    y[3, 5], y[10, 100] = float("nan"), float("inf")
    got = w4q.moe_w4a16(y, layer.router, layer.w13, layer.w2, 256, 2)
    keep = [i for i in range(12) if i not in (3, 10)]
    assert torch.equal(got[keep], want[keep])


def test_repeated_calls_and_graph_replay_are_bitwise_equal(cuda):
    layer = Layer(1024, 512, 32)
    ws = torch.full((w4q.moe_workspace_bytes(64, 1024, 512, 32, 4),), 255, dtype=torch.uint8, device="cuda")
    for tokens in (1, 40, 5, 64):
        x = layer.x(tokens)
        call = lambda out=None: w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 512, 4, out=out, workspace=ws)  # noqa: E731, B023
        a = call()
        for _ in range(5):
            assert torch.equal(call(), a)
        out = torch.zeros_like(a)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)


@pytest.mark.parametrize("tokens,topk,inter", [(1, 1, 256), (1, 3, 256), (5, 1, 768), (8, 2, 256), (2, 4, 512)])
def test_few_terms_are_not_rounded_between_the_products(cuda, tokens, topk, inter):
    """tokens * topk * inter up to 4096: the bound of check() without the 2^-8 of h's rounding."""
    layer = Layer(512, inter, 6)
    x = layer.x(tokens)
    ids, weights = torch.empty(tokens, topk, dtype=torch.int32, device=cuda), torch.empty(tokens, topk, device=cuda)
    out = w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, inter, topk, ids=ids, weights=weights)
    ref, mag = layer.reference(x, ids.long(), weights)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * mag).all()


@pytest.mark.parametrize("topk,hidden,inter", [(1, 256, 256), (2, 256, 512), (8, 512, 256)])
def test_workspace_grows_with_the_tokens(cuda, topk, hidden, inter):
    sizes = [w4q.moe_workspace_bytes(m, hidden, inter, 16, topk) for m in range(1, 65)]
    assert sizes == sorted(sizes)


def test_on_a_stream_of_its_own(cuda):
    layer = Layer(512, 256, 8)
    x = layer.x(4)
    want = w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2, stream=stream)
    stream.synchronize()
    assert torch.equal(got, want)


def test_refused_calls_write_nothing(cuda):
    layer = Layer(256, 256, 4)
    x = layer.x(2)
    out = torch.full_like(x, 7.0)
    with pytest.raises(w4q.W4QError) as err:
        w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2, out=out, workspace=torch.zeros(16, dtype=torch.uint8, device=cuda))
    assert err.value.status == 4
    with pytest.raises(w4q.W4QError):
        w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 5, out=out)
    with pytest.raises(w4q.W4QError):
        w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2, 256, 2, bias=layer.bias, out=out)
    with pytest.raises(ValueError):
        w4q.moe_w4a16(x, layer.router, layer.w13, layer.w2[:-16], 256, 2, out=out)
    with pytest.raises(ValueError):
        w4q.moe_w4a16(x.float(), layer.router, layer.w13, layer.w2, 256, 2, out=out)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
