"""Drawing without drafts: of equal logits with equal noise the lowest index wins, wherever the row's other logits lie and
however the row is cut."""
import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,vocab", [(3, 600), (64, 5000), (300, 9001), (2, 151936), (40, 50257)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heat", [None, 0.7, 0.037, 5.0])
def test_equal_elements_below_the_maximum(cuda, seqs, vocab, dtype, heat):
    """The tied elements have logits between -3 T and 3 T below a maximum of some 4 to 5 deviations, and noise that lets
    them win by a factor of 1000."""
    g = torch.Generator(device=cuda).manual_seed(seqs + vocab)
    t = 1.0 if heat is None else heat
    for _ in range(10):
        logits = (torch.randn(seqs, 1, vocab, generator=g, device=cuda) * t).to(dtype)
        noise = 0.5 + torch.rand(seqs, vocab, generator=g, device=cuda)
        places = torch.rand(seqs, vocab, generator=g, device=cuda).topk(4, 1).indices
        value = (torch.rand(seqs, generator=g, device=cuda) * 6 - 3) * t
        rows = torch.arange(seqs, device=cuda)[:, None]
        logits[rows, 0, places] = value[:, None].to(dtype)
        # e^(5.5 + 3) of the largest over the least of them, and a factor of 1000
        noise[rows, places] = (1e-7 * (1 + torch.rand(seqs, generator=g, device=cuda)))[:, None]
        none = torch.empty(seqs, 0, device=cuda)
        tokens, _ = w4q.verify_drafts(logits, none.int(), none, noise,
                                      temperature=None if heat is None else torch.full((seqs,), heat, device=cuda))
        assert torch.equal(tokens[:, 0].long(), places.amin(1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_batch_does_not_decide(cuda, dtype):
    """Rows of few different logits and noises, full of ties and near ties: the same tokens one by one, in a batch, and in
    rows that lie apart."""
    g = torch.Generator(device=cuda).manual_seed(5)
    seqs, vocab = 96, 20011
    logits = (torch.randint(-40, 12, (seqs, 1, vocab), generator=g, device=cuda) / 8).to(dtype)
    noise = 1.0 + torch.randint(0, 4, (seqs, vocab), generator=g, device=cuda) / 4
    noise[logits[:, 0].float() > 0.5] *= 8                # most ties that win lie below the row's maximum
    none = torch.empty(seqs, 0, device=cuda)
    heat = 0.3 + torch.rand(seqs, generator=g, device=cuda)

    def draw(at, rows):
        return w4q.verify_drafts(rows, none[at].int(), none[at], noise[at].clone(), temperature=heat[at].clone())[0][:, 0]

    want = draw(slice(None), logits)
    wide = torch.zeros(seqs, 1, vocab + 21, dtype=dtype, device=cuda)
    wide[..., :vocab] = logits
    assert torch.equal(draw(slice(None), wide[..., :vocab]), want)
    alone = torch.cat([draw(slice(i, i + 1), logits[i:i + 1].clone()) for i in range(seqs)])
    assert torch.equal(alone, want)
    # and in fp64 by the definition: equal logits with equal noise are equal there too
    score = logits.double()[:, 0] / heat.double()[:, None] - noise.double().log()
    best = score.amax(1, keepdim=True)
    assert torch.equal(want.long(), (score >= best - 1e-9).int().argmax(1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [40, 4099, 33000, 151936])
@pytest.mark.parametrize("n", [0, 2])
def test_a_greedy_sequences_noise_does_not_matter(cuda, dtype, vocab, n):
    g = torch.Generator(device=cuda).manual_seed(vocab)
    logits = torch.randint(-30, 20, (6, n + 1, vocab), generator=g, device=cuda).to(dtype)
    heat = torch.tensor([0.0, 1.0, -1.0, 0.0, 0.5, float("nan")], device=cuda)
    noise = torch.empty(6, vocab, device=cuda).exponential_(generator=g)
    drafts, u = torch.zeros(6, n, dtype=torch.int32, device=cuda), torch.ones(6, n, device=cuda)
    want = w4q.verify_drafts(logits, drafts, u, noise, temperature=heat)
    greedy = ~(heat > 0)
    first = want[0][greedy, want[1][greedy].long()]
    rows = logits[greedy, want[1][greedy].long()].float()
    assert torch.equal(first.long(), (rows == rows.amax(1, keepdim=True)).int().argmax(1))
    noise[greedy] = torch.tensor([float("nan"), 0.0, float("inf"), -1.0], device=cuda)[torch.randint(4, (4, vocab), generator=g, device=cuda)]
    got = w4q.verify_drafts(logits, drafts, u, noise, temperature=heat)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
