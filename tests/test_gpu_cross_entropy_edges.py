"""The loss over the vocabulary where roundings and fillers could show: very
confident tokens, vocabulary rows of -infinity, and the tiles of the largest calls."""
import sys

import pytest
import torch

from tests import step_util as U
from tests.test_gpu_cross_entropy import check, inputs

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("tokens,vocab,scale", [(40, 500, 1.0), (64, 9000, 0.7), (300, 500, 1.25), (1500, 3001, 1.0)])
def test_confident_tokens_lose_nothing(device, tokens, vocab, scale):
    """No log-probability is above zero.  Where the target's logit is the largest, the loss is the logarithm of one and
    the other exponentials' sum: each of them off by the two logits' errors (step_util.loss_tolerance), the sum by 2^-24
    for each addition, and nothing of the logit's own size."""
    import fp4_rollout_guided_amd as tr
    _say("case confident tokens", tokens, vocab, scale)
    g = torch.Generator(device=device)
    g.manual_seed(tokens)
    k = 128
    w = (torch.randn(vocab, k, generator=g, device=device) / k ** 0.5).to(torch.bfloat16)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    lean = 1 + 79 * torch.rand(tokens, 1, generator=g, device=device) / scale
    x = (lean * w[targets].float()).to(torch.bfloat16)
    loss, lse = tr.linear_cross_entropy(x, w, targets, scale)
    want, want_lse, has = U.loss(x, w, targets, scale)
    z = U.logits(x, w, scale)
    tol = U.loss_tolerance(x, w, has, scale, want_lse)
    assert ((lse.double() - want_lse).abs() <= tol).all()
    assert (loss >= 0).all(), float(loss.min())
    largest = z.gather(1, targets.unsqueeze(1)).squeeze(1) >= z.amax(1)
    assert int(largest.sum()) > tokens // 2
    size = (x.double().abs() @ w.double().abs().t().contiguous()).amax(1) * scale
    each = torch.expm1(2 * size * ((k + 3) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -21)
    near = want * each + (100 + vocab / 64) * 2.0 ** -24 + want * 2.0 ** -22
    assert ((loss.double() - want).abs() <= near)[largest].all()


@pytest.mark.parametrize("tokens", [256, 300, 1100])
def test_vocabulary_rows_of_minus_infinity(device, tokens):
    """An entry whose logit is -infinity for every token has no probability: the loss and the other rows' gradients are
    those without it, and its own row's gradient is zero, however the rows fill their tiles."""
    import fp4_rollout_guided_amd as tr
    _say("case rows of -infinity", tokens)
    g = torch.Generator(device=device)
    g.manual_seed(tokens)
    vocab, k = 700, 96
    x = torch.randn(tokens, k, generator=g, device=device).to(torch.bfloat16)
    x[:, 0] = 1.0
    w = (torch.randn(vocab, k, generator=g, device=device) / k ** 0.5).to(torch.bfloat16)
    targets = torch.randint(5, vocab - 5, (tokens,), generator=g, device=device)
    targets = torch.where(targets == 300, 301, targets)
    grad = torch.randn(tokens, generator=g, device=device)
    gone = [3, 300, vocab - 1]
    w[gone, 0] = -float("inf")
    loss, lse = tr.linear_cross_entropy(x, w, targets)
    without = w.clone()
    without[gone] = 0
    keep = torch.ones(vocab, dtype=torch.bool, device=device)
    keep[gone] = False
    place = torch.cumsum(keep, 0) - 1
    want, want_lse, has = U.loss(x, w[keep], place[targets])
    tol = U.loss_tolerance(x, w[keep], has, 1.0, want_lse)
    assert ((lse.double() - want_lse).abs() <= tol).all() and ((loss.double() - want).abs() <= 2 * tol).all()
    _, gw = tr.linear_cross_entropy_bwd(grad, x, w, targets, lse, want_x=False)
    _, ww, _, sw = U.loss_gradients(grad, x, w[keep], place[targets])
    assert not gw[gone].any()
    U.gradients_close(gw[keep], ww, sw, tokens + 8, x, w[keep], 1.0, ("minus infinity", "grad_w"))


# the products in tiles of 256 (grad_w of the last case in those of 128), over more stages than the ring holds: k past whole
# tiles and with a last half stage, grad_x in parts, a last slice shorter than the others, ignored tokens
@pytest.mark.parametrize("tokens,vocab,k,ignored", [(4000, 20000, 2080, 0.3), (4096, 33000, 2048, 0.0), (33000, 16600, 1056, 0.2)])
def test_tiles_of_the_largest_calls(device, tokens, vocab, k, ignored):
    import fp4_rollout_guided_amd as tr
    _say("case largest tiles", tokens, vocab, k)
    check(tr, *inputs(tokens, vocab, k, device, ignored=ignored), 0.8, (tokens, vocab, k))


# few tokens whose rows are multiples of 4 KiB: each workgroup begins at a place of its own in k, several tiles to a share
@pytest.mark.parametrize("tokens,vocab,k", [(1, 65536 + 333, 2048), (33, 131072 + 77, 2048), (64, 100003, 4096), (16, 140000, 4096),
                                            (32, 70000, 6144), (5, 300, 2048), (64, 17, 2048)])
def test_few_tokens_of_long_rows(device, tokens, vocab, k):
    import fp4_rollout_guided_amd as tr
    _say("case few tokens, long rows", tokens, vocab, k)
    check(tr, *inputs(tokens, vocab, k, device, ignored=0.2 if tokens > 1 else 0.0), 1.1, (tokens, vocab, k))
