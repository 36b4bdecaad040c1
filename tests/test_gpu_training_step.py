"""The operators together, as a training step of a routed policy uses them: router,
sorted rows, the experts' microscaled product, the weighted sum, the loss over the
vocabulary, the gradients of all of it, and the optimiser step, against the same
step in 64 bits with the same roundings of the operands passed straight through."""
import sys

import pytest
import torch

from tests import step_util as U
from tests.product_util import values

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


class _Straight(torch.autograd.Function):
    """A rounded operand's values in the forward, its gradient where the clip mask is set."""

    @staticmethod
    def forward(ctx, x, rounded, keep):
        ctx.save_for_backward(keep)
        return rounded

    @staticmethod
    def backward(ctx, g):
        return g * ctx.saved_tensors[0], None, None


def _rounded(tr, fmt, x, cols):
    scales, codes, mask = (tr.mx_quantize if fmt == "mx" else tr.mx8_quantize)(x, want_mask=True)
    keep = ((mask.unsqueeze(-1) >> torch.arange(8, device=x.device, dtype=torch.uint8)) & 1).flatten().double()
    return values(fmt, scales, codes, cols).view(x.shape), keep.view(x.shape)


def test_training_step(device):
    import fp4_rollout_guided_amd as tr
    _say("case training step")
    g = torch.Generator(device=device)
    g.manual_seed(11)
    tokens, cols, experts, topk, vocab = 240, 128, 8, 2, 700
    new = lambda *s, by=1.0: (torch.randn(*s, generator=g, device=device) * by).to(torch.bfloat16)  # noqa: E731
    x, router, w, head = new(tokens, cols), new(experts, cols, by=0.3), new(experts, cols, cols, by=0.09), new(vocab, cols, by=0.3)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    targets[::5] = -100
    valid = torch.rand(tokens, generator=g, device=device) < 0.9
    params = [torch.nn.Parameter(p) for p in (router, w, head)]
    opt = tr.AdamW(params, lr=1e-3, states="mx8", seed=3)
    count = int((targets >= 0).sum())

    def loss_of():
        r, we, h = params
        z = x.float() @ r.float().t()
        ids, weights, counts, balance = tr.ExpertRoute.apply(z, topk, True, valid)
        offsets, row_index, slot = tr.expert_sort(ids, experts)
        rows = tr.ExpertDispatch.apply(x, row_index, slot)
        y = tr.MxMatmul.apply(rows, we, offsets, "mx8")
        out = tr.ExpertCombine.apply(y, slot, weights, offsets)
        hidden = x + out
        loss = tr.LinearCrossEntropy.apply(hidden, h, targets, 1.0)
        return loss.sum() / count + 0.01 * balance.sum(), ids, rows, offsets, slot, hidden

    total, ids, rows, offsets, slot, hidden = loss_of()
    total.backward()
    got = [p.grad.clone() for p in params]

    # the same in 64 bits: the operands' roundings are the kernels' own, everything else is exact
    r64, w64, h64 = (p.detach().double().requires_grad_(True) for p in params)
    z = x.double() @ r64.t()
    at = ids.clamp(min=0)
    there = (ids >= 0).double()
    weights = torch.softmax(z.gather(1, at), 1) * there
    p = torch.softmax(z, 1) * (ids[:, :1] >= 0)
    counts = torch.bincount(ids[ids >= 0], minlength=experts).double()
    balance = experts * (counts / counts.sum() * p.sum(0) / (ids[:, 0] >= 0).sum()).sum()
    aq, _ = _rounded(tr, "mx8", rows, cols)
    wq, keep = _rounded(tr, "mx", w, cols)
    ws = _Straight.apply(w64, wq, keep)
    y = torch.zeros(tokens * topk, cols, dtype=torch.float64, device=device)
    o = offsets.tolist()
    y = torch.cat([aq[o[e]:o[e + 1]] @ ws[e].t() for e in range(experts)] + [y[o[-1]:]])
    out = (y[slot.clamp(min=0)] * (weights * (slot >= 0)).unsqueeze(-1)).sum(1)
    loss, _, has = U.loss(x.double() + out, h64, targets)
    want_total = loss.sum() / has.sum() + 0.01 * balance
    want = torch.autograd.grad(want_total, (r64, w64, h64))

    # each activation on the way is rounded to bf16 (y, out, hidden: 2^-8 of itself each), and so is each gradient (P, to
    # hidden, to y, the result): eight roundings in all, of at most 2^-8, whose sum bounds the norm of the difference
    total, want_total = float(total.detach()), float(want_total.detach())
    assert abs(total - want_total) < 8 * 2.0 ** -8 * abs(want_total)
    for a, b, name in zip(got, want, ("router", "experts", "head")):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel < 8 * 2.0 ** -8, (name, rel)
    before = [p.detach().clone() for p in params]
    opt.step()
    # the first step: m / sqrt(v) is the gradient's sign (g / |g|), so each weight moves by lr and its rounding, up to a
    # step of bf16 (2^-7 of itself), less its decay
    for p, b, gr in zip(params, before, got):
        moved = p.detach().double() - b.double()
        want_move = -1e-3 * torch.sign(gr.double()) - 1e-5 * b.double()
        far = (gr.double().abs() > 1e-5) & ((moved - want_move).abs() > 2.0 ** -7 * b.double().abs() + 2e-5)
        assert not far.any(), float((moved - want_move).abs().max())
    opt.zero_grad()
    again, *_ = loss_of()
    again.backward()
    opt.step()
    assert opt.steps == 2 and all(p.isfinite().all() for p in params)
