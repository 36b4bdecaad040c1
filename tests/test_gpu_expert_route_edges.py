"""The router's gradients for pairs that were taken out after the forward."""
import sys

import pytest
import torch

from tests.test_gpu_expert_route import logits

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("experts,topk", [(40, 4), (40, 20), (300, 6)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_first_pairs_taken_out(device, dtype, experts, topk, renormalize):
    """A row counts as long as one of its pairs stands, whichever it is (a limit of an expert's rows took the others).
    Against the 64-bit gradient of the pairs that stand; the tolerance is that of test_gpu_expert_route.check."""
    import fp4_rollout_guided_amd as tr
    _say("case pairs taken out", dtype, experts, topk, renormalize)
    tokens = 61
    z = logits(tokens, experts, dtype, device)
    ids, _, counts, _, _ = tr.expert_route(z, topk)
    ids[::3, 0] = -1
    ids[1::6, :topk - 1] = -1
    ids[5::7] = -1
    there = ids >= 0
    some = there.any(1)
    zd = z.double().requires_grad_(True)
    p = torch.softmax(zd, 1)
    sel = torch.where(there, zd.gather(1, ids.clamp(min=0)), -float("inf"))[some]
    w = torch.softmax(sel, 1) if renormalize else torch.where(there, p.gather(1, ids.clamp(min=0)), 0.0)[some]
    weights = torch.zeros(tokens, topk, dtype=torch.float64, device=device)
    weights[some] = w.detach()
    gw = torch.where(there, torch.randn(tokens, topk, device=device), float("nan"))
    clean = torch.where(there, gw, 0.0).double()
    gb = torch.full((1,), 0.3 * tokens, device=device)
    c = counts[:-1].double()
    slope = float(gb) * experts * c / c.sum() / float(counts[-1])
    rel, half = 2.0 ** -18, 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for a, b in ((gw, gb), (gw, None), (None, gb)):
        got = tr.expert_route_bwd(a, b, z, ids, weights.float(), counts, renormalize=renormalize)
        total = (w * clean[some]).sum() if a is not None else 0.0
        if b is not None:
            total = total + (p[some] * slope).sum()
        want, = torch.autograd.grad(total, zd, retain_graph=True)
        size, pd = torch.zeros_like(want), p.detach()
        if a is not None:
            part = weights * clean.abs()
            size += pd * part.sum(1, keepdim=True)
            size.scatter_add_(1, ids.clamp(min=0), part + weights * part.sum(1, keepdim=True))
        if b is not None:
            size += pd * (slope + (pd * slope).sum(1, keepdim=True))
        tol = 16 * rel * size
        tol = tol + half * (want.abs() + tol) + 2.0 ** -126
        assert ((got.double() - want).abs() <= tol).all(), (a is None, b is None)
        assert not got[~some].any()
