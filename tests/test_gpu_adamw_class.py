"""AdamW's class: copies of the weights, their gradients, states that move, and checkpoints."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def test_copies_given_up(device):
    """Copies that the optimiser has no more are not written to."""
    import fp4_rollout_guided_amd as tr
    _say("case copies given up")
    params = [torch.randn(n, device=device) for n in (100, 5000, 3)]
    copies = [torch.empty(n, dtype=torch.bfloat16, device=device) for n in (100, 5000, 3)]
    opt = tr.AdamW(params, lr=0.1, copies=copies)
    grads = [torch.randn_like(p) for p in params]
    opt.step(grads)
    assert all(torch.equal(c, p.to(torch.bfloat16)) for c, p in zip(copies, params))
    former = [c.clone() for c in copies]
    opt.copies = None
    opt.step(grads)
    assert all(torch.equal(c, f) for c, f in zip(copies, former))
    assert not torch.equal(params[1].to(torch.bfloat16), former[1])
    opt.copies = copies
    opt.step(grads)
    assert all(torch.equal(c, p.to(torch.bfloat16)) for c, p in zip(copies, params))
