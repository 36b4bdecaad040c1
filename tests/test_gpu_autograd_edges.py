"""The autograd functions of the products and the routed rows at the edges of
what they take."""
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu


def _gen(device, *key):
    g = torch.Generator(device=device)
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _bf16(rows, cols, g, dev):
    return torch.randn(rows, cols, generator=g, device=dev).to(torch.bfloat16)


@pytest.mark.parametrize("which", ["matmul", "dispatch", "combine"])
def test_second_derivatives_are_refused(device, which):
    """Their gradients are written by kernels that leave no graph: a second
    derivative through them is an error, not a term that is missing."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, which)
    x = _bf16(12, 64, g, device).requires_grad_()
    if which == "matmul":
        out = tr.MxMatmul.apply(x, _bf16(32, 64, g, device).requires_grad_())
    else:
        ids = torch.randint(0, 3, (12, 2) if which == "dispatch" else (6, 2), generator=g, device=device)
        off, index, slot = tr.expert_sort(ids, 3)
        if which == "dispatch":
            out = tr.ExpertDispatch.apply(x, index, slot)
        else:
            out = tr.ExpertCombine.apply(x, slot, torch.rand(6, 2, generator=g, device=device), off)
    gx, = torch.autograd.grad(out, x, torch.ones_like(out).requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.float().sum().backward()
