"""The autograd functions of the products and the routed rows, and the products
of empty contractions, at the edges of what they take."""
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


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
def test_empty_contractions(device, fmt):
    """k == 0: sums of nothing, as the C entry points give them."""
    import fp4_rollout_guided_amd as tr
    matmul, grouped, bwd_weight, grouped_bwd = (
        (tr.mx_matmul, tr.grouped_mx_matmul, tr.mx_matmul_bwd_weight, tr.grouped_mx_matmul_bwd_weight) if fmt == "mx" else
        (tr.mx8_matmul, tr.grouped_mx8_matmul, tr.mx8_matmul_bwd_weight, tr.grouped_mx8_matmul_bwd_weight))
    none = torch.empty(0, dtype=torch.uint8, device=device)
    off = torch.tensor([0, 2, 4], device=device)
    y = torch.full((5, 32), 7.0, device=device).bfloat16()
    assert matmul(none, none, none, none, 32, 0, y=y) is y and (y == 0).all()
    y.fill_(7)
    assert (grouped(none, none, off, none, none, 32, 0, y=y) == 0).all()
    got = grouped(none, none, off, none, none, 32, 0, row_index=torch.zeros(5, dtype=torch.int64, device=device))
    assert got.shape == (5, 32) and (got == 0).all()
    with pytest.raises(ValueError, match="y must be given"):
        matmul(none, none, none, none, 32, 0)
    gy = torch.ones(5, 32, dtype=torch.bfloat16, device=device)
    assert bwd_weight(gy, none, none, 0).shape == (32, 0)
    assert grouped_bwd(gy, off, none, none, 0).shape == (2, 32, 0)
    x = torch.empty(2, 3, 0, dtype=torch.bfloat16, device=device, requires_grad=True)
    w = torch.empty(32, 0, dtype=torch.bfloat16, device=device, requires_grad=True)
    out = tr.MxMatmul.apply(x, w, None, fmt)
    assert out.shape == (2, 3, 32) and (out == 0).all()
    out.backward(torch.ones_like(out))
    assert x.grad.shape == x.shape and w.grad.shape == w.shape


def test_combine_without_weights(device):
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "no weights")
    ids = torch.randint(0, 4, (10, 3), generator=g, device=device)
    off, _, slot = tr.expert_sort(ids, 3)
    y, go = _bf16(30, 64, g, device).requires_grad_(), _bf16(10, 64, g, device)
    out = tr.ExpertCombine.apply(y, slot, None, off)
    assert torch.equal(out, tr.expert_combine(y.detach(), slot))
    out.backward(go)
    want = go.new_zeros(30, 64)
    t, j = (slot >= 0).nonzero(as_tuple=True)
    want[slot[t, j]] = go[t]
    assert torch.equal(y.grad, want)
