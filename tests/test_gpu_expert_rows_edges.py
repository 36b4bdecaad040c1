"""The routed rows where pairs have been dropped from the sorted order: their
rows' gradients, which no slot names, and results that hold NaN."""
import sys
import zlib

import pytest
import torch

from tests.product_util import close

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _gen(device, *key):
    g = torch.Generator(device=device)
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


@pytest.mark.parametrize("tokens,topk,cols", [(1, 1, 16), (5, 2, 48), (40, 8, 2048), (700, 4, 528), (1024, 8, 144),
                                              (1025, 8, 144), (5003, 5, 1040)])
@pytest.mark.parametrize("drop", [0.3, 1.0])
def test_gradients_of_dropped_pairs_are_zeros(device, tokens, topk, cols, drop):
    """Pairs over an expert's capacity, taken out of slot: their rows lie inside
    the groups, and their gradient is zero whatever the memory held."""
    import fp4_rollout_guided_amd as tr
    _say("case dropped", tokens, topk, cols, drop)
    g = _gen(device, tokens, topk, cols, drop)
    ids = torch.randint(-1, 9, (tokens, topk), generator=g, device=device)
    off, _, slot = tr.expert_sort(ids, 8)
    slot[torch.rand(tokens, topk, generator=g, device=device) < drop] = -1
    y = torch.randn(tokens * topk, cols, generator=g, device=device).to(torch.bfloat16)
    go = torch.randn(tokens, cols, generator=g, device=device).to(torch.bfloat16)
    wt = torch.randn(tokens, topk, generator=g, device=device)
    want = torch.zeros(y.shape, dtype=torch.float64, device=device)
    t, j = (slot >= 0).nonzero(as_tuple=True)
    want[slot[t, j]] = go.double()[t] * wt.double()[t, j].unsqueeze(1)
    named = torch.zeros(y.shape[0], dtype=torch.bool, device=device)
    named[slot[t, j]] = True
    guard = torch.full((y.shape[0] + 3, cols), float("nan"), dtype=torch.bfloat16, device=device)
    gy, gw = tr.expert_combine_bwd(go, y, slot, wt, off, grad_y=guard[:-3])
    assert guard[-3:].isnan().all()
    close(gy, want, want.abs(), 1)
    assert (gy[~named].view(torch.int16) == 0).all() and (gw[slot < 0] == 0).all()
    # memory of the allocator's that was not zeros
    junk = torch.full_like(y, float("nan"))
    del junk
    leaf, leaf_w = y.clone().requires_grad_(), wt.clone().requires_grad_()
    tr.ExpertCombine.apply(leaf, slot, leaf_w, off).backward(go)
    assert torch.equal(leaf.grad.view(torch.int16), gy.view(torch.int16)) and torch.equal(leaf_w.grad, gw)


@pytest.mark.parametrize("more", [0, 9000])  # pairs looked through, and rows marked
def test_no_gradient_is_taken_for_a_row_without_one(device, more):
    """Rows of NaN, of every kind of payload, stay NaN where a slot names them."""
    import fp4_rollout_guided_amd as tr
    cols = 64
    bits = torch.tensor([0x7F81, 0x7FBF, 0x7FC0, 0xFF81 - 65536, 0x7FFF, 0x7FC1], device=device)
    bits = bits.repeat(1 + more // len(bits))
    go = bits.to(torch.int16).unsqueeze(1).repeat(1, cols).contiguous().view(torch.bfloat16)
    tokens = go.shape[0]
    slot = torch.arange(tokens, device=device).flip(0).unsqueeze(1).contiguous()
    off = torch.tensor([0, tokens, tokens], device=device)
    y = torch.ones(tokens + 2, cols, dtype=torch.bfloat16, device=device)
    for wt in (None, torch.ones(tokens, 1, device=device), torch.full((tokens, 1), -2.0, device=device)):
        gy, gw = tr.expert_combine_bwd(go, y, slot, wt, off)
        assert gy[:tokens].isnan().all() and (gy[tokens:] == 0).all() and gw.isnan().all()


@pytest.mark.parametrize("tokens", [333, 3000])
def test_dropped_pairs_in_a_graph_and_in_the_small_grid_build(device, tokens):
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "dropped graph", tokens)
    topk, cols = 4, 272
    ids = torch.randint(0, 13, (tokens, topk), generator=g, device=device)
    off, _, slot = tr.expert_sort(ids, 12)
    y = torch.randn(tokens * topk, cols, generator=g, device=device).to(torch.bfloat16)
    go = torch.randn(tokens, cols, generator=g, device=device).to(torch.bfloat16)
    kept = torch.empty_like(slot)

    def run():
        return tr.expert_combine_bwd(go, y, kept, None, off)

    def drop():
        kept.copy_(torch.where(torch.rand(slot.shape, generator=g, device=device) < 0.4, -1, slot))

    drop()
    want = run()
    held = tr.lib
    try:
        tr.lib = tr.load_library(tr.SMALLGRID_LIB_PATH)
        got = run()
        torch.cuda.synchronize()
    finally:
        tr.lib = held
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        drop()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, run())), i
