"""The routed rows on the GPU: the sort of (token, expert) pairs, the gather
into packed order, the weighted sum back and its gradients, against plain
forms, with experts that are not held, empty experts, one chunk of pairs and
many, and repeated experts."""
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


def _sorted(ids, experts):
    """The definition, on the host."""
    flat = ids.flatten().tolist()
    topk = ids.shape[1]
    order = [p for e in range(experts) for p in range(len(flat)) if flat[p] == e] if len(flat) < 300 else \
        sorted((p for p in range(len(flat)) if 0 <= flat[p] < experts), key=lambda p: (flat[p], p))
    counts = [0] * experts
    for e in flat:
        if 0 <= e < experts:
            counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    slot = [-1] * len(flat)
    for s, p in enumerate(order):
        slot[p] = s
    index = [p // topk for p in order] + [-1] * (len(flat) - len(order))
    return torch.tensor(offsets), torch.tensor(index, dtype=torch.int64), torch.tensor(slot, dtype=torch.int64).view(ids.shape)


@pytest.mark.parametrize("tokens,topk,experts,pool", [
    (0, 2, 8, "all"), (1, 1, 1, "all"), (1, 8, 128, "all"), (24, 8, 128, "all"), (63, 3, 5, "half"), (100, 2, 1, "none"),
    (256, 8, 128, "all"), (257, 8, 127, "half"), (300, 7, 1024, "all"), (3000, 4, 9, "one"), (5000, 6, 200, "half"),
    (16384, 8, 128, "all"), (33, 64, 64, "all"), (700, 3, 1023, "half"),
    (32769, 8, 40, "half"), (262145, 8, 9, "half")])
def test_sort(device, tokens, topk, experts, pool):
    import fp4_rollout_guided_amd as tr
    _say("case sort", tokens, topk, experts, pool)
    g = _gen(device, tokens, topk, experts, pool)
    lo, hi = {"all": (0, experts), "half": (-experts // 2 - 1, 2 * experts), "none": (experts, experts + 5),
              "one": (experts - 1, experts)}[pool]
    ids = torch.randint(lo, hi, (tokens, topk), generator=g, device=device)
    if ids.numel() > 4:
        ids.view(-1)[3] = 1 << 40 if pool != "one" else experts - 1  # past 32 bits: not held
        ids.view(-1)[4] = -(1 << 40) if pool != "one" else experts - 1
    got = tr.expert_sort(ids, experts)
    for a, b in zip(got, _sorted(ids.cpu(), experts)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("tokens,topk,cols,rows_short", [(1, 1, 16, 0), (5, 2, 48, 0), (37, 8, 2048, 0), (200, 3, 7168, 0),
                                                         (64, 64, 32, 0), (130, 6, 272, 11)])
def test_dispatch_combine_and_gradients(device, tokens, topk, cols, rows_short):
    import fp4_rollout_guided_amd as tr
    _say("case rows", tokens, topk, cols)
    g = _gen(device, tokens, topk, cols)
    experts = 9
    ids = torch.randint(-1, experts + 1, (tokens, topk), generator=g, device=device)
    off, index, slot = tr.expert_sort(ids, experts)
    x = torch.randn(tokens, cols, generator=g, device=device).to(torch.bfloat16)
    rows = tr.expert_dispatch(x, index)
    there = index >= 0
    assert torch.equal(rows, x[index.clamp(min=0)] * there.unsqueeze(1))
    y = torch.randn(tokens * topk, cols, generator=g, device=device).to(torch.bfloat16)
    y[int(off[-1]):] = float("nan")  # rows of no expert are not read
    if rows_short:
        y = y[:-rows_short].contiguous()  # slots past y are left out
    wt = torch.randn(tokens, topk, generator=g, device=device)
    ok = (slot >= 0) & (slot < y.shape[0])
    yt = torch.where(ok.unsqueeze(-1), y[slot.clamp(0, y.shape[0] - 1)].double(), 0.0)
    for w in (wt, None):
        wd = wt.double() if w is not None else torch.ones_like(wt).double()
        close(tr.expert_combine(y, slot, w), (yt * wd.unsqueeze(-1)).sum(1), (yt * wd.unsqueeze(-1)).abs().sum(1), topk)
        go = torch.randn(tokens, cols, generator=g, device=device).to(torch.bfloat16)
        gy, gw = tr.expert_combine_bwd(go, y, slot, w, off)
        prod = yt * go.double().unsqueeze(1)
        # cols products, each rounded once when added: 2^-24 of the partial sums' size
        close(gw, prod.sum(-1), prod.abs().sum(-1), cols + 16, step=2.0 ** -24)
        want = torch.zeros(y.shape, dtype=torch.float64, device=device)
        t, j = ok.nonzero(as_tuple=True)
        want[slot[t, j]] = go.double()[t] * wd[t, j].unsqueeze(1)
        close(gy, want, want.abs(), 1)
        assert (gy[int(off[-1]):].view(torch.int16) == 0).all()


def test_combine_gradients_against_differences(device):
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "combine differences")
    tokens, topk, cols = 6, 3, 32
    ids = torch.randint(0, 4, (tokens, topk), generator=g, device=device)
    off, index, slot = tr.expert_sort(ids, 4)
    y = torch.randn(tokens * topk, cols, generator=g, device=device).to(torch.bfloat16).requires_grad_()
    w = torch.randn(tokens, topk, generator=g, device=device).requires_grad_()
    go = torch.randn(tokens, cols, generator=g, device=device).to(torch.bfloat16)
    tr.ExpertCombine.apply(y, slot, w, off).backward(go)
    loss = lambda y, w: ((y[slot.flatten()].view(tokens, topk, cols) * w.unsqueeze(-1)).sum(1) * go.double()).sum()  # noqa: E731
    yd, wd = y.detach().double(), w.detach().double()
    base = loss(yd, wd)
    for r, c in ((0, 0), (7, 5), (17, 31)):
        moved = yd.clone()
        moved[r, c] += 1.0
        diff = loss(moved, wd) - base
        assert abs(diff - y.grad[r, c].double()) <= 2.0 ** -8 * abs(diff) + 1e-9
    for t, j in ((0, 0), (5, 2), (2, 1)):
        moved = wd.clone()
        moved[t, j] += 1.0
        assert abs(loss(yd, moved) - base - w.grad[t, j].double()) <= 1e-4


def test_dispatch_gradient_sums_a_tokens_rows(device):
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "dispatch grad")
    tokens, topk, cols, experts = 50, 4, 64, 6
    ids = torch.randint(-2, experts, (tokens, topk), generator=g, device=device)
    off, index, slot = tr.expert_sort(ids, experts)
    x = torch.randn(tokens, cols, generator=g, device=device).to(torch.bfloat16).requires_grad_()
    gr = torch.randn(tokens * topk, cols, generator=g, device=device).to(torch.bfloat16)
    tr.ExpertDispatch.apply(x, index, slot).backward(gr)
    rows = torch.where((slot >= 0).unsqueeze(-1), gr[slot.clamp(min=0)].double(), 0.0)
    close(x.grad, rows.sum(1), rows.abs().sum(1), topk)


def test_combine_bwd_leaves_unnamed_rows(device):
    """Without offsets, rows that no slot names stay as they were."""
    import fp4_rollout_guided_amd as tr
    y = torch.ones(6, 16, dtype=torch.bfloat16, device=device)
    slot = torch.tensor([[4], [1], [-1]], device=device)
    gy = torch.full((6, 16), 9.0, dtype=torch.bfloat16, device=device)
    go = torch.ones(3, 16, dtype=torch.bfloat16, device=device)
    out, gw = tr.expert_combine_bwd(go, y, slot, None, grad_y=gy)
    assert out[[1, 4]].eq(1).all() and out[[0, 2, 3, 5]].eq(9).all() and gw.flatten().tolist() == [16.0, 16.0, 0.0]
    fresh, _ = tr.expert_combine_bwd(go, y, slot, None)
    assert fresh[[0, 2, 3, 5]].eq(0).all()


def test_small_grid_build_gives_the_same(device):
    """The test build sends every row past the cache and runs its grid-stride
    loops several times: the same bits."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "small grid")
    tokens, topk, experts, cols = 333, 4, 12, 528
    ids = torch.randint(0, experts + 3, (tokens, topk), generator=g, device=device)
    x = torch.randn(tokens, cols, generator=g, device=device).to(torch.bfloat16)
    wt = torch.rand(tokens, topk, generator=g, device=device)

    def run():
        off, index, slot = tr.expert_sort(ids, experts)
        rows = tr.expert_dispatch(x, index)
        return [off, index, slot, rows, tr.expert_combine(rows, slot, wt), *tr.expert_combine_bwd(x, rows, slot, wt, off)]

    want = run()
    held = tr.lib
    try:
        tr.lib = tr.load_library(tr.SMALLGRID_LIB_PATH)
        got = run()
        torch.cuda.synchronize()
    finally:
        tr.lib = held
    for a, b in zip(got, want):
        assert torch.equal(a, b)
