"""The router against its 64-bit form: experts below, at and past the kernels'
widths, ties, masked rows and experts, NaN and infinities, the balance loss, its
gradient against the formula's and differences, and its way into the sorted rows."""
import sys

import pytest
import torch

from tests import step_util as U
from tests.test_gpu_gridstride import _small_grid

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def logits(tokens, experts, dtype, device, seed=0, grid=None):
    g = torch.Generator(device=device)
    g.manual_seed(seed + 7919 * tokens + experts)
    z = torch.randn(tokens, experts, generator=g, device=device) * 2
    if grid:
        z = (z * grid).round() / grid  # many equal ones
    return z.to(dtype)


def check(tr, z, topk, renormalize, valid=None, grads=True):
    """weights: two exponentials (off by |z| 2^-23 of their argument's rounding and an ulp each), their sum over up to
    1024 terms (a lane adds 16, the lanes six times) and a division: 2^-18 of the value is three times that for |z| below
    16.  probs: sums of such, relative to themselves, plus an addition for each row a lane has.  The gradient: products of
    those with factors whose sums' sizes bound it."""
    got = tr.expert_route(z, topk, renormalize=renormalize, valid=valid)
    ids, weights, counts, probs, balance = got
    want = U.route(z, topk, renormalize, valid)
    assert torch.equal(ids.cpu(), want[0])
    assert torch.equal(counts.cpu(), want[2])
    rel = 2.0 ** -18
    assert ((weights.cpu().double() - want[1]).abs() <= rel * want[1] + 2.0 ** -126).all()
    assert ((probs.cpu().double() - want[3]).abs() <= 4 * rel * want[3] + 2.0 ** -120).all()
    assert abs(float(balance) - float(want[4])) <= 4 * rel * float(want[4])
    if not grads:
        return got
    tokens = z.shape[0]
    gw = torch.randn(tokens, topk, device=z.device)
    gw = torch.where(ids >= 0, gw, torch.full_like(gw, float("nan")))  # not read beside id -1
    gb = torch.full((1,), 0.3 * max(1, tokens), device=z.device)
    clean = torch.where(ids >= 0, gw, torch.zeros_like(gw))
    for a, b in ((gw, gb), (gw, None), (None, gb), (None, None)):
        out = tr.expert_route_bwd(a, b, z, ids, weights, counts, renormalize=renormalize)
        exact = U.route_gradient(z, ids, counts, renormalize, None if a is None else clean, b)
        exact = torch.zeros(z.shape, dtype=torch.float64) if exact is None else exact.nan_to_num(0.0)
        half = 2.0 ** -8 if z.dtype == torch.bfloat16 else 2.0 ** -24
        p = torch.softmax(z.double().cpu(), 1).nan_to_num(0.0)
        size = torch.zeros(z.shape, dtype=torch.float64)
        if a is not None:
            w = want[1] * clean.double().cpu().abs()
            size += p * w.sum(1, keepdim=True)
            size.scatter_add_(1, want[0].clamp(min=0), w + want[1] * w.sum(1, keepdim=True))
        if b is not None and int(counts[-1]):
            c = float(b) * z.shape[1] * counts[:-1].double().cpu() / float(counts[:-1].sum()) / float(counts[-1])
            size += p * (c + (p * c).sum(1, keepdim=True))
        tol = 16 * rel * size
        tol = tol + half * (exact.abs() + tol) + 2.0 ** -126
        assert ((out.cpu().double() - exact).abs() <= tol).all(), (a is None, b is None)
        assert not out[(ids[:, 0] < 0)].any()
    return got


SIZES = [(1, 1, 1), (5, 2, 2), (24, 128, 8), (63, 7, 3), (64, 16, 16), (65, 63, 1), (66, 64, 6), (70, 65, 8), (130, 127, 4),
         (257, 129, 8), (33, 255, 10), (40, 256, 6), (41, 257, 8), (20, 511, 64), (21, 512, 9), (22, 513, 3), (9, 1000, 64),
         (10, 1023, 33), (12, 1024, 64), (1030, 128, 8), (4099, 60, 4)]


@pytest.mark.parametrize("tokens,experts,topk", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_sizes(device, tokens, experts, topk, dtype, renormalize):
    import fp4_rollout_guided_amd as tr
    _say("case route", tokens, experts, topk, dtype, renormalize)
    z = logits(tokens, experts, dtype, device)
    valid = torch.rand(tokens, device=device) < 0.8 if tokens % 2 else None
    check(tr, z, topk, renormalize, valid)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("experts", [60, 128, 131, 640])
def test_ties(device, dtype, experts):
    import fp4_rollout_guided_amd as tr
    _say("case ties", dtype, experts)
    check(tr, logits(200, experts, dtype, device, grid=1), 8, True)
    check(tr, torch.zeros(70, experts, dtype=dtype, device=device), 5, False)
    z = torch.zeros(3, experts, dtype=dtype, device=device)
    z[0, ::2], z[1] = -0.0, -0.0  # the two zeros are equal
    assert tr.expert_route(z, 4)[0].cpu().tolist() == [[0, 1, 2, 3]] * 3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("experts", [20, 128, 600])
def test_masked_experts_and_rows(device, dtype, experts):
    import fp4_rollout_guided_amd as tr
    _say("case masks", dtype, experts)
    z = logits(150, experts, dtype, device)
    z[::3, 5:] = -float("inf")      # five experts left for a top eight
    z[7] = -float("inf")            # none
    z[8, 1:] = torch.finfo(dtype).min
    check(tr, z, 8, True)
    check(tr, z, 8, False)
    for valid in (torch.zeros(150, dtype=torch.uint8, device=device), torch.zeros(150, dtype=torch.bool, device=device)):
        ids, weights, counts, probs, balance = tr.expert_route(z, 8, valid=valid)
        assert (ids == -1).all() and not weights.any() and not counts.any() and not probs.any() and not balance.any()
        g = tr.expert_route_bwd(torch.ones(150, 8, device=device), torch.ones(1, device=device), z, ids, weights, counts)
        assert not g.any()
    # rows that are left out hold anything
    valid = torch.rand(150, device=device) < 0.5
    a = tr.expert_route(z, 8, valid=valid)
    z2 = z.clone()
    z2[~valid] = float("nan")
    b = tr.expert_route(z2, 8, valid=valid)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    gw = torch.randn(150, 8, device=device)
    assert torch.equal(tr.expert_route_bwd(gw, a[4], z, *a[:3]), tr.expert_route_bwd(gw, a[4], z2, *b[:3]))


def test_nan_and_infinity(device):
    import fp4_rollout_guided_amd as tr
    _say("case NaN")
    z = logits(40, 128, torch.float32, device)
    z[3, 100], z[3, 20], z[5, 60] = float("nan"), float("nan"), float("inf")
    ids, weights, counts, probs, balance = tr.expert_route(z, 4)
    assert torch.equal(ids.cpu(), U.route(z, 4, True)[0])
    assert ids[3, 0] == 20 and ids[3, 1] == 100 and ids[5, 0] == 60
    other = torch.ones(40, dtype=torch.bool, device=device)
    other[3] = other[5] = False
    assert weights[3].isnan().all() and weights[5].isnan().any() and not weights[other].isnan().any()
    assert probs.isnan().all() and balance.isnan() and int(counts[-1]) == 40


def test_pairs_that_the_forward_does_not_make(device):
    """ids past the last expert are passed over, the same expert twice gets both gradients."""
    import fp4_rollout_guided_amd as tr
    _say("case odd pairs")
    z = logits(30, 40, torch.float32, device)
    ids, weights, counts, _, _ = tr.expert_route(z, 4)
    gw = torch.randn(30, 4, device=device)
    odd = ids.clone()
    odd[:10, 1], odd[10:20, 2], odd[20:, 3] = 40, 2 ** 40 + 3, odd[20:, 1]
    for renormalize in (True, False):
        g = tr.expert_route_bwd(gw, None, z, odd, weights, counts, renormalize=renormalize)
        w, d, p = weights.double(), gw.double(), torch.softmax(z.double(), 1)
        s = (w * d).sum(1, keepdim=True)
        add = w * (d - s) if renormalize else w * d
        want = torch.zeros_like(p) if renormalize else -p * s
        there = odd < 40
        want.scatter_add_(1, torch.where(there, odd, 0), torch.where(there, add, 0.0))
        # products and sums of a few fp32 terms of their sizes
        size = p * (w * d.abs()).sum(1, keepdim=True)
        size.scatter_add_(1, torch.where(there, odd, 0), w * (d.abs() + (w * d.abs()).sum(1, keepdim=True)))
        assert ((g.double() - want).abs() <= 2.0 ** -18 * size + 2.0 ** -126).all()


def test_no_rows(device):
    import fp4_rollout_guided_amd as tr
    _say("case no rows")
    ids, weights, counts, probs, balance = tr.expert_route(torch.empty(0, 128, device=device), 8)
    assert ids.shape == (0, 8) and weights.shape == (0, 8)
    assert not counts.any() and not probs.any() and not balance.any()
    assert tr.expert_route_bwd(None, balance, torch.empty(0, 128, device=device), ids, weights, counts).shape == (0, 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_unaligned_rows(device, dtype):
    """Logits at any multiple of their own size: the kernels of single loads against those of vectors."""
    import fp4_rollout_guided_amd as tr
    _say("case unaligned", dtype)
    for experts in (64, 128, 256, 512, 1024):
        z = logits(90, experts, dtype, device)
        a = tr.expert_route(z, 4)
        gw = torch.randn(90, 4, device=device)
        g = tr.expert_route_bwd(gw, a[4], z, *a[:3])
        room = torch.zeros(90 * experts + 8, dtype=dtype, device=device)
        for shift in (1, 3):
            there = room[shift:shift + 90 * experts].view(90, experts)
            there.copy_(z)
            b = tr.expert_route(there, 4)
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
            for x, y in zip(a, b):  # sums in another order
                assert torch.allclose(x.double(), y.double(), rtol=2.0 ** -18, atol=0)
            out = torch.empty_like(room)[shift:shift + 90 * experts].view(90, experts)
            h = tr.expert_route_bwd(gw, a[4], there, *a[:3], grad_logits=out)
            assert torch.allclose(g.double(), h.double(), rtol=2.0 ** -7, atol=1e-6)
            assert torch.equal(tr.expert_route_bwd(gw, a[4], there, *a[:3], grad_logits=there), h)  # in place


def test_many_rows_and_small_grids(device):
    import fp4_rollout_guided_amd as tr
    _say("case many rows")
    for tokens, experts, topk, dtype in ((70001, 128, 8, torch.float32), (40003, 300, 6, torch.bfloat16)):
        z = logits(tokens, experts, dtype, device)
        a = check(tr, z, topk, True, grads=tokens < 50000)
        assert all(torch.equal(x, y) for x, y in zip(a, tr.expert_route(z, topk)))  # the same bits every time
    z = logits(3001, 128, torch.float32, device)
    want = tr.expert_route(z, 8)
    gw = torch.randn(3001, 8, device=device)
    g = tr.expert_route_bwd(gw, want[4], z, *want[:3])
    with _small_grid():
        got = tr.expert_route(z, 8)
        h = tr.expert_route_bwd(gw, want[4], z, *want[:3])
    assert all(torch.equal(x, y) for x, y in zip(want[:3], got[:3])) and torch.equal(g, h)
    # the probabilities' sums go over other workgroups there: 3001 rows, 2^-24 of the sum for each
    assert torch.allclose(want[3], got[3], rtol=3001 * 2.0 ** -24) and torch.allclose(want[4], got[4], rtol=3001 * 2.0 ** -23)


def test_gradient_against_differences(device):
    import fp4_rollout_guided_amd as tr
    _say("case differences")
    z = logits(50, 128, torch.float32, device)
    for renormalize in (True, False):
        ids, weights, counts, _, balance = tr.expert_route(z, 8, renormalize=renormalize)
        gw = torch.randn(50, 8, device=device)
        g = tr.expert_route_bwd(gw, torch.ones(1, device=device), z, ids, weights, counts, renormalize=renormalize)
        d = torch.randn(50, 128, dtype=torch.float64)

        def f(s):
            zd = z.double().cpu() + s * d
            p = torch.softmax(zd, 1)
            at = ids.cpu()
            w = torch.softmax(zd.gather(1, at), 1) if renormalize else p.gather(1, at)
            c = counts.cpu().double()
            return float((w * gw.double().cpu()).sum() + 128 * (c[:128] / c[:128].sum() * p.sum(0) / c[128]).sum())
        h = 1e-5
        slope = (f(h) - f(-h)) / (2 * h)  # off by h^2 and by 1e-16 / h
        assert abs(float((g.double().cpu() * d).sum()) - slope) < 1e-4 * (1 + abs(slope))


def test_autograd_and_rows(device):
    """The router before the rows it chooses: weights reach expert_combine, and their gradients come back through it."""
    import fp4_rollout_guided_amd as tr
    _say("case router and rows")
    torch.manual_seed(5)
    tokens, experts, topk, cols = 90, 16, 4, 64
    z = torch.randn(tokens, experts, device=device, requires_grad=True)
    x = torch.randn(tokens, cols, device=device).to(torch.bfloat16)
    valid = torch.rand(tokens, device=device) < 0.9
    ids, weights, counts, balance = tr.ExpertRoute.apply(z, topk, True, valid)
    assert not ids.requires_grad and not counts.requires_grad and weights.requires_grad and balance.requires_grad
    offsets, row_index, slot = tr.expert_sort(ids, experts)
    assert torch.equal((offsets[1:] - offsets[:-1]), counts[:-1])
    rows = tr.expert_dispatch(x, row_index)
    scaled = (rows.float() * (1 + torch.arange(rows.shape[0], device=device).unsqueeze(1) % 7)).to(torch.bfloat16)
    out = tr.ExpertCombine.apply(scaled, slot, weights, offsets)
    grad = torch.randn(tokens, cols, device=device).to(torch.bfloat16)
    (out.float() * grad.float()).sum().backward(retain_graph=True)
    alone = z.grad.clone()
    dots = torch.where(slot >= 0, (scaled[slot.clamp(min=0)].double() * grad.double().unsqueeze(1)).sum(-1), 0.0)
    want = U.route_gradient(z, ids, counts, True, dots, None)
    assert torch.allclose(alone.double().cpu(), want, rtol=1e-4, atol=1e-4)
    assert not alone[~valid].any()
    z.grad = None
    (0.01 * balance.sum()).backward()
    want = U.route_gradient(z, ids, counts, True, None, torch.tensor([0.01]))
    assert torch.allclose(z.grad.double().cpu(), want, rtol=1e-4, atol=1e-9)


def test_counts_of_several_ranks(device):
    """Two halves of a batch, their counts and probabilities added, give the whole batch's balance gradient."""
    import fp4_rollout_guided_amd as tr
    _say("case ranks")
    z = logits(120, 64, torch.float32, device)
    whole = tr.expert_route(z, 4)
    gb = torch.full((1,), 2.0, device=device)
    want = tr.expert_route_bwd(None, gb, z, *whole[:3])
    halves = [tr.expert_route(h, 4) for h in (z[:50], z[50:])]
    counts = halves[0][2] + halves[1][2]
    assert torch.equal(counts, whole[2])
    got = torch.cat([tr.expert_route_bwd(None, gb, h, r[0], r[1], counts) for h, r in zip((z[:50], z[50:]), halves)])
    assert torch.equal(got, want)


def test_graph_replays_and_streams(device):
    import fp4_rollout_guided_amd as tr
    _say("case graph and streams")
    z = logits(5000, 128, torch.float32, device)
    want = list(tr.expert_route(z, 8))
    gw = torch.randn(5000, 8, device=device)
    want.append(tr.expert_route_bwd(gw, want[4], z, *want[:3]))
    need = tr.lib.trace_expert_route_workspace_bytes(5000, 128)

    def buffers():
        return [torch.empty_like(v) for v in want] + [torch.empty(need, dtype=torch.uint8, device=device)]

    def run(o):
        tr.expert_route(z, 8, ids=o[0], weights=o[1], counts=o[2], probs=o[3], balance=o[4], workspace=o[6])
        tr.expert_route_bwd(gw, o[4], z, *o[:3], grad_logits=o[5])
    outs, streams = [buffers() for _ in range(2)], [torch.cuda.Stream(device=device) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for o, s in zip(outs, streams):
            with torch.cuda.stream(s):
                run(o)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(want, o))
    o = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(o)
    for _ in range(4):
        for b in o:
            b.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, o))
    del graph


def test_binding_refusals(device):
    import fp4_rollout_guided_amd as tr
    _say("case refusals")
    z = logits(20, 16, torch.float32, device)
    for args in ((z, 0), (z, 17), (z, True), (z, 2.0), (z.double(), 2), (z.t(), 2), (z.cpu(), 2), (z[:, :0], 1)):
        with pytest.raises((TypeError, ValueError)):
            tr.expert_route(*args)
    with pytest.raises(ValueError):
        tr.expert_route(torch.zeros(2, 1025, device=device), 2)
    for valid in (torch.ones(19, dtype=torch.bool, device=device), torch.ones(20, device=device), torch.ones(20, dtype=torch.bool)):
        with pytest.raises((TypeError, ValueError)):
            tr.expert_route(z, 2, valid=valid)
    ids, weights, counts, probs, balance = tr.expert_route(z, 2)
    gw = torch.zeros(20, 2, device=device)
    for bad in ((gw[:19], balance, z, ids, weights, counts), (gw, probs, z, ids, weights, counts),
                (gw, balance, z[:19], ids, weights, counts), (gw, balance, z, ids[0], weights, counts),
                (gw, balance, z, ids.int(), weights, counts), (gw, balance, z, ids, weights[:3], counts),
                (gw, balance, z, ids, weights, counts[:-1])):
        with pytest.raises((TypeError, ValueError)):
            tr.expert_route_bwd(*bad)
