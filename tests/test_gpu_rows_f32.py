"""Packed rows in fp32: the grouped products' and their input gradient's sums
as they are, and the tokens' sums of them, against plain 64-bit forms, in every
tile, with empty and uneven groups, gathered rows, masks, rows behind the last
group and guards behind the results."""
import sys
import zlib

import pytest
import torch

from tests.product_util import close, groups_of, random_record, unbits, values

pytestmark = pytest.mark.gpu

# the cut of an MXFP8 product's terms, as in test_gpu_mx_product.py
CUT = {"mx": 0.0, "mx8": 7 * 2.0 ** -13}
F32 = 2.0 ** -24  # half a step of fp32


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _gen(device, *key):
    g = torch.Generator(device=device)
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _offsets(groups, rows, tail, g, dev):
    """Offsets of uneven groups, empty ones among them, and `tail` rows behind them."""
    cuts = torch.randint(0, rows - tail + 1, (groups - 1,), generator=g, device=dev).sort().values
    return torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows - tail)])


# (groups, rows, rows behind the groups, n, k): few rows in each of its tiles, many rows in 128 x 128 and 128 x 256
SHAPES = [(1, 1, 0, 16, 32), (8, 8, 1, 64, 96), (4, 100, 7, 64, 4128), (40, 300, 0, 1040, 160), (64, 1280, 30, 1040, 1056),
          (5, 400, 129, 272, 544), (3, 2000, 0, 144, 1120), (6, 16420, 5000, 1040, 544)]


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("groups,rows,tail,n,k", SHAPES)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_matmul(device, fmt, groups, rows, tail, n, k, gather):
    import fp4_rollout_guided_amd as tr
    _say("case f32", fmt, groups, rows, tail, n, k, gather)
    g = _gen(device, fmt, groups, rows, n, k, gather, "f32")
    src = rows // 2 + 1 if gather else rows
    sa, ca = random_record(fmt, src, k, g, device)
    sw, cw = random_record("mx", groups * n, k, g, device)
    off = _offsets(groups, rows, tail, g, device)
    index = torch.randint(-1, src + 1, (rows,), generator=g, device=device) if gather else None
    mm = tr.grouped_mx_matmul if fmt == "mx" else tr.grouped_mx8_matmul
    out = torch.full((rows + 3, n), 7.0, device=device)
    y = mm(sa, ca, off, sw, cw, n, k, row_index=index, y=out, dtype=torch.float32)
    assert y is out and (out[rows:] == 7).all()
    a, w = values(fmt, sa, ca, k), values("mx", sw, cw, k).view(groups, n, k)
    if gather:
        a = a[index.clamp(0, src - 1)] * ((index >= 0) & (index < src)).unsqueeze(1)
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        if lo < hi:
            want, size = a[lo:hi] @ w[e].T.contiguous(), a[lo:hi].abs() @ w[e].abs().T.contiguous()
            close(y[lo:hi], want, size, 1, step=F32, product=k * 2.0 ** -24 + CUT[fmt])
    assert (y[rows - tail:rows].view(torch.int32) == 0).all()
    # the bf16 result is this one, rounded
    assert torch.equal(mm(sa, ca, off, sw, cw, n, k, row_index=index).view(torch.int16),
                       y[:rows].to(torch.bfloat16).view(torch.int16))


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
def test_grouped_linear(device, fmt):
    import fp4_rollout_guided_amd as tr
    g = _gen(device, fmt, "f32 linear")
    tokens, topk, experts, n, k = 200, 4, 6, 272, 288
    x = torch.randn(tokens, k, generator=g, device=device).to(torch.bfloat16)
    ids = torch.randint(-1, experts + 1, (tokens, topk), generator=g, device=device)
    sw, cw = random_record("mx", experts * n, k, g, device)
    off, index, slot = tr.expert_sort(ids, experts)
    quantize, mm, lin = ((tr.mx_quantize, tr.grouped_mx_matmul, tr.grouped_mx_linear) if fmt == "mx" else
                         (tr.mx8_quantize, tr.grouped_mx8_matmul, tr.grouped_mx8_linear))
    sa, ca, _ = quantize(x)
    want = mm(sa, ca, off, sw, cw, n, k, row_index=index, dtype=torch.float32)
    assert torch.equal(lin(x, off, sw, cw, n, row_index=index, dtype=torch.float32), want)
    assert torch.equal(lin(tr.expert_dispatch(x, index), off, sw, cw, n, dtype=torch.float32), want)


@pytest.mark.parametrize("groups,rows,tail,n,k", SHAPES)
@pytest.mark.parametrize("masked", [False, True])
def test_grouped_grad_input(device, groups, rows, tail, n, k, masked):
    import fp4_rollout_guided_amd as tr
    _say("case f32 grad input", groups, rows, tail, n, k, masked)
    g = _gen(device, groups, rows, n, k, masked, "f32 gx")
    gy = torch.randn(rows, n, generator=g, device=device).to(torch.bfloat16)
    gy[rows - tail:] = float("nan")  # rows of no group are not read
    sw, cw = random_record("mx", groups * n, k, g, device)
    off = _offsets(groups, rows, tail, g, device)
    mask = torch.randint(0, 256, (rows * k // 8,), generator=g, device=device, dtype=torch.uint8) if masked else None
    keep = unbits(mask, (rows, k)) if masked else torch.ones(rows, k, dtype=torch.bool, device=device)
    out = torch.full((rows + 2, k), 3.0, device=device)
    gx = tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k, mask=mask, grad_x=out, dtype=torch.float32)
    w = values("mx", sw, cw, k).view(groups, n, k)
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        if lo < hi:
            gd = gy[lo:hi].double()
            close(gx[lo:hi], (gd @ w[e]) * keep[lo:hi], (gd.abs() @ w[e].abs()) * keep[lo:hi], n, step=F32)
    assert (gx[rows - tail:rows].view(torch.int32) == 0).all() and (gx[rows:] == 3).all()
    assert (gx[:rows][~keep].view(torch.int32) == 0).all()
    assert torch.equal(tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k, mask=mask).view(torch.int16),
                       gx[:rows].to(torch.bfloat16).view(torch.int16))


@pytest.mark.parametrize("tokens,topk,cols,rows_short", [(1, 1, 16, 0), (5, 2, 48, 0), (37, 8, 2048, 0), (64, 64, 32, 0),
                                                         (130, 6, 272, 11)])
def test_combine(device, tokens, topk, cols, rows_short):
    import fp4_rollout_guided_amd as tr
    _say("case f32 combine", tokens, topk, cols)
    g = _gen(device, tokens, topk, cols, "f32 combine")
    ids = torch.randint(-1, 10, (tokens, topk), generator=g, device=device)
    off, _, slot = tr.expert_sort(ids, 9)
    y = torch.randn(tokens * topk, cols, generator=g, device=device)
    y[int(off[-1]):] = float("nan")  # rows of no expert are not read
    if rows_short:
        y = y[:-rows_short].contiguous()  # slots past y are left out
    wt = torch.randn(tokens, topk, generator=g, device=device)
    ok = (slot >= 0) & (slot < y.shape[0])
    yt = torch.where(ok.unsqueeze(-1), y[slot.clamp(0, y.shape[0] - 1)].double(), 0.0)
    for w in (wt, None):
        wd = (wt if w is not None else torch.ones_like(wt)).double().unsqueeze(-1)
        out = tr.expert_combine(y, slot, w)
        assert out.dtype == torch.bfloat16
        close(out, (yt * wd).sum(1), (yt * wd).abs().sum(1), topk)
    # bf16 rows held in fp32 give the bf16 rows' result
    yb = y.to(torch.bfloat16)
    assert torch.equal(tr.expert_combine(yb.float(), slot, wt).view(torch.int16), tr.expert_combine(yb, slot, wt).view(torch.int16))


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
def test_layer_rounds_once(device, fmt):
    """The second product's rows, weighted and summed, and the gradient's rows,
    summed: both within one rounding of the 64-bit form."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, fmt, "once")
    tokens, topk, experts, n, k = 300, 8, 16, 208, 544
    ids = torch.topk(torch.rand(tokens, experts + 4, generator=g, device=device), topk).indices.contiguous()
    off, index, slot = tr.expert_sort(ids, experts)
    rows, end = tokens * topk, int(off[-1])
    sa, ca = random_record(fmt, rows, k, g, device)
    sw, cw = random_record("mx", experts * n, k, g, device)
    wt = torch.rand(tokens, topk, generator=g, device=device)
    a, w = values(fmt, sa, ca, k), values("mx", sw, cw, k).view(experts, n, k)
    y, size = (torch.zeros(rows, n, dtype=torch.float64, device=device) for _ in range(2))
    gx, gsize = (torch.zeros(rows, k, dtype=torch.float64, device=device) for _ in range(2))
    gy = torch.randn(rows, n, generator=g, device=device).to(torch.bfloat16)
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        y[lo:hi], size[lo:hi] = a[lo:hi] @ w[e].T.contiguous(), a[lo:hi].abs() @ w[e].abs().T.contiguous()
        gx[lo:hi], gsize[lo:hi] = gy[lo:hi].double() @ w[e], gy[lo:hi].double().abs() @ w[e].abs()
    mm = tr.grouped_mx_matmul if fmt == "mx" else tr.grouped_mx8_matmul
    out = tr.expert_combine(mm(sa, ca, off, sw, cw, n, k, dtype=torch.float32), slot, wt)
    there = (slot >= 0).unsqueeze(-1)
    pick = lambda t: torch.where(there, t[slot.clamp(min=0)], 0.0)  # noqa: E731
    wd = wt.double().unsqueeze(-1)
    # k terms a row, cut once; then topk weighted rows
    close(out, (pick(y) * wd).sum(1), (pick(size) * wd).sum(1), 1, product=(k + topk + 1) * 2.0 ** -24 + CUT[fmt])
    gxo = tr.expert_combine(tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k, dtype=torch.float32), slot)
    close(gxo, pick(gx).sum(1), pick(gsize).sum(1), n + topk)
    assert end < rows


def test_refusals(device):
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "f32 refusals")
    rows, n, k = 8, 32, 64
    sa, ca = random_record("mx", rows, k, g, device)
    sw, cw = random_record("mx", 2 * n, k, g, device)
    off = torch.tensor([0, 3, rows], device=device)
    with pytest.raises(TypeError, match="dtype"):
        tr.grouped_mx_matmul(sa, ca, off, sw, cw, n, k, dtype=torch.float16)
    with pytest.raises(TypeError, match="y must be"):
        tr.grouped_mx_matmul(sa, ca, off, sw, cw, n, k, y=torch.empty(rows, n, device=device))
    with pytest.raises(TypeError, match="y must be"):
        tr.grouped_mx_matmul(sa, ca, off, sw, cw, n, k, dtype=torch.float32,
                             y=torch.empty(rows, n, device=device, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="at least"):
        tr.grouped_mx_matmul(sa, ca, off, sw, cw, n, k, dtype=torch.float32, y=torch.empty(rows - 1, n, device=device))
    slot = torch.zeros(4, 2, dtype=torch.int64, device=device)
    with pytest.raises(ValueError, match="contiguous"):
        tr.expert_combine(torch.zeros(n, rows, device=device).T, slot)
    with pytest.raises(TypeError, match="y must be bf16"):  # its gradients are bf16 rows'
        tr.ExpertCombine.apply(torch.zeros(rows, n, device=device), slot, torch.ones(4, 2, device=device), None)


def test_in_a_graph_and_in_the_small_grid_build(device):
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "f32 graph")
    tokens, topk, experts, n, k = 160, 4, 4, 272, 544
    ids = torch.randint(0, experts + 1, (tokens, topk), generator=g, device=device)
    x = torch.randn(tokens, k, generator=g, device=device).to(torch.bfloat16)
    gy = torch.randn(tokens * topk, n, generator=g, device=device).to(torch.bfloat16)
    wt = torch.rand(tokens, topk, generator=g, device=device)
    sw, cw = random_record("mx", experts * n, k, g, device)

    def run():
        off, index, slot = tr.expert_sort(ids, experts)
        y = tr.grouped_mx_linear(x, off, sw, cw, n, row_index=index, dtype=torch.float32)
        gr = tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k, dtype=torch.float32)
        return y, tr.expert_combine(y, slot, wt), gr, tr.expert_combine(gr, slot)

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
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        x.copy_(torch.randn(tokens, k, generator=g, device=device))
        ids.copy_(torch.randint(0, experts + 1, (tokens, topk), generator=g, device=device))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, run()):
            assert torch.equal(a, b), i
