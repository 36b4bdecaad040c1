"""The microscaled operands, their products and the products' gradients on the
GPU, against ``oracle`` (quantisers, bit for bit) and plain 64-bit forms
(products), at sizes around the kernels' tiles, with empty and uneven groups,
gathered rows, extreme scale bytes, masks, odd alignments of the scale rows,
streams, graph replays and the autograd function."""
import sys
import zlib

import numpy as np
import pytest
import torch

import oracle
from oracle import formats as F
from tests.gpu_util import from_np_u16, to_np_u8
from tests.product_util import close, groups_of, random_record, unbits, values

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _gen(device, *key):
    g = torch.Generator(device=device)
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def _bf16(rows, cols, g, dev, scale=1.0):
    return (torch.randn(rows, cols, generator=g, device=dev) * scale).to(torch.bfloat16)


# The terms of an MXFP8 product: the matrix instruction adds the products of
# eight neighbouring k on one grid, cutting each to a multiple of 2^-13 of the
# largest's power of two.  Each of the seven others is then off by less than
# 2^-13 of the largest, so a group by less than 7 * 2^-13 of its terms' total.
CUT = {"mx": 0.0, "mx8": 7 * 2.0 ** -13}


def _check_product(fmt, y, a, w):
    want, size = a @ w.T.contiguous(), a.abs() @ w.abs().T.contiguous()
    if CUT[fmt]:
        close(y, want, size, 1, product=a.shape[1] * 2.0 ** -24 + CUT[fmt])
    else:
        close(y, want, size, a.shape[1])


# ---------------------------------------------------------------------------
# quantisers
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (37, 2048), (5, 7168)])
def test_quantize_matches_the_capture_and_the_rne_mask(device, fmt, shape):
    import fp4_rollout_guided_amd as tr
    _say("case quantize", fmt, shape)
    rng = np.random.default_rng(shape[0] * 7919 + shape[1])
    v = rng.standard_t(3, shape) * 2.0 ** rng.integers(-130, 118, (shape[0], 1))
    x = F.f32_to_bf16_rne(v.astype(np.float32).reshape(-1))
    at = rng.choice(x.size, max(1, x.size // 40), replace=False)
    x[at] = rng.choice(np.array([0x7F80, 0xFF80, 0x7FC1, 0xFFC0, 0x8000, 0x0000, 0x0001, 0x8001, 0x7F7F], np.uint16),
                       at.size)
    if x.size > 64:
        x[32:64] = 0x7FC0  # a block of NaN alone
    xd = from_np_u16(x, device, shape)
    sc, cd, mk = (tr.mx_quantize if fmt == "mx" else tr.mx8_quantize)(xd, want_mask=True)
    torch.cuda.synchronize()
    cap = (oracle.mx_capture if fmt == "mx" else oracle.mx8_capture)(x, with_codes=True)
    rne = (oracle.mx_rne_fwd if fmt == "mx" else oracle.mx8_rne_fwd)(x, cap["scales"])
    assert np.array_equal(to_np_u8(sc), cap["scales"])
    assert np.array_equal(to_np_u8(cd), cap["codes"])
    assert np.array_equal(to_np_u8(mk), rne["mask"])


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

SHAPES = [(1, 16, 32), (1, 48, 160), (2, 2048, 4096), (7, 80, 96), (16, 16, 128), (33, 272, 544), (64, 128, 256),
          (127, 144, 768), (129, 256, 2080), (255, 528, 1056), (257, 272, 512), (300, 1024, 640), (1021, 768, 2048),
          (64, 4112, 96), (2100, 592, 96), (2100, 592, 544), (16390, 1040, 544), (16400, 1024, 1184)]


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("rows,n,k", SHAPES)
def test_matmul(device, fmt, rows, n, k):
    import fp4_rollout_guided_amd as tr
    _say("case matmul", fmt, rows, n, k)
    g = _gen(device, fmt, rows, n, k)
    sa, ca = random_record(fmt, rows, k, g, device)
    sw, cw = random_record("mx", n, k, g, device)
    y = (tr.mx_matmul if fmt == "mx" else tr.mx8_matmul)(sa, ca, sw, cw, n, k)
    assert y.shape == (rows, n) and y.dtype == torch.bfloat16
    _check_product(fmt, y, values(fmt, sa, ca, k), values("mx", sw, cw, k))


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
def test_matmul_at_extreme_and_nan_scales(device, fmt):
    import fp4_rollout_guided_amd as tr
    _say("case scales", fmt)
    rows, n, k = 37, 48, 256
    g = _gen(device, fmt, "scales")
    mm = tr.mx_matmul if fmt == "mx" else tr.mx8_matmul
    # factors 2^-124 .. 2^-117 against 2^113 .. 2^120: products of ordinary size
    sa, ca = random_record(fmt, rows, k, g, device, 3, 10)
    sw, cw = random_record("mx", n, k, g, device, 240, 247)
    _check_product(fmt, mm(sa, ca, sw, cw, n, k), values(fmt, sa, ca, k), values("mx", sw, cw, k))
    # a NaN scale in one row of A and one of W, zero codes under it
    sa, ca = random_record(fmt, rows, k, g, device)
    sw, cw = random_record("mx", n, k, g, device)
    sa.view(rows, -1)[5, 3] = 255
    ca.view(rows, -1)[5] = 0
    sw.view(n, -1)[17, 0] = 255
    y = mm(sa, ca, sw, cw, n, k)
    assert y[5].isnan().all() and y[:, 17].isnan().all()
    ok = torch.ones_like(y, dtype=torch.bool)
    ok[5] = False
    ok[:, 17] = False
    assert not y[ok].isnan().any()


def _uneven(groups, rows, kind):
    """Offsets of `groups` groups in `rows` packed rows."""
    if kind == "even":
        o = [rows * i // groups for i in range(groups + 1)]
    elif kind == "one":  # every row in one of the groups
        o = [0] * (groups // 2 + 1) + [rows] * (groups - groups // 2)
    elif kind == "tail":  # rows behind the last group
        o = [(rows * 2 // 3) * i // groups for i in range(groups + 1)]
    else:  # skewed: sizes 0, 1, 2, 4, ...
        o = [0]
        for i in range(groups):
            o.append(min(rows, o[-1] + (0 if i % 3 == 0 else 1 << (i % 9))))
    return torch.tensor(o, dtype=torch.int64)


GROUPED = [(1, 1, 16, 32, "even"), (5, 40, 48, 96, "skewed"), (3, 257, 144, 544, "tail"), (8, 700, 272, 256, "one"),
           (70, 300, 64, 160, "skewed"), (130, 1500, 256, 768, "even"), (6, 0, 32, 64, "even"),
           (4, 1200, 512, 1024, "tail"), (9, 90, 2048, 768, "even"), (64, 300, 336, 192, "tail"),
           (64, 300, 336, 192, "one"),
           (5, 16500, 1040, 544, "skewed"), (6, 16420, 1024, 1056, "tail")]


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("groups,rows,n,k,kind", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_matmul(device, fmt, groups, rows, n, k, kind, gather):
    import fp4_rollout_guided_amd as tr
    _say("case grouped", fmt, groups, rows, n, k, kind, gather)
    g = _gen(device, fmt, groups, rows, n, k, gather)
    src = rows // 2 + 1 if gather else rows
    sa, ca = random_record(fmt, src, k, g, device)
    sw, cw = random_record("mx", groups * n, k, g, device)
    off = _uneven(groups, rows, kind).to(device)
    index = torch.randint(-1, src + 1, (rows,), generator=g, device=device) if gather else None
    mm = tr.grouped_mx_matmul if fmt == "mx" else tr.grouped_mx8_matmul
    out = torch.full((rows + 3, n), 7.0, dtype=torch.bfloat16, device=device)
    y = mm(sa, ca, off, sw, cw, n, k, row_index=index, y=out)
    assert (out[rows:] == 7).all()  # nothing past the packed rows is written
    a, w = values(fmt, sa, ca, k), values("mx", sw, cw, k).view(groups, n, k)
    if gather:
        a = a[index.clamp(0, src - 1)] * ((index >= 0) & (index < src)).unsqueeze(1)
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        if lo < hi:
            _check_product(fmt, y[lo:hi], a[lo:hi], w[e])
    assert (y[int(off[-1]):rows].view(torch.int16) == 0).all()


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("rows,n,k", [(1, 16, 32), (4, 2048, 4096), (16, 4112, 1024), (3, 528, 96), (37, 96, 544), (300, 256, 1056)])
def test_linear_is_quantize_and_matmul(device, fmt, rows, n, k):
    import fp4_rollout_guided_amd as tr
    _say("case linear", fmt, rows, n, k)
    g = _gen(device, fmt, rows, n, k, "linear")
    x = _bf16(rows, k, g, device)
    x[0, 0] = float("nan")
    x[-1, -1] = float("inf")
    sw, cw = random_record("mx", n, k, g, device)
    quant, mm, lin = ((tr.mx_quantize, tr.mx_matmul, tr.mx_linear) if fmt == "mx" else
                      (tr.mx8_quantize, tr.mx8_matmul, tr.mx8_linear))
    sa, ca, _ = quant(x)
    y = lin(x, sw, cw, n)
    a, w = values(fmt, sa, ca, k), values("mx", sw, cw, k)
    _check_product(fmt, y[:-1], a[:-1], w)
    _check_product(fmt, mm(sa, ca, sw, cw, n, k)[:-1], a[:-1], w)
    assert torch.equal(lin(x.view(1, rows, k), sw, cw, n).view(rows, n).view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("tokens,topk,experts,n,k", [(1, 2, 8, 32, 64), (24, 8, 128, 256, 512), (200, 4, 6, 272, 288)])
def test_grouped_linear_on_routed_rows(device, fmt, tokens, topk, experts, n, k):
    import fp4_rollout_guided_amd as tr
    _say("case grouped linear", fmt, tokens, topk, experts, n, k)
    g = _gen(device, fmt, tokens, experts, n, k)
    x = _bf16(tokens, k, g, device)
    ids = torch.stack([torch.randperm(experts + 2, generator=g, device=device)[:topk] for _ in range(tokens)]) - 1
    sw, cw = random_record("mx", experts * n, k, g, device)
    off, index, slot = tr.expert_sort(ids, experts)
    quant, lin = ((tr.mx_quantize, tr.grouped_mx_linear) if fmt == "mx" else (tr.mx8_quantize, tr.grouped_mx8_linear))
    y = lin(x, off, sw, cw, n, row_index=index)
    sa, ca, _ = quant(x)
    a, w = values(fmt, sa, ca, k), values("mx", sw, cw, k).view(experts, n, k)
    for e, (lo, hi) in enumerate(groups_of(off, tokens * topk)):
        if lo < hi:
            _check_product(fmt, y[lo:hi], a[index[lo:hi]], w[e])
    assert (y[int(off[-1]):].view(torch.int16) == 0).all()
    packed = tr.expert_dispatch(x, index)
    packed[int(off[-1]):] = float("nan")  # rows behind the last group are not read
    assert torch.equal(lin(packed, off, sw, cw, n).view(torch.int16), y.view(torch.int16))


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,n,k", [(1, 16, 32), (5, 48, 160), (127, 256, 128), (129, 144, 544), (300, 512, 1024),
                                      (1021, 768, 2048), (16400, 80, 1056)])
@pytest.mark.parametrize("masked", [False, True])
def test_grad_input(device, rows, n, k, masked):
    import fp4_rollout_guided_amd as tr
    _say("case grad input", rows, n, k, masked)
    g = _gen(device, rows, n, k, masked)
    gy = _bf16(rows, n, g, device)
    sw, cw = random_record("mx", n, k, g, device)
    mask = torch.randint(0, 256, (rows * k // 8,), generator=g, device=device, dtype=torch.uint8) if masked else None
    gx = tr.mx_matmul_bwd_input(gy, sw, cw, k, mask=mask)
    w = values("mx", sw, cw, k)
    keep = unbits(mask, (rows, k)) if masked else torch.ones(rows, k, device=device)
    close(gx, (gy.double() @ w) * keep, (gy.double().abs() @ w.abs()) * keep, n)
    if masked:
        assert (gx[~keep].view(torch.int16) == 0).all()


@pytest.mark.parametrize("groups,rows,n,k,kind", GROUPED)
def test_grouped_grad_input(device, groups, rows, n, k, kind):
    import fp4_rollout_guided_amd as tr
    _say("case grouped grad input", groups, rows, n, k, kind)
    g = _gen(device, groups, rows, n, k, kind)
    gy = _bf16(rows, n, g, device)
    sw, cw = random_record("mx", groups * n, k, g, device)
    off = _uneven(groups, rows, kind).to(device)
    end = int(off[-1])
    gy[end:] = float("nan")  # rows of no group are not read
    out = torch.full((rows + 2, k), 3.0, dtype=torch.bfloat16, device=device)
    gx = tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k, grad_x=out)
    w = values("mx", sw, cw, k).view(groups, n, k)
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        if lo < hi:
            close(gx[lo:hi], gy[lo:hi].double() @ w[e], gy[lo:hi].double().abs() @ w[e].abs(), n)
    assert (gx[end:rows].view(torch.int16) == 0).all() and (gx[rows:] == 3).all()


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("rows,n,k", [(0, 32, 64), (1, 16, 32), (31, 48, 160), (33, 272, 128), (300, 144, 544),
                                      (1021, 768, 512), (5000, 128, 256), (9001, 64, 96), (70, 2064, 8192), (4100, 1040, 2080)])
@pytest.mark.parametrize("masked", [False, True])
def test_grad_weight(device, fmt, rows, n, k, masked):
    import fp4_rollout_guided_amd as tr
    _say("case grad weight", fmt, rows, n, k, masked)
    g = _gen(device, fmt, rows, n, k, masked)
    gy = _bf16(rows, n, g, device)
    sa, ca = random_record(fmt, rows, k, g, device)
    mask = torch.randint(0, 256, (n * k // 8,), generator=g, device=device, dtype=torch.uint8) if masked else None
    gw = (tr.mx_matmul_bwd_weight if fmt == "mx" else tr.mx8_matmul_bwd_weight)(gy, sa, ca, k, mask=mask)
    a = values(fmt, sa, ca, k)
    keep = unbits(mask, (n, k)) if masked else torch.ones(n, k, device=device)
    close(gw, (gy.double().T.contiguous() @ a) * keep, (gy.double().abs().T.contiguous() @ a.abs()) * keep, rows)


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("groups,rows,n,k,kind", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_grad_weight(device, fmt, groups, rows, n, k, kind, gather):
    import fp4_rollout_guided_amd as tr
    _say("case grouped grad weight", fmt, groups, rows, n, k, kind, gather)
    g = _gen(device, fmt, groups, rows, n, k, gather, "gw")
    src = rows // 2 + 1 if gather else rows
    gy = _bf16(rows, n, g, device)
    sa, ca = random_record(fmt, src, k, g, device)
    off = _uneven(groups, rows, kind).to(device)
    gy[int(off[-1]):] = float("nan")
    index = torch.randint(-1, src + 1, (rows,), generator=g, device=device) if gather else None
    mask = torch.randint(0, 256, (groups * n * k // 8,), generator=g, device=device, dtype=torch.uint8)
    bw = tr.grouped_mx_matmul_bwd_weight if fmt == "mx" else tr.grouped_mx8_matmul_bwd_weight
    gw = bw(gy, off, sa, ca, k, row_index=index, mask=mask)
    keep = unbits(mask, (groups, n, k))
    a = values(fmt, sa, ca, k)
    if gather:
        a = a[index.clamp(0, src - 1)] * ((index >= 0) & (index < src)).unsqueeze(1)
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        gt = gy[lo:hi].double().T.contiguous()
        close(gw[e], (gt @ a[lo:hi]) * keep[e], (gt.abs() @ a[lo:hi].abs()) * keep[e], max(1, hi - lo))


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["mx", "mx8"])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("guided", [False, True])
def test_autograd_function(device, fmt, grouped, guided):
    """y and the gradients equal the formula's: the product of the rounded
    operands, and grad_y times the other operand inside the clip range."""
    import fp4_rollout_guided_amd as tr
    _say("case autograd", fmt, grouped, guided)
    g = _gen(device, fmt, grouped, guided)
    rows, n, k, groups = 75, 64, 160, 3
    x = _bf16(rows, k, g, device).requires_grad_()
    w = (_bf16(groups * n, k, g, device, 0.1).view(groups, n, k) if grouped else _bf16(n, k, g, device, 0.1))
    w.requires_grad_()
    off = torch.tensor([0, 20, 20, 70], device=device) if grouped else None
    gy = _bf16(rows, n, g, device)
    scales = bits = None
    if guided:
        roll = (x.detach().float() * 1.05).to(torch.bfloat16)
        scales, bits, _ = (tr.mx_capture if fmt == "mx" else tr.mx8_capture)(roll)
        fwd = tr.mx_guided_fakequant_fwd if fmt == "mx" else tr.mx8_guided_fakequant_fwd
        xq, xm, _ = fwd(x.detach(), scales, bits)
        xq = xq.double()
    else:
        sa, ca, xm = (tr.mx_quantize if fmt == "mx" else tr.mx8_quantize)(x.detach(), want_mask=True)
        xq = values(fmt, sa, ca, k)
    sw, cw, wm = tr.mx_quantize(w.detach(), want_mask=True)
    wq = values("mx", sw, cw, k).view(-1, n, k)
    y = tr.MxMatmul.apply(x, w, off, fmt, scales, bits)
    y.backward(gy)
    xk, wk = unbits(xm, (rows, k)), unbits(wm, (-1, n, k))
    for e, (lo, hi) in enumerate(groups_of(off, rows) if grouped else [(0, rows)]):
        if lo < hi:
            _check_product(fmt, y[lo:hi].detach(), xq[lo:hi], wq[e])
        gd = gy[lo:hi].double()
        close(x.grad[lo:hi], (gd @ wq[e]) * xk[lo:hi], (gd.abs() @ wq[e].abs()) * xk[lo:hi], n)
        gt = gd.T.contiguous()
        close(w.grad.view(-1, n, k)[e], (gt @ xq[lo:hi]) * wk[e], (gt.abs() @ xq[lo:hi].abs()) * wk[e], max(1, hi - lo))
    if grouped:
        assert (x.grad[70:] == 0).all() and (y[70:] == 0).all()


def test_gradients_match_differences(device):
    """The product is linear in the decoded operands: one code of A or W
    moved to another value changes <gy, y> by the gradient times the move."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "differences")
    rows, n, k = 19, 32, 96
    sa, ca = random_record("mx", rows, k, g, device, 125, 129)
    sw, cw = random_record("mx", n, k, g, device, 125, 129)
    gy = _bf16(rows, n, g, device)
    gx = tr.mx_matmul_bwd_input(gy, sw, cw, k).double()
    gw = tr.mx_matmul_bwd_weight(gy, sa, ca, k).double()
    a, w = values("mx", sa, ca, k), values("mx", sw, cw, k)
    loss = lambda a, w: (gy.double() * (a @ w.T.contiguous())).sum()  # noqa: E731
    base = loss(a, w)
    for i, j in ((0, 0), (7, 31), (18, 95), (3, 64)):
        for which, grad in ((a, gx), (w, gw)):
            moved = which.clone()
            moved[i, j] += 1.0
            diff = (loss(moved, w) if which is a else loss(a, moved)) - base
            # the difference is exact in 64 bits; the gradient is a bf16
            assert abs(diff - grad[i, j]) <= 2.0 ** -8 * abs(diff) + 1e-4


def test_empty_contractions_give_zeros(device):
    import fp4_rollout_guided_amd as tr
    none = torch.empty(0, dtype=torch.uint8, device=device)
    x, y = torch.empty(5, 0, dtype=torch.bfloat16, device=device), torch.full((5, 32), 7.0, device=device).bfloat16()
    for lin in (tr.mx_linear, tr.mx8_linear):
        assert lin(x, none, none, 32, y=y) is y and (y == 0).all()
        y.fill_(7)
    off = torch.tensor([0, 2, 4], device=device)
    assert (tr.grouped_mx_linear(x, off, none, none, 32, y=y) == 0).all()
    gx = torch.full((5, 64), 7.0, device=device).bfloat16()
    assert (tr.mx_matmul_bwd_input(x, none, none, 64, grad_x=gx) == 0).all()
    with pytest.raises(ValueError, match="rows of"):
        tr.MxMatmul.apply(_bf16(4, 64, _gen(device, "k"), device), _bf16(16, 32, _gen(device, "k"), device))


# ---------------------------------------------------------------------------
# streams, graphs, devices
# ---------------------------------------------------------------------------

def test_products_on_a_side_stream_and_in_a_graph(device):
    """One layer's forward and backward, captured once and replayed on new
    inputs, with eager work between the replays, equals the eager results."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "graph")
    tokens, topk, experts, n, k = 40, 4, 8, 64, 128
    x = _bf16(tokens, k, g, device)
    ids = torch.topk(torch.rand(tokens, experts, generator=g, device=device), topk).indices.contiguous()
    wt = torch.rand(tokens, topk, generator=g, device=device)
    go = _bf16(tokens, n, g, device)
    sw, cw = random_record("mx", experts * n, k, g, device)

    def layer():
        off, index, slot = tr.expert_sort(ids, experts)
        sa, ca, mask = tr.mx_quantize(x, want_mask=True)
        y = tr.grouped_mx_matmul(sa, ca, off, sw, cw, n, k, row_index=index)
        out = tr.expert_combine(y, slot, wt)
        gy, gwt = tr.expert_combine_bwd(go, y, slot, wt, off)
        gx = tr.ste_bwd(tr.expert_combine(tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k), slot), mask)
        gw = tr.grouped_mx_matmul_bwd_weight(gy, off, sa, ca, k, row_index=index)
        return out, gwt, gx, gw

    side = torch.cuda.Stream(device)
    side.wait_stream(torch.cuda.current_stream(device))
    with torch.cuda.stream(side):
        on_side = layer()
    torch.cuda.current_stream(device).wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(on_side, layer()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for i in range(4):
        x.copy_(_bf16(tokens, k, g, device))
        go.copy_(_bf16(tokens, n, g, device))
        ids.copy_(torch.topk(torch.rand(tokens, experts, generator=g, device=device), topk).indices)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, layer()):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("fmt", ["mx", "mx8"])
def test_autograd_in_a_graph(device, fmt):
    """Token rounded in the product, routed rows and both gradients through
    autograd, captured after an eager pass whose graph is gone."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, fmt, "autograd graph")
    tokens, topk, experts, n, k = 24, 2, 4, 64, 96
    x, w = _bf16(tokens, k, g, device), _bf16(experts * n, k, g, device, 0.1).view(experts, n, k)
    ids = torch.topk(torch.rand(tokens, experts, generator=g, device=device), topk).indices.contiguous()
    wt, go = torch.rand(tokens, topk, generator=g, device=device), _bf16(tokens, n, g, device)
    sw, cw = random_record("mx", n, k, g, device)

    def layer():
        leaves = [t.detach().requires_grad_() for t in (x, w, wt)]
        off, index, slot = tr.expert_sort(ids, experts)
        y = tr.MxMatmul.apply(tr.ExpertDispatch.apply(leaves[0], index, slot), leaves[1], off, fmt)
        out = tr.ExpertCombine.apply(y, slot, leaves[2], off)
        one = (tr.mx_linear if fmt == "mx" else tr.mx8_linear)(x[:1], sw, cw, n)
        return [out.detach(), one, *torch.autograd.grad(out, leaves, go)]

    side = torch.cuda.Stream(device)
    side.wait_stream(torch.cuda.current_stream(device))
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream(device).wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for i in range(4):
        x.copy_(_bf16(tokens, k, g, device))
        go.copy_(_bf16(tokens, n, g, device))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, layer()):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [5, -7, 1 << 40, 30], [90, 90, 0, 0], [0, 90, 0, 90]])
@pytest.mark.parametrize("rows", [90, 300])
def test_offsets_out_of_order_stay_in_bounds(device, offsets, rows):
    """Their results are unspecified, but nothing past the arrays is written."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, rows, *offsets)
    n, k, groups = 80, 544, 3
    off = torch.tensor(offsets, device=device)
    x, gy = _bf16(rows, k, g, device), _bf16(rows, n, g, device)
    sa, ca = random_record("mx", rows, k, g, device)
    sw, cw = random_record("mx", groups * n, k, g, device)
    for shape, call in (((rows, n), lambda t: tr.grouped_mx_linear(x, off, sw, cw, n, y=t)),
                        ((rows, n), lambda t: tr.grouped_mx_matmul(sa, ca, off, sw, cw, n, k, y=t)),
                        ((rows, k), lambda t: tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k, grad_x=t)),
                        ((groups * n, k), lambda t: tr.grouped_mx_matmul_bwd_weight(gy, off, sa, ca, k, grad_w=t))):
        buf = torch.full((shape[0] + 200, shape[1]), 7.0, dtype=torch.bfloat16, device=device)
        call(buf[:shape[0]])
        assert (buf[shape[0]:] == 7).all()


def test_results_do_not_change_between_calls(device):
    """The same call twice gives the same bits (no order of atomics in them)."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "twice")
    rows, n, k = 700, 272, 1056
    sa, ca = random_record("mx8", rows, k, g, device)
    sw, cw = random_record("mx", n, k, g, device)
    gy = _bf16(rows, n, g, device)
    for f in (lambda: tr.mx8_matmul(sa, ca, sw, cw, n, k), lambda: tr.mx_matmul_bwd_input(gy, sw, cw, k),
              lambda: tr.mx8_matmul_bwd_weight(gy, sa, ca, k)):
        assert torch.equal(f(), f())


def test_small_grid_build_gives_the_same(device):
    """The test build sends every result past the cache and runs its grid-stride
    loops several times: the same bits."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "small grid")
    groups, rows, n, k = 4, 1500, 272, 1056
    off = torch.tensor([0, 700, 700, 1400, 1450], device=device)
    sa, ca = random_record("mx8", rows, k, g, device)
    sw, cw = random_record("mx", groups * n, k, g, device)
    gy, gz = _bf16(rows, n, g, device), _bf16(2100, 592, g, device)
    wm = torch.randint(0, 256, (groups * n * k // 8,), generator=g, device=device, dtype=torch.uint8)
    sb, cb = random_record("mx", 2100, 544, g, device)
    sv, cv = random_record("mx", 592, 544, g, device)
    calls = [lambda: tr.grouped_mx8_matmul(sa, ca, off, sw, cw, n, k),
             lambda: tr.mx_matmul(sb, cb, sv, cv, 592, 544), lambda: tr.mx_matmul_bwd_input(gz, sv, cv, 544),
             lambda: tr.mx_matmul_bwd_weight(gz, sb, cb, 544),
             lambda: tr.grouped_mx_matmul_bwd_input(gy, off, sw, cw, k),
             lambda: tr.grouped_mx8_matmul_bwd_weight(gy, off, sa, ca, k, mask=wm)]
    want = [f() for f in calls]
    held = tr.lib
    try:
        tr.lib = tr.load_library(tr.SMALLGRID_LIB_PATH)
        got = [f() for f in calls]
        torch.cuda.synchronize()
    finally:
        tr.lib = held
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), i


def test_binding_refusals(device):
    """The binding turns down tensors of the wrong device, type, shape or size
    before the C ABI, which sees bare pointers, is called."""
    import fp4_rollout_guided_amd as tr
    g = _gen(device, "refusals")
    rows, n, k = 8, 32, 64
    x = _bf16(rows, k, g, device)
    gy = _bf16(rows, n, g, device)
    sa, ca = random_record("mx", rows, k, g, device)
    sw, cw = random_record("mx", n, k, g, device)
    off = torch.tensor([0, 3, rows], device=device)
    with pytest.raises(ValueError, match="multiple of 16"):
        tr.mx_matmul(sa, ca, sw, cw, 24, k)
    with pytest.raises(ValueError, match="multiple of 32"):
        tr.mx_matmul(sa, ca, sw, cw, n, 48)
    with pytest.raises(ValueError, match="elements"):
        tr.mx_matmul(sa, ca, sw[:-1], cw, n, k)
    with pytest.raises(ValueError, match="elements"):
        tr.mx_matmul(sa, ca[:-1], sw, cw, n, k)
    with pytest.raises(ValueError, match="elements"):
        tr.mx8_matmul(sa, ca, sw, cw, n, k)  # MXFP4 codes where MXFP8's are wanted
    with pytest.raises(ValueError, match="must be on"):
        tr.mx_matmul(sa, ca, sw.cpu(), cw, n, k)
    with pytest.raises(ValueError, match="at least"):
        tr.mx_matmul(sa, ca, sw, cw, n, k, y=torch.empty(rows - 1, n, dtype=torch.bfloat16, device=device))
    with pytest.raises(TypeError):
        tr.mx_matmul(sa, ca, sw, cw, n, k, y=torch.empty(rows, n, device=device))
    with pytest.raises(ValueError, match="elements"):
        tr.grouped_mx_matmul(sa, ca, off, sw, cw, n, k)  # one weight for two groups
    with pytest.raises(ValueError, match="at most"):
        tr.grouped_mx_matmul(sa, ca, torch.zeros(4098, dtype=torch.int64, device=device), sw, cw, n, k)
    with pytest.raises(TypeError):
        tr.mx_linear(x.float(), sw, cw, n)
    with pytest.raises(ValueError, match="contiguous"):
        tr.mx_linear(_bf16(k, rows, g, device).T, sw, cw, n)
    with pytest.raises(ValueError, match="at least"):
        tr.mx_linear(_bf16(24, k, g, device), sw, cw, n, workspace=torch.empty(16, dtype=torch.uint8, device=device))
    with pytest.raises(TypeError):
        tr.grouped_mx_linear(x, off.int(), sw, cw, n)
    with pytest.raises(ValueError, match="at least"):
        tr.mx_matmul_bwd_input(gy, sw, cw, k, mask=torch.empty(rows * k // 8 - 1, dtype=torch.uint8, device=device))
    with pytest.raises(ValueError, match="rows"):
        tr.mx_matmul_bwd_weight(gy[:-1], sa, ca, k)
    with pytest.raises(ValueError, match="elements"):
        tr.grouped_mx_matmul_bwd_weight(gy, off, sa, ca, k, row_index=torch.zeros(rows - 1, dtype=torch.int64, device=device))
    ids = torch.zeros(4, 2, dtype=torch.int64, device=device)
    with pytest.raises(ValueError, match="experts"):
        tr.expert_sort(ids, 1025)
    with pytest.raises(TypeError):
        tr.expert_sort(ids.int(), 4)
    with pytest.raises(ValueError, match="topk"):
        tr.expert_sort(torch.zeros(1, 65, dtype=torch.int64, device=device), 4)
    with pytest.raises(ValueError, match="tokens, topk"):
        tr.expert_combine(x, ids.view(-1))
    with pytest.raises(ValueError, match="elements"):
        tr.expert_combine(x, ids, torch.ones(7, device=device))
    with pytest.raises(ValueError, match="grad_out"):
        tr.expert_combine_bwd(x, x, ids, None)
    with pytest.raises(ValueError, match='fmt must be'):
        tr.MxMatmul.apply(x, x, None, "fp8")
