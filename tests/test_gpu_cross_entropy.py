"""The loss over the vocabulary and its gradients against their 64-bit forms:
sizes below, at and past the tiles' (128 and 256), one slice of the vocabulary
and several, tokens without a target whose rows hold anything, captured graphs,
other streams, and the refusals of the binding."""
import sys

import pytest
import torch

from tests import step_util as U
from tests.test_gpu_gridstride import _small_grid

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def inputs(tokens, vocab, k, device, seed=0, ignored=0.25, spread=1.0):
    g = torch.Generator(device=device)
    g.manual_seed(1000 * seed + tokens + vocab + k)
    w = (torch.randn(vocab, k, generator=g, device=device) * spread / k ** 0.5).to(torch.bfloat16)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    lean = torch.rand(tokens, 1, generator=g, device=device) * 6
    x = (torch.randn(tokens, k, generator=g, device=device) + lean * w[targets].float()).to(torch.bfloat16)
    off = torch.rand(tokens, generator=g, device=device)
    targets = torch.where(off < ignored, torch.where(off < ignored / 2, -100, vocab + 3), targets)
    grad = torch.randn(tokens, generator=g, device=device) / tokens
    return x, w, targets, grad


def check(tr, x, w, targets, grad, scale=1.0, ctx=None):
    loss, lse = tr.linear_cross_entropy(x, w, targets, scale)
    want, want_lse, has = U.loss(x, w, targets, scale)
    tol = U.loss_tolerance(x, w, has, scale, want_lse)
    assert (loss[~has] == 0).all() and (lse[~has] == 0).all(), ctx
    assert ((lse.double() - want_lse).abs() <= tol).all(), (ctx, float((lse.double() - want_lse).abs().max()))
    assert ((loss.double() - want).abs() <= 2 * tol).all(), (ctx, float((loss.double() - want).abs().max()))
    gx, gw = tr.linear_cross_entropy_bwd(grad, x, w, targets, lse, scale)
    wx, ww, sx, sw = U.loss_gradients(grad, x, w, targets, scale)
    U.gradients_close(gx, wx, sx, w.shape[0] + 32, x, w, scale, (ctx, "grad_x"))
    U.gradients_close(gw, ww, sw, x.shape[0] + 8, x, w, scale, (ctx, "grad_w"))
    assert (gx[~has] == 0).all(), ctx
    return loss, lse, gx, gw


SIZES = [(1, 1, 32), (1, 17, 64), (2, 130, 96), (16, 128, 32), (31, 256, 64), (32, 1000, 160), (33, 129, 128), (64, 300, 224),
         (65, 257, 96), (127, 1023, 64), (128, 128, 64), (129, 2050, 128), (256, 256, 256), (257, 1000, 1056), (300, 65, 544),
         (511, 4097, 288), (1021, 700, 96)]


@pytest.mark.parametrize("tokens,vocab,k", SIZES)
@pytest.mark.parametrize("scale,ignored", [(1.0, 0.3), (-0.7, 0.0)])
def test_sizes(device, tokens, vocab, k, scale, ignored):
    import fp4_rollout_guided_amd as tr
    _say("case cross entropy", tokens, vocab, k, scale, ignored)
    check(tr, *inputs(tokens, vocab, k, device, ignored=ignored), scale, (tokens, vocab, k))


# the large tiles (their turns fill the units), a last half stage of k, one token past a tile
@pytest.mark.parametrize("tokens,vocab,k,ignored", [(4096, 33000, 96, 0.0), (4097, 20481, 64, 0.4), (2047, 66000, 32, 0.1)])
def test_large_tiles(device, tokens, vocab, k, ignored):
    import fp4_rollout_guided_amd as tr
    _say("case large tiles", tokens, vocab, k)
    check(tr, *inputs(tokens, vocab, k, device, ignored=ignored), 1.25, (tokens, vocab, k))


@pytest.mark.parametrize("vocab", [8192 + 100, 16384])
def test_several_slices(device, vocab):
    """More than 32768 tokens: slices of 8192 columns."""
    import fp4_rollout_guided_amd as tr
    _say("case several slices", vocab)
    check(tr, *inputs(32768 + 40, vocab, 64, device, ignored=0.5), 1.0, vocab)


# up to 64 tokens: more rows of w to a workgroup than a tile's, and shares that end inside one
@pytest.mark.parametrize("tokens,vocab,k", [(5, 200003, 32), (32, 65536 + 197, 96), (33, 131072 + 77, 64), (50, 300007, 32),
                                            (64, 65, 64), (64, 1024 * 64 + 1, 32)])
def test_few_tokens_and_long_vocabularies(device, tokens, vocab, k):
    import fp4_rollout_guided_amd as tr
    _say("case few tokens", tokens, vocab, k)
    check(tr, *inputs(tokens, vocab, k, device, ignored=0.2), 0.9, (tokens, vocab, k))


# grad_x's parts go by the tokens that have targets: few of many, one, all, and a last slice shorter than the parts
@pytest.mark.parametrize("tokens,vocab,k,ignored", [(2000, 9000, 256, 0.6), (700, 20000, 96, 0.97), (1000, 10007, 288, 0.0),
                                                    (300, 5000, 64, 0.996), (66000, 8192 + 70, 32, 0.999)])
def test_parts(device, tokens, vocab, k, ignored):
    import fp4_rollout_guided_amd as tr
    _say("case parts", tokens, vocab, k, ignored)
    check(tr, *inputs(tokens, vocab, k, device, ignored=ignored), 1.0, (tokens, vocab, k))


def test_long_rows(device):
    """k past the tiles, the largest hidden size of the workloads."""
    import fp4_rollout_guided_amd as tr
    _say("case long rows")
    check(tr, *inputs(96, 600, 7168, device), 1.0, "7168")
    check(tr, *inputs(3, 4099, 7168, device, ignored=0.0), 1.0, "7168, few")


def test_confident_and_spread_out(device):
    """Logits far apart: probabilities of one and of nearly nothing."""
    import fp4_rollout_guided_amd as tr
    _say("case confident")
    x, w, targets, grad = inputs(200, 900, 128, device, spread=12.0)
    check(tr, (x.float() * 3).to(torch.bfloat16), w, targets, grad, 1.0, "confident")


def test_equal_gradients(device):
    """A mean: each entry near one of P is rounded alike, and must not take the gradients with it."""
    import fp4_rollout_guided_amd as tr
    _say("case mean")
    x, w, targets, _ = inputs(700, 3000, 256, device, ignored=0.0)
    for g in (1 / 700, -3e-30, 5e30):
        grad = torch.full((700,), g, device=device)
        _, lse = tr.linear_cross_entropy(x, w, targets)
        gx, gw = tr.linear_cross_entropy_bwd(grad, x, w, targets, lse)
        wx, ww, _, _ = U.loss_gradients(grad, x, w, targets)
        # the result's own rounding is 2^-8 / sqrt(3) of a value at most on average, with x's as much again for grad_w; P's
        # entries add a little
        for got, want, most in ((gx, wx, 1.1), (gw, ww, 1.5)):
            assert float((got.double() - want).norm() / want.norm()) < most * 2.0 ** -8 / 3 ** 0.5, g
    zero = torch.zeros(700, device=device)
    gx, gw = tr.linear_cross_entropy_bwd(zero, x, w, targets, lse)
    assert (gx == 0).all() and (gw == 0).all()


def test_ignored_rows_hold_anything(device):
    import fp4_rollout_guided_amd as tr
    _say("case ignored rows")
    for tokens in (40, 300):
        x, w, targets, grad = inputs(tokens, 500, 96, device)
        has = (targets >= 0) & (targets < 500)
        want = tr.linear_cross_entropy(x, w, targets)
        want += tr.linear_cross_entropy_bwd(grad, x, w, targets, want[1])
        bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device=device)
        fill = bad[torch.arange(tokens, device=device) % 4]
        x2 = torch.where(has.unsqueeze(1), x, fill.unsqueeze(1).to(torch.bfloat16))
        grad2, lse2 = torch.where(has, grad, fill), torch.where(has, want[1], fill)
        got = tr.linear_cross_entropy(x2, w, targets)
        got += tr.linear_cross_entropy_bwd(grad2, x2, w, targets, lse2)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        # only ignored tokens, and targets at the ends of their type
        none = torch.full_like(targets, -1)
        none[0], none[1] = 2 ** 63 - 1, -2 ** 63
        loss, lse = tr.linear_cross_entropy(x2, w, none)
        gx, gw = tr.linear_cross_entropy_bwd(grad2, x2, w, none, lse)
        assert not loss.any() and not lse.any() and not gx.any() and not gw.any()


def test_nan_stays_in_its_row(device):
    import fp4_rollout_guided_amd as tr
    _say("case NaN row")
    x, w, targets, grad = inputs(300, 500, 96, device, ignored=0.0)
    want, lse = tr.linear_cross_entropy(x, w, targets)
    gx, _ = tr.linear_cross_entropy_bwd(grad, x, w, targets, lse)
    x[7, 3] = float("nan")
    got, lse2 = tr.linear_cross_entropy(x, w, targets)
    gx2, gw2 = tr.linear_cross_entropy_bwd(grad, x, w, targets, lse2)
    other = torch.arange(300, device=device) != 7
    assert got[7].isnan() and torch.equal(got[other], want[other])
    assert gx2[7].isnan().all() and torch.equal(gx2[other], gx[other]) and gw2.isnan().all()
    grad[9] = float("nan")
    x[7, 3] = 0
    _, lse = tr.linear_cross_entropy(x, w, targets)
    gx3, _ = tr.linear_cross_entropy_bwd(grad, x, w, targets, lse)
    other[9] = False
    assert gx3[9].isnan().all() and torch.equal(gx3[other], gx[other])


def test_no_tokens_and_parts_of_the_gradients(device):
    import fp4_rollout_guided_amd as tr
    _say("case no tokens")
    w = torch.randn(70, 64, device=device).to(torch.bfloat16)
    x, t, f = torch.empty(0, 64, dtype=torch.bfloat16, device=device), torch.empty(0, dtype=torch.int64, device=device), torch.empty(0, device=device)
    loss, lse = tr.linear_cross_entropy(x, w, t)
    gx, gw = tr.linear_cross_entropy_bwd(f, x, w, t, lse)
    assert loss.numel() == 0 and gx.shape == x.shape and gw.shape == w.shape and not gw.any()
    x, w, t, g = inputs(150, 333, 64, device)
    _, lse = tr.linear_cross_entropy(x, w, t)
    gx, gw = tr.linear_cross_entropy_bwd(g, x, w, t, lse)
    only_x = tr.linear_cross_entropy_bwd(g, x, w, t, lse, want_w=False)
    only_w = tr.linear_cross_entropy_bwd(g, x, w, t, lse, want_x=False)
    assert only_x[1] is None and only_w[0] is None
    assert torch.equal(only_x[0], gx) and torch.equal(only_w[1], gw)


def test_neighbouring_memory_is_left(device):
    """Outputs and workspace inside larger buffers: what lies around them stays."""
    import fp4_rollout_guided_amd as tr
    _say("case neighbours")
    for tokens, vocab, k in ((5, 131, 96), (259, 515, 96)):
        x, w, t, g = inputs(tokens, vocab, k, device)
        want = tr.linear_cross_entropy(x, w, t)
        want += tr.linear_cross_entropy_bwd(g, x, w, t, want[1])

        def inside(numel, dtype):
            whole = torch.full((numel + 512,), 77, dtype=dtype, device=device)
            return whole, whole[256:256 + numel]
        held = []
        for n, d in ((tokens, torch.float32), (tokens, torch.float32), (tokens * k, torch.bfloat16), (vocab * k, torch.bfloat16),
                     (tr.lib.trace_linear_cross_entropy_workspace_bytes(tokens, vocab, k), torch.uint8),
                     (tr.lib.trace_linear_cross_entropy_bwd_workspace_bytes(tokens, vocab, k), torch.uint8)):
            held.append(inside(n, d))
        part = [p for _, p in held]
        tr.linear_cross_entropy(x, w, t, loss=part[0], lse=part[1], workspace=part[4])
        tr.linear_cross_entropy_bwd(g, x, w, t, part[1], grad_x=part[2], grad_w=part[3], workspace=part[5])
        for (whole, p), v in zip(held, want):
            assert torch.equal(p, v.flatten())
        for whole, p in held:
            assert (whole[:256] == 77).all() and (whole[256 + p.numel():] == 77).all()


def test_same_bits_every_time_and_small_grids(device):
    import fp4_rollout_guided_amd as tr
    _say("case repeated and small grids")
    x, w, t, g = inputs(777, 2500, 160, device)

    def run():
        loss, lse = tr.linear_cross_entropy(x, w, t)
        return (loss, lse) + tr.linear_cross_entropy_bwd(g, x, w, t, lse)
    first = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
    with _small_grid():
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


def test_autograd(device):
    import fp4_rollout_guided_amd as tr
    _say("case autograd")
    x, w, t, _ = inputs(130, 301, 64, device)
    weight = torch.randn(130, device=device)
    xs = x.view(2, 65, 64).transpose(0, 1).contiguous().transpose(0, 1).detach().requires_grad_(True)  # strided
    ws = w.detach().requires_grad_(True)
    loss = tr.LinearCrossEntropy.apply(xs, ws, t.view(2, 65), 0.9)
    assert loss.shape == (2, 65)
    (loss * weight.view(2, 65)).sum().backward()
    wx, ww, sx, sw = U.loss_gradients(weight, x, w, t, 0.9)
    U.gradients_close(xs.grad.reshape(130, 64), wx, sx, 333, x, w, 0.9, ("autograd", "grad_x"))
    U.gradients_close(ws.grad, ww, sw, 138, x, w, 0.9, ("autograd", "grad_w"))
    only = x.detach().requires_grad_(True)
    tr.LinearCrossEntropy.apply(only, w, t).sum().backward()  # a frozen weight
    assert only.grad is not None
    y = tr.LinearCrossEntropy.apply(xs, ws, t.view(2, 65))
    gx, = torch.autograd.grad(y.sum(), xs, create_graph=True)
    with pytest.raises(RuntimeError):  # a second derivative is refused
        torch.autograd.grad(gx.float().sum(), ws)


def test_gradient_against_differences(device):
    """The kernel's gradient along a direction against central differences of the 64-bit loss: their own error is of
    the order of h^2, 1e-8, far below the gradients' roundings."""
    import fp4_rollout_guided_amd as tr
    _say("case differences")
    x, w, t, g = inputs(90, 211, 96, device)
    _, lse = tr.linear_cross_entropy(x, w, t, 1.1)
    gx, gw = tr.linear_cross_entropy_bwd(g, x, w, t, lse, 1.1)
    wx, ww, sx, sw = U.loss_gradients(g, x, w, t, 1.1)
    f = lambda a, b: float((U.loss(a, b, t, 1.1)[0] * g.double()).sum())  # noqa: E731
    h = 1e-4
    for got, size, move in ((gx, sx, lambda d, s: (x.double() + s * h * d, w.double())),
                            (gw, sw, lambda d, s: (x.double(), w.double() + s * h * d))):
        d = torch.randn(got.shape, device=device, dtype=torch.float64)
        slope = (f(*move(d, 1)) - f(*move(d, -1))) / (2 * h)
        # each element's roundings, 2^-8 of itself or of the sum's size, have random signs: the sums of their sizes bound
        # them, and a sixth of that is already out of reach
        assert abs(float((got.double() * d).sum()) - slope) <= float((size * d.abs()).sum()) * 2.0 ** -8 / 6 + 1e-6


def test_graph_replays_and_streams(device):
    import fp4_rollout_guided_amd as tr
    _say("case graph and streams")
    x, w, t, g = inputs(400, 1100, 128, device)
    want = tr.linear_cross_entropy(x, w, t)
    want += tr.linear_cross_entropy_bwd(g, x, w, t, want[1])
    need = (tr.lib.trace_linear_cross_entropy_workspace_bytes(400, 1100, 128),
            tr.lib.trace_linear_cross_entropy_bwd_workspace_bytes(400, 1100, 128))

    def buffers():
        return [torch.empty_like(v) for v in want] + [torch.empty(n, dtype=torch.uint8, device=device) for n in need]

    def run(o):
        tr.linear_cross_entropy(x, w, t, loss=o[0], lse=o[1], workspace=o[4])
        tr.linear_cross_entropy_bwd(g, x, w, t, o[1], grad_x=o[2], grad_w=o[3], workspace=o[5])
    # two streams at once, each with buffers of its own
    outs, streams = [buffers() for _ in range(2)], [torch.cuda.Stream(device=device) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o, s in zip(outs, streams):
            with torch.cuda.stream(s):
                run(o)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, o))
    o = buffers()
    with torch.cuda.stream(streams[0]):
        run(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(o)
    for _ in range(4):
        for b in o:
            b.fill_(85)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, o))
    del graph


@pytest.mark.parametrize("tokens,vocab,k", [(20, 70000, 96), (700, 5000, 64), (1500, 3001, 64)])
def test_replays_with_other_targets(device, tokens, vocab, k):
    """What a captured pass lists, packs and splits is the replay's own: as many targets as it finds."""
    import fp4_rollout_guided_amd as tr
    _say("case replays with other targets", tokens)
    x, w, t, g = inputs(tokens, vocab, k, device)

    def run():
        loss, lse = tr.linear_cross_entropy(x, w, t)
        return loss, lse, *tr.linear_cross_entropy_bwd(g, x, w, t, lse)
    stream = torch.cuda.Stream(device=device)
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    first = t.clone()
    for keep in (tokens, 1, tokens // 2, 0, tokens):
        t.copy_(torch.where(torch.arange(tokens, device=device) < keep, first.clamp(0, vocab - 1), -1))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        assert all(torch.equal(a, b) for a, b in zip(run(), got)), keep
    del graph


def test_binding_refusals(device):
    import fp4_rollout_guided_amd as tr
    _say("case refusals")
    x, w, t, g = inputs(20, 40, 64, device)
    lse = torch.zeros(20, device=device)
    for bad in ((x, w[:, :32], t), (x[:, :32], w, t), (x, w, t[:19]), (x, w, t.int()), (x.float(), w, t), (x, w.cpu(), t),
                (x, w, t.cpu()), (x, w[:0], t), (x, w.view(-1), t), (x[:, :0], w[:, :0], t), (x.t(), w, t)):
        with pytest.raises((TypeError, ValueError)):
            tr.linear_cross_entropy(*bad)
        with pytest.raises((TypeError, ValueError)):
            tr.linear_cross_entropy_bwd(g, *bad, lse)
    for bad in (g[:10], g.double(), g.cpu()):
        with pytest.raises((TypeError, ValueError)):
            tr.linear_cross_entropy_bwd(bad, x, w, t, lse)
        with pytest.raises((TypeError, ValueError)):
            tr.linear_cross_entropy_bwd(g, x, w, t, bad)
    with pytest.raises(ValueError):
        tr.linear_cross_entropy(x, w, t, workspace=torch.empty(8, dtype=torch.uint8, device=device))
    with pytest.raises(tr.TraceError):
        tr.linear_cross_entropy(x, w, t, loss=lse, lse=lse)
