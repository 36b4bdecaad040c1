"""The optimiser step against the same fp32 operations in numpy, bit for bit:
every type, sizes around the blocks of 32 and the chunks of 4096, lists longer than
a launch's, random roundings, NaN and infinities, and its refusals."""
import copy
import sys

import numpy as np
import pytest
import torch

from tests import step_util as U
from tests.test_gpu_gridstride import _small_grid

pytestmark = pytest.mark.gpu

SIZES = [1, 3, 4, 5, 7, 8, 31, 32, 33, 63, 64, 100, 0, 1021, 4095, 4096, 4097, 8192 + 40, 20000]


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy().view(np.uint32)


def to(a, device, bf16=False):
    if bf16:
        return torch.from_numpy(a.view(np.int16).copy()).to(device).view(torch.bfloat16)
    return torch.from_numpy(a.copy()).to(device)


class Case:
    """Tensors on the GPU and what numpy holds of them."""

    def __init__(self, sizes, param_bf16, grad_bf16, mx8, device, seed=0, copies=False):
        rng = np.random.default_rng(seed)
        self.sizes, self.param_bf16, self.grad_bf16, self.mx8, self.device = sizes, param_bf16, grad_bf16, mx8, device
        self.copies = copies
        self.p, self.g, self.m, self.v = [], [], [], []
        for n in sizes:
            own = np.exp(rng.standard_normal(n) * 2).astype(np.float32) * np.float32(1e-3)
            p = rng.standard_normal(n).astype(np.float32) * np.float32(0.02)
            g = rng.standard_normal(n).astype(np.float32) * own
            self.p.append(U.widen(U.bf16_bits(p)) if param_bf16 else p)
            self.g.append(U.widen(U.bf16_bits(g)) if grad_bf16 else g)
            m, r = (rng.standard_normal(n).astype(np.float32) * own * np.float32(0.3), own * np.float32(0.9))
            if mx8:
                half = np.full(n, 32768)
                m, r = U.encode(m, half), U.encode(r, half)
                self.m.append(m), self.v.append(r)
            else:
                self.m.append(m), self.v.append(r * r)
        self.put()

    def put(self):
        d = self.device
        self.tp = [to(U.bf16_bits(p), d, True) if self.param_bf16 else to(p, d) for p in self.p]
        self.tg = [to(U.bf16_bits(g), d, True) if self.grad_bf16 else to(g, d) for g in self.g]
        if self.mx8:
            self.tm = [tuple(to(a, d) for a in m) for m in self.m]
            self.tv = [tuple(to(a, d) for a in v) for v in self.v]
        else:
            self.tm, self.tv = [to(m, d) for m in self.m], [to(v, d) for v in self.v]
        self.tc = [torch.zeros(n, dtype=torch.bfloat16, device=d) for n in self.sizes] if self.copies else None

    def numpy_step(self, step, lr, betas, eps, weight_decay, grad_scale, seed):
        place = 0
        self.c = []
        for i, n in enumerate(self.sizes):
            m, v = self.m[i], self.v[i]
            if self.mx8:
                m, r = U.decode(*m), U.decode(*v)
                with np.errstate(all="ignore"):
                    v = r * r
            p, m, v, root = U.adamw(self.p[i], self.g[i], m, v, step, lr, betas, eps, weight_decay, grad_scale)
            u = U.random_bits(seed or 0, place, n)
            self.c.append(U.bf16_bits(p))
            if self.param_bf16:
                h = U.bf16_bits(p) if seed is None else U.bf16_bits_random(p, U.mix(u.astype(np.uint64)) >> np.uint32(16))
                p = U.widen(h)
            self.p[i] = p
            if self.mx8:
                self.m[i], self.v[i] = U.encode(m, u & np.uint32(0xFFFF)), U.encode(root, u >> np.uint32(16))
            else:
                self.m[i], self.v[i] = m, v
            place += -(-n // 32) * 32

    def same(self, ctx):
        def eq(got, want, name, i):
            both_nan = False
            if want.dtype == np.uint32:
                both_nan = np.isnan(got.view(np.float32)) & np.isnan(want.view(np.float32))
            elif want.dtype == np.uint16:
                both_nan = np.isnan(U.widen(got)) & np.isnan(U.widen(want))
            bad = (got != want) & ~both_nan
            assert not bad.any(), (ctx, name, i, self.sizes[i], int(bad.sum()), int(bad.argmax()), got[bad][:3], want[bad][:3])
        for i in range(len(self.sizes)):
            eq(bits(self.tp[i]), U.bf16_bits(self.p[i]) if self.param_bf16 else self.p[i].view(np.uint32), "param", i)
            if self.copies:
                eq(bits(self.tc[i]), self.c[i], "copy", i)
            for got, want, name in ((self.tm[i], self.m[i], "avg"), (self.tv[i], self.v[i], "sq")):
                if self.mx8:
                    eq(got[0].cpu().numpy(), want[0], name + " scales", i)
                    ok = np.repeat(want[0], 32)[: self.sizes[i]] != 255  # a NaN block's codes are NaN, of either sign
                    eq(got[1].cpu().numpy()[ok], want[1][ok], name + " codes", i)
                    assert (got[1].cpu().numpy()[~ok] & 127 == 127).all()
                else:
                    eq(bits(got), want.view(np.uint32), name, i)


OPT = dict(lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


@pytest.mark.parametrize("param_bf16", [False, True], ids=["p32", "p16"])
@pytest.mark.parametrize("grad_bf16", [False, True], ids=["g32", "g16"])
@pytest.mark.parametrize("mx8", [False, True], ids=["s32", "s8"])
def test_types_and_sizes(device, param_bf16, grad_bf16, mx8):
    import fp4_rollout_guided_amd as tr
    _say("case adamw", param_bf16, grad_bf16, mx8)
    c = Case(SIZES, param_bf16, grad_bf16, mx8, device, copies=not param_bf16)
    scale = torch.full((1,), 0.7, device=device)
    for step, seed, gs in ((1, 7, None), (2, 2 ** 63 + 11, scale), (1000, 0 if mx8 else None, scale)):
        tr.adamw_step(c.tp, c.tg, c.tm, c.tv, step, grad_scale=gs, copies=c.tc, seed=seed, **OPT)
        c.numpy_step(step, OPT["lr"], OPT["betas"], OPT["eps"], OPT["weight_decay"], None if gs is None else 0.7, seed)
        c.same((step, seed))


@pytest.mark.parametrize("mx8", [False, True], ids=["s32", "s8"])
def test_many_tensors(device, mx8):
    """More than one launch's tensors: places in the list count on."""
    import fp4_rollout_guided_amd as tr
    _say("case many tensors", mx8)
    rng = np.random.default_rng(3)
    sizes = [int(n) for n in rng.integers(1, 700, 130)] + [5000, 1, 32]
    c = Case(sizes, True, True, mx8, device)
    tr.adamw_step(c.tp, c.tg, c.tm, c.tv, 5, seed=3, **OPT)
    c.numpy_step(5, OPT["lr"], OPT["betas"], OPT["eps"], OPT["weight_decay"], None, 3)
    c.same("many")
    tr.adamw_step(tuple(c.tp), (g for g in c.tg), c.tm, c.tv, 6, seed=4, **OPT)
    c.numpy_step(6, OPT["lr"], OPT["betas"], OPT["eps"], OPT["weight_decay"], None, 4)
    c.same("many, other containers")


def test_large_and_small_grids(device):
    """Past 256 MiB in all (streamed), and the build that streams everything."""
    import fp4_rollout_guided_amd as tr
    _say("case large")
    n = 24_000_000
    for mx8 in (False, True):
        g = torch.Generator(device=device)
        g.manual_seed(1)
        new = lambda: [torch.randn(n, generator=g, device=device) * 0.02, torch.randn(n, generator=g, device=device) * 1e-3]  # noqa: E731
        p, grad = new()
        zero = lambda k: torch.zeros(k, dtype=torch.uint8, device=device)  # noqa: E731
        state = ([(zero(n // 32), zero(n))] if mx8 else [torch.zeros(n, device=device)])
        sets = []
        for part in (None, [0, 1_000_000, 9_999_968, n]):  # whole, and in three tensors at the same places
            q = p.clone()
            s = copy.deepcopy(state), copy.deepcopy(state)
            cut = (lambda t, k=1: [t]) if part is None else (lambda t, k=1: [t[a // k:b // k] for a, b in zip(part, part[1:])])
            lists = [cut(q), cut(grad)]
            for one in s:
                lists.append([*zip(cut(one[0][0], 32), cut(one[0][1]))] if mx8 else cut(one[0]))
            tr.adamw_step(*lists, 1, 1e-3, seed=9)
            sets.append((q, s))
        for a, b in ((sets[0], sets[1]),):
            assert torch.equal(a[0], b[0])
            for x, y in zip(a[1], b[1]):
                for u, v in zip(x[0], y[0]) if mx8 else ((x[0], y[0]),):
                    assert torch.equal(u, v)
    c, d = (Case(SIZES, True, False, True, device, seed=4) for _ in range(2))
    tr.adamw_step(c.tp, c.tg, c.tm, c.tv, 3, seed=8, **OPT)
    with _small_grid():
        tr.adamw_step(d.tp, d.tg, d.tm, d.tv, 3, seed=8, **OPT)
    d.p = [U.widen(bits(t)) for t in c.tp]
    d.m, d.v = ([tuple(a.cpu().numpy() for a in s) for s in ss] for ss in (c.tm, c.tv))
    d.same("small grid")


def test_extremes(device):
    """Zeros, the smallest and largest numbers, NaN and infinities: each in its block alone."""
    import fp4_rollout_guided_amd as tr
    _say("case extremes")
    for param_bf16 in (False, True):
        for mx8 in (False, True):
            c = Case([256, 40], param_bf16, False, mx8, device, seed=2)
            c.g[0][:32] = 0
            c.g[0][32:64] = np.float32(1e-45) * np.arange(32, dtype=np.float32)
            c.g[0][64:96] = np.float32(1e-20)
            c.g[0][96] = np.inf
            c.g[0][130] = np.nan
            c.g[0][161] = np.float32(3e38)
            c.g[0][200:224] = np.float32(2.0) ** -np.arange(24, dtype=np.float32)
            c.p[0][3], c.p[0][4] = np.float32(np.inf), np.float32(np.nan)
            c.put()
            for step in (1, 2, 3):
                tr.adamw_step(c.tp, c.tg, c.tm, c.tv, step, lr=1e-2, weight_decay=0.0, seed=step)
                c.numpy_step(step, 1e-2, (0.9, 0.999), 1e-8, 0.0, None, step)
                c.same((param_bf16, mx8, step))
    # nothing to divide by: 0 / 0 is the formula's NaN, with eps zero there is none
    p = torch.ones(8, device=device)
    zero = [torch.zeros(8, device=device) for _ in range(3)]
    tr.adamw_step([p], [zero[0]], [zero[1]], [zero[2]], 1, 1e-3, weight_decay=0.0)
    assert (p == 1).all()
    tr.adamw_step([p], [zero[0]], [zero[1]], [zero[2]], 1, 1e-3, eps=0.0, weight_decay=0.0)
    assert p.isnan().all()


def test_random_roundings_keep_the_mean(device):
    """65536 equal elements that no code holds: their mean after one rounding is the value within six standard deviations
    of a rounding's, half a step of the code over 256 (each is a coin with two sides one step apart)."""
    import fp4_rollout_guided_amd as tr
    _say("case means")
    n = 65536
    grad = torch.full((n,), 0.0317, device=device)
    p = torch.full((n,), 1.2345, device=device).to(torch.bfloat16)
    rec = lambda: (torch.zeros(n // 32, dtype=torch.uint8, device=device), torch.zeros(n, dtype=torch.uint8, device=device))  # noqa: E731
    m, r = rec(), rec()
    tr.adamw_step([p], [grad], [m], [r], 1, lr=1e-3, betas=(0.9, 0.999), weight_decay=0.0, seed=77)
    for state, want in ((m, 0.00317), (r, 0.0317 * (1 - 0.999) ** 0.5)):
        v = U.decode(*(a.cpu().numpy() for a in state)).astype(np.float64)
        steps = np.unique(v)
        assert len(steps) == 2 and steps[0] < want < steps[1]
        assert abs(v.mean() - want) < 6 * (steps[1] - steps[0]) / 2 / 256 + 1e-6 * want
    want = float(p.new_full((1,), 1.2345).float()) - 1e-3
    v = p.float().cpu().numpy().astype(np.float64)
    steps = np.unique(v)
    assert len(steps) == 2 and abs(v.mean() - want) < 6 * (steps[1] - steps[0]) / 2 / 256 + 1e-6
    # a root that falls by less than a code's step still falls
    for t in range(2, 402):
        tr.adamw_step([p], [torch.zeros(n, device=device)], [m], [r], t, lr=0.0, betas=(0.9, 0.999), weight_decay=0.0, seed=t)
    v = U.decode(*(a.cpu().numpy() for a in r)).astype(np.float64)
    expect = 0.0317 * (0.001 * 0.999 ** 400) ** 0.5
    # a rounding keeps the root's mean, which each step takes by sqrt(0.999).  One step moves a root by 0.0005 of itself,
    # so it goes down a code (an eighth of it at most) with a chance whose variance is 0.0005 / 8 of its square: 400 of
    # them leave 0.16 of the root for each element, 0.0006 for the mean of 65536, and six times that is allowed
    assert abs(v.mean() / expect - 1) < 0.004


def test_state_class(device):
    """AdamW against adamw_step, its saved states, gradients of its parameters and changed storage."""
    import fp4_rollout_guided_amd as tr
    _say("case class")
    for states, seed, dtype in (("fp32", None, torch.float32), ("mx8", 5, torch.bfloat16), ("mx8", 5, torch.float32)):
        torch.manual_seed(1)
        params = [torch.nn.Parameter(torch.randn(s, device=device).to(dtype)) for s in ((33, 7), (4100,), (1,))]
        other = [p.detach().clone() for p in params]
        opt = tr.AdamW(params, lr=1e-2, states=states, seed=seed)
        if states == "fp32":
            m, v = ([torch.zeros_like(p) for p in other] for _ in range(2))
        else:
            rec = lambda p: (torch.zeros(-(-p.numel() // 32), dtype=torch.uint8, device=device), torch.zeros(p.numel(), dtype=torch.uint8, device=device))  # noqa: E731
            m, v = ([rec(p) for p in other] for _ in range(2))
        for t in range(1, 4):
            grads = [torch.randn_like(p) for p in other]
            for p, g in zip(params, grads):
                p.grad = g
            before = [p._version for p in params]
            opt.step()
            assert all(p._version > b for p, b in zip(params, before))
            tr.adamw_step(other, grads, m, v, t, 1e-2, seed=None if seed is None else seed + t)
            assert all(torch.equal(a, b) for a, b in zip(params, other))
        saved = copy.deepcopy(opt.state_dict())
        again = tr.AdamW(params, lr=1e-2, states=states, seed=1)
        again.load_state_dict(saved)
        params[1].data = params[1].data.clone()  # another storage
        again.step(grads, grad_scale=torch.ones(1, device=device))
        tr.adamw_step(other, grads, m, v, 4, 1e-2, seed=None if seed is None else seed + 4)
        assert again.steps == 4 and all(torch.equal(a, b) for a, b in zip(params, other))
        again.zero_grad()
        assert all(p.grad is None for p in params)
        with pytest.raises(ValueError):
            again.step()
        with pytest.raises((TypeError, ValueError)):
            tr.AdamW(params, states="fp32" if states == "mx8" else "mx8", seed=3).load_state_dict(saved)
        params[0].data = torch.zeros(5, device=device, dtype=dtype)
        with pytest.raises(ValueError):
            again.step(grads)
    with pytest.raises(ValueError):
        tr.AdamW([torch.zeros(4, device=device)], states="mx8")
    with pytest.raises(ValueError):
        tr.AdamW([])


def test_backward_sees_the_step(device):
    """A graph whose saved weight has been stepped refuses its backward pass, as after any other in-place change."""
    import fp4_rollout_guided_amd as tr
    _say("case versions")
    w = torch.nn.Parameter(torch.randn(8, 8, device=device))
    y = (torch.randn(8, 8, device=device, requires_grad=True) @ w).sum()
    tr.AdamW([w]).step([torch.ones_like(w)])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_graph_replays_and_streams(device):
    import fp4_rollout_guided_amd as tr
    _say("case graph")
    c, d = (Case(SIZES, True, True, True, device, seed=6) for _ in range(2))
    side = torch.cuda.Stream(device=device)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.adamw_step(c.tp, c.tg, c.tm, c.tv, 4, seed=6, **OPT)
    c.same("captured, not run")
    for rep in range(4):
        graph.replay()
        with torch.cuda.stream(side):
            tr.adamw_step(d.tp, d.tg, d.tm, d.tv, 4, seed=6, **OPT)
        torch.cuda.synchronize()
        c.numpy_step(4, OPT["lr"], OPT["betas"], OPT["eps"], OPT["weight_decay"], None, 6)
        c.same(("replay", rep))
        d.p, d.m, d.v = c.p, c.m, c.v
        d.same(("stream", rep))
    del graph


def test_refusals(device):
    import fp4_rollout_guided_amd as tr
    _say("case refusals")
    z = lambda n, dtype=torch.float32: torch.zeros(n, dtype=dtype, device=device)  # noqa: E731
    p, g, m, v = ([z(64), z(33)] for _ in range(4))
    rec = [(z(2, torch.uint8), z(64, torch.uint8)), (z(2, torch.uint8), z(33, torch.uint8))]
    rec2 = [(z(2, torch.uint8), z(64, torch.uint8)), (z(2, torch.uint8), z(33, torch.uint8))]
    tr.adamw_step(p, g, m, v, 1, 1e-3)
    tr.adamw_step(p, g, rec, rec2, 1, 1e-3, seed=0)
    for bad in ((p, g[:1], m, v), (p, g, m[:1], v), (p, [g[0], z(32)], m, v), (p, [g[0], z(33, torch.bfloat16)], m, v),
                (p, [z(64, torch.float16), z(33, torch.float16)], m, v), (p, g, [m[0], m[1].to(torch.bfloat16)], v),
                (p, g, rec, v), (p, g, m, rec), (p, g, [rec[0], rec[1][::-1]], rec2), (p, g, [rec[0], rec[1][:1]], rec2),
                (p, [g[0], g[1].cpu()], m, v), ([p[0], p[1].cpu()], g, m, v), ([p[0], z(66)[::2]], g, m, v), (p, g, m, None),
                ([p[0], 3], g, m, v), (p, [g[0], None], m, v)):
        with pytest.raises((TypeError, ValueError)):
            tr.adamw_step(*bad, 1, 1e-3, seed=1)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=True), dict(seed=1.5), dict(grad_scale=z(2)),
               dict(grad_scale=torch.ones(1)), dict(copies=[z(64), z(33)]), dict(copies=[z(64, torch.bfloat16)])):
        with pytest.raises((TypeError, ValueError)):
            tr.adamw_step(p, g, m, v, 1, 1e-3, **kw)
    with pytest.raises(ValueError):
        tr.adamw_step(p, g, rec, rec2, 1, 1e-3)  # records without a seed
    with pytest.raises(ValueError):
        tr.adamw_step([z(64, torch.bfloat16)], [z(64)], [z(64)], [z(64)], 1, 1e-3, copies=[z(64, torch.bfloat16)])
    for args in ((0, 1e-3), (1, float("nan"))):
        with pytest.raises(tr.TraceError):
            tr.adamw_step(p, g, m, v, *args)
    for lists in (([p[0], p[0]], [z(64), z(64)], [z(64), z(64)], [z(64), z(64)]), (p, p, m, v), (p, g, m, m), (p, g, p, v)):
        with pytest.raises(tr.TraceError):  # an element of two tensors
            tr.adamw_step(*lists, 1, 1e-3)
    with pytest.raises(tr.TraceError):
        tr.adamw_step([z(66)[1:65]], [z(64)], [z(64)], [z(64)], 1, 1e-3)  # not 16-byte aligned
