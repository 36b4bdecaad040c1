"""Plain 64-bit forms of the vocabulary loss and the router, and the optimiser
step in fp32 operations of numpy (each of them one IEEE rounding), shared by
their tests."""
import numpy as np
import torch


# ---------------------------------------------------------------------------
# the vocabulary loss
# ---------------------------------------------------------------------------

def logits(x, w, scale):
    return (x.double() @ w.double().t().contiguous()) * scale


def loss(x, w, targets, scale=1.0):
    """(loss, lse, which tokens count) in float64."""
    has = (targets >= 0) & (targets < w.shape[0])
    xv = torch.where(has.unsqueeze(1), x, torch.zeros_like(x))
    z = logits(xv, w, scale)
    lse = torch.logsumexp(z, 1)
    hit = z.gather(1, torch.where(has, targets, 0).unsqueeze(1)).squeeze(1)
    zero = torch.zeros_like(lse)
    return torch.where(has, lse - hit, zero), torch.where(has, lse, zero), has


def loss_tolerance(x, w, has, scale, lse):
    """How far loss and lse may be off.  A logit is a sum of k fp32 terms whose
    products are exact: k 2^-24 of their total size, and two more roundings for the
    scale.  lse is off by no more than its worst logit, plus the sum of the
    exponentials: its terms are off by |z| 2^-23 (the exponent's rounding) and
    2^-22 (the instruction's), its additions by 2^-24 for each of up to
    64 + 32 in a tile's column and one per tile; then two roundings of lse."""
    k = x.shape[1]
    xv = torch.where(has.unsqueeze(1), x, torch.zeros_like(x)).double()
    size = (xv.abs() @ w.double().abs().t().contiguous()).amax(1) * abs(scale)
    tiles = -(-w.shape[0] // 128)
    return size * (k + 3) * 2.0 ** -24 + size * 2.0 ** -22 + 2.0 ** -21 + (100 + tiles) * 2.0 ** -24 + lse.abs() * 2.0 ** -22


def loss_gradients(grad_loss, x, w, targets, scale=1.0):
    """(grad_x, grad_w, and the sizes of their sums' terms) in float64."""
    _, lse, has = loss(x, w, targets, scale)
    xv = torch.where(has.unsqueeze(1), x, torch.zeros_like(x)).double()
    p = torch.exp(logits(xv, w, scale) - lse.unsqueeze(1))
    g = torch.where(has, grad_loss.double() * scale, torch.zeros_like(lse)).unsqueeze(1)
    hot = torch.zeros_like(p)
    hot[torch.arange(len(targets), device=x.device), torch.where(has, targets, 0)] = 1.0
    d, s = g * (p - hot), g.abs() * (p + hot)
    wd = w.double()
    # what P's entries below the smallest normal number come to, see gradients_close
    tiny = float(g.abs().max()) * 2.0 ** -125 if len(targets) else 0.0
    return (d @ wd, d.t().contiguous() @ xv, s @ wd.abs() + tiny / STEP * wd.abs().sum(0),
            s.t().contiguous() @ xv.abs() + tiny / STEP * xv.abs().sum(0))


STEP = 2.0 ** -8  # half a step of bf16


def gradients_close(got, want, size, terms, x, w, scale, ctx):
    """bf16 gradients.  Each of P's entries is off by the logit's error (relative,
    as above, k + 3 + 4 steps of the largest logit's size), by 8 roundings of its
    own arithmetic and by half a step of bf16, 2^-8; for grad_w x times the row's
    factor is rounded by half a step too; their sum by `terms` additions; the result
    by half a step.  An entry of P over |p - 1| that is below 2^-126 counts as zero
    (the exponential gives no subnormal numbers, the matrix instruction takes none), a
    product of two factors near it as well: 2^-125 of the largest gradient for each
    term, which `size` has in it, over the 2^-8 below."""
    k = x.shape[1]
    largest = float((x.double().abs().nan_to_num(0, 0, 0) @ w.double().abs().t().contiguous()).max()) * abs(scale)
    each = (2 if ctx[-1] == "grad_w" else 1) * STEP + 12 * 2.0 ** -24 + (k + 7) * 2.0 ** -24 * largest + largest * 2.0 ** -21
    tol = size * (each + terms * 2.0 ** -24)
    tol = tol + STEP * (want.abs() + tol) + 2.0 ** -133
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError((ctx, int(bad.sum()), i, got[i].item(), want[i].item(), tol[i].item()))
    # as a whole: the result's rounding, at most 2^-8, and for grad_w as much again from x, independent of each other
    rel = float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
    assert rel < 2.0 ** -7.5, (ctx, rel)


# ---------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------

def route(z, topk, renormalize, valid=None):
    """(ids, weights, counts, probs, balance), float64, on the CPU, row by row."""
    z = z.double().cpu()
    tokens, experts = z.shape
    ids = torch.full((tokens, topk), -1, dtype=torch.int64)
    weights = torch.zeros(tokens, topk, dtype=torch.float64)
    counts = torch.zeros(experts + 1, dtype=torch.int64)
    probs = torch.zeros(experts, dtype=torch.float64)
    if tokens:
        key = torch.where(z.isnan(), torch.full_like(z, float("inf")), z)
        order = torch.sort(key, dim=1, descending=True, stable=True).indices
        # NaN above +infinity: among equals of the replaced keys NaN comes first
        rows_with_nan = z.isnan().any(1).nonzero().flatten().tolist()
        for t in rows_with_nan:
            nan = z[t].isnan()
            rest = torch.sort(torch.where(nan, torch.full_like(z[t], -float("inf")), z[t]), descending=True, stable=True).indices
            rest = rest[~nan[rest]]
            order[t] = torch.cat([nan.nonzero().flatten(), rest])
        ok = ~(z == -float("inf")).gather(1, order)
        keep = torch.ones(tokens, dtype=torch.bool) if valid is None else valid.cpu().bool()
        ids = torch.where(ok[:, :topk] & keep.unsqueeze(1), order[:, :topk], -1)
        routed = ids[:, 0] >= 0
        p = torch.softmax(z, 1)
        chosen = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
        if renormalize:
            sel = torch.where(ids >= 0, z.gather(1, ids.clamp(min=0)), -float("inf"))
            chosen = torch.where(ids >= 0, torch.softmax(sel, 1), 0.0)
        weights = torch.where(routed.unsqueeze(1), chosen, torch.zeros_like(chosen))
        for e in ids[ids >= 0].tolist():
            counts[e] += 1
        counts[experts] = int(routed.sum())
        probs = p[routed].sum(0) if bool(routed.any()) else probs
    pairs, rows = int(counts[:experts].sum()), int(counts[experts])
    balance = experts * (counts[:experts].double() / pairs * probs / rows).sum() if pairs else torch.zeros((), dtype=torch.float64)
    return ids, weights, counts, probs, balance


def route_gradient(z, ids, counts, renormalize, grad_weights, grad_balance):
    """The logits' gradient by autograd in float64; ids' choice is not differentiated."""
    z = z.detach().double().cpu().requires_grad_(True)
    ids, counts = ids.cpu(), counts.cpu().double()
    experts = z.shape[1]
    routed = ids[:, 0] >= 0
    there = ids >= 0
    zr = z[routed]
    p = torch.softmax(zr, 1)
    total = torch.zeros((), dtype=torch.float64)
    if grad_weights is not None:
        sel = torch.where(there, z.gather(1, ids.clamp(min=0)), -float("inf"))[routed]
        w = torch.softmax(sel, 1) if renormalize else p.gather(1, ids[routed].clamp(min=0))
        g = torch.where(there, grad_weights.double().cpu(), 0.0)[routed]
        total = total + (torch.where(there[routed], w, 0.0) * g).sum()
    if grad_balance is not None and bool(routed.any()):
        c = counts[:experts]
        total = total + grad_balance.double().cpu().sum() * experts * (c / c.sum() * p.sum(0) / counts[experts]).sum()
    return torch.autograd.grad(total, z, allow_unused=True)[0] if total.requires_grad else torch.zeros_like(z)


# ---------------------------------------------------------------------------
# the optimiser step
# ---------------------------------------------------------------------------

F, U = np.float32, np.uint32


def mix(h):
    h = h.astype(np.uint64)
    h ^= h >> np.uint64(16)
    h = (h * np.uint64(0x6A09E667)) & np.uint64(0xFFFFFFFF)
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0xBB67AE85)) & np.uint64(0xFFFFFFFF)
    return (h ^ (h >> np.uint64(16))).astype(U)


def random_bits(seed, first, n):
    """32 bits for each of n elements from place `first` on."""
    at = np.uint64(first) + np.arange(n, dtype=np.uint64)
    one = lambda v: mix(np.array([v & 0xFFFFFFFF], np.uint64))  # noqa: E731
    key = int(one(int(one(seed & 0xFFFFFFFF)[0]) + (seed >> 32))[0])
    keys = mix((np.uint64(key) + (at >> np.uint64(32))) & np.uint64(0xFFFFFFFF))
    return mix((mix(at & np.uint64(0xFFFFFFFF)).astype(np.uint64) + keys) & np.uint64(0xFFFFFFFF))


def _e4m3_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


E4M3 = _e4m3_table()


def decode(scales, codes):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    with np.errstate(all="ignore"):
        return (E4M3[codes] * np.repeat(s, 32)[: codes.size]).astype(F)


def encode(v, u):
    """(scales, codes) of fp32 v, each element rounded by 16 random bits u, by a
    search in the grid's values in place of the kernel's bit arithmetic.  Below
    2^-6 the rounding sees the element in steps of 2^-29 (half to even)."""
    n = v.size
    blocks = -(-n // 32)
    full = np.zeros(blocks * 32, F)
    full[:n] = v
    with np.errstate(all="ignore"):
        top = np.abs(full).reshape(-1, 32).max(1)
        bad = ~np.isfinite(full).reshape(-1, 32).all(1)
        e = np.zeros(blocks, np.int64)
        for b in range(blocks):
            if bad[b]:
                e[b] = 128
                continue
            e[b] = -127
            if top[b] > 448 * 2.0 ** -127:
                e[b] = int(np.ceil(np.log2(float(top[b]) / 448.0)))
                while float(top[b]) > 448 * 2.0 ** float(e[b]):
                    e[b] += 1
                while e[b] > -127 and float(top[b]) <= 448 * 2.0 ** float(e[b] - 1):
                    e[b] -= 1
        s = np.repeat(2.0 ** e.astype(np.float64), 32)[:n]
        z = np.abs(v.astype(np.float64)) / s
        z = z.astype(F).astype(np.float64)  # scaled in fp32: below its range steps of 2^-149
        z = np.where(z < 2.0 ** -6, np.rint(z * 2.0 ** 29) * 2.0 ** -29, z)
        grid = E4M3[:127]
        lo = np.clip(np.searchsorted(grid, z, side="right") - 1, 0, 126)
        hi = np.minimum(lo + 1, 126)
        width = np.where(hi > lo, grid[hi] - grid[lo], 1.0)
        share = np.floor((z - grid[lo]) / width * 2.0 ** 20)  # what the code's step leaves, in 20 bits
        up = share + (u.astype(np.int64) << 4) >= 2.0 ** 20
        code = np.where(up, hi, lo)
        code = np.where(np.repeat(bad, 32)[:n], 127, code)
    sign = (v.view(U) >> 31).astype(np.int64) << 7
    return (e + 127).astype(np.uint8), (code | sign).astype(np.uint8)


def bf16_bits(v):
    """Nearest, ties to even, of fp32 v."""
    b = v.view(U).astype(np.uint64)
    r = ((b + np.uint64(0x7FFF) + ((b >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)).astype(np.uint16)
    return np.where(np.isnan(v), (b >> np.uint64(16)).astype(np.uint16) | np.uint16(0x40), r)


def bf16_bits_random(v, u):
    b = v.view(U).astype(np.uint64)
    finite = (b & np.uint64(0x7F800000)) != np.uint64(0x7F800000)
    return ((b + np.where(finite, u, 0).astype(np.uint64)) >> np.uint64(16)).astype(np.uint16)


def widen(bits):
    return (bits.astype(U) << 16).view(F)


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=None):
    """fp32 p, g, m and v: (p, m, v, root) after the step."""
    b1, b2 = betas
    with np.errstate(all="ignore"):
        g = g * F(1.0 if grad_scale is None else grad_scale)
        m = m * F(b1) + g * F(1 - b1)
        v = v * F(b2) + (g * g) * F(1 - b2)
        root = np.sqrt(v)
        rate, by = F(lr / (1 - b1 ** step)), F(1 / np.sqrt(1 - b2 ** step))
        p = p * F(1 - lr * weight_decay) - (m / (root * by + F(eps))) * rate
    return p, m, v, root
