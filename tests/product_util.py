"""Plain 64-bit forms of the microscaled products and the routed rows, shared
by their tests, and the tolerances of bf16 results of fp32 sums."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3_values():
    """The value of every E4M3FN byte (NaN for 0x7F and 0xFF)."""
    c = torch.arange(256)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(c >= 128, -v, v)


def values(fmt, scales, codes, cols):
    """float64 [rows, cols] that scale and code bytes stand for (0xFF: NaN)."""
    dev = codes.device
    if fmt == "mx":
        c = torch.stack([codes & 15, codes >> 4], -1).flatten().long()
        v = E2M1.to(dev)[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    else:
        v = e4m3_values().to(dev)[codes.long()]
    s = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return (v.view(-1, 32) * s.view(-1, 1)).reshape(-1, cols)


def random_record(fmt, rows, cols, g, dev, lo=118, hi=132):
    """Random codes (no NaN codes) under scale bytes lo..hi-1."""
    n = rows * cols
    codes = torch.randint(0, 256, (n // 2 if fmt == "mx" else n,), generator=g, device=dev, dtype=torch.uint8)
    if fmt == "mx8":
        codes = torch.where((codes & 127) == 127, codes & 128, codes)
    scales = torch.randint(lo, hi, (n // 32,), generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
    return scales, codes


def unbits(mask, shape):
    f = (mask.unsqueeze(-1) >> torch.arange(8, device=mask.device, dtype=torch.uint8)) & 1
    return f.reshape(shape).bool()


def groups_of(offsets, rows):
    """[(first, end)] of the groups' packed rows, host integers."""
    o = [min(max(int(v), 0), rows) for v in offsets.cpu()]
    return list(zip(o, o[1:]))


def close(got, want, size, terms, step=2.0 ** -8, product=2.0 ** -24):
    """Every element of got (bf16: step 2^-8, half a step of its rounding;
    fp32: 2^-24) within its tolerance of want (float64).  A sum of `terms`
    fp32 terms of total magnitude `size` is off by at most terms * product *
    size: each of its additions rounds a partial sum of at most `size` by half
    a step, 2^-24 of it.  The result is then rounded once."""
    got = got.double()
    tol = terms * product * size
    tol = tol + step * (want.abs() + tol) + 2.0 ** -133
    bad = ~((got - want).abs() <= tol)
    bad &= ~(got.isnan() & want.isnan())
    if bad.any():
        i = bad.flatten().nonzero()[0].item()
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off; first at {i}: got {got.flatten()[i].item()!r} "
                             f"want {want.flatten()[i].item()!r} tol {tol.flatten()[i].item()!r}")
