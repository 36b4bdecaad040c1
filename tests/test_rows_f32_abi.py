"""Refusals of the entry points on fp32 packed rows, and of sizes past one
launch, on the CPU: every bad argument is turned down before any HIP call (the
device addresses below are never dereferenced)."""
import pytest
import torch

import fp4_rollout_guided_amd as tr

L = tr.lib
OK, E_NULL, E_SHAPE, E_ALIGN, E_ALIAS = 0, 1, 2, 3, 4
A = 0x7F0000000000
STEP = 0x1000000  # 16 MiB between fake buffers


def buf(i, shift=0):
    return A + i * STEP + shift


def call(fn, spec, **change):
    assert set(change) <= set(spec), change
    return getattr(L, fn)(*{**spec, **change}.values())


MM = dict(a_scales=buf(0), a_codes=buf(1), src_rows=40, row_index=buf(5), rows=64, offsets=buf(6), groups=3,
          w_scales=buf(2), w_codes=buf(3), n=48, k=96, y=buf(4), stream=None)
LIN = dict(x=buf(0), src_rows=40, row_index=buf(5), rows=64, offsets=buf(6), groups=3, w_scales=buf(2), w_codes=buf(3),
           n=48, k=96, workspace=buf(7), workspace_bytes=1 << 20, y=buf(4), stream=None)
GX = dict(grad_y=buf(0), rows=64, offsets=buf(6), groups=3, w_scales=buf(2), w_codes=buf(3), n=48, k=96, mask=buf(5),
          grad_x=buf(4), stream=None)


@pytest.mark.parametrize("fn,spec,out", [
    ("trace_grouped_mx_matmul_f32", MM, "y"), ("trace_grouped_mx8_matmul_f32", MM, "y"),
    ("trace_grouped_mx_linear_f32", LIN, "y"), ("trace_grouped_mx8_linear_f32", LIN, "y"),
    ("trace_grouped_mx_matmul_bwd_input_f32", GX, "grad_x")])
def test_products(fn, spec, out):
    c = lambda **k: call(fn, spec, **k)  # noqa: E731
    assert c(rows=0, **{out: None}) == OK
    for bad in ({"rows": -1}, {"rows": 1 << 31}, {"n": 8}, {"k": 48}, {"groups": 0}, {"groups": 4097}):
        assert c(**bad) == E_SHAPE, bad
    assert c(offsets=None) == c(offsets=None, groups=0) == E_NULL  # packed rows only
    for name, v in spec.items():
        if name in ("mask", "row_index", "stream") or not isinstance(v, int) or v < A:
            continue
        assert c(**{name: None}) == E_NULL, name
        if name not in ("workspace", out):
            assert c(**{out: v}) == E_ALIAS, name
    assert c(**{out: buf(4, 8)}) == E_ALIGN
    # the result is four bytes an element: an input behind its bf16 size overlaps it
    elements = 64 * (96 if spec is GX else 48)
    assert c(w_scales=buf(4, 4 * elements - 16)) == E_ALIAS


COMB = dict(y=buf(0), rows=60, cols=48, slot=buf(1), weights=buf(2), tokens=30, topk=2, out=buf(3), stream=None)


def test_combine():
    c = lambda **k: call("trace_expert_combine_f32", COMB, **k)  # noqa: E731
    assert c(tokens=0) == c(cols=0) == OK
    assert c(rows=-1) == c(cols=40) == c(topk=0) == c(topk=65) == c(tokens=-1) == E_SHAPE
    assert c(y=None) == c(slot=None) == c(out=None) == E_NULL
    assert c(y=buf(0, 8)) == c(slot=buf(1, 4)) == c(weights=buf(2, 2)) == c(out=buf(3, 8)) == E_ALIGN
    assert c(out=buf(0)) == c(out=buf(1)) == c(out=buf(2)) == c(out=buf(0, 4 * 60 * 48 - 16)) == E_ALIAS


def test_binding():
    with pytest.raises(ValueError, match="device tensor"):
        tr.expert_combine(torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(TypeError, match="y must be bf16"):
        tr.expert_combine(torch.zeros(4, 64, dtype=torch.float16), torch.zeros(4, 2, dtype=torch.int64))


@pytest.mark.parametrize("fn", ["trace_mx_linear", "trace_mx8_linear", "trace_grouped_mx_linear_f32",
                                "trace_grouped_mx8_linear_f32"])
def test_sizes_past_one_launch_are_refused_before_the_rounding(fn):
    """Without a GPU, a launch would answer TRACE_E_HIP."""
    rows = (1 << 31) - 1
    at = [(1 << 46) + (i << 42) for i in range(6)]
    grouped = fn.endswith("_f32")
    for k in (32, 512):
        need = getattr(L, fn.replace("grouped_", "").replace("_f32", "") + "_workspace_bytes")(rows, rows, int(grouped), k)
        n = 16 if k == 32 else 1024
        assert getattr(L, fn)(at[0], rows, None, rows, at[1] if grouped else None, int(grouped), at[2], at[3], n, k, at[4],
                              need, at[5], None) == E_SHAPE, k
