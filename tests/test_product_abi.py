"""Refusals of the microscaled products and of the routed rows, on the CPU:
every bad argument is turned down before any HIP call (the device addresses
below are never dereferenced)."""
import ctypes

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
    """Call fn with spec's arguments (an ordered dict) and some changed."""
    assert set(change) <= set(spec), change
    return getattr(L, fn)(*{**spec, **change}.values())


QUANT = dict(x=buf(0), rows=64, cols=256, scales=buf(1), codes=buf(2), mask=buf(3), stream=None)


@pytest.mark.parametrize("fn", ["trace_mx_quantize", "trace_mx8_quantize"])
def test_quantize(fn):
    c = lambda **k: call(fn, QUANT, **k)  # noqa: E731
    assert c(rows=0) == OK and c(cols=0, x=None, scales=None, codes=None) == OK
    assert c(rows=-1) == c(cols=-32) == c(cols=48) == c(rows=1 << 40, cols=1 << 30) == E_SHAPE
    assert c(x=None) == c(scales=None) == c(codes=None) == E_NULL
    assert c(x=buf(0, 8)) == c(codes=buf(2, 8)) == c(mask=buf(3, 1)) == E_ALIGN
    assert c(scales=buf(0, 64)) == c(codes=buf(0)) == c(mask=buf(2, 2)) == c(scales=buf(2, 16)) == E_ALIAS


MM = dict(a_scales=buf(0), a_codes=buf(1), rows=64, w_scales=buf(2), w_codes=buf(3), n=48, k=96, y=buf(4), stream=None)
GMM = dict(a_scales=buf(0), a_codes=buf(1), src_rows=40, row_index=buf(5), rows=64, offsets=buf(6), groups=3,
           w_scales=buf(2), w_codes=buf(3), n=48, k=96, y=buf(4), stream=None)


@pytest.mark.parametrize("fn,spec", [("trace_mx_matmul", MM), ("trace_mx8_matmul", MM),
                                     ("trace_grouped_mx_matmul", GMM), ("trace_grouped_mx8_matmul", GMM)])
def test_matmul(fn, spec):
    c = lambda **k: call(fn, spec, **k)  # noqa: E731
    assert c(rows=0, y=None) == c(n=0, y=None) == OK
    for bad in ({"rows": -1}, {"rows": 1 << 31}, {"n": 8}, {"n": -16}, {"n": 1 << 24}, {"k": 48}, {"k": -32}, {"k": 1 << 24}):
        assert c(**bad) == E_SHAPE, bad
    for name in ("a_scales", "a_codes", "w_scales", "w_codes", "y"):
        assert c(**{name: None}) == E_NULL, name
    assert c(a_codes=buf(1, 8)) == c(w_codes=buf(3, 8)) == c(y=buf(4, 2)) == E_ALIGN
    for name in ("a_scales", "a_codes", "w_scales", "w_codes"):
        assert c(y=spec[name]) == E_ALIAS, name
    if spec is GMM:
        assert c(offsets=None) == E_NULL
        assert c(groups=0) == c(groups=4097) == c(groups=-1) == c(src_rows=-1) == E_SHAPE
        assert c(row_index=None) == E_SHAPE  # src_rows != rows
        assert c(offsets=buf(6, 4)) == c(row_index=buf(5, 4)) == E_ALIGN
        assert c(y=buf(5)) == c(y=buf(6)) == E_ALIAS


LIN = dict(x=buf(0), src_rows=40, row_index=buf(5), rows=64, offsets=buf(6), groups=3, w_scales=buf(2), w_codes=buf(3),
           n=48, k=96, workspace=buf(7), workspace_bytes=1 << 20, y=buf(4), stream=None)


@pytest.mark.parametrize("fn", ["trace_mx_linear", "trace_mx8_linear"])
def test_linear(fn):
    c = lambda **k: call(fn, LIN, **k)  # noqa: E731
    assert c(rows=0, y=None) == OK
    assert c(n=24) == c(k=16) == c(groups=5000) == c(row_index=None) == c(workspace_bytes=16) == E_SHAPE
    assert c(x=None) == c(workspace=None) == c(y=None) == c(w_codes=None) == c(offsets=None) == E_NULL
    assert c(x=buf(0, 2)) == c(workspace=buf(7, 8)) == E_ALIGN
    assert c(workspace=buf(0)) == c(workspace=buf(4)) == c(y=buf(7, 64)) == c(y=buf(0)) == E_ALIAS


def test_results_past_one_launch():
    at = [(1 << 44) + (i << 40) for i in range(5)]
    f = L.trace_mx_matmul
    assert f(at[0], at[1], (1 << 31) - 1, at[2], at[3], 16, 32, at[4], None) == E_SHAPE


def test_linear_workspace():
    f, f8 = L.trace_mx_linear_workspace_bytes, L.trace_mx8_linear_workspace_bytes
    assert f(40, 40, 0, 96) == 40 * 48 + 128 and f8(40, 40, 0, 96) == 40 * 96 + 128
    assert f(40, 64, 3, 96) == 40 * 48 + 128  # the tokens' record, not the packed rows'
    assert f(16, 16, 0, 96) == f8(1, 1, 0, 4096) == 0  # rounded by the product itself
    assert f(16, 16, 0, 4096) == 16 * 2048 + 2048 and f(24, 192, 128, 2048) == 24 * 1024 + 1536
    assert f(0, 0, 0, 96) == f(-1, 4, 0, 96) == f8(40, 40, 0, 40) == f(40, 40, 5000, 96) == 0


GX = dict(grad_y=buf(0), rows=64, offsets=buf(6), groups=3, w_scales=buf(2), w_codes=buf(3), n=48, k=96, mask=buf(5),
          grad_x=buf(4), stream=None)


def test_grad_input():
    c = lambda **k: call("trace_mx_matmul_bwd_input", GX, **k)  # noqa: E731
    assert c(rows=0) == c(k=0) == OK
    assert c(rows=-1) == c(n=40) == c(k=80) == c(groups=0) == c(groups=4097) == E_SHAPE
    assert c(grad_y=None) == c(w_scales=None) == c(w_codes=None) == c(grad_x=None) == c(offsets=None) == E_NULL
    assert c(grad_y=buf(0, 8)) == c(w_codes=buf(3, 8)) == c(mask=buf(5, 1)) == c(grad_x=buf(4, 8)) == E_ALIGN
    assert c(grad_x=buf(0)) == c(grad_x=buf(5)) == c(grad_x=buf(3)) == E_ALIAS


GW = dict(grad_y=buf(0), rows=64, offsets=buf(6), groups=3, a_scales=buf(1), a_codes=buf(2), src_rows=40,
          row_index=buf(5), n=48, k=96, mask=buf(7), grad_w=buf(4), workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("fn", ["trace_mx_matmul_bwd_weight", "trace_mx8_matmul_bwd_weight"])
def test_grad_weight(fn):
    c = lambda **k: call(fn, GW, **k)  # noqa: E731
    assert c(n=0) == c(k=0) == OK
    assert c(rows=-1) == c(n=40) == c(k=80) == c(groups=0) == c(groups=4097) == c(row_index=None) == E_SHAPE
    assert c(grad_y=None) == c(a_scales=None) == c(a_codes=None) == c(grad_w=None) == c(offsets=None) == E_NULL
    assert c(grad_y=buf(0, 8)) == c(a_codes=buf(2, 8)) == c(mask=buf(7, 1)) == c(grad_w=buf(4, 8)) == E_ALIGN
    assert c(grad_w=buf(0)) == c(grad_w=buf(7)) == c(grad_w=buf(2)) == c(grad_w=buf(5)) == E_ALIAS


def test_grad_weight_workspace():
    f = L.trace_mx_matmul_bwd_weight_workspace_bytes
    assert f(-1, 0, 64, 64) == f(8, 0, 40, 64) == f(8, 5000, 64, 64) == 0
    assert f(100, 8, 64, 64) == 0  # groups are not split
    need = f(16384, 0, 64, 64)
    assert need % (4 * 64 * 64) == 0
    if need:
        spec = dict(GW, offsets=None, groups=0, rows=16384, src_rows=16384, row_index=None, n=64, k=64, workspace=buf(8),
                    workspace_bytes=need)
        c = lambda **k: call("trace_mx_matmul_bwd_weight", spec, **k)  # noqa: E731
        assert c(workspace=None) == E_NULL and c(workspace_bytes=need - 1) == E_SHAPE
        assert c(workspace=buf(8, 8)) == E_ALIGN and c(workspace=buf(4)) == E_ALIAS


SORT = dict(ids=buf(0), tokens=1000, topk=8, experts=128, workspace=buf(1), workspace_bytes=1 << 20, offsets=buf(2),
            row_index=buf(3), slot=buf(4), stream=None)


def test_sort():
    c = lambda **k: call("trace_expert_sort", SORT, **k)  # noqa: E731
    for bad in ({"tokens": -1}, {"topk": 0}, {"topk": 65}, {"experts": 0}, {"experts": 1025}, {"tokens": 1 << 28},
                {"workspace_bytes": 4}):
        assert c(**bad) == E_SHAPE, bad
    for name in ("ids", "workspace", "offsets", "row_index", "slot"):
        assert c(**{name: None}) == E_NULL, name
        assert c(**{name: SORT[name] + 2}) == E_ALIGN, name
    for name in ("workspace", "offsets", "row_index", "slot"):
        assert c(**{name: buf(0)}) == E_ALIAS, name
    assert c(slot=buf(3)) == E_ALIAS
    f = L.trace_expert_sort_workspace_bytes
    assert f(256, 8, 128) == 0 and f(257, 8, 128) == 3 * 129 * 4 and f(-1, 8, 128) == f(4, 8, 2000) == 0
    assert f(32768, 8, 128) == 256 * 129 * 4 and f(32769, 8, 128) == 129 * 129 * 4


DISP = dict(x=buf(0), tokens=30, cols=48, row_index=buf(1), rows=60, out=buf(2), stream=None)
COMB = dict(y=buf(0), rows=60, cols=48, slot=buf(1), weights=buf(2), tokens=30, topk=2, out=buf(3), stream=None)
CBWD = dict(grad_out=buf(0), y=buf(1), rows=60, cols=48, slot=buf(2), weights=buf(3), tokens=30, topk=2, offsets=buf(4),
            groups=5, grad_y=buf(5), grad_weights=buf(6), stream=None)


def test_dispatch_and_combine():
    c = lambda **k: call("trace_expert_dispatch", DISP, **k)  # noqa: E731
    assert c(rows=0) == c(cols=0) == OK
    assert c(rows=-1) == c(tokens=-1) == c(cols=40) == c(cols=1 << 24) == E_SHAPE
    assert c(x=None) == c(row_index=None) == c(out=None) == E_NULL
    assert c(x=buf(0, 8)) == c(row_index=buf(1, 4)) == c(out=buf(2, 8)) == E_ALIGN
    assert c(out=buf(0)) == c(out=buf(1)) == E_ALIAS
    c = lambda **k: call("trace_expert_combine", COMB, **k)  # noqa: E731
    assert c(tokens=0) == c(cols=0) == OK
    assert c(rows=-1) == c(cols=40) == c(topk=0) == c(topk=65) == c(tokens=-1) == E_SHAPE
    assert c(y=None) == c(slot=None) == c(out=None) == E_NULL
    assert c(y=buf(0, 8)) == c(slot=buf(1, 4)) == c(weights=buf(2, 2)) == c(out=buf(3, 8)) == E_ALIGN
    assert c(out=buf(0)) == c(out=buf(1)) == c(out=buf(2)) == E_ALIAS


def test_combine_bwd():
    c = lambda **k: call("trace_expert_combine_bwd", CBWD, **k)  # noqa: E731
    assert c(tokens=0, rows=0) == c(tokens=0, offsets=None, groups=0) == OK
    assert c(rows=-1) == c(cols=40) == c(topk=0) == c(tokens=-1) == c(groups=0) == c(groups=4097) == E_SHAPE
    for name in ("grad_out", "y", "slot", "offsets", "grad_y", "grad_weights"):
        assert c(**{name: None}) == E_NULL, name
    for name in ("grad_out", "y", "slot", "weights", "offsets", "grad_y", "grad_weights"):
        assert c(**{name: CBWD[name] + 2}) == E_ALIGN, name
    for name in ("grad_out", "y", "slot", "weights", "offsets"):
        assert c(grad_y=CBWD[name]) == E_ALIAS and c(grad_weights=CBWD[name]) == E_ALIAS, name
    assert c(grad_y=buf(6)) == E_ALIAS


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(128, dtype=torch.uint8)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    for f in (lambda: tr.mx_quantize(x), lambda: tr.mx8_quantize(x), lambda: tr.mx_linear(x, u8, u8, 16),
              lambda: tr.mx_matmul(u8, u8, u8, u8, 16, 64), lambda: tr.mx_matmul_bwd_input(x, u8, u8, 64),
              lambda: tr.mx_matmul_bwd_weight(x, u8, u8, 64), lambda: tr.expert_sort(ids, 4),
              lambda: tr.expert_dispatch(x, ids), lambda: tr.expert_combine(x, ids)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    with pytest.raises(ValueError, match="offsets is required"):
        tr.grouped_mx_matmul(u8, u8, None, u8, u8, 16, 64)
