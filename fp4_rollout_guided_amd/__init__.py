"""Python binding for libtrace (rollout-guided FP4 rounding on MI355X).

Argument marshalling only: every step of the path runs in the HIP kernels of
``libtrace.so`` (built by ``python fp4_rollout_guided_amd/build.py``).  PyTorch
supplies device memory and the current stream.  There is no CPU fallback:
importing this package fails if the library has not been built.

Functions mirror the C ABI in ``include/trace.h``:

    tensor_scale(x)                                  -> ts (fp32[1])
    tensor_scale_noalloc(x)                          -> ts, without a workspace
    capture(x_roll, ts, want_codes=False)            -> (scales, bits, codes)
    guided_fakequant_fwd(x_train, scales, ts, bits)  -> (y, mask, qcodes)
    rne_fakequant_fwd(x_train, scales, ts)           -> (y, mask, qcodes)
    full_info_fakequant_fwd(x_train, scales, ts, codes) -> (y, mask, qcodes)
    gather_records(bits, scales, codes, cols, row_index) -> (bits, scales, codes)
    grouped_tensor_scale(x, offsets)                 -> ts (fp32[groups])
    grouped_capture / grouped_guided_fakequant_fwd / grouped_rne_fakequant_fwd /
    grouped_full_info_fakequant_fwd: as above, with one tensor scale per group
    of rows (per-expert scales of packed MoE rows; offsets int64[groups + 1])
    mx_capture / mx_guided_fakequant_fwd / mx_rne_fakequant_fwd /
    mx_full_info_fakequant_fwd: the MXFP4 variant (32-element blocks, E8M0
    scales, no tensor scale)
    mx8_capture / mx8_guided_fakequant_fwd / mx8_rne_fakequant_fwd /
    mx8_full_info_fakequant_fwd: the MXFP8 (E4M3) activation grid of the W4A8
    setting (32-element blocks, E8M0 scales, one code byte per element)
    tensor_scale_batch(xs)                           -> [ts, ...] (up to 8 sites, one pass)
    capture_batch(xs, tss, want_codes=False)         -> [(scales, bits, codes), ...] (one launch)
    capture_lowbits(x_roll, ts, nbits)               -> (scales, planes, codes)
    lowbits_fakequant_fwd(x_train, scales, ts, nbits, planes) -> (y, mask, qcodes)
    ste_bwd(grad_out, mask)                          -> grad_in
    mismatch_stats(x_train, scales, ts, bits, codes, stats=None) -> stats (int64[20], added to)

products of the rounded operands (weights in MXFP4; activations in MXFP4, or
in MXFP8 with the mx8_ forms; grouped_ forms: one weight per group of rows):

    mx_quantize(x, want_mask=False)                  -> (scales, codes, mask)   (and mx8_quantize)
    mx_matmul(a_scales, a_codes, w_scales, w_codes, n, k) -> y bf16 [rows, n]   (mx8_, grouped_)
    mx_linear(x, w_scales, w_codes, n)               -> y: quantise, then multiply (mx8_, grouped_)
    mx_matmul_bwd_input(grad_y, w_scales, w_codes, k, mask=None)  -> grad_x     (grouped_)
    mx_matmul_bwd_weight(grad_y, a_scales, a_codes, k, mask=None) -> grad_w     (mx8_, grouped_)

routed rows (the groups of the grouped_ forms):

    expert_sort(ids, experts)                        -> (offsets, row_index, slot)
    expert_dispatch(x, row_index)                    -> packed rows
    expert_combine(y, slot, weights=None)            -> the tokens' weighted sums (y bf16, or fp32 from the grouped_
                                                        products with dtype=torch.float32)
    expert_combine_bwd(grad_out, y, slot, weights, offsets=None) -> (grad_y, grad_weights)

the rest of a policy's training step:

    expert_route(logits, topk, renormalize=True, valid=None) -> (ids, weights, counts, probs, balance): the router's
                                                        choices for expert_sort and expert_combine, the balance loss
    expert_route_bwd(grad_weights, grad_balance, logits, ids, weights, counts) -> grad_logits
    linear_cross_entropy(x, w, targets, scale=1.0)   -> (loss, lse) of the logits scale * x W^T, which are not kept
    linear_cross_entropy_bwd(grad_loss, x, w, targets, lse, scale=1.0) -> (grad_x, grad_w)
    adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr) -> one AdamW step over many tensors, in place, states
                                                        in fp32 or as MXFP8 records

and ``GuidedFakeQuant``, ``MxMatmul``, ``ExpertDispatch``, ``ExpertCombine``,
``ExpertRoute`` and ``LinearCrossEntropy`` wrap the forward/backward pairs as
autograd functions; ``AdamW`` keeps the optimiser's states.
"""
import ctypes
import importlib
import math
import os
from array import array

import torch
from torch.autograd.function import once_differentiable

__all__ = [
    "TraceError", "LIB_PATH", "SMALLGRID_LIB_PATH", "lib", "load_library", "abi_version", "abi_revision",
    "tensor_scale", "tensor_scale_noalloc", "capture",
    "guided_fakequant_fwd", "rne_fakequant_fwd", "full_info_fakequant_fwd", "ste_bwd", "gather_records",
    "gathered_guided_fakequant_fwd", "gathered_rne_fakequant_fwd", "gathered_full_info_fakequant_fwd",
    "grouped_tensor_scale", "grouped_capture", "grouped_guided_fakequant_fwd", "grouped_rne_fakequant_fwd",
    "grouped_full_info_fakequant_fwd", "mx_capture", "mx_guided_fakequant_fwd", "mx_rne_fakequant_fwd",
    "mx_full_info_fakequant_fwd", "mx8_capture", "mx8_guided_fakequant_fwd", "mx8_rne_fakequant_fwd",
    "mx8_full_info_fakequant_fwd", "capture_lowbits", "lowbits_fakequant_fwd", "mismatch_stats", "STAT_FIELDS",
    "GuidedFakeQuant", "tensor_scale_batch", "capture_batch", "MAX_BATCH_SITES",
    "mx_quantize", "mx8_quantize", "mx_matmul", "mx8_matmul", "grouped_mx_matmul", "grouped_mx8_matmul", "mx_linear",
    "mx8_linear", "grouped_mx_linear", "grouped_mx8_linear", "mx_matmul_bwd_input", "grouped_mx_matmul_bwd_input",
    "mx_matmul_bwd_weight", "mx8_matmul_bwd_weight", "grouped_mx_matmul_bwd_weight", "grouped_mx8_matmul_bwd_weight",
    "expert_sort", "expert_dispatch", "expert_combine", "expert_combine_bwd", "MxMatmul", "ExpertDispatch",
    "ExpertCombine", "MAX_EXPERTS", "MAX_TOPK", "MAX_PRODUCT_GROUPS",
    "expert_route", "expert_route_bwd", "ExpertRoute", "linear_cross_entropy", "linear_cross_entropy_bwd",
    "LinearCrossEntropy", "adamw_step", "AdamW", "step_revision",
    "STATUS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtrace.so")
# the same sources with tiny grid caps, for the tests of the grid-stride paths
SMALLGRID_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtrace_smallgrid.so")

STATUS = {0: "TRACE_OK", 1: "TRACE_E_NULL", 2: "TRACE_E_SHAPE", 3: "TRACE_E_ALIGN",
          4: "TRACE_E_ALIAS", 5: "TRACE_E_HIP"}


class TraceError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = lib.trace_status_string(status).decode()
        if status == 5:
            msg += f" (hipError_t {lib.trace_last_hip_error()})"
        super().__init__(f"{what}: {msg}")


def load_library(path):
    """Load a libtrace build and declare its entry points' signatures."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python fp4_rollout_guided_amd/build.py` "
            "(libtrace has no CPU fallback)")
    L = ctypes.CDLL(path)
    p, i64, st, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "trace_abi_version": ([], ctypes.c_int),
        "trace_abi_revision": ([], ctypes.c_int),
        "trace_status_string": ([st], ctypes.c_char_p),
        "trace_last_hip_error": ([], ctypes.c_int),
        "trace_tensor_scale_workspace_bytes": ([i64], sz),
        "trace_tensor_scale": ([p, i64, p, sz, p, p], st),
        "trace_tensor_scale_noalloc": ([p, i64, p, p], st),
        "trace_capture": ([p, i64, i64, p, p, p, p, p], st),
        "trace_guided_fakequant_fwd": ([p, i64, i64, p, p, p, p, p, p, p], st),
        "trace_rne_fakequant_fwd": ([p, i64, i64, p, p, p, p, p, p], st),
        "trace_full_info_fakequant_fwd": ([p, i64, i64, p, p, p, p, p, p, p], st),
        "trace_ste_bwd": ([p, p, i64, p, p], st),
        "trace_gather_records": ([p, p, p, i64, i64, p, i64, p, p, p, p], st),
        "trace_gathered_guided_fakequant_fwd": ([p, i64, i64, p, i64, p, i64, p, p, p, p, p, p, p], st),
        "trace_gathered_full_info_fakequant_fwd": ([p, i64, i64, p, i64, p, i64, p, p, p, p, p, p, p], st),
        "trace_gathered_rne_fakequant_fwd": ([p, i64, i64, p, i64, p, i64, p, p, p, p, p, p], st),
        "trace_grouped_tensor_scale_workspace_bytes": ([i64], sz),
        "trace_grouped_tensor_scale": ([p, i64, i64, p, i64, p, sz, p, p], st),
        "trace_grouped_capture": ([p, i64, i64, p, i64, p, p, p, p, p], st),
        "trace_grouped_guided_fakequant_fwd": ([p, i64, i64, p, i64, p, p, p, p, p, p, p], st),
        "trace_grouped_rne_fakequant_fwd": ([p, i64, i64, p, i64, p, p, p, p, p, p], st),
        "trace_grouped_full_info_fakequant_fwd": ([p, i64, i64, p, i64, p, p, p, p, p, p, p], st),
        "trace_mx_capture": ([p, i64, i64, p, p, p, p], st),
        "trace_capture_lowbits": ([p, i64, i64, p, ctypes.c_int32, p, p, p, p], st),
        "trace_lowbits_fakequant_fwd": ([p, i64, i64, p, p, ctypes.c_int32, p, p, p, p, p], st),
        "trace_mx_guided_fakequant_fwd": ([p, i64, i64, p, p, p, p, p, p], st),
        "trace_mx_rne_fakequant_fwd": ([p, i64, i64, p, p, p, p, p], st),
        "trace_mx_full_info_fakequant_fwd": ([p, i64, i64, p, p, p, p, p, p], st),
        "trace_mx8_capture": ([p, i64, i64, p, p, p, p], st),
        "trace_mismatch_stats": ([p, i64, i64, p, p, p, p, p, p], st),
        "trace_mx8_guided_fakequant_fwd": ([p, i64, i64, p, p, p, p, p, p], st),
        "trace_mx8_rne_fakequant_fwd": ([p, i64, i64, p, p, p, p, p], st),
        "trace_mx8_full_info_fakequant_fwd": ([p, i64, i64, p, p, p, p, p, p], st),
        "trace_tensor_scale_batch_workspace_bytes": ([p, ctypes.c_int32], sz),
        "trace_tensor_scale_batch": ([p, ctypes.c_int32, p, sz, p], st),
        "trace_capture_batch": ([p, ctypes.c_int32, p], st),
        "trace_mx_quantize": ([p, i64, i64, p, p, p, p], st),
        "trace_mx_matmul": ([p, p, i64, p, p, i64, i64, p, p], st),
        "trace_grouped_mx_matmul": ([p, p, i64, p, i64, p, i64, p, p, i64, i64, p, p], st),
        "trace_mx_linear_workspace_bytes": ([i64, i64, i64, i64], sz),
        "trace_mx_linear": ([p, i64, p, i64, p, i64, p, p, i64, i64, p, sz, p, p], st),
        "trace_mx_matmul_bwd_input": ([p, i64, p, i64, p, p, i64, i64, p, p, p], st),
        "trace_mx_matmul_bwd_weight_workspace_bytes": ([i64, i64, i64, i64], sz),
        "trace_mx_matmul_bwd_weight": ([p, i64, p, i64, p, p, i64, p, i64, i64, p, p, p, sz, p], st),
        "trace_expert_sort_workspace_bytes": ([i64, i64, i64], sz),
        "trace_expert_sort": ([p, i64, i64, i64, p, sz, p, p, p, p], st),
        "trace_expert_dispatch": ([p, i64, i64, p, i64, p, p], st),
        "trace_expert_combine": ([p, i64, i64, p, p, i64, i64, p, p], st),
        "trace_expert_combine_bwd": ([p, p, i64, i64, p, p, i64, i64, p, i64, p, p, p], st),
        "trace_step_revision": ([], ctypes.c_int),
        "trace_linear_cross_entropy_workspace_bytes": ([i64, i64, i64], sz),
        "trace_linear_cross_entropy": ([p, p, p, i64, i64, i64, ctypes.c_float, p, sz, p, p, p], st),
        "trace_linear_cross_entropy_bwd_workspace_bytes": ([i64, i64, i64], sz),
        "trace_linear_cross_entropy_bwd": ([p, p, p, p, p, i64, i64, i64, ctypes.c_float, p, sz, p, p, p], st),
        "trace_expert_route_workspace_bytes": ([i64, i64], sz),
        "trace_expert_route": ([p, p, i64, i64, i64, ctypes.c_int, p, sz, p, p, p, p, p, p], st),
        "trace_expert_route_bwd": ([p, p, p, p, p, p, i64, i64, i64, ctypes.c_int, p, p], st),
        "trace_adamw_step": ([p, ctypes.c_int32, p, p, p], st),
    }
    for name in ("quantize", "matmul", "linear_workspace_bytes", "linear", "matmul_bwd_weight"):
        sig["trace_mx8_" + name] = sig["trace_mx_" + name]
    sig["trace_grouped_mx8_matmul"] = sig["trace_grouped_mx_matmul"]
    for name, like in (("grouped_mx_matmul", "grouped_mx_matmul"), ("grouped_mx8_matmul", "grouped_mx_matmul"),
                       ("grouped_mx_linear", "mx_linear"), ("grouped_mx8_linear", "mx_linear"),
                       ("grouped_mx_matmul_bwd_input", "mx_matmul_bwd_input"), ("expert_combine", "expert_combine"),
                       ("expert_route", "expert_route"), ("expert_route_bwd", "expert_route_bwd")):
        sig[f"trace_{name}_f32"] = sig["trace_" + like]  # the same on fp32 rows
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


lib = load_library(LIB_PATH)
try:
    _tensor_lists = importlib.import_module(__name__ + "._tensor_lists")
except ImportError as e:
    class _Missing:
        """In the module's place: everything that does not use it is there all the same."""

        def __init__(self, why):
            self._why = why

        def __getattr__(self, name):
            raise ImportError(f"{self._why}: build it with `python fp4_rollout_guided_amd/build.py`")

    _tensor_lists = _Missing(str(e))


def abi_version() -> int:
    return lib.trace_abi_version()


def abi_revision() -> int:
    """Additions within ``abi_version``: 1 has the products and the routed rows."""
    return lib.trace_abi_revision()


def step_revision() -> int:
    """1: the library has the router, the vocabulary loss and the optimiser step."""
    return lib.trace_step_revision()


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _bf16(t, name):
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{name} must be bf16 (or its raw 16-bit pattern), got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_I64 = (torch.int64,)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _arg(t, name, like, dtypes, numel):
    """Check a tensor argument before its pointer reaches the C ABI (which
    sees no sizes or devices): on ``like``'s device, contiguous, of one of
    ``dtypes``, and holding at least ``numel`` elements.  A host tensor
    beside device data, or a short buffer, would otherwise be read or
    written out of bounds by a kernel."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device} (the data's device), got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} needs at least {numel} elements, got {t.numel()}")
    return t


def _rows_cols(t):
    cols = t.shape[-1] if t.dim() > 0 else 1
    rows = t.numel() // cols if cols else 0
    return rows, cols


def _u8(n, like, out, name):
    if out is None:
        return torch.empty(n, dtype=torch.uint8, device=like.device)
    return _arg(out, name, like, _U8, n)


def _bf16_out(out, like, n, name):
    if out is None:
        return torch.empty_like(like)
    return _arg(out, name, like, _BF16, n)


def _check(status, what):
    if status != 0:
        raise TraceError(status, what)


# --------------------------------------------------------------------------
# entry points
# --------------------------------------------------------------------------

def tensor_scale(x, out=None, workspace=None):
    """ts = fl32(max|x| / 2688) as a float32[1] device tensor."""
    _bf16(x, "x")
    n = x.numel()
    need = lib.trace_tensor_scale_workspace_bytes(n)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _arg(workspace, "workspace", x, _U8, need)
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    _arg(out, "out", x, _F32, 1)
    _check(lib.trace_tensor_scale(_ptr(x), n, _ptr(workspace), workspace.numel(), _ptr(out), _stream(x)),
           "trace_tensor_scale")
    return out


def tensor_scale_noalloc(x, out=None):
    """``tensor_scale`` without a workspace: the library's per-GPU scratch
    array holds the partial maxima (for callers that cannot allocate; calls
    that overlap on one GPU race)."""
    _bf16(x, "x")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    _arg(out, "out", x, _F32, 1)
    _check(lib.trace_tensor_scale_noalloc(_ptr(x), x.numel(), _ptr(out), _stream(x)), "trace_tensor_scale_noalloc")
    return out


def capture(x_roll, ts, want_codes=False, scales=None, bits=None, codes=None):
    """Compact rollout record of one site tensor: (scales u8[n/16],
    bits u8[n/8], codes u8[n/2] or None)."""
    _bf16(x_roll, "x_roll")
    rows, cols = _rows_cols(x_roll)
    n = rows * cols
    _arg(ts, "ts", x_roll, _F32, 1)
    scales = _u8(n // 16, x_roll, scales, "scales")
    bits = _u8(n // 8, x_roll, bits, "bits")
    if want_codes or codes is not None:
        codes = _u8(n // 2, x_roll, codes, "codes")
    _check(lib.trace_capture(_ptr(x_roll), rows, cols, _ptr(ts), _ptr(scales), _ptr(bits), _ptr(codes),
                             _stream(x_roll)), "trace_capture")
    return scales, bits, codes


class _Site(ctypes.Structure):
    """trace_site of include/trace.h."""
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ts", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("bits", ctypes.c_void_p),
                ("codes", ctypes.c_void_p)]


MAX_BATCH_SITES = 8


def _sites(xs, tss, records=None):
    if len(xs) > MAX_BATCH_SITES:
        raise ValueError(f"at most {MAX_BATCH_SITES} sites per batch, got {len(xs)}")
    arr = (_Site * max(1, len(xs)))()
    if len(tss) != len(xs) or (records is not None and len(records) != len(xs)):
        raise ValueError("one tensor scale (and record) per site is required")
    for i, x in enumerate(xs):
        _bf16(x, f"xs[{i}]")
        rows, cols = _rows_cols(x)
        n = rows * cols
        _arg(tss[i], f"ts[{i}]", x, _F32, 1)
        sc, bt, cd = records[i] if records is not None else (None, None, None)
        if records is not None:
            _arg(sc, f"scales[{i}]", x, _U8, n // 16)
            _arg(bt, f"bits[{i}]", x, _U8, n // 8)
            if cd is not None:
                _arg(cd, f"codes[{i}]", x, _U8, n // 2)
        arr[i] = _Site(x.data_ptr() if x.numel() else None, rows, cols, tss[i].data_ptr(),
                       None if sc is None else sc.data_ptr(), None if bt is None else bt.data_ptr(),
                       None if cd is None else cd.data_ptr())
    return arr


def tensor_scale_batch(xs, outs=None, workspace=None):
    """Tensor scales of up to 8 site tensors in one pass: a list of
    float32[1] device tensors, each equal to tensor_scale(x)."""
    if not xs:
        return []
    dev = xs[0].device
    outs = outs if outs is not None else [torch.empty(1, dtype=torch.float32, device=dev) for _ in xs]
    arr = _sites(xs, outs)
    need = lib.trace_tensor_scale_batch_workspace_bytes(arr, len(xs))
    if workspace is None:
        workspace = torch.empty(max(4, need), dtype=torch.uint8, device=dev)
    _arg(workspace, "workspace", xs[0], _U8, need)
    _check(lib.trace_tensor_scale_batch(arr, len(xs), _ptr(workspace), workspace.numel(), _stream(xs[0])),
           "trace_tensor_scale_batch")
    return outs


def capture_batch(xs, tss, want_codes=False, records=None):
    """Compact records of up to 8 site tensors in one launch: a list of
    (scales, bits, codes or None), each equal to capture(x, ts)."""
    if not xs:
        return []
    if records is None:
        records = []
        for x in xs:
            n = x.numel()
            records.append((_u8(n // 16, x, None, "scales"), _u8(n // 8, x, None, "bits"),
                            _u8(n // 2, x, None, "codes") if want_codes else None))
    arr = _sites(xs, tss, records)
    _check(lib.trace_capture_batch(arr, len(xs), _stream(xs[0])), "trace_capture_batch")
    return records


def _fwd(mode, x, scales, ts, side, y, mask, want_codes, qcodes):
    _bf16(x, "x_train")
    rows, cols = _rows_cols(x)
    n = rows * cols
    _arg(scales, "scales", x, _U8, n // 16)
    _arg(ts, "ts", x, _F32, 1)
    if mode != "rne":
        _arg(side, "bits" if mode == "guided" else "codes", x, _U8, n // 8 if mode == "guided" else n // 2)
    y = _bf16_out(y, x, n, "y")
    mask = _u8(n // 8, x, mask, "mask")
    if want_codes or qcodes is not None:
        qcodes = _u8(n // 2, x, qcodes, "qcodes")
    if mode == "guided":
        st = lib.trace_guided_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), _ptr(ts), _ptr(side), _ptr(y),
                                            _ptr(mask), _ptr(qcodes), _stream(x))
    elif mode == "full":
        st = lib.trace_full_info_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), _ptr(ts), _ptr(side), _ptr(y),
                                               _ptr(mask), _ptr(qcodes), _stream(x))
    else:
        st = lib.trace_rne_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), _ptr(ts), _ptr(y), _ptr(mask),
                                         _ptr(qcodes), _stream(x))
    _check(st, {"guided": "trace_guided_fakequant_fwd", "full": "trace_full_info_fakequant_fwd",
                "rne": "trace_rne_fakequant_fwd"}[mode])
    return y, mask, qcodes


def guided_fakequant_fwd(x_train, scales, ts, bits, y=None, mask=None, want_codes=False, qcodes=None):
    """Rollout-guided fake-quant forward: (y bf16, mask u8[n/8], qcodes)."""
    return _fwd("guided", x_train, scales, ts, bits, y, mask, want_codes, qcodes)


def rne_fakequant_fwd(x_train, scales, ts, y=None, mask=None, want_codes=False, qcodes=None):
    """Plain round-to-nearest-even fake-quant forward: (y, mask, qcodes)."""
    return _fwd("rne", x_train, scales, ts, None, y, mask, want_codes, qcodes)


def full_info_fakequant_fwd(x_train, scales, ts, codes, y=None, mask=None, want_codes=False, qcodes=None):
    """Full-information guided forward from the rollout's 4-bit codes: (y, mask, qcodes)."""
    return _fwd("full", x_train, scales, ts, codes, y, mask, want_codes, qcodes)


def ste_bwd(grad_out, mask, grad_in=None):
    """Straight-through estimator backward: grad_out where mask is set."""
    _bf16(grad_out, "grad_out")
    n = grad_out.numel()
    _arg(mask, "mask", grad_out, _U8, n // 8)
    grad_in = _bf16_out(grad_in, grad_out, n, "grad_in")
    _check(lib.trace_ste_bwd(_ptr(grad_out), _ptr(mask), grad_out.numel(), _ptr(grad_in), _stream(grad_out)),
           "trace_ste_bwd")
    return grad_in


def gather_records(bits, scales, codes, cols, row_index):
    """Records in the trainer's row order: row r of the result is source row
    row_index[r] (int64 device tensor); out-of-range indices give zero rows."""
    if not row_index.is_cuda or row_index.dtype != torch.int64 or not row_index.is_contiguous():
        raise ValueError("row_index must be a contiguous int64 device tensor")
    src_rows = scales.numel() * 16 // cols if cols else 0
    dst_rows = row_index.numel()
    n = dst_rows * cols
    n_src = src_rows * cols
    _arg(scales, "scales", row_index, _U8, n_src // 16)
    _arg(bits, "bits", row_index, _U8, n_src // 8)
    if codes is not None:
        _arg(codes, "codes", row_index, _U8, n_src // 2)
    bits_d = torch.empty(n // 8, dtype=torch.uint8, device=bits.device)
    scales_d = torch.empty(n // 16, dtype=torch.uint8, device=bits.device)
    codes_d = torch.empty(n // 2, dtype=torch.uint8, device=bits.device) if codes is not None else None
    _check(lib.trace_gather_records(_ptr(bits), _ptr(scales), _ptr(codes), src_rows, cols, _ptr(row_index),
                                    dst_rows, _ptr(bits_d), _ptr(scales_d), _ptr(codes_d), _stream(bits)),
           "trace_gather_records")
    return bits_d, scales_d, codes_d


def _gathered_fwd(mode, x, row_index, scales, ts, side, offsets, y, mask, want_codes, qcodes):
    _bf16(x, "x_train")
    rows, cols = _rows_cols(x)
    _arg(row_index, "row_index", x, _I64, rows)
    if row_index.numel() != rows:
        raise ValueError(f"row_index needs one entry per row of x_train ({rows}), got {row_index.numel()}")
    _arg(scales, "scales", x, _U8, 0)
    src_rows = scales.numel() * 16 // cols if cols else 0
    n, n_src = rows * cols, src_rows * cols
    groups = 0
    if offsets is not None:
        groups = _offsets(offsets, x)
    _arg(ts, "ts", x, _F32, max(groups, 1))
    if mode != "rne":
        _arg(side, "bits" if mode == "guided" else "codes", x, _U8, n_src // 8 if mode == "guided" else n_src // 2)
    y = _bf16_out(y, x, n, "y")
    mask = _u8(n // 8, x, mask, "mask")
    if want_codes or qcodes is not None:
        qcodes = _u8(n // 2, x, qcodes, "qcodes")
    head = (_ptr(x), rows, cols, _ptr(row_index), src_rows, _ptr(offsets), groups, _ptr(scales), _ptr(ts))
    tail = (_ptr(y), _ptr(mask), _ptr(qcodes), _stream(x))
    name = {"guided": "trace_gathered_guided_fakequant_fwd", "full": "trace_gathered_full_info_fakequant_fwd",
            "rne": "trace_gathered_rne_fakequant_fwd"}[mode]
    fn = getattr(lib, name)
    _check(fn(*head, *tail) if mode == "rne" else fn(*head, _ptr(side), *tail), name)
    return y, mask, qcodes


def gathered_guided_fakequant_fwd(x_train, row_index, scales, ts, bits, offsets=None, y=None, mask=None,
                                  want_codes=False, qcodes=None):
    """``guided_fakequant_fwd`` of x_train row r on source row row_index[r]
    of the record (scales, bits; the source's row count is
    scales.numel() * 16 / cols) without a gathered copy; ts is one tensor
    scale, or one per group of source rows when ``offsets`` is given.
    Out-of-range indices give zero-scale blocks."""
    return _gathered_fwd("guided", x_train, row_index, scales, ts, bits, offsets, y, mask, want_codes, qcodes)


def gathered_rne_fakequant_fwd(x_train, row_index, scales, ts, offsets=None, y=None, mask=None, want_codes=False,
                               qcodes=None):
    """``rne_fakequant_fwd`` on source rows row_index[r] of the record's
    scale bytes, as ``gathered_guided_fakequant_fwd``."""
    return _gathered_fwd("rne", x_train, row_index, scales, ts, None, offsets, y, mask, want_codes, qcodes)


def gathered_full_info_fakequant_fwd(x_train, row_index, scales, ts, codes, offsets=None, y=None, mask=None,
                                     want_codes=False, qcodes=None):
    """``full_info_fakequant_fwd`` on source rows row_index[r] of the record
    (scales, codes), as ``gathered_guided_fakequant_fwd``."""
    return _gathered_fwd("full", x_train, row_index, scales, ts, codes, offsets, y, mask, want_codes, qcodes)


def _offsets(offsets, x):
    _arg(offsets, "offsets", x, _I64, 2)
    if offsets.dim() != 1:
        raise ValueError("offsets must be a 1-D int64 device tensor of groups + 1 entries")
    groups = offsets.numel() - 1
    if groups < 1:
        raise ValueError("at least one group is required")
    return groups


def grouped_tensor_scale(x, offsets, out=None, workspace=None):
    """One tensor scale per group of rows: ts[g] = fl32(amax over rows
    [offsets[g], offsets[g+1]) / 2688), as a float32[groups] device tensor."""
    _bf16(x, "x")
    rows, cols = _rows_cols(x)
    groups = _offsets(offsets, x)
    need = lib.trace_grouped_tensor_scale_workspace_bytes(rows)
    if workspace is None:
        workspace = torch.empty(max(need, 4), dtype=torch.uint8, device=x.device)
    _arg(workspace, "workspace", x, _U8, need)
    if out is None:
        out = torch.empty(groups, dtype=torch.float32, device=x.device)
    _arg(out, "out", x, _F32, groups)
    _check(lib.trace_grouped_tensor_scale(_ptr(x), rows, cols, _ptr(offsets), groups, _ptr(workspace),
                                          workspace.numel(), _ptr(out), _stream(x)), "trace_grouped_tensor_scale")
    return out


def grouped_capture(x_roll, offsets, ts, want_codes=False, scales=None, bits=None, codes=None):
    """``capture`` with ts[group of the row] as each row's tensor scale."""
    _bf16(x_roll, "x_roll")
    rows, cols = _rows_cols(x_roll)
    groups = _offsets(offsets, x_roll)
    n = rows * cols
    _arg(ts, "ts", x_roll, _F32, groups)
    scales = _u8(n // 16, x_roll, scales, "scales")
    bits = _u8(n // 8, x_roll, bits, "bits")
    if want_codes or codes is not None:
        codes = _u8(n // 2, x_roll, codes, "codes")
    _check(lib.trace_grouped_capture(_ptr(x_roll), rows, cols, _ptr(offsets), groups, _ptr(ts), _ptr(scales),
                                     _ptr(bits), _ptr(codes), _stream(x_roll)), "trace_grouped_capture")
    return scales, bits, codes


def _grouped_fwd(mode, x, offsets, scales, ts, side, y, mask, want_codes, qcodes):
    _bf16(x, "x_train")
    rows, cols = _rows_cols(x)
    groups = _offsets(offsets, x)
    n = rows * cols
    _arg(scales, "scales", x, _U8, n // 16)
    _arg(ts, "ts", x, _F32, groups)
    if mode != "rne":
        _arg(side, "bits" if mode == "guided" else "codes", x, _U8, n // 8 if mode == "guided" else n // 2)
    y = _bf16_out(y, x, n, "y")
    mask = _u8(n // 8, x, mask, "mask")
    if want_codes or qcodes is not None:
        qcodes = _u8(n // 2, x, qcodes, "qcodes")
    head = (_ptr(x), rows, cols, _ptr(offsets), groups, _ptr(scales), _ptr(ts))
    tail = (_ptr(y), _ptr(mask), _ptr(qcodes), _stream(x))
    if mode == "guided":
        st, name = lib.trace_grouped_guided_fakequant_fwd(*head, _ptr(side), *tail), "trace_grouped_guided_fakequant_fwd"
    elif mode == "full":
        st, name = (lib.trace_grouped_full_info_fakequant_fwd(*head, _ptr(side), *tail),
                    "trace_grouped_full_info_fakequant_fwd")
    else:
        st, name = lib.trace_grouped_rne_fakequant_fwd(*head, *tail), "trace_grouped_rne_fakequant_fwd"
    _check(st, name)
    return y, mask, qcodes


def grouped_guided_fakequant_fwd(x_train, offsets, scales, ts, bits, y=None, mask=None, want_codes=False,
                                 qcodes=None):
    """``guided_fakequant_fwd`` with one tensor scale per group of rows."""
    return _grouped_fwd("guided", x_train, offsets, scales, ts, bits, y, mask, want_codes, qcodes)


def grouped_rne_fakequant_fwd(x_train, offsets, scales, ts, y=None, mask=None, want_codes=False, qcodes=None):
    """``rne_fakequant_fwd`` with one tensor scale per group of rows."""
    return _grouped_fwd("rne", x_train, offsets, scales, ts, None, y, mask, want_codes, qcodes)


def grouped_full_info_fakequant_fwd(x_train, offsets, scales, ts, codes, y=None, mask=None, want_codes=False,
                                    qcodes=None):
    """``full_info_fakequant_fwd`` with one tensor scale per group of rows."""
    return _grouped_fwd("full", x_train, offsets, scales, ts, codes, y, mask, want_codes, qcodes)


def capture_lowbits(x_roll, ts, nbits, want_codes=False, scales=None, planes=None, codes=None):
    """Capture keeping b = nbits low bits per element: (scales u8[n/16],
    planes u8[nbits * n/8], codes or None)."""
    _bf16(x_roll, "x_roll")
    rows, cols = _rows_cols(x_roll)
    n = rows * cols
    _arg(ts, "ts", x_roll, _F32, 1)
    scales = _u8(n // 16, x_roll, scales, "scales")
    planes = _u8(max(0, nbits) * (n // 8), x_roll, planes, "planes")
    if want_codes or codes is not None:
        codes = _u8(n // 2, x_roll, codes, "codes")
    _check(lib.trace_capture_lowbits(_ptr(x_roll), rows, cols, _ptr(ts), nbits, _ptr(scales), _ptr(planes),
                                     _ptr(codes), _stream(x_roll)), "trace_capture_lowbits")
    return scales, planes, codes


def lowbits_fakequant_fwd(x_train, scales, ts, nbits, planes, y=None, mask=None, want_codes=False, qcodes=None):
    """Guided forward from b = nbits cached low bits: (y, mask, qcodes)."""
    _bf16(x_train, "x_train")
    rows, cols = _rows_cols(x_train)
    n = rows * cols
    _arg(scales, "scales", x_train, _U8, n // 16)
    _arg(ts, "ts", x_train, _F32, 1)
    _arg(planes, "planes", x_train, _U8, max(0, nbits) * (n // 8))
    y = _bf16_out(y, x_train, n, "y")
    mask = _u8(n // 8, x_train, mask, "mask")
    if want_codes or qcodes is not None:
        qcodes = _u8(n // 2, x_train, qcodes, "qcodes")
    _check(lib.trace_lowbits_fakequant_fwd(_ptr(x_train), rows, cols, _ptr(scales), _ptr(ts), nbits, _ptr(planes),
                                           _ptr(y), _ptr(mask), _ptr(qcodes), _stream(x_train)),
           "trace_lowbits_fakequant_fwd")
    return y, mask, qcodes


def mx_capture(x_roll, want_codes=False, scales=None, bits=None, codes=None):
    """MXFP4 capture: (scales u8[n/32] E8M0, bits u8[n/8], codes u8[n/2] or None)."""
    _bf16(x_roll, "x_roll")
    rows, cols = _rows_cols(x_roll)
    n = rows * cols
    scales = _u8(n // 32, x_roll, scales, "scales")
    bits = _u8(n // 8, x_roll, bits, "bits")
    if want_codes or codes is not None:
        codes = _u8(n // 2, x_roll, codes, "codes")
    _check(lib.trace_mx_capture(_ptr(x_roll), rows, cols, _ptr(scales), _ptr(bits), _ptr(codes), _stream(x_roll)),
           "trace_mx_capture")
    return scales, bits, codes


def _mx_fwd(mode, x, scales, side, y, mask, want_codes, qcodes):
    _bf16(x, "x_train")
    rows, cols = _rows_cols(x)
    n = rows * cols
    _arg(scales, "scales", x, _U8, n // 32)
    if mode != "rne":
        _arg(side, "bits" if mode == "guided" else "codes", x, _U8, n // 8 if mode == "guided" else n // 2)
    y = _bf16_out(y, x, n, "y")
    mask = _u8(n // 8, x, mask, "mask")
    if want_codes or qcodes is not None:
        qcodes = _u8(n // 2, x, qcodes, "qcodes")
    tail = (_ptr(y), _ptr(mask), _ptr(qcodes), _stream(x))
    if mode == "guided":
        st, name = lib.trace_mx_guided_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), _ptr(side), *tail), \
            "trace_mx_guided_fakequant_fwd"
    elif mode == "full":
        st, name = lib.trace_mx_full_info_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), _ptr(side), *tail), \
            "trace_mx_full_info_fakequant_fwd"
    else:
        st, name = lib.trace_mx_rne_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), *tail), \
            "trace_mx_rne_fakequant_fwd"
    _check(st, name)
    return y, mask, qcodes


def mx_guided_fakequant_fwd(x_train, scales, bits, y=None, mask=None, want_codes=False, qcodes=None):
    """Rollout-guided forward on MXFP4 scales: (y, mask, qcodes)."""
    return _mx_fwd("guided", x_train, scales, bits, y, mask, want_codes, qcodes)


def mx_rne_fakequant_fwd(x_train, scales, y=None, mask=None, want_codes=False, qcodes=None):
    """Round-to-nearest-even forward on MXFP4 scales: (y, mask, qcodes)."""
    return _mx_fwd("rne", x_train, scales, None, y, mask, want_codes, qcodes)


def mx_full_info_fakequant_fwd(x_train, scales, codes, y=None, mask=None, want_codes=False, qcodes=None):
    """Full-information guided forward on MXFP4 scales: (y, mask, qcodes)."""
    return _mx_fwd("full", x_train, scales, codes, y, mask, want_codes, qcodes)


def mx8_capture(x_roll, want_codes=False, scales=None, bits=None, codes=None):
    """MXFP8 capture: (scales u8[n/32] E8M0, bits u8[n/8], codes u8[n] E4M3FN or None)."""
    _bf16(x_roll, "x_roll")
    rows, cols = _rows_cols(x_roll)
    n = rows * cols
    scales = _u8(n // 32, x_roll, scales, "scales")
    bits = _u8(n // 8, x_roll, bits, "bits")
    if want_codes or codes is not None:
        codes = _u8(n, x_roll, codes, "codes")
    _check(lib.trace_mx8_capture(_ptr(x_roll), rows, cols, _ptr(scales), _ptr(bits), _ptr(codes), _stream(x_roll)),
           "trace_mx8_capture")
    return scales, bits, codes


def _mx8_fwd(mode, x, scales, side, y, mask, want_codes, qcodes):
    _bf16(x, "x_train")
    rows, cols = _rows_cols(x)
    n = rows * cols
    _arg(scales, "scales", x, _U8, n // 32)
    if mode != "rne":
        _arg(side, "bits" if mode == "guided" else "codes", x, _U8, n // 8 if mode == "guided" else n)
    y = _bf16_out(y, x, n, "y")
    mask = _u8(n // 8, x, mask, "mask")
    if want_codes or qcodes is not None:
        qcodes = _u8(n, x, qcodes, "qcodes")
    tail = (_ptr(y), _ptr(mask), _ptr(qcodes), _stream(x))
    if mode == "guided":
        name = "trace_mx8_guided_fakequant_fwd"
        st = lib.trace_mx8_guided_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), _ptr(side), *tail)
    elif mode == "full":
        name = "trace_mx8_full_info_fakequant_fwd"
        st = lib.trace_mx8_full_info_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), _ptr(side), *tail)
    else:
        name = "trace_mx8_rne_fakequant_fwd"
        st = lib.trace_mx8_rne_fakequant_fwd(_ptr(x), rows, cols, _ptr(scales), *tail)
    _check(st, name)
    return y, mask, qcodes


def mx8_guided_fakequant_fwd(x_train, scales, bits, y=None, mask=None, want_codes=False, qcodes=None):
    """Rollout-guided forward on the MXFP8 grid: (y, mask, qcodes u8[n])."""
    return _mx8_fwd("guided", x_train, scales, bits, y, mask, want_codes, qcodes)


def mx8_rne_fakequant_fwd(x_train, scales, y=None, mask=None, want_codes=False, qcodes=None):
    """Round-to-nearest-even forward on the MXFP8 grid: (y, mask, qcodes u8[n])."""
    return _mx8_fwd("rne", x_train, scales, None, y, mask, want_codes, qcodes)


def mx8_full_info_fakequant_fwd(x_train, scales, codes, y=None, mask=None, want_codes=False, qcodes=None):
    """Full-information forward on the MXFP8 grid (codes: rollout E4M3FN bytes,
    u8[n]): (y, mask, qcodes u8[n])."""
    return _mx8_fwd("full", x_train, scales, codes, y, mask, want_codes, qcodes)


# Layout of the agreement statistics: hist[0..14], then these counters.
STAT_FIELDS = ("straddle", "crossed", "recovered", "violations", "elements")


def mismatch_stats(x_train, scales, ts, bits, codes, stats=None):
    """Agreement statistics of x_train's RNE / guided / full-information
    codes with the rollout codes, ADDED to ``stats`` (an int64[20] device
    tensor, zeroed here when not given): [0..14] histogram of signed grid
    steps between rollout and RNE codes, then straddle, crossed, recovered,
    violations, elements (the counts are below 2^63)."""
    _bf16(x_train, "x_train")
    rows, cols = _rows_cols(x_train)
    n = rows * cols
    _arg(scales, "scales", x_train, _U8, n // 16)
    _arg(ts, "ts", x_train, _F32, 1)
    _arg(bits, "bits", x_train, _U8, n // 8)
    _arg(codes, "codes", x_train, _U8, n // 2)
    if stats is None:
        stats = torch.zeros(20, dtype=torch.int64, device=x_train.device)
    _arg(stats, "stats", x_train, _I64, 20)
    _check(lib.trace_mismatch_stats(_ptr(x_train), rows, cols, _ptr(scales), _ptr(ts), _ptr(bits), _ptr(codes),
                                    _ptr(stats), _stream(x_train)), "trace_mismatch_stats")
    return stats


class GuidedFakeQuant(torch.autograd.Function):
    """y = s * q* in the forward, straight-through (clip-masked) gradient in
    the backward; the rollout record (scales, ts, bits) is not differentiated."""

    @staticmethod
    def forward(ctx, x_train, scales, ts, bits):
        y, mask, _ = guided_fakequant_fwd(x_train.contiguous(), scales, ts, bits)
        ctx.save_for_backward(mask)
        return y

    @staticmethod
    def backward(ctx, grad_out):
        (mask,) = ctx.saved_tensors
        return ste_bwd(grad_out.contiguous(), mask), None, None, None


# --------------------------------------------------------------------------
# products of microscaled operands
# --------------------------------------------------------------------------

MAX_EXPERTS = 1024
MAX_TOPK = 64
MAX_PRODUCT_GROUPS = 4096


def _addr(t):
    return None if t is None else t.data_ptr()


def _bytes(workspace):
    return 0 if workspace is None else workspace.numel()


# A device's current stream as an integer.  A Stream object for each call would
# take a microsecond of the ten that a small product's call takes.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(name, like, *args):
    """Call an entry point on ``like``'s device and its current stream."""
    dev = like.device.index
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _launch(name, like, *args)
    status = getattr(lib, name)(*args, _current_stream(dev))
    if status != 0:
        raise TraceError(status, name)


def _matrix(t, name, dtypes=_BF16):
    """A contiguous bf16 (or fp32) device tensor as (rows, cols) over its last dimension."""
    if dtypes is _BF16:
        _bf16(t, name)
    else:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        _arg(t, name, t, dtypes, 0)
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    return math.prod(t.shape[:-1]), t.shape[-1]


def _dim(v, name, multiple):
    if isinstance(v, bool) or not isinstance(v, int) or v < 0 or v % multiple:
        raise ValueError(f"{name} must be a non-negative multiple of {multiple}, got {v!r}")
    return v


def _fit(t, name, like, dtypes, numel):
    """``_arg`` for a tensor that must hold exactly ``numel`` elements."""
    _arg(t, name, like, dtypes, numel)
    if t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
    return t


def _code_bytes(fmt, n):
    return n // 2 if fmt == "mx" else n


def _out(t, name, like, shape, dtype):
    n = 1
    for d in shape:
        n *= d
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    return _arg(t, name, like, _BF16 if dtype == torch.bfloat16 else (dtype,), n)


def _outs(like, workspace_bytes, workspace, *outs):
    """Several outputs, each (given, name, shape, dtype), and the workspace
    after them: those that were given checked, the others made at once."""
    if workspace is None and all(o[0] is None for o in outs):
        wanted = []
        for _, _, shape, dtype in outs:
            wanted += (shape, dtype)
        return _tensor_lists.empties(like, *wanted, workspace_bytes, torch.uint8)
    return (*(_out(t, name, like, shape, dtype) for t, name, shape, dtype in outs),
            _workspace(workspace, like, workspace_bytes))


def _rows_type(dtype):
    """The suffix of the entry points for packed rows in dtype."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    return "_f32" if dtype == torch.float32 else ""


def _workspace(t, like, need):
    if t is None:
        return like.new_empty(need, dtype=torch.uint8) if need else None
    return _arg(t, "workspace", like, _U8, need)


def _groups(offsets, like):
    """(address, groups, weights) of a product's groups; offsets None: one weight."""
    if offsets is None:
        return None, 0, 1
    groups = _offsets(offsets, like)
    if groups > MAX_PRODUCT_GROUPS:
        raise ValueError(f"at most {MAX_PRODUCT_GROUPS} groups, got {groups}")
    return offsets.data_ptr(), groups, groups


def _quantize(fmt, x, want_mask, scales, codes, mask):
    rows, cols = _matrix(x, "x")
    n = rows * cols
    scales = _u8(n // 32, x, scales, "scales")
    codes = _u8(_code_bytes(fmt, n), x, codes, "codes")
    if want_mask or mask is not None:
        mask = _u8(n // 8, x, mask, "mask")
    _launch(f"trace_{fmt}_quantize", x, _addr(x), rows, cols, _addr(scales), _addr(codes), _addr(mask))
    return scales, codes, mask


def mx_quantize(x, want_mask=False, scales=None, codes=None, mask=None):
    """MXFP4 operand of a product: (scales u8[n/32], codes u8[n/2], clip mask
    u8[n/8] or None), the scales and codes of ``mx_capture`` in one pass."""
    return _quantize("mx", x, want_mask, scales, codes, mask)


def mx8_quantize(x, want_mask=False, scales=None, codes=None, mask=None):
    """MXFP8 operand of a product: (scales u8[n/32], codes u8[n], clip mask
    u8[n/8] or None), the scales and codes of ``mx8_capture`` in one pass."""
    return _quantize("mx8", x, want_mask, scales, codes, mask)


def _record(fmt, scales, codes, like, k, prefix, rows):
    """Rows of a stored operand [rows, k]; with k == 0, which leaves nothing to
    count them by, the ``rows`` that the caller knows of."""
    _arg(scales, f"{prefix}_scales", like, _U8, 0)
    if k > 0:
        rows = scales.numel() * 32 // k
    elif rows is None:
        raise ValueError("k is 0: y must be given, for its rows")
    _fit(scales, f"{prefix}_scales", like, _U8, rows * (k // 32))
    _fit(codes, f"{prefix}_codes", like, _U8, _code_bytes(fmt, rows * k))
    return rows


def _weight(w_scales, w_codes, like, weights, n, k):
    _fit(w_scales, "w_scales", like, _U8, weights * n * (k // 32))
    _fit(w_codes, "w_codes", like, _U8, weights * n * k // 2)


def _index(row_index, like):
    _arg(row_index, "row_index", like, _I64, 0)
    return row_index.numel()


def _matmul(fmt, a_scales, a_codes, offsets, w_scales, w_codes, n, k, row_index, y, dtype=torch.bfloat16, rows=None):
    if not isinstance(a_codes, torch.Tensor) or not a_codes.is_cuda:
        raise ValueError("a_codes must be a device tensor")
    _dim(n, "n", 16)
    _dim(k, "k", 32)
    if k == 0 and rows is None:
        rows = 0 if row_index is not None else y.numel() // n if isinstance(y, torch.Tensor) and n else None
    src_rows = _record(fmt, a_scales, a_codes, a_codes, k, "a", rows)
    at, groups, weights = _groups(offsets, a_codes)
    _weight(w_scales, w_codes, a_codes, weights, n, k)
    rows = src_rows if row_index is None else _index(row_index, a_codes)
    rows_type = _rows_type(dtype)
    y = _out(y, "y", a_codes, (rows, n), dtype)
    if offsets is None:
        _launch(f"trace_{fmt}_matmul", a_codes, _addr(a_scales), _addr(a_codes), rows, _addr(w_scales), _addr(w_codes),
                n, k, _addr(y))
    else:
        _launch(f"trace_grouped_{fmt}_matmul{rows_type}", a_codes, _addr(a_scales), _addr(a_codes), src_rows,
                _addr(row_index), rows, at, groups, _addr(w_scales), _addr(w_codes), n, k, _addr(y))
    return y


def mx_matmul(a_scales, a_codes, w_scales, w_codes, n, k, y=None):
    """y = A W^T (bf16 [rows, n]) of MXFP4 activations [rows, k] and an MXFP4
    weight [n, k]; n % 16 == 0, k % 32 == 0.  k == 0 gives zeros in the y
    passed in."""
    return _matmul("mx", a_scales, a_codes, None, w_scales, w_codes, n, k, None, y)


def mx8_matmul(a_scales, a_codes, w_scales, w_codes, n, k, y=None):
    """``mx_matmul`` with MXFP8 activations (W4A8)."""
    return _matmul("mx8", a_scales, a_codes, None, w_scales, w_codes, n, k, None, y)


def grouped_mx_matmul(a_scales, a_codes, offsets, w_scales, w_codes, n, k, row_index=None, y=None,
                      dtype=torch.bfloat16):
    """``mx_matmul`` of packed rows [offsets[g], offsets[g+1]) with the g-th of
    the weights [groups, n, k].  Packed row r is row r of the activations, or,
    with ``row_index`` (int64, one per packed row), row row_index[r].  Rows
    behind the last group give zeros.  dtype torch.float32: the sums as they
    are, for rows that ``expert_combine`` sums further (in bf16 each row is
    rounded once more on the way)."""
    return _matmul("mx", a_scales, a_codes, _need(offsets), w_scales, w_codes, n, k, row_index, y, dtype)


def grouped_mx8_matmul(a_scales, a_codes, offsets, w_scales, w_codes, n, k, row_index=None, y=None,
                       dtype=torch.bfloat16):
    """``grouped_mx_matmul`` with MXFP8 activations (W4A8)."""
    return _matmul("mx8", a_scales, a_codes, _need(offsets), w_scales, w_codes, n, k, row_index, y, dtype)


def _need(offsets):
    if offsets is None:
        raise ValueError("offsets is required")
    return offsets


def _linear(fmt, x, offsets, w_scales, w_codes, n, row_index, workspace, y, dtype=torch.bfloat16):
    src_rows, k = _matrix(x, "x")
    _dim(n, "n", 16)
    at, groups, weights = _groups(offsets, x)
    _weight(w_scales, w_codes, x, weights, n, k)
    rows = src_rows if row_index is None else _index(row_index, x)
    shape = (rows, n) if row_index is not None else (*x.shape[:-1], n)
    rows_type = _rows_type(dtype)
    y = _out(y, "y", x, shape, dtype)
    workspace = _workspace(workspace, x, getattr(lib, f"trace_{fmt}_linear_workspace_bytes")(src_rows, rows, groups, k))
    name = f"trace_grouped_{fmt}_linear_f32" if rows_type else f"trace_{fmt}_linear"
    _launch(name, x, _addr(x), src_rows, _addr(row_index), rows, at, groups, _addr(w_scales), _addr(w_codes), n, k,
            _addr(workspace), 0 if workspace is None else workspace.numel(), _addr(y))
    return y


def mx_linear(x, w_scales, w_codes, n, workspace=None, y=None):
    """y = q(x) W^T: bf16 activations x [..., k] rounded to MXFP4 (as
    ``mx_quantize``) and multiplied by the MXFP4 weight [n, k]."""
    return _linear("mx", x, None, w_scales, w_codes, n, None, workspace, y)


def mx8_linear(x, w_scales, w_codes, n, workspace=None, y=None):
    """``mx_linear`` with the activations rounded to MXFP8 (W4A8)."""
    return _linear("mx8", x, None, w_scales, w_codes, n, None, workspace, y)


def grouped_mx_linear(x, offsets, w_scales, w_codes, n, row_index=None, workspace=None, y=None, dtype=torch.bfloat16):
    """``mx_linear`` per group of packed rows, as ``grouped_mx_matmul``: with
    ``row_index``, x holds the tokens, each rounded once for all its experts."""
    return _linear("mx", x, _need(offsets), w_scales, w_codes, n, row_index, workspace, y, dtype)


def grouped_mx8_linear(x, offsets, w_scales, w_codes, n, row_index=None, workspace=None, y=None, dtype=torch.bfloat16):
    """``grouped_mx_linear`` with the activations rounded to MXFP8 (W4A8)."""
    return _linear("mx8", x, _need(offsets), w_scales, w_codes, n, row_index, workspace, y, dtype)


def _bwd_input(grad_y, offsets, w_scales, w_codes, k, mask, grad_x, dtype=torch.bfloat16):
    rows, n = _matrix(grad_y, "grad_y")
    _dim(k, "k", 32)
    at, groups, weights = _groups(offsets, grad_y)
    _weight(w_scales, w_codes, grad_y, weights, n, k)
    if mask is not None:
        _arg(mask, "mask", grad_y, _U8, rows * k // 8)
    rows_type = _rows_type(dtype)
    grad_x = _out(grad_x, "grad_x", grad_y, (*grad_y.shape[:-1], k), dtype)
    name = "trace_grouped_mx_matmul_bwd_input_f32" if rows_type else "trace_mx_matmul_bwd_input"
    _launch(name, grad_y, _addr(grad_y), rows, at, groups, _addr(w_scales), _addr(w_codes), n, k, _addr(mask),
            _addr(grad_x))
    return grad_x


def mx_matmul_bwd_input(grad_y, w_scales, w_codes, k, mask=None, grad_x=None):
    """grad_x = grad_y W (bf16 [..., k]), zero where the activations' clip
    mask is 0; for MXFP4 and MXFP8 activations alike."""
    return _bwd_input(grad_y, None, w_scales, w_codes, k, mask, grad_x)


def grouped_mx_matmul_bwd_input(grad_y, offsets, w_scales, w_codes, k, mask=None, grad_x=None, dtype=torch.bfloat16):
    """``mx_matmul_bwd_input`` per group of packed rows, in packed order (sum
    the rows of a token with ``expert_combine``; dtype torch.float32 keeps
    them unrounded until then)."""
    return _bwd_input(grad_y, _need(offsets), w_scales, w_codes, k, mask, grad_x, dtype)


def _bwd_weight(fmt, grad_y, offsets, a_scales, a_codes, k, row_index, mask, grad_w, workspace):
    rows, n = _matrix(grad_y, "grad_y")
    _dim(k, "k", 32)
    at, groups, weights = _groups(offsets, grad_y)
    src_rows = _record(fmt, a_scales, a_codes, grad_y, k, "a", rows)
    if row_index is not None:
        _fit(row_index, "row_index", grad_y, _I64, rows)
    elif src_rows != rows:
        raise ValueError(f"grad_y has {rows} rows, the activations {src_rows}")
    if mask is not None:
        _arg(mask, "mask", grad_y, _U8, weights * n * k // 8)
    grad_w = _out(grad_w, "grad_w", grad_y, (n, k) if offsets is None else (weights, n, k), torch.bfloat16)
    workspace = _workspace(workspace, grad_y, lib.trace_mx_matmul_bwd_weight_workspace_bytes(rows, groups, n, k))
    _launch(f"trace_{fmt}_matmul_bwd_weight", grad_y, _addr(grad_y), rows, at, groups, _addr(a_scales), _addr(a_codes),
            src_rows, _addr(row_index), n, k, _addr(mask), _addr(grad_w), _addr(workspace),
            0 if workspace is None else workspace.numel())
    return grad_w


def mx_matmul_bwd_weight(grad_y, a_scales, a_codes, k, mask=None, grad_w=None, workspace=None):
    """grad_w = grad_y^T A (bf16 [n, k]) with MXFP4 activations A, zero where
    the weight's clip mask is 0."""
    return _bwd_weight("mx", grad_y, None, a_scales, a_codes, k, None, mask, grad_w, workspace)


def mx8_matmul_bwd_weight(grad_y, a_scales, a_codes, k, mask=None, grad_w=None, workspace=None):
    """``mx_matmul_bwd_weight`` with MXFP8 activations."""
    return _bwd_weight("mx8", grad_y, None, a_scales, a_codes, k, None, mask, grad_w, workspace)


def grouped_mx_matmul_bwd_weight(grad_y, offsets, a_scales, a_codes, k, row_index=None, mask=None, grad_w=None,
                                 workspace=None):
    """``mx_matmul_bwd_weight`` per group of packed rows: bf16 [groups, n, k],
    zeros for a group without rows."""
    return _bwd_weight("mx", grad_y, _need(offsets), a_scales, a_codes, k, row_index, mask, grad_w, workspace)


def grouped_mx8_matmul_bwd_weight(grad_y, offsets, a_scales, a_codes, k, row_index=None, mask=None, grad_w=None,
                                  workspace=None):
    """``grouped_mx_matmul_bwd_weight`` with MXFP8 activations."""
    return _bwd_weight("mx8", grad_y, _need(offsets), a_scales, a_codes, k, row_index, mask, grad_w, workspace)


# --------------------------------------------------------------------------
# routed rows
# --------------------------------------------------------------------------

def _pairs(t, name, like, dtypes):
    """A contiguous [tokens, topk] device tensor as (tokens, topk)."""
    _arg(t, name, like, dtypes, 0)
    if t.dim() != 2:
        raise ValueError(f"{name} must be [tokens, topk], got {tuple(t.shape)}")
    tokens, topk = t.shape
    if not 1 <= topk <= MAX_TOPK:
        raise ValueError(f"topk must be 1 to {MAX_TOPK}, got {topk}")
    return tokens, topk


def expert_sort(ids, experts, offsets=None, row_index=None, slot=None, workspace=None):
    """Stable sort of the (token, expert) pairs by expert.  ids: int64
    [tokens, topk]; pairs whose id lies outside [0, experts) are left out.
    Returns (offsets int64[experts + 1]: the experts' packed rows, row_index
    int64[tokens*topk]: the token of each packed row, -1 behind the last
    group, slot int64[tokens, topk]: the packed row of each pair or -1)."""
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise ValueError("ids must be a device tensor")
    tokens, topk = _pairs(ids, "ids", ids, _I64)
    if isinstance(experts, bool) or not isinstance(experts, int) or not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"experts must be 1 to {MAX_EXPERTS}, got {experts!r}")
    offsets = _out(offsets, "offsets", ids, (experts + 1,), torch.int64)
    row_index = _out(row_index, "row_index", ids, (tokens * topk,), torch.int64)
    slot = _out(slot, "slot", ids, (tokens, topk), torch.int64)
    workspace = _workspace(workspace, ids, lib.trace_expert_sort_workspace_bytes(tokens, topk, experts))
    _launch("trace_expert_sort", ids, _addr(ids), tokens, topk, experts, _addr(workspace),
            0 if workspace is None else workspace.numel(), _addr(offsets), _addr(row_index), _addr(slot))
    return offsets, row_index, slot


def expert_dispatch(x, row_index, out=None):
    """Packed rows: row r is row row_index[r] of x (bf16 [..., cols]), zeros
    for an index outside x."""
    tokens, cols = _matrix(x, "x")
    rows = _index(row_index, x)
    out = _out(out, "out", x, (rows, cols), torch.bfloat16)
    _launch("trace_expert_dispatch", x, _addr(x), tokens, cols, _addr(row_index), rows, _addr(out))
    return out


def expert_combine(y, slot, weights=None, out=None):
    """The tokens' sums of their packed rows, out[t] = sum over j of
    weights[t, j] * y[slot[t, j]] (fp32 weights; None: ones; y in bf16 or
    fp32, out in bf16); pairs whose slot lies outside y are left out."""
    f32 = isinstance(y, torch.Tensor) and y.dtype == torch.float32
    rows, cols = _matrix(y, "y", _F32 if f32 else _BF16)
    tokens, topk = _pairs(slot, "slot", y, _I64)
    if weights is not None:
        _fit(weights, "weights", y, _F32, tokens * topk)
    out = _out(out, "out", y, (tokens, cols), torch.bfloat16)
    name = "trace_expert_combine_f32" if f32 else "trace_expert_combine"
    _launch(name, y, _addr(y), rows, cols, _addr(slot), _addr(weights), tokens, topk, _addr(out))
    return out


def expert_combine_bwd(grad_out, y, slot, weights, offsets=None, grad_y=None, grad_weights=None):
    """Gradients of ``expert_combine``: (grad_y bf16, packed as y; grad_weights
    fp32 [tokens, topk]).  Rows that no slot names are zeros; without
    ``offsets`` they are left as they are in a grad_y passed in.  No two slots
    may name the same row."""
    rows, cols = _matrix(y, "y")
    tokens, topk = _pairs(slot, "slot", y, _I64)
    t, c = _matrix(grad_out, "grad_out")
    if grad_out.device != y.device or (t, c) != (tokens, cols):
        raise ValueError(f"grad_out must be [{tokens}, {cols}] on {y.device}, got {tuple(grad_out.shape)}")
    if weights is not None:
        _fit(weights, "weights", y, _F32, tokens * topk)
    at, groups, _ = _groups(offsets, y)
    if grad_y is None and offsets is None:
        grad_y = torch.zeros_like(y)
    grad_y = _out(grad_y, "grad_y", y, tuple(y.shape), torch.bfloat16)
    grad_weights = _out(grad_weights, "grad_weights", y, (tokens, topk), torch.float32)
    _launch("trace_expert_combine_bwd", y, _addr(grad_out), _addr(y), rows, cols, _addr(slot), _addr(weights), tokens,
            topk, at, groups, _addr(grad_y), _addr(grad_weights))
    return grad_y, grad_weights


class MxMatmul(torch.autograd.Function):
    """y = q(x) q(w)^T with both operands rounded in the forward and the
    gradients passed straight through inside the clip ranges.

    x: bf16 [rows, k]; w: bf16 [n, k], or [groups, n, k] with ``offsets`` (the
    packed rows' groups).  fmt: "mx" (MXFP4 activations) or "mx8" (MXFP8).
    scales, bits: the rollout's record of x in that format; x is then rounded
    by the rollout-guided rule instead of to nearest.  y and both gradients are
    bf16; the grouped functions themselves also give fp32 rows."""

    @staticmethod
    def forward(ctx, x, w, offsets=None, fmt="mx", scales=None, bits=None):
        if fmt not in ("mx", "mx8"):
            raise ValueError(f'fmt must be "mx" or "mx8", got {fmt!r}')
        x, w = x.contiguous(), w.contiguous()
        n, k = w.shape[-2:]
        if x.shape[-1] != k:
            raise ValueError(f"x has rows of {x.shape[-1]}, w of {k}")
        if scales is None:
            a_scales, a_codes, a_mask = _quantize(fmt, x, True, None, None, None)
        else:
            guided = mx_guided_fakequant_fwd if fmt == "mx" else mx8_guided_fakequant_fwd
            a_scales, (_, a_mask, a_codes) = scales, guided(x, scales, bits, want_codes=True)
        w_scales, w_codes, w_mask = mx_quantize(w, want_mask=True)
        ctx.save_for_backward(a_scales, a_codes, a_mask, w_scales, w_codes, w_mask, offsets)
        ctx.fmt, ctx.k = fmt, k
        y = _matmul(fmt, a_scales, a_codes, offsets, w_scales, w_codes, n, k, None, None, rows=math.prod(x.shape[:-1]))
        return y.view(*x.shape[:-1], n)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        a_scales, a_codes, a_mask, w_scales, w_codes, w_mask, offsets = ctx.saved_tensors
        grad_y = grad_y.contiguous()
        grad_x = grad_w = None
        if ctx.needs_input_grad[0]:
            grad_x = _bwd_input(grad_y, offsets, w_scales, w_codes, ctx.k, a_mask, None)
        if ctx.needs_input_grad[1]:
            grad_w = _bwd_weight(ctx.fmt, grad_y, offsets, a_scales, a_codes, ctx.k, None, w_mask, None, None)
        return grad_x, grad_w, None, None, None, None


class ExpertDispatch(torch.autograd.Function):
    """``expert_dispatch`` of the packed rows of ``expert_sort``'s (row_index,
    slot); the gradient sums a token's packed rows.  They arrive in bf16, as
    torch hands every gradient on in its tensor's type: each is rounded once
    before the sum (``grouped_mx_matmul_bwd_input`` with dtype torch.float32 and
    ``expert_combine`` leave that out)."""

    @staticmethod
    def forward(ctx, x, row_index, slot):
        ctx.save_for_backward(slot)
        ctx.shape = x.shape
        return expert_dispatch(x.contiguous(), row_index)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        (slot,) = ctx.saved_tensors
        return expert_combine(grad.contiguous(), slot).view(ctx.shape), None, None


class ExpertCombine(torch.autograd.Function):
    """``expert_combine`` of bf16 rows with gradients to the rows and the
    weights (None: ones).  As for ``expert_combine_bwd``, no two slots may name
    the same row."""

    @staticmethod
    def forward(ctx, y, slot, weights, offsets):
        y = _bf16(y.contiguous(), "y")  # the gradients' type too
        weights = None if weights is None else weights.contiguous()
        ctx.save_for_backward(y, slot, weights, offsets)
        return expert_combine(y, slot, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        y, slot, weights, offsets = ctx.saved_tensors
        grad_y, grad_weights = expert_combine_bwd(grad_out.contiguous(), y, slot, weights, offsets)
        return grad_y, None, None if weights is None else grad_weights, None


# --------------------------------------------------------------------------
# the router
# --------------------------------------------------------------------------

def _router(logits, topk):
    """(suffix of the entry points, tokens, experts) of router logits."""
    f32 = isinstance(logits, torch.Tensor) and logits.dtype == torch.float32
    tokens, experts = _matrix(logits, "logits", _F32 if f32 else _BF16)
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"experts must be 1 to {MAX_EXPERTS}, got {experts}")
    if isinstance(topk, bool) or not isinstance(topk, int) or not 1 <= topk <= min(MAX_TOPK, experts):
        raise ValueError(f"topk must be 1 to {min(MAX_TOPK, experts)}, got {topk!r}")
    return "_f32" if f32 else "", tokens, experts


def expert_route(logits, topk, renormalize=True, valid=None, ids=None, weights=None, counts=None, probs=None,
                 balance=None, workspace=None):
    """Each row's topk experts by its router logits (bf16 or fp32
    [..., experts]; ties go to the lowest index, NaN is above all, -infinity is
    never taken).  valid: bool or uint8, one per row; rows where it is 0 are
    left out.  Returns

    ids int64 [tokens, topk]: what ``expert_sort`` takes; -1 for rows left out;
    weights fp32 [tokens, topk]: the softmax at ids, divided by its sum over
    them with ``renormalize``; what ``expert_combine`` takes;
    counts int64 [experts + 1]: the experts' pairs, then the rows routed;
    probs fp32 [experts]: the softmaxes summed over the rows routed;
    balance fp32 [1]: experts * sum of (counts / their sum) * (probs / rows)."""
    suffix, tokens, experts = _router(logits, topk)
    if valid is not None:
        _fit(valid, "valid", logits, (torch.bool, torch.uint8), tokens)
    ids, weights, counts, probs, balance, workspace = _outs(
        logits, lib.trace_expert_route_workspace_bytes(tokens, experts), workspace,
        (ids, "ids", (tokens, topk), torch.int64), (weights, "weights", (tokens, topk), torch.float32),
        (counts, "counts", (experts + 1,), torch.int64), (probs, "probs", (experts,), torch.float32),
        (balance, "balance", (1,), torch.float32))
    _launch("trace_expert_route" + suffix, logits, _addr(logits), _addr(valid), tokens, experts, topk,
            int(bool(renormalize)), _addr(workspace), _bytes(workspace), _addr(ids), _addr(weights), _addr(counts),
            _addr(probs), _addr(balance))
    return ids, weights, counts, probs, balance


def expert_route_bwd(grad_weights, grad_balance, logits, ids, weights, counts, renormalize=True, grad_logits=None):
    """The gradient to the logits, of their type, from those of the weights
    (fp32 [tokens, topk]) and of the balance loss (fp32 [1]); None: zeros.
    ids, weights: the forward's; counts: the forward's, or summed over ranks.
    grad_logits may be the logits themselves."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be [tokens, topk]")
    suffix, tokens, experts = _router(logits, ids.shape[1])
    topk = ids.shape[1]
    pairs = tokens * topk
    if weights is None or counts is None or not _tensor_lists.fits(  # otherwise: which one, and why
            logits, ids, torch.int64, pairs, weights, torch.float32, pairs, counts, torch.int64, experts + 1,
            grad_weights, torch.float32, pairs, grad_balance, torch.float32, 1):
        _fit(ids, "ids", logits, _I64, pairs)
        _fit(weights, "weights", logits, _F32, pairs)
        _fit(counts, "counts", logits, _I64, experts + 1)
        if grad_weights is not None:
            _fit(grad_weights, "grad_weights", logits, _F32, pairs)
        if grad_balance is not None:
            _fit(grad_balance, "grad_balance", logits, _F32, 1)
    dtype = torch.float32 if suffix else torch.bfloat16
    if grad_logits is None:
        grad_logits, = _tensor_lists.empties(logits, tuple(logits.shape), dtype)
    else:
        _out(grad_logits, "grad_logits", logits, tuple(logits.shape), dtype)
    _launch("trace_expert_route_bwd" + suffix, logits, _addr(grad_weights), _addr(grad_balance), _addr(logits),
            _addr(ids), _addr(weights), _addr(counts), tokens, experts, topk, int(bool(renormalize)),
            _addr(grad_logits))
    return grad_logits


class ExpertRoute(torch.autograd.Function):
    """``expert_route`` as (ids, weights, counts, balance), with gradients from
    the weights and the balance loss to the logits."""

    @staticmethod
    def forward(ctx, logits, topk, renormalize=True, valid=None):
        logits = logits.contiguous()
        ids, weights, counts, _, balance = expert_route(logits, topk, renormalize, valid)
        ctx.save_for_backward(logits, ids, weights, counts)
        ctx.renormalize = renormalize
        ctx.mark_non_differentiable(ids, counts)
        ctx.set_materialize_grads(False)
        return ids, weights, counts, balance

    @staticmethod
    @once_differentiable
    def backward(ctx, _ids, grad_weights, _counts, grad_balance):
        logits, ids, weights, counts = ctx.saved_tensors
        if grad_weights is not None:
            grad_weights = grad_weights.contiguous()
        if grad_balance is not None:
            grad_balance = grad_balance.contiguous()
        return expert_route_bwd(grad_weights, grad_balance, logits, ids, weights, counts, ctx.renormalize), None, None, None


# --------------------------------------------------------------------------
# the loss over the vocabulary
# --------------------------------------------------------------------------

def _logits_of(x, w, targets):
    """(tokens, vocab, k) of the logits x W^T."""
    tokens, k = _matrix(x, "x")
    _bf16(w, "w")
    if w.device != x.device or w.dim() != 2 or w.shape[1] != k:
        raise ValueError(f"w must be [vocab, {k}] on {x.device}, got {tuple(w.shape)} on {w.device}")
    if k == 0 or k % 32:
        raise ValueError(f"rows must be a multiple of 32 long, got {k}")
    if w.shape[0] == 0:
        raise ValueError("the vocabulary is empty")
    _fit(targets, "targets", x, _I64, tokens)
    return tokens, w.shape[0], k


def linear_cross_entropy(x, w, targets, scale=1.0, loss=None, lse=None, workspace=None):
    """Softmax cross entropy of the logits scale * x W^T over the vocabulary,
    without keeping them: (loss, lse), fp32, one per token.  x: bf16 [..., k];
    w: bf16 [vocab, k], k % 32 == 0; targets: int64, one per token.  loss is
    minus the target's log-probability; tokens whose target lies outside
    [0, vocab) are ignored, with loss and lse 0."""
    tokens, vocab, k = _logits_of(x, w, targets)
    shape = tuple(x.shape[:-1])
    loss, lse, workspace = _outs(x, lib.trace_linear_cross_entropy_workspace_bytes(tokens, vocab, k), workspace,
                                 (loss, "loss", shape, torch.float32), (lse, "lse", shape, torch.float32))
    _launch("trace_linear_cross_entropy", x, _addr(x), _addr(w), _addr(targets), tokens, vocab, k, scale,
            _addr(workspace), _bytes(workspace), _addr(loss), _addr(lse))
    return loss, lse


def linear_cross_entropy_bwd(grad_loss, x, w, targets, lse, scale=1.0, grad_x=None, grad_w=None, workspace=None,
                             want_x=True, want_w=True):
    """Gradients of ``linear_cross_entropy``'s loss, the logits computed again a
    slice of the vocabulary at a time: (grad_x as x, grad_w as w, in bf16; None
    where not wanted).  grad_loss: fp32, one per token, not read where the token
    is ignored; lse: the forward's."""
    tokens, vocab, k = _logits_of(x, w, targets)
    _fit(grad_loss, "grad_loss", x, _F32, tokens)
    _fit(lse, "lse", x, _F32, tokens)
    grad_x = _out(grad_x, "grad_x", x, tuple(x.shape), torch.bfloat16) if want_x else None
    grad_w = _out(grad_w, "grad_w", x, tuple(w.shape), torch.bfloat16) if want_w else None
    workspace = _workspace(workspace, x, lib.trace_linear_cross_entropy_bwd_workspace_bytes(tokens, vocab, k))
    _launch("trace_linear_cross_entropy_bwd", x, _addr(grad_loss), _addr(x), _addr(w), _addr(targets), _addr(lse),
            tokens, vocab, k, scale, _addr(workspace), _bytes(workspace), _addr(grad_x),
            _addr(grad_w))
    return grad_x, grad_w


class LinearCrossEntropy(torch.autograd.Function):
    """``linear_cross_entropy``'s loss per token, with gradients to x and w."""

    @staticmethod
    def forward(ctx, x, w, targets, scale=1.0):
        x, w, targets = x.contiguous(), w.contiguous(), targets.contiguous()
        loss, lse = linear_cross_entropy(x, w, targets, scale)
        ctx.save_for_backward(x, w, targets, lse)
        ctx.scale = scale
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss):
        x, w, targets, lse = ctx.saved_tensors
        grad_x, grad_w = linear_cross_entropy_bwd(grad_loss.contiguous(), x, w, targets, lse, ctx.scale,
                                                  want_x=ctx.needs_input_grad[0], want_w=ctx.needs_input_grad[1])
        return grad_x, grad_w, None, None


# --------------------------------------------------------------------------
# the optimiser step
# --------------------------------------------------------------------------

class _AdamwOptions(ctypes.Structure):
    """trace_adamw_options of include/trace.h."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint64)] + [
        (n, ctypes.c_int32) for n in ("param_bf16", "grad_bf16", "states_mx8", "randomly")]


# Words of trace_adamw_tensor: param, grad, avg, sq, avg_scales, sq_scales, copy, n
_TENSOR_WORDS = 8
_F32_OR_BF16 = (torch.float32, torch.bfloat16)
_BF16_ONLY = (torch.bfloat16,)


def _list(ts):
    return ts if isinstance(ts, (list, tuple)) else list(ts)


class _Step:
    """The words of a list of parameters: their checks and addresses, one call
    for each list."""

    def __init__(self, params):
        if not isinstance(params[0], torch.Tensor):
            raise TypeError(f"params[0] must be a tensor, got {type(params[0]).__name__}")
        self.device = params[0].get_device()
        if self.device < 0:
            raise ValueError("params must be device tensors")
        self.count = len(params)
        self.numels = array("q", bytes(8 * self.count))
        self.words = array("q", bytes(8 * _TENSOR_WORDS * self.count))
        _tensor_lists.check(params, -1, "params", _F32_OR_BF16, self.device, self.numels, None, 0, 0)
        self.words[7::_TENSOR_WORDS] = self.numels
        self.blocks, self.copied = None, False

    def put(self, ts, column, name, dtypes, part=-1, numels=None):
        return _tensor_lists.check(ts, part, name, dtypes, self.device, self.numels if numels is None else numels,
                                   self.words, _TENSOR_WORDS, column)

    def put_states(self, avgs, sqs):
        self.states = avgs, sqs
        self.mx8 = len(avgs) > 0 and isinstance(avgs[0], (tuple, list))
        if not self.mx8:
            self.put(avgs, 2, "exp_avgs", _F32)
            self.put(sqs, 3, "exp_avg_sqs", _F32)
            return
        if self.blocks is None:
            self.blocks = array("q", [(n + 31) // 32 for n in self.numels])
        for ts, name, column in ((avgs, "exp_avgs", 2), (sqs, "exp_avg_sqs", 3)):
            self.put(ts, column, name + " codes", _U8, 1)
            self.put(ts, column + 2, name + " scales", _U8, 0, self.blocks)

    def run(self, params, grads, copies, step, lr, betas, eps, weight_decay, grad_scale, seed):
        param = self.put(params, 0, "params", _F32_OR_BF16)
        grad = self.put(grads, 1, "grads", _F32_OR_BF16)
        if copies is not None:
            if param == torch.bfloat16:
                raise ValueError("copies are for fp32 parameters")
            self.put(copies, 6, "copies", _BF16_ONLY)
        elif self.copied:  # the addresses of an earlier step's
            self.words[6::_TENSOR_WORDS] = array("q", bytes(8 * self.count))
        self.copied = copies is not None
        if grad_scale is not None:
            _fit(grad_scale, "grad_scale", params[0], _F32, 1)
        if self.mx8 and seed is None:
            raise ValueError("8-bit states are rounded at random: seed is required")
        if seed is not None and (isinstance(seed, bool) or not isinstance(seed, int) or not 0 <= seed < 1 << 64):
            raise ValueError(f"seed must be an integer of 64 bits, got {seed!r}")
        options = _AdamwOptions(lr, betas[0], betas[1], eps, weight_decay, step, seed or 0, param == torch.bfloat16,
                                grad == torch.bfloat16, self.mx8, seed is not None)
        _launch("trace_adamw_step", params[0], self.words.buffer_info()[0], self.count, ctypes.addressof(options),
                _addr(grad_scale))
        for written in (params, copies or (), *self.states):
            _tensor_lists.changed(written)


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
               grad_scale=None, copies=None, seed=None):
    """One AdamW step over lists of tensors, in place, in fp32 throughout.

    params: all fp32 or all bf16; grads: likewise, independently.  exp_avgs,
    exp_avg_sqs: fp32 tensors, or MXFP8 records (scales u8[ceil(n/32)], codes
    u8[n]) of the first moment and of the second one's square root, zeros to
    begin with (the root keeps its mean; its square settles some 5% above that
    of fp32 states with beta2 = 0.999).  step: 1 for the first.  grad_scale: fp32[1] on the device, a
    factor of every gradient (clipping, unscaling).  copies: bf16 tensors that
    fp32 parameters are rounded into (the forward's weights).  seed: random
    roundings of the records and of bf16 parameters, which keep their means;
    another one for each step.  Without it bf16 parameters go to nearest, and
    records are refused: rounded to nearest they would stand still.

    The numbers are those of the call: a captured graph replays them."""
    params = _list(params)
    if len(params) == 0:
        return
    words = _Step(params)
    words.put_states(_list(exp_avgs), _list(exp_avg_sqs))
    words.run(params, _list(grads), None if copies is None else _list(copies), step, lr, betas, eps, weight_decay,
              grad_scale, seed)


class AdamW:
    """``adamw_step`` with the states of its parameters: fp32 (states="fp32") or
    MXFP8 records (states="mx8").  The random bits of step t are those of seed
    + t; seed None: fp32 states, bf16 parameters rounded to nearest.  lr, betas,
    eps and weight_decay are plain attributes, read at each step.  copies: as for
    ``adamw_step``; a forward pass through them leaves the gradients with them,
    and the step takes a copy's .grad where its parameter has none."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, states="fp32", copies=None,
                 seed=None):
        self.params = list(params)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.copies = None if copies is None else list(copies)
        self.steps, self.seed = 0, seed
        if states not in ("fp32", "mx8"):
            raise ValueError(f'states must be "fp32" or "mx8", got {states!r}')
        if states == "mx8" and seed is None:
            raise ValueError("8-bit states are rounded at random: seed is required")
        if not self.params:
            raise ValueError("no parameters")
        self._words = _Step(self.params)
        self._mx8 = states == "mx8"

        def zeros(p):
            if not self._mx8:
                return torch.zeros(p.shape, dtype=torch.float32, device=p.device)
            n = p.numel()
            return (torch.zeros((n + 31) // 32, dtype=torch.uint8, device=p.device),
                    torch.zeros(n, dtype=torch.uint8, device=p.device))

        self._avgs, self._sqs = [zeros(p) for p in self.params], [zeros(p) for p in self.params]

    def step(self, grads=None, grad_scale=None):
        """One step with these gradients, or the .grad of each parameter or else of
        its copy."""
        params = self.params
        if grads is None:
            grads = [p.grad for p in params]
            if self.copies is not None:
                grads = [c.grad if g is None else g for g, c in zip(grads, self.copies)]
            if any(g is None for g in grads):
                raise ValueError("a parameter has no gradient")
        t = self.steps + 1
        seed = None if self.seed is None else (self.seed + t) % (1 << 64)
        self._words.put_states(self._avgs, self._sqs)  # where they lie now: their storage is the user's to move
        self._words.run(params, _list(grads), self.copies, t, self.lr, self.betas, self.eps, self.weight_decay,
                        grad_scale, seed)
        self.steps = t

    def zero_grad(self):
        for p in (*self.params, *(self.copies or ())):
            p.grad = None

    def state_dict(self):
        """The states themselves, not copies."""
        return {"steps": self.steps, "seed": self.seed, "exp_avgs": list(self._avgs), "exp_avg_sqs": list(self._sqs)}

    def load_state_dict(self, state):
        """Copies states of the same kind and sizes, on any device, into these."""
        pairs = []
        for name, mine in (("exp_avgs", self._avgs), ("exp_avg_sqs", self._sqs)):
            if len(state[name]) != len(mine):
                raise ValueError(f"{name} must be one for each parameter")
            for i, (to, of) in enumerate(zip(mine, state[name])):
                if isinstance(of, (tuple, list)) != self._mx8 or (self._mx8 and len(of) != 2):
                    raise TypeError("the states are of the other kind")
                for a, b in zip(to, of) if self._mx8 else ((to, of),):
                    if not isinstance(b, torch.Tensor) or b.dtype != a.dtype:
                        raise TypeError(f"{name}[{i}] must be of {a.dtype}")
                    if b.numel() != a.numel():
                        raise ValueError(f"{name}[{i}] must hold {a.numel()} elements, got {b.numel()}")
                    pairs.append((a, b))
        for a, b in pairs:  # nothing is changed before all are known to fit
            a.copy_(b.reshape(a.shape))
        self.steps, self.seed = state["steps"], state["seed"]
