"""Refusals of the vocabulary loss, the router and the optimiser step, on the CPU:
every bad argument is turned down before any HIP call (the device addresses
below are never dereferenced)."""
import ctypes

import pytest
import torch

import fp4_rollout_guided_amd as tr
from tests.test_product_abi import E_ALIAS, E_ALIGN, E_NULL, E_SHAPE, OK, buf, call

L = tr.lib


def test_revision():
    assert tr.step_revision() == 1


CE = dict(x=buf(0), w=buf(1), targets=buf(2), tokens=100, vocab=1000, k=96, scale=1.0, workspace=buf(3),
          workspace_bytes=1 << 23, loss=buf(4), lse=buf(5), stream=None)


def test_linear_cross_entropy():
    c = lambda **k: call("trace_linear_cross_entropy", CE, **k)  # noqa: E731
    assert c(tokens=0, x=None, loss=None, lse=None, targets=None, workspace=None) == OK
    for bad in ({"tokens": -1}, {"tokens": 1 << 31}, {"vocab": 0}, {"vocab": -5}, {"vocab": 1 << 31}, {"k": 0}, {"k": 16},
                {"k": 48}, {"k": -32}, {"k": 1 << 20}, {"workspace_bytes": 64}):
        assert c(**bad) == E_SHAPE, bad
    for name in ("x", "w", "targets", "workspace", "loss", "lse"):
        assert c(**{name: None}) == E_NULL, name
    assert c(x=buf(0, 8)) == c(w=buf(1, 2)) == c(targets=buf(2, 4)) == c(workspace=buf(3, 8)) == E_ALIGN
    assert c(loss=buf(4, 2)) == c(lse=buf(5, 1)) == E_ALIGN
    for name in ("x", "w", "targets", "workspace", "lse"):
        assert c(loss=CE[name]) == E_ALIAS, name
    assert c(workspace=buf(1)) == c(lse=buf(0)) == E_ALIAS
    need = L.trace_linear_cross_entropy_workspace_bytes
    assert need(0, 1000, 96) == need(100, 0, 96) == need(100, 1000, 40) == 0
    assert need(1, 32768, 2048) < 1 << 16 and c(workspace_bytes=need(100, 1000, 96) - 1) == E_SHAPE
    # sizes past one launch: refused before anything is enqueued (fake addresses)
    big = dict(x=1 << 44, w=1 << 46, targets=1 << 45, tokens=(1 << 31) - 256, vocab=1 << 20, k=32,
               workspace=1 << 47, workspace_bytes=1 << 46, loss=1 << 42, lse=1 << 43)
    assert c(**big) == E_SHAPE


CEB = dict(grad_loss=buf(6), x=buf(0), w=buf(1), targets=buf(2), lse=buf(5), tokens=100, vocab=1000, k=96, scale=1.0,
           workspace=buf(30), workspace_bytes=1 << 27, grad_x=buf(8), grad_w=buf(9), stream=None)


def test_linear_cross_entropy_bwd():
    c = lambda **k: call("trace_linear_cross_entropy_bwd", CEB, **k)  # noqa: E731
    assert c(grad_x=None, grad_w=None) == OK and c(tokens=0, grad_w=None) == OK
    for bad in ({"tokens": -1}, {"vocab": 0}, {"k": 48}, {"k": 0}, {"workspace_bytes": 64}):
        assert c(**bad) == E_SHAPE, bad
    for name in ("grad_loss", "x", "w", "targets", "lse", "workspace"):
        assert c(**{name: None}) == E_NULL, name
    for name, shift in (("x", 8), ("w", 8), ("grad_x", 8), ("grad_w", 8), ("workspace", 8), ("targets", 4),
                        ("grad_loss", 2), ("lse", 2)):
        assert c(**{name: CEB[name] + shift}) == E_ALIGN, name
    for name in ("grad_loss", "x", "w", "targets", "lse", "workspace", "grad_w"):
        assert c(grad_x=CEB[name]) == E_ALIAS, name
    assert L.trace_linear_cross_entropy_bwd_workspace_bytes(100, 1000, 40) == 0


RT = dict(logits=buf(0), valid=buf(1), tokens=1000, experts=128, topk=8, renormalize=1, workspace=buf(2),
          workspace_bytes=1 << 20, ids=buf(3), weights=buf(4), counts=buf(5), probs=buf(6), balance=buf(7), stream=None)


@pytest.mark.parametrize("fn,each", [("trace_expert_route", 2), ("trace_expert_route_f32", 4)])
def test_expert_route(fn, each):
    c = lambda **k: call(fn, RT, **k)  # noqa: E731
    for bad in ({"tokens": -1}, {"tokens": 1 << 30}, {"experts": 0}, {"experts": 1025}, {"topk": 0}, {"topk": 129},
                {"topk": 65, "experts": 1024}, {"topk": 9, "experts": 8}, {"workspace_bytes": 16}):
        assert c(**bad) == E_SHAPE, bad
    for name in ("logits", "ids", "weights", "counts", "probs", "balance", "workspace"):
        assert c(**{name: None}) == E_NULL, name
    assert c(logits=buf(0, each // 2)) == c(ids=buf(3, 4)) == c(weights=buf(4, 2)) == c(counts=buf(5, 4)) == E_ALIGN
    assert c(probs=buf(6, 2)) == c(balance=buf(7, 2)) == c(workspace=buf(2, 8)) == E_ALIGN
    for name in ("logits", "valid", "workspace", "weights", "counts"):
        assert c(ids=RT[name]) == E_ALIAS, name
    assert c(balance=buf(6, 4)) == E_ALIAS


RTB = dict(grad_weights=buf(1), grad_balance=buf(2), logits=buf(0), ids=buf(3), weights=buf(4), counts=buf(5),
           tokens=1000, experts=128, topk=8, renormalize=1, grad_logits=buf(6), stream=None)


@pytest.mark.parametrize("fn,each", [("trace_expert_route_bwd", 2), ("trace_expert_route_bwd_f32", 4)])
def test_expert_route_bwd(fn, each):
    c = lambda **k: call(fn, RTB, **k)  # noqa: E731
    assert c(tokens=0, logits=None, grad_logits=None) == OK
    assert c(tokens=-1) == c(experts=0) == c(experts=2000) == c(topk=0) == c(topk=65) == E_SHAPE
    for name in ("logits", "ids", "weights", "counts", "grad_logits"):
        assert c(**{name: None}) == E_NULL, name
    for name in ("grad_weights", "grad_balance", "ids", "weights", "counts"):
        assert c(grad_logits=RTB[name]) == E_ALIAS, name
        assert c(**{name: RTB[name] + 1}) == E_ALIGN, name
    assert c(grad_logits=buf(0, 64)) == E_ALIAS  # in place is exact or not at all


class Tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "avg", "sq", "avg_scales", "sq_scales", "copy")] + [
        ("n", ctypes.c_int64)]


def step(tensors, scale=None, count=None, **options):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, seed=5, param_bf16=0, grad_bf16=0,
             states_mx8=0, randomly=0)
    assert set(options) <= set(o)
    o = tr._AdamwOptions(*{**o, **options}.values())
    many = (Tensor * max(1, len(tensors)))(*[Tensor(*t) for t in tensors])
    return L.trace_adamw_step(many, len(tensors) if count is None else count, ctypes.byref(o), scale, None)


ONE = (buf(0), buf(1), buf(2), buf(3), None, None, None, 1000)
REC = (buf(0), buf(1), buf(2), buf(3), buf(4), buf(5), None, 1000)


def but(t, i, v):
    return t[:i] + (v,) + t[i + 1:]


def test_adamw_step():
    assert step([]) == OK and step([but(ONE, 7, 0)]) == OK
    assert L.trace_adamw_step(None, 1, None, None, None) == E_NULL
    assert step([ONE], count=-1) == E_SHAPE and step([but(ONE, 7, -1)]) == E_SHAPE
    for bad in ({"step": 0}, {"step": -3}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0}, {"beta2": float("nan")},
                {"eps": -1.0}, {"eps": float("inf")}, {"lr": float("nan")}, {"weight_decay": float("inf")}):
        assert step([ONE], **bad) == E_SHAPE, bad
    for i in range(4):
        assert step([but(ONE, i, None)]) == E_NULL, i
        assert step([but(ONE, i, ONE[i] + 8)]) == E_ALIGN, i
        assert step([but(REC, i, REC[i] + 4)], states_mx8=1) == E_ALIGN, i
    assert step([but(REC, 4, None)], states_mx8=1) == step([but(REC, 5, None)], states_mx8=1) == E_NULL
    assert step([but(ONE, 6, buf(6))], param_bf16=1) == E_SHAPE  # copies are of fp32 parameters
    assert step([but(ONE, 6, buf(6, 8))]) == E_ALIGN
    assert step([ONE], scale=buf(7, 2)) == E_ALIGN


def test_adamw_step_overlaps():
    for i in range(4):
        for j in range(4):
            if i < j:
                assert step([but(ONE, j, ONE[i])]) == E_ALIAS, (i, j)
    assert step([but(ONE, 6, buf(1, 16))]) == E_ALIAS  # the copy on the gradients
    other = tuple(a + (1 << 22) if a else a for a in ONE[:7]) + (1000,)
    for i in (0, 2, 3):
        assert step([ONE, but(other, i, ONE[i])]) == E_ALIAS, i  # an element of two tensors
        assert step([ONE, but(other, i, ONE[i] + 4000 - 16)]) == E_ALIAS, i
    assert step([ONE], scale=buf(3, 400)) == E_ALIAS
    assert step([REC, but(tuple(a + (1 << 22) if a else a for a in REC[:7]) + (1000,), 4, buf(4, 31))],
                states_mx8=1) == E_ALIAS
    many = [tuple(a + (i << 12) if a else a for a in ONE[:7]) + (1000,) for i in range(40)]
    assert step(many[::-1] + [many[17]]) == E_ALIAS


def test_binding_refuses_host_tensors():
    x, w, t = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        tr.linear_cross_entropy(x, w, t)
    with pytest.raises(ValueError):
        tr.expert_route(torch.zeros(4, 8), 2)
    f = [torch.zeros(8)]
    with pytest.raises(ValueError):
        tr.adamw_step(f, f, f, f, 1, 1e-3)
    with pytest.raises(ValueError):
        tr.AdamW(f)
    with pytest.raises(TypeError):
        tr.adamw_step([1], f, f, f, 1, 1e-3)
    assert tr.adamw_step([], [], [], [], 1, 1e-3) is None
