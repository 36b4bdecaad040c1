"""AdamW's class: copies of the weights, their gradients, states that move, and checkpoints."""
import copy
import io
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def test_copies_given_up(device):
    """Copies that the optimiser has no more are not written to."""
    import fp4_rollout_guided_amd as tr
    _say("case copies given up")
    params = [torch.randn(n, device=device) for n in (100, 5000, 3)]
    copies = [torch.empty(n, dtype=torch.bfloat16, device=device) for n in (100, 5000, 3)]
    opt = tr.AdamW(params, lr=0.1, copies=copies)
    grads = [torch.randn_like(p) for p in params]
    opt.step(grads)
    assert all(torch.equal(c, p.to(torch.bfloat16)) for c, p in zip(copies, params))
    former = [c.clone() for c in copies]
    opt.copies = None
    opt.step(grads)
    assert all(torch.equal(c, f) for c, f in zip(copies, former))
    assert not torch.equal(params[1].to(torch.bfloat16), former[1])
    opt.copies = copies
    opt.step(grads)
    assert all(torch.equal(c, p.to(torch.bfloat16)) for c, p in zip(copies, params))


@pytest.mark.parametrize("states", ["fp32", "mx8"])
def test_states_that_moved(device, states):
    """A step works on the states where they lie now, not where they lay when they were made."""
    import fp4_rollout_guided_amd as tr
    _say("case moved states", states)
    make = lambda: [torch.nn.Parameter(torch.linspace(-1, 1, n, device=device)) for n in (70, 4100)]  # noqa: E731
    grads = [torch.randn(n, device=device) for n in (70, 4100)]
    a, b = make(), make()
    one, two = (tr.AdamW(p, lr=0.1, states=states, seed=3) for p in (a, b))
    one.step(grads), two.step(grads)
    flat = lambda o: [t for k in ("exp_avgs", "exp_avg_sqs") for s in o.state_dict()[k]  # noqa: E731
                      for t in (s if isinstance(s, tuple) else (s,))]
    former = [t.data for t in flat(two)]
    held = [t.clone() for t in former]
    for t in flat(two):
        t.data = t.data.clone()
    one.step(grads), two.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(x, y) for x, y in zip(flat(one), flat(two)))
    assert all(torch.equal(x, y) for x, y in zip(former, held))
    for t in flat(two):
        t.data = t.data.cpu()
    with pytest.raises(ValueError):
        two.step(grads)
    assert two.steps == 2
    for t in flat(two):
        t.data = t.data.to(device)
    one.step(grads), two.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("states", ["fp32", "mx8"])
def test_backward_sees_all_that_the_step_writes(device, states):
    """A graph that saved a copy refuses its backward pass; states count their writes as well."""
    import fp4_rollout_guided_amd as tr
    _say("case versions of copies", states)
    w = torch.randn(64, 64, device=device)
    c = w.to(torch.bfloat16)
    if states == "fp32":
        m, v = torch.zeros_like(w), torch.zeros_like(w)
        written = [m, v]
    else:
        m, v = ((torch.zeros(128, dtype=torch.uint8, device=device), torch.zeros(4096, dtype=torch.uint8, device=device)) for _ in range(2))
        written = [*m, *v]
    y = (torch.randn(64, 64, device=device).to(torch.bfloat16).requires_grad_(True) @ c).sum()
    before = [t._version for t in written]
    tr.adamw_step([w], [torch.ones_like(w)], [m], [v], 1, 1e-3, copies=[c], seed=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    assert all(t._version > b for t, b in zip(written, before))


def test_gradients_of_copies(device):
    """The forward's weights are the copies: their gradients are the step's, and zero_grad clears them."""
    import fp4_rollout_guided_amd as tr
    _say("case gradients of copies")
    masters = [torch.nn.Parameter(torch.randn(s, device=device)) for s in ((48, 32), (48,))]
    other = [p.detach().clone() for p in masters]
    copies = [p.detach().to(torch.bfloat16).requires_grad_(True) for p in masters]
    opt = tr.AdamW(masters, lr=0.1, copies=(c for c in copies))
    m, v = ([torch.zeros_like(p) for p in other] for _ in range(2))
    x = torch.randn(7, 32, device=device).to(torch.bfloat16)
    for t in (1, 2):
        opt.zero_grad()
        assert all(c.grad is None for c in copies)
        (x @ copies[0].t() + copies[1]).float().square().sum().backward()
        grads = [c.grad.clone() for c in copies]
        opt.step()
        tr.adamw_step(other, grads, m, v, t, 0.1)
        assert all(torch.equal(a, b) for a, b in zip(masters, other))
        assert all(torch.equal(c, p.to(torch.bfloat16)) for c, p in zip(copies, other))
    # a parameter's own gradient comes first
    for p in masters:
        p.grad = torch.ones_like(p)
    opt.step()
    tr.adamw_step(other, [torch.ones_like(p) for p in other], m, v, 3, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(masters, other))
    opt.zero_grad()
    assert all(t.grad is None for t in (*masters, *copies))
    with pytest.raises(ValueError):
        opt.step()


@pytest.mark.parametrize("states", ["fp32", "mx8"])
def test_checkpoint_on_the_host(device, states):
    """States saved, read back to the host, and loaded."""
    import fp4_rollout_guided_amd as tr
    _say("case checkpoint", states)
    make = lambda: [torch.nn.Parameter(torch.linspace(-1, 1, n, device=device).view(-1, 10)) for n in (70, 4100)]  # noqa: E731
    a, b = make(), make()
    grads = [torch.randn_like(p) for p in a]
    one, two = tr.AdamW(a, lr=0.1, states=states, seed=3), tr.AdamW(b, lr=0.1, states=states, seed=8)
    one.step(grads)
    file = io.BytesIO()
    torch.save(one.state_dict(), file)
    file.seek(0)
    saved = torch.load(file, map_location="cpu", weights_only=True)
    for p, q in zip(b, a):
        p.data.copy_(q.data)
    lists = copy.deepcopy(saved)
    if states == "mx8":  # as other containers give them back
        lists["exp_avgs"] = [list(s) for s in lists["exp_avgs"]]
    for state in (saved, lists):
        two.load_state_dict(state)
        assert two.steps == 1 and two.seed == 3
        for x, y in zip(one.state_dict()["exp_avgs"] + one.state_dict()["exp_avg_sqs"],
                        two.state_dict()["exp_avgs"] + two.state_dict()["exp_avg_sqs"]):
            for s, t in zip(x, y) if states == "mx8" else ((x, y),):
                assert t.is_cuda and torch.equal(s, t)
    one.step(grads), two.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    short = dict(saved, exp_avgs=saved["exp_avgs"][:1])
    with pytest.raises((TypeError, ValueError)):
        two.load_state_dict(short)
    with pytest.raises((TypeError, ValueError)):
        two.load_state_dict(dict(saved, exp_avg_sqs=saved["exp_avg_sqs"][::-1]))
    assert two.steps == 2
