"""The operators around a policy's layers on a training step, as a user calls them, in cases of real sizes.

The router picks experts for `expert_sort` and weights for `expert_combine`; the loss over the vocabulary starts the
backward pass; the optimiser step ends it. Kinds of cases:

  score      hidden states, output weight, tokens -> each token's loss (minus its log-probability) and log-sum-exp
  score_bwd  the losses' gradients -> the gradients of the hidden states and of the output weight
  route      router logits -> experts, their weights, the experts' counts and the balance loss
  route_bwd  the gradients of the weights and of the balance loss -> the logits' gradients
  adamw      one optimiser step over many tensors, with states in fp32 or in 8-bit records

With `own` false, `run` is the plain form: elementary torch operations in 32 bits.
"""
import itertools
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the token that a rollout has just drawn, scored: latency and the weight's bytes count
        {"name": "score_token", "kind": "score", "tokens": 1, "k": 2048, "vocab": 32768, "ignored": 0.0, "scale": 1.0},
        # a short answer scored on the large hidden size, odd vocabulary, drawn at temperature 0.8
        {"name": "score_answer", "kind": "score", "tokens": 61, "k": 7168, "vocab": 100003, "ignored": 0.0,
         "scale": 1.25},
        # a batch of trajectories scored, prompts and padding ignored
        {"name": "score_batch", "kind": "score", "tokens": 8192, "k": 2048, "vocab": 131072, "ignored": 0.3,
         "scale": 1.0},
        # a short ragged training step
        {"name": "score_bwd_ragged", "kind": "score_bwd", "tokens": 509, "k": 1056, "vocab": 10007, "ignored": 0.1,
         "scale": 1.0},
        # a training step's gradients, prompts and padding ignored
        {"name": "score_bwd", "kind": "score_bwd", "tokens": 8192, "k": 2048, "vocab": 131072, "ignored": 0.3,
         "scale": 1.0},
        # a decoding batch through the router of the MoE layer
        {"name": "route_decode", "kind": "route", "tokens": 24, "experts": 128, "topk": 8, "dtype": "bf16",
         "renormalize": True, "ignored": 0.0},
        # the MoE layer's tokens, padded rows masked
        {"name": "route_layer", "kind": "route", "tokens": 16384, "experts": 128, "topk": 8, "dtype": "fp32",
         "renormalize": True, "ignored": 0.1},
        # the gradients of the same
        {"name": "route_bwd", "kind": "route_bwd", "tokens": 16384, "experts": 128, "topk": 8, "dtype": "fp32",
         "renormalize": True, "ignored": 0.1},
        # a long batch over more experts, weights straight from the softmax
        {"name": "route_bwd_wide", "kind": "route_bwd", "tokens": 65573, "experts": 256, "topk": 6, "dtype": "bf16",
         "renormalize": False, "ignored": 0.0},
        # the norms, gains and biases of a deep model: many small tensors, latency counts
        {"name": "adamw_small", "kind": "adamw", "sizes": "80x2048 40x128 3x1 5x1021", "params": "fp32",
         "grads": "fp32", "states": "fp32", "copies": False},
        # one of eight expert-parallel ranks' experts of a layer and its attention projections, fp32 masters
        {"name": "adamw_layer", "kind": "adamw", "sizes": "16x3145728 16x1572864 2x8388608 2x1048576 2x2048 1x262144",
         "params": "fp32", "grads": "bf16", "states": "fp32", "copies": True},
        # the same with 8-bit states on bf16 weights
        {"name": "adamw_layer_8bit", "kind": "adamw",
         "sizes": "16x3145728 16x1572864 2x8388608 2x1048576 2x2048 1x262144", "params": "bf16", "grads": "bf16",
         "states": "mx8", "copies": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["score", "score", "score_bwd", "route", "route_bwd", "adamw", "adamw"])
    if kind in ("score", "score_bwd"):
        k, vocab = 32 * _log(rng, 4, 224), _log(rng, 128, 131072)
        most = min(8192, 8192 * 2048 * 131072 // (2 * k * vocab))
        tokens = _log(rng, 1 if kind == "score" else 16, max(16, most))
        return {"kind": kind, "tokens": tokens, "k": k, "vocab": vocab, "ignored": round(rng.uniform(0.0, 0.5), 2),
                "scale": rng.choice([1.0, 1.25, 0.7])}
    if kind in ("route", "route_bwd"):
        experts = _log(rng, 4, 512)
        return {"kind": kind, "tokens": _log(rng, 1, 65573 * 256 // max(256, experts)), "experts": experts,
                "topk": rng.randint(1, min(experts, 10)), "dtype": rng.choice(["fp32", "bf16"]),
                "renormalize": rng.random() < 0.5, "ignored": round(rng.uniform(0.0, 0.4), 2)}
    sizes, left = [], 60_000_000
    for _ in range(rng.randint(1, 6)):
        each = _log(rng, 1, 8_000_000)
        count = max(1, min(_log(rng, 1, 60), left // each))
        left -= count * each
        sizes.append(f"{count}x{each}")
        if left < 8_000_000:
            break
    params = rng.choice(["fp32", "bf16"])
    return {"kind": kind, "sizes": " ".join(sizes), "params": params, "grads": rng.choice(["fp32", "bf16"]),
            "states": rng.choice(["fp32", "mx8"]), "copies": params == "fp32" and rng.random() < 0.5}


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _numels(case):
    return [int(n) for part in case["sizes"].split() for c, n in [part.split("x")] for _ in range(int(c))]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 3e-4, 0.1


def _score_inputs(case, g, dev):
    """Hidden states that lean towards their token's row of the output weight, as a trained policy's do."""
    tokens, k, vocab = case["tokens"], case["k"], case["vocab"]
    w = (torch.randn(vocab, k, generator=g, device=dev) * (1.5 / math.sqrt(k))).to(torch.bfloat16)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device=dev)
    lean = torch.rand(tokens, 1, generator=g, device=dev) * 8.0
    x = torch.randn(tokens, k, generator=g, device=dev)
    x += w[targets].float() * lean
    ignored = torch.rand(tokens, generator=g, device=dev) < case["ignored"]
    return {"x": x.to(torch.bfloat16), "w": w, "targets": torch.where(ignored, -100, targets)}


def _route_inputs(case, g, dev):
    popular = torch.randn(case["experts"], generator=g, device=dev) * 0.5
    z = torch.randn(case["tokens"], case["experts"], generator=g, device=dev) * 1.5 + popular
    return {"logits": z.to(_type(case["dtype"])),
            "valid": torch.rand(case["tokens"], generator=g, device=dev) >= case["ignored"]}


def _adamw_inputs(case, g, dev):
    """Parameters, gradients and states after some steps, every tensor a part of one buffer of its kind that starts at
    a multiple of 32 elements; what lies between the parts is zero."""
    numels = _numels(case)
    starts = [0, *itertools.accumulate((n + 31) // 32 * 32 for n in numels)]
    total = starts[-1]
    there = torch.zeros(total + 1, dtype=torch.int32, device=dev)
    there[torch.tensor(starts[:-1], device=dev)] = 1
    ends = torch.tensor([s + n for s, n in zip(starts, numels)], device=dev)
    there.index_add_(0, ends, there.new_full(ends.shape, -1))
    there = there.cumsum(0)[:total].bool()
    p = torch.randn(total, generator=g, device=dev) * 0.02 * there
    loud = torch.exp(torch.randn(total, generator=g, device=dev)) * 1e-3  # each weight's own size of gradients
    grad = torch.randn(total, generator=g, device=dev) * loud * there
    m = torch.randn(total, generator=g, device=dev) * 0.3 * loud * there
    r = loud * there * (0.8 + 0.4 * torch.rand(total, generator=g, device=dev))
    s = {"numels": numels, "starts": starts, "p": p.to(_type(case["params"])), "grad": grad.to(_type(case["grads"])),
         "grad_scale": torch.full((1,), 0.7, device=dev), "step": 100, "seed": 20261 + int(case["copies"])}
    if case["copies"]:
        s["copies"] = s["p"].to(torch.bfloat16)
    if case["states"] == "fp32":
        s["m"], s["v"] = m, r * r
    else:
        s["m_scales"], s["m_codes"] = _record(m, torch.full_like(m, 0.5))
        s["r_scales"], s["r_codes"] = _record(r, torch.full_like(r, 0.5))
    s["params"], s["grads"] = _parts(s, "p"), _parts(s, "grad")
    s["copy_list"] = _parts(s, "copies") if case["copies"] else None
    if case["states"] == "fp32":
        s["states"] = _parts(s, "m"), _parts(s, "v")
    else:
        s["states"] = tuple(list(zip(_parts(s, n + "_scales", 32), _parts(s, n + "_codes"))) for n in ("m", "r"))
    return s


def _parts(s, name, block=1):
    """The tensors of a buffer: of one element, or of one byte for a block, each."""
    return [s[name][a // block:a // block + (n + block - 1) // block] for a, n in zip(s["starts"], s["numels"])]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kind = case["kind"]
    if kind in ("score", "score_bwd"):
        s = _score_inputs(case, g, dev)
        if kind == "score_bwd":  # the forward has been; the policy's advantages over the batch's tokens
            s["lse"] = _score(s, case)["lse"]
            s["grad_loss"] = torch.randn(case["tokens"], generator=g, device=dev) / case["tokens"]
    elif kind in ("route", "route_bwd"):
        s = _route_inputs(case, g, dev)
        if kind == "route_bwd":
            s |= _route(s, case)
            s["grad_weights"] = torch.randn(case["tokens"], case["topk"], generator=g, device=dev) * 0.1
            s["grad_balance"] = torch.full((1,), 0.01 * case["tokens"], device=dev)
    else:
        s = _adamw_inputs(case, g, dev)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _score(s, case):
    valid = (s["targets"] >= 0) & (s["targets"] < case["vocab"])
    z = (s["x"].float() @ s["w"].float().T) * case["scale"]
    top = z.amax(1)
    at = z.gather(1, torch.where(valid, s["targets"], 0).unsqueeze(1)).squeeze(1)
    lse = top + torch.log(torch.exp(z - top.unsqueeze(1)).sum(1))
    return {"loss": torch.where(valid, lse - at, 0.0), "lse": torch.where(valid, lse, 0.0)}


def _score_bwd(s, case):
    valid = (s["targets"] >= 0) & (s["targets"] < case["vocab"])
    at = torch.where(valid, s["targets"], 0)
    x, w = s["x"].float() * valid.unsqueeze(1), s["w"].float()
    p = torch.exp((x @ w.T) * case["scale"] - s["lse"].unsqueeze(1))
    p[torch.arange(at.numel(), device=at.device), at] -= 1.0
    p *= torch.where(valid, s["grad_loss"] * case["scale"], 0.0).unsqueeze(1)
    return {"grad_x": (p @ w).to(torch.bfloat16), "grad_w": (p.T @ x).to(torch.bfloat16)}


def _softmax(z):
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route(s, case):
    experts, topk = case["experts"], case["topk"]
    z, valid = s["logits"].float(), s["valid"].unsqueeze(1)
    p = _softmax(z) * valid
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :topk]
    weights = p.gather(1, order)
    if case["renormalize"]:
        weights = torch.where(valid, weights / weights.sum(1, keepdim=True), 0.0)
    counts = torch.bincount(torch.where(valid, order, experts).flatten(), minlength=experts + 1)
    counts[experts] = s["valid"].sum()
    probs = p.double().sum(0)
    c = counts.double()
    balance = experts * (c[:experts] * probs).sum() / (c[:experts].sum() * c[experts]).clamp(min=1.0)
    return {"ids": torch.where(valid, order, -1), "weights": weights, "counts": counts, "probs": probs.float(),
            "balance": balance.float().view(1)}


def _route_bwd(s, case):
    experts = case["experts"]
    valid, at = s["ids"] >= 0, s["ids"].clamp(min=0)
    p = _softmax(s["logits"].float())
    gw = torch.where(valid, s["grad_weights"], 0.0)
    c = s["counts"].double()
    gp = (s["grad_balance"].double() * experts * c[:experts] / (c[:experts].sum() * c[experts]).clamp(min=1.0)).float()
    gz = p * (gp - (p * gp).sum(1, keepdim=True))
    if case["renormalize"]:  # the weights are the softmax of the chosen logits alone
        w = s["weights"]
        gz.scatter_add_(1, at, w * (gw - (w * gw).sum(1, keepdim=True)))
    else:
        pg = p.gather(1, at) * gw
        gz -= p * pg.sum(1, keepdim=True)
        gz.scatter_add_(1, at, pg)
    return {"grad_logits": (gz * valid[:, :1]).to(_type(case["dtype"]))}


def _mix(h):
    """A 32-bit integer to another one, each bit of which depends on all of its bits."""
    h = h & 0xFFFFFFFF
    h = h ^ (h >> 16)
    h = (h * 0x6A09E667) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * 0xBB67AE85) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random_bits(seed, n, dev):
    """32 random bits for each of n elements, by the seed and their place."""
    at = torch.arange(n, device=dev)
    key = _mix(_mix(_mix(seed & 0xFFFFFFFF) + (seed >> 32)) + (at >> 32))
    return _mix(_mix(at) + key)


def _record(a, u):
    """(E8M0 bytes of 32-element blocks, E4M3 bytes) of a: each element goes to one of its two neighbours on the grid,
    to the one away from zero where the share of the step that it has come passes 1 - u."""
    b = a.view(-1, 32)
    amax = b.abs().amax(1)
    f, e = torch.frexp(amax)
    e = torch.where(amax > 0, (e - torch.where(f > 0.875, 8, 9)).clamp(-127, 127), -127).to(torch.int32)
    z = torch.ldexp(b.abs(), -e.unsqueeze(1))
    step = (torch.frexp(z).exponent - 1).clamp(min=-6) - 3
    z = torch.ldexp(torch.floor(torch.ldexp(z, -step) + u.view(-1, 32)), step)
    codes = torch.copysign(z, b).to(torch.float8_e4m3fn).view(torch.uint8)
    return (e + 127).to(torch.uint8), codes.flatten()


def _of_record(scales, codes):
    z = codes.view(torch.float8_e4m3fn).float().view(-1, 32)
    return torch.ldexp(z, scales.to(torch.int32).unsqueeze(1) - 127).flatten()


def _bf16_up_or_down(p, u):
    """p to one of its two neighbours in bf16, by 16 random bits u."""
    b = p.view(torch.int32)
    return ((b + u.to(torch.int32)) >> 16).to(torch.int16).view(torch.bfloat16)


def _adamw(s, case):
    mx8 = case["states"] == "mx8"
    step, p = s["step"], s["p"].float()
    g = s["grad"].float() * s["grad_scale"]
    m = _of_record(s["m_scales"], s["m_codes"]) if mx8 else s["m"]
    r = _of_record(s["r_scales"], s["r_codes"]) if mx8 else None
    v = r * r if mx8 else s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    r = torch.sqrt(v)
    rate, root = LR / (1 - BETA1 ** step), 1 / math.sqrt(1 - BETA2 ** step)
    p = p * (1 - LR * DECAY) - (m / (r * root + EPS)) * rate
    if mx8 or case["params"] == "bf16":
        bits = _random_bits(s["seed"], p.numel(), p.device)
    s["p"].copy_(_bf16_up_or_down(p, _mix(bits) >> 16) if case["params"] == "bf16" else p)
    if case["copies"]:
        s["copies"].copy_(p)
    if mx8:
        scales, codes = _record(m, (bits & 0xFFFF).float() * 2.0 ** -16)
        s["m_scales"].copy_(scales), s["m_codes"].copy_(codes)
        scales, codes = _record(r, (bits >> 16).float() * 2.0 ** -16)
        s["r_scales"].copy_(scales), s["r_codes"].copy_(codes)
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    return _adamw_outputs(s, case)


def _adamw_outputs(s, case):
    """The whole buffers; records as the values of their scale and code bytes."""
    out = {"p": s["p"]}
    if case["copies"]:
        out["copies"] = s["copies"]
    if case["states"] == "fp32":
        return out | {"m": s["m"], "v": s["v"]}
    for name in ("m", "r"):
        out[name + "_scales"] = s[name + "_scales"].view(torch.float8_e8m0fnu)
        out[name + "_codes"] = s[name + "_codes"].view(torch.float8_e4m3fn)
    return out


def _plain(s):
    case = s["case"]
    if case["kind"] == "route":
        return _route(s, case)
    return {"score": _score, "score_bwd": _score_bwd, "route_bwd": _route_bwd, "adamw": _adamw}[case["kind"]](s, case)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _calls(s):
    import fp4_rollout_guided_amd as tr
    case = s["case"]
    kind = case["kind"]
    if kind == "score":
        loss, lse = tr.linear_cross_entropy(s["x"], s["w"], s["targets"], scale=case["scale"])
        return {"loss": loss, "lse": lse}
    if kind == "score_bwd":
        gx, gw = tr.linear_cross_entropy_bwd(s["grad_loss"], s["x"], s["w"], s["targets"], s["lse"],
                                             scale=case["scale"])
        return {"grad_x": gx, "grad_w": gw}
    if kind == "route":
        ids, weights, counts, probs, balance = tr.expert_route(s["logits"], case["topk"],
                                                               renormalize=case["renormalize"], valid=s["valid"])
        return {"ids": ids, "weights": weights, "counts": counts, "probs": probs, "balance": balance}
    if kind == "route_bwd":
        return {"grad_logits": tr.expert_route_bwd(s["grad_weights"], s["grad_balance"], s["logits"], s["ids"],
                                                   s["weights"], s["counts"], renormalize=case["renormalize"])}
    tr.adamw_step(s["params"], s["grads"], *s["states"], step=s["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
                  weight_decay=DECAY, grad_scale=s["grad_scale"], copies=s["copy_list"], seed=s["seed"])
    return _adamw_outputs(s, case)


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    """Inputs once, outputs once; of the tokens those that are not ignored."""
    kind = case["kind"]
    if kind in ("score", "score_bwd"):
        k, vocab = case["k"], case["vocab"]
        rows = max(1.0, case["tokens"] * (1 - case["ignored"]))
        if kind == "score":
            return {"bytes": 2 * k * (rows + vocab) + 16 * case["tokens"], "flops": 2 * rows * vocab * k}
        return {"bytes": 4 * k * (rows + vocab) + 16 * case["tokens"], "flops": 6 * rows * vocab * k}
    if kind in ("route", "route_bwd"):
        tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
        each = 2 if case["dtype"] == "bf16" else 4
        if kind == "route":
            return {"bytes": tokens * (each * experts + 12 * topk + 1) + 12 * experts, "flops": 4 * tokens * experts}
        return {"bytes": tokens * (2 * each * experts + 16 * topk) + 8 * experts, "flops": 8 * tokens * experts}
    n = sum(_numels(case))
    each = {"fp32": 8, "bf16": 4}[case["params"]] + {"fp32": 4, "bf16": 2}[case["grads"]] + 2 * case["copies"]
    return {"bytes": n * (each + (16 if case["states"] == "fp32" else 4 + 4 / 32)), "flops": 16 * n}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def _exact_score(s, case):
    """A slice of the vocabulary at a time."""
    rows = torch.nonzero((s["targets"] >= 0) & (s["targets"] < case["vocab"])).flatten()
    x, w, at = s["x"][rows].double(), s["w"], s["targets"][rows]
    slices = [(a, min(a + 16384, case["vocab"])) for a in range(0, case["vocab"], 16384)]
    logits = lambda a, b: torch.mm(x, w[a:b].double().t().contiguous()) * case["scale"]  # noqa: E731
    if case["kind"] == "score":
        lse = torch.stack([torch.logsumexp(logits(a, b), 1) for a, b in slices]).logsumexp(0)
        hit = (x * w[at].double()).sum(1) * case["scale"]
        out = {"loss": lse - hit, "lse": lse}
        return {n: torch.zeros(case["tokens"], dtype=torch.float64, device=x.device).index_copy_(0, rows, v)
                for n, v in out.items()}
    g = s["grad_loss"][rows].double().unsqueeze(1) * case["scale"]
    gx, gw = torch.zeros_like(x), torch.empty(w.shape, dtype=torch.float64, device=x.device)
    for a, b in slices:
        p = torch.exp(logits(a, b) - s["lse"][rows].double().unsqueeze(1))
        p -= (at.unsqueeze(1) == torch.arange(a, b, device=at.device)).double()
        p *= g
        gx += torch.mm(p, w[a:b].double())
        gw[a:b] = torch.mm(p.t().contiguous(), x)
    full = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device=x.device)
    return {"grad_x": full.index_copy_(0, rows, gx), "grad_w": gw}


def _exact_route(s, case):
    experts, topk = case["experts"], case["topk"]
    z = s["logits"].double()
    p = torch.softmax(z, 1)
    if case["kind"] == "route":
        valid = s["valid"]
        left, ids = z.clone(), []
        for _ in range(topk):
            best = left.amax(1, keepdim=True)
            ids.append(torch.where(left == best, torch.arange(experts, device=z.device), experts).amin(1))
            left.scatter_(1, ids[-1].unsqueeze(1), -math.inf)
        ids = torch.stack(ids, 1)
        w = torch.softmax(z.gather(1, ids), 1) if case["renormalize"] else p.gather(1, ids)
        pairs = [(ids[valid] == e).sum() for e in range(experts)]
        counts = torch.stack(pairs + [valid.sum()])
        probs = p[valid].sum(0)
        rows = max(1, int(valid.sum()))
        balance = experts * (counts[:experts].double() / max(1, int(sum(pairs))) * (probs / rows)).sum()
        return {"ids": torch.where(valid.unsqueeze(1), ids, -1), "weights": w * valid.unsqueeze(1), "counts": counts,
                "probs": probs, "balance": balance.view(1)}
    z.requires_grad_(True)
    valid, at = s["ids"][:, 0] >= 0, s["ids"].clamp(min=0)
    p = torch.softmax(z, 1)
    w = torch.softmax(z.gather(1, at), 1) if case["renormalize"] else p.gather(1, at)
    c = s["counts"].double()
    balance = experts * (c[:experts] / c[:experts].sum() * (p * valid.unsqueeze(1)).sum(0) / c[experts]).sum()
    total = (w * s["grad_weights"].double() * valid.unsqueeze(1)).sum()
    if bool(valid.any()):
        total = total + balance * s["grad_balance"].double()
    return {"grad_logits": torch.autograd.grad(total.sum(), z)[0]}


def _exact_adamw(s, case):
    step, g, p = s["step"], s["grad"].double() * s["grad_scale"].double(), s["p"].double()
    m = s["m"].double() if "m" in s else _of_record(s["m_scales"], s["m_codes"]).double()
    v = s["v"].double() if "v" in s else _of_record(s["r_scales"], s["r_codes"]).double().square()
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    m_hat, v_hat = m / (1 - BETA1 ** step), v / (1 - BETA2 ** step)
    p = p - LR * DECAY * p - LR * m_hat / (v_hat.sqrt() + EPS)
    bits = _random_bits(s["seed"], p.numel(), p.device)
    if case["params"] == "bf16":
        out = {"p": _exact_up_or_down(p, 8, _mix(bits) >> 16)}
    else:
        out = {"p": p}
    if case["copies"]:
        out["copies"] = p
    if case["states"] == "fp32":
        return out | {"m": m, "v": v}
    for name, a, u in (("m", m, bits & 0xFFFF), ("r", v.sqrt(), bits >> 16)):
        amax = a.abs().view(-1, 32).amax(1)
        e = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0)).clamp(-127, 127), -127.0)
        scale = torch.exp2(e)
        out[name + "_scales"] = scale
        out[name + "_codes"] = _exact_up_or_down(a / scale.repeat_interleave(32), 4, u, 2.0 ** -6)
    return out


def _exact_up_or_down(a, digits, u, least=2.0 ** -126):
    """a in so many binary digits, to one of its two neighbours by 16 random bits; subnormal below `least`."""
    e = torch.floor(torch.log2(a.abs().clamp(min=least)))
    e = e + (torch.exp2(e + 1) <= a.abs()).double() - ((torch.exp2(e) > a.abs()) & (e > math.log2(least))).double()
    step = torch.exp2(e - (digits - 1))
    return torch.copysign(torch.floor(a.abs() / step + u.double() / 65536) * step, a)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("score"):
        return _exact_score(s, case)
    return _exact_route(s, case) if kind.startswith("route") else _exact_adamw(s, case)
