"""Measured work of the expert permutation and the gradient norm: the plain forms and the library's calls.

Five operators of a mixture-of-experts model's training step and of its serving:

* ``moe_sort``        the slots [T, k] that a router filled, sorted by expert (stable), each expert's
  rows padded to a multiple of ``align`` where a tiled product wants that: the plan;
* ``moe_dispatch``    the tokens' rows [T, H] in the plan's order ("dispatch" cases with ``train`` run
  its gradient too, the sum over a token's slots);
* ``moe_combine``     the experts' rows back by token, weighted and summed ("combine"; ``train`` runs the
  gradients of the rows and of the weights too);
* ``grad_norm``       the norm of all of a model's gradients;
* ``clip_grad_norm``  the gradients scaled so that this norm is at most ``max_norm``.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token of a decoding sequence, 8 of 128 experts: latency
        dict(name="sort_1x8of128", op="sort", T=1, E=128, k=8, padded=0.0, align=1),
        # a whole training step's tokens of a large mixture, segments padded to the rows of a product's tile
        dict(name="sort_131072x8of256", op="sort", T=131072, E=256, k=8, padded=0.02, align=128),
        # one token of a decoding sequence: its row copied to 8 experts
        dict(name="dispatch_1x2048", op="dispatch", T=1, E=128, k=8, H=2048, dtype="bf16", padded=0.0,
             align=1, pad=0, train=False),
        # a training micro-batch, 4 of 60 experts: rows out, and the gradient back
        dict(name="dispatch_train_8192x2048", op="dispatch", T=8192, E=60, k=4, H=2048, dtype="bf16",
             padded=0.05, align=128, pad=0, train=True),
        # decoding a batch of sequences
        dict(name="combine_33x4096", op="combine", T=33, E=64, k=4, H=4096, dtype="f16", padded=0.0,
             align=1, pad=0, train=False),
        # a long prompt through a large mixture
        dict(name="combine_16384x4096", op="combine", T=16384, E=256, k=8, H=4096, dtype="bf16",
             padded=0.0, align=1, pad=0, train=False),
        # odd rows in full precision, part of them padding: rows that do not start on 16-byte boundaries
        dict(name="combine_train_777x1001", op="combine", T=777, E=17, k=2, H=1001, dtype="f32",
             padded=0.3, align=1, pad=0, train=True),
        # a training step's tokens, forward and both gradients
        dict(name="combine_train_16384x2048", op="combine", T=16384, E=128, k=8, H=2048, dtype="bf16",
             padded=0.02, align=128, pad=0, train=True),
        # a small model's gradients in full precision: latency
        dict(name="norm_small", op="norm", layers=2, width=96, hidden=384, vocab=1000, dtype="f32",
             kind="2", size=3.0, packed=False),
        # a whole model's gradients, matrices in bf16 and vectors in fp32
        dict(name="norm_1e9", op="norm", layers=24, width=2048, hidden=5504, vocab=32000, dtype="mixed",
             kind="2", size=20.0, packed=False),
        # odd sizes packed without gaps into the buffer that the optimiser reads
        dict(name="clip_odd", op="clip", layers=6, width=333, hidden=1001, vocab=5003, dtype="bf16",
             kind="inf", size=20.0, packed=True),
        # a whole model's gradients, clipped into the optimiser's buffers
        dict(name="clip_1e9", op="clip", layers=24, width=2048, hidden=5504, vocab=32000, dtype="mixed",
             kind="2", size=20.0, packed=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "combine", "norm", "clip"])
    if op in ("norm", "clip"):
        width = _spread(rng, 16, 2048)
        case = dict(op=op, layers=rng.randint(1, 24), width=width, hidden=_spread(rng, width, 3 * width - 1),
                    vocab=_spread(rng, 100, 32000), dtype=rng.choice(["f32", "bf16", "f16", "mixed"]),
                    kind=rng.choice(["2", "2", "1", "inf"]), size=rng.choice([0.3, 20.0]),
                    packed=rng.random() < 0.3)
        while work(case)["bytes"] > 5e9:
            case["layers"] -= 1
        return case
    E = _spread(rng, 2, 512)
    k = rng.randint(1, min(8, E))
    case = dict(op=op, T=_spread(rng, 1, 131072 if op == "sort" else 16384), E=E, k=k,
                padded=rng.choice([0.0, 0.05, 0.4]), align=rng.choice([1, 1, 16, 128]))
    if op == "sort":
        return case
    H = 8 * _spread(rng, 2, 512)
    if rng.random() < 0.2:
        H -= rng.randint(1, 7)  # rows that do not start on 16-byte boundaries
    train = rng.random() < 0.6
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    while case["T"] * k * H * (2 if dtype == "f32" else 1) * (2 if train else 1) > 5e8:
        case["T"] = (case["T"] + 1) // 2
    case.update(H=H, dtype=dtype, pad=rng.choice([0, 0, 8, 200]), train=train)
    return case


def _padded_tokens(case):
    return min(case["T"] - 1, round(case["T"] * case["padded"]))


def _plan_rows(case):
    """Rows of a plan: enough for every slot, with any choice of experts."""
    slots, align = case["T"] * case["k"], case["align"]
    return -(-(slots + min(case["E"], slots) * (align - 1)) // align) * align


def _shapes(case):
    """The parameters of a plain decoder: attention and gated projections, norms, embedding and head."""
    w, h = case["width"], case["hidden"]
    layer = [(w, w), (w, w), (w, w), (w, w), (h, w), (h, w), (w, h), (w,), (w,)]
    return [(case["vocab"], w)] + layer * case["layers"] + [(w,), (case["vocab"], w)]


def _type(case, shape):
    if case["dtype"] == "mixed":
        return torch.float32 if len(shape) == 1 else torch.bfloat16
    return TYPES[case["dtype"]]


def _max_norm(case):
    """1, the usual limit; a sum of absolute values grows with the root of their number more."""
    return math.sqrt(sum(math.prod(shape) for shape in _shapes(case))) if case["kind"] == "1" else 1.0


def _buffers(case):
    """For each parameter its buffer and its place there: one buffer a type, places apart by 16 values."""
    used, places = {}, []
    for shape in _shapes(case):
        dt, n = _type(case, shape), math.prod(shape)
        at = used.get(dt, 0)
        places.append((dt, at, shape))
        used[dt] = at + (n if case["packed"] else -(-n // 16) * 16)
    return used, places


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] in ("norm", "clip"):
        used, places = _buffers(case)
        total = sum(math.prod(shape) for _, _, shape in places)
        # gradients whose norm comes out near `size` times the limit, layers of different sizes
        each = case["size"] * (0.18 if case["kind"] == "inf" else total ** -0.5)
        grads = []
        for i, (dt, _, shape) in enumerate(places):
            grads.append(normal(*shape).mul_(each * (0.5 + (i * 7 % 10) / 9)).to(dt))
        state = dict(case=case, grads=grads)
        if case["op"] == "clip":
            state["flat"] = {str(dt): torch.zeros(n, device="cuda", dtype=dt) for dt, n in used.items()}
            state["outs"] = [state["flat"][str(dt)][at:at + math.prod(shape)].view(shape)
                             for dt, at, shape in places]
        return state
    T, E, k = case["T"], case["E"], case["k"]
    # a router's choice with some experts ahead of the others, and its normalised weights
    top = (normal(T, E) + 0.7 * normal(E)).topk(k, dim=1)
    experts = top.indices.contiguous()
    experts[torch.randperm(T, device="cuda", generator=gen)[:_padded_tokens(case)]] = -1
    state = dict(case=case, experts=experts)
    if case["op"] == "sort":
        return state
    state["plan"] = _plain_sort(experts, case)
    H, R, dt = case["H"], _plan_rows(case), TYPES[case["dtype"]]

    def rows(n):
        buf = torch.empty(n, H + case["pad"], device="cuda", dtype=dt)
        buf[:, :H] = normal(n, H).to(dt)
        return buf[:, :H]

    if case["op"] == "dispatch":
        state["x"] = rows(T)
        if case["train"]:
            state["d_rows"] = rows(R)
    else:
        state["y"] = rows(R)
        state["weights"] = torch.softmax(top.values, 1).contiguous()
        if case["train"]:
            state["d_out"] = rows(T)
    return state


# --- the plain forms -------------------------------------------------------------------------------


def _plain_sort(experts, case):
    E, align, R = case["E"], case["align"], _plan_rows(case)
    dev, slots = experts.device, experts.numel()
    key = torch.where(experts >= 0, experts, E).reshape(-1)
    by_expert, order = torch.sort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=dev).scatter_add(0, key, torch.ones_like(key))
    segment = (counts[:E] + align - 1) // align * align
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    offsets[1:] = segment.cumsum(0)
    first = counts.cumsum(0) - counts
    row = offsets[by_expert] + torch.arange(slots, device=dev) - first[by_expert]
    live = by_expert < E
    position = torch.empty(slots, dtype=torch.int64, device=dev)
    position[order] = torch.where(live, row, -1)
    source = torch.full((R + 1,), -1, dtype=torch.int64, device=dev)
    source[torch.where(live, row, R)] = order
    return {"position": position.view_as(experts).int(), "source": source[:R].int(), "offsets": offsets.int(),
            "counts": counts[:E].int()}


def _plain_dispatch(x, plan, k):
    token = plan["source"].long() // k
    live = (plan["source"] >= 0)[:, None]
    return torch.where(live, x[token.clamp_min(0)], 0.0)


def _plain_combine(y, plan, weights):
    p = plan["position"].long()
    live = p >= 0
    terms = torch.where(live[:, :, None], y[p.clamp_min(0)].float(), 0.0)
    if weights is not None:
        terms = terms * torch.where(live, weights, 0.0)[:, :, None]
    return terms.sum(1).to(y.dtype)


def _plain_combine_bwd(d_out, y, plan, weights):
    p, s = plan["position"].long(), plan["source"].long()
    live = p >= 0
    dot = (d_out.float()[:, None, :] * y[p.clamp_min(0)].float()).sum(2)
    at = s.clamp_min(0)
    w = torch.where(s >= 0, weights.reshape(-1)[at], 0.0)
    d_y = (w[:, None] * d_out[at // p.shape[1]].float()).to(y.dtype)
    return d_y, torch.where(live, dot, 0.0)


def _plain_norm(grads, kind):
    if kind == "inf":
        return torch.stack([g.abs().amax().float() for g in grads]).amax()
    if kind == "1":
        return torch.stack([g.float().abs().sum(dtype=torch.float64) for g in grads]).sum().float()
    return torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt().float()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return {"norm": _plain_norm(s["grads"], case["kind"])}
    if op == "clip":
        norm = _plain_norm(s["grads"], case["kind"])
        factor = (_max_norm(case) / (norm + EPS)).clamp_max(1.0)
        [o.copy_(g.float() * factor) for o, g in zip(s["outs"], s["grads"])]
        return {"norm": norm, "clipped": s["flat"]}
    if op == "sort":
        return _plain_sort(s["experts"], case)
    if op == "dispatch":
        out = {"rows": _plain_dispatch(s["x"], s["plan"], case["k"])}
        if case["train"]:
            out["d_x"] = _plain_combine(s["d_rows"], s["plan"], None)
        return out
    out = {"out": _plain_combine(s["y"], s["plan"], s["weights"])}
    if case["train"]:
        out["d_y"], out["d_weights"] = _plain_combine_bwd(s["d_out"], s["y"], s["plan"], s["weights"])
    return out


def _own(s):
    import cross_entropy_loss_ce_gb300 as gbce
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return {"norm": gbce.grad_norm(s["grads"], float(case["kind"]))}
    if op == "clip":
        norm = gbce.clip_grad_norm(s["grads"], _max_norm(case), float(case["kind"]), EPS, outs=s["outs"])
        return {"norm": norm, "clipped": s["flat"]}
    if op == "sort":
        plan = gbce.moe_sort(s["experts"], case["E"], case["align"])
        return {"position": plan.position, "source": plan.source, "offsets": plan.offsets, "counts": plan.counts}
    p = s["plan"]
    plan = gbce.MoePlan(p["position"], p["source"], p["offsets"], p["counts"], case["align"])
    if op == "dispatch":
        out = {"rows": gbce.moe_dispatch(s["x"], plan)}
        if case["train"]:
            out["d_x"] = gbce.moe_combine(s["d_rows"], plan)
        return out
    out = {"out": gbce.moe_combine(s["y"], plan, s["weights"])}
    if case["train"]:
        out["d_y"], out["d_weights"] = gbce.moe_combine_bwd(s["d_out"], s["y"], plan, s["weights"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# --- the definitions in 64 bits --------------------------------------------------------------------


def _exact_plan(experts, case):
    """Expert by expert: where its slots stand, in their order."""
    E, align, R = case["E"], case["align"], _plan_rows(case)
    flat = experts.reshape(-1)
    position, source = torch.full_like(flat, -1), flat.new_full((R,), -1)
    offsets, counts, at = [0], [], 0
    for e in range(E):
        slots = (flat == e).nonzero().squeeze(1)
        n = slots.numel()
        position[slots] = torch.arange(at, at + n, device=flat.device)
        source[at:at + n] = slots
        at += -(-n // align) * align
        offsets.append(at)
        counts.append(n)
    new = dict(device=flat.device, dtype=torch.int32)
    return {"position": position.view_as(experts).int(), "source": source.int(),
            "offsets": torch.tensor(offsets, **new), "counts": torch.tensor(counts, **new)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip"):
        sizes = [g.double() for g in s["grads"]] if sum(g.numel() for g in s["grads"]) < 3e8 else None
        order = float(case["kind"])
        if sizes is not None:
            norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g, order) for g in sizes]), order)
        else:  # a gradient at a time
            norm = torch.linalg.vector_norm(torch.stack(
                [torch.linalg.vector_norm(g, order, dtype=torch.float64) for g in s["grads"]]), order)
        if op == "norm":
            return {"norm": norm}
        factor = min(1.0, _max_norm(case) / (float(norm) + EPS))
        flat = {name: torch.zeros_like(f, dtype=torch.float64) for name, f in s["flat"].items()}
        for g, (dt, at, shape) in zip(s["grads"], _buffers(case)[1]):
            flat[str(dt)][at:at + g.numel()] = g.reshape(-1).double() * factor
        return {"norm": norm, "clipped": flat}
    plan = _exact_plan(s["experts"], case)
    if op == "sort":
        return plan
    T, k, H = case["T"], case["k"], case["H"]
    live = (plan["position"] >= 0).reshape(-1)
    at = plan["position"].reshape(-1).long()[live]
    token = torch.arange(T, device=at.device).repeat_interleave(k)[live]
    if op == "dispatch":
        rows = torch.zeros(_plan_rows(case), H, dtype=torch.float64, device=at.device)
        rows[at] = s["x"].double()[token]
        if not case["train"]:
            return {"rows": rows}
        d_x = torch.zeros(T, H, dtype=torch.float64, device=at.device)
        return {"rows": rows, "d_x": d_x.index_add_(0, token, s["d_rows"].double()[at])}
    y = s["y"].double().requires_grad_(case["train"])
    w = s["weights"].double().requires_grad_(case["train"])
    out = torch.zeros(T, H, dtype=torch.float64, device=at.device)
    out = out.index_add(0, token, y[at] * w.reshape(-1)[live][:, None])
    if not case["train"]:
        return {"out": out}
    d_y, d_w = torch.autograd.grad(out, (y, w), s["d_out"].double())
    return {"out": out.detach(), "d_y": d_y, "d_weights": d_w}


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        values = sum(math.prod(shape) for shape in _shapes(case))
        size = sum(math.prod(shape) * (4 if _type(case, shape) == torch.float32 else 2) for shape in _shapes(case))
        # read once; clipped gradients written once
        return {"bytes": size * (2 if op == "clip" else 1) + 4, "flops": (3.0 if op == "clip" else 2.0) * values}
    T, E, k, R = case["T"], case["E"], case["k"], _plan_rows(case)
    live = T - _padded_tokens(case)
    if op == "sort":
        return {"bytes": T * k * 8 + T * k * 4 + R * 4 + (2 * E + 1) * 4, "flops": 0.0}
    row = case["H"] * (4 if case["dtype"] == "f32" else 2)
    if op == "dispatch":
        size = live * row + R * row + T * k * 4
        if case["train"]:
            size += live * k * row + T * row
        return {"bytes": size, "flops": float(live * k * case["H"]) if case["train"] else 0.0}
    size, flops = live * k * row + T * row + T * k * 8, 2.0 * live * k * case["H"]
    if case["train"]:
        size, flops = size + live * row + R * row + T * k * 4, 5.0 * live * k * case["H"]
    return {"bytes": size, "flops": flops}
