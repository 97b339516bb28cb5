"""Measured work of the output-layer and router losses: the plain forms and the library's calls.

Four operators of a language model's training step and of its answer:

* ``linear_ce_fwd``  cross-entropy of hidden states [M, K] through the output layer's weights [V, K],
  the logits [M, V] never stored: the loss, the row losses and the log-sum-exp of each row;
* ``linear_ce_bwd``  its gradients for the hidden states and the weights ("train" cases run both);
* ``linear_greedy``  the most probable token of each row and its log-probability (decoding);
* ``moe_balance``    a router's balance loss and z-loss with per-expert counts and the logits' gradient.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORE = -100
BALANCE, ZLOSS = 1e-2, 1e-3  # the coefficients that mixture-of-experts training commonly uses


def listed():
    return [
        # evaluation / scoring forward of a large-vocabulary model, 2% of the tokens padding
        dict(name="fwd_8192x128256", op="fwd", M=8192, V=128256, K=4096, dtype="bf16", ignored=0.02,
             reduction="mean", pad=0),
        # scoring a ragged batch whose prompts do not count: odd rows, odd vocabulary, per-row losses
        dict(name="fwd_777x32001_none", op="fwd", M=777, V=32001, K=1000, dtype="f16", ignored=0.3,
             reduction="none", pad=24),
        # a handful of tokens of a small model: latency
        dict(name="fwd_7x1000", op="fwd", M=7, V=1000, K=64, dtype="bf16", ignored=0.0,
             reduction="mean", pad=0),
        # one pre-training step of the 32000-token workload (batch 4 x sequence 2048), 5% ignored
        dict(name="train_8192x32000", op="train", M=8192, V=32000, K=2048, dtype="bf16", ignored=0.05,
             reduction="mean", pad=0),
        # one fine-tuning step on a large vocabulary: half of the tokens are prompt
        dict(name="train_4096x128256_half", op="train", M=4096, V=128256, K=4096, dtype="bf16",
             ignored=0.5, reduction="mean", pad=0),
        # a small head in fp16 with a gradient of its own for each row (weighted tokens)
        dict(name="train_500x5003_none", op="train", M=500, V=5003, K=504, dtype="f16", ignored=0.1,
             reduction="none", pad=0),
        # greedy decoding, one sequence: reading the weights is the whole cost
        dict(name="greedy_1x128256", op="greedy", M=1, V=128256, K=4096, dtype="bf16", pad=0),
        # greedy decoding of a batch whose hidden states are the last positions of longer rows
        dict(name="greedy_33x32000", op="greedy", M=33, V=32000, K=2048, dtype="f16", pad=4096),
        # verifying drafted tokens of many sequences at once
        dict(name="greedy_256x128256", op="greedy", M=256, V=128256, K=2048, dtype="bf16", pad=0),
        # a small mixture's router on a micro-batch: latency
        dict(name="moe_64x8", op="moe", T=64, E=8, k=2, dtype="f32", padded=0.0),
        # a router of 60 experts (rows that are no whole vectors) with a padded batch
        dict(name="moe_8192x60", op="moe", T=8192, E=60, k=4, dtype="bf16", padded=0.1),
        # a large mixture on a whole step's tokens
        dict(name="moe_131072x256", op="moe", T=131072, E=256, k=8, dtype="f32", padded=0.02),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "train", "train", "greedy", "moe", "moe"])
    if op == "moe":
        E = _spread(rng, 4, 512)
        return dict(op=op, T=_spread(rng, 1, 65536), E=E, k=rng.randint(1, min(8, E)),
                    dtype=rng.choice(["f32", "bf16", "f16"]), padded=rng.choice([0.0, 0.05, 0.4]))
    V, K = _spread(rng, 500, 130000), 8 * _spread(rng, 8, 512)
    if rng.random() < 0.15:
        K -= rng.randint(1, 7)  # rows that do not start on 16-byte boundaries
    M = _spread(rng, 1, 256 if op == "greedy" else 8192)
    while op == "train" and M * V * K > 1e12:
        M = (M + 1) // 2
    case = dict(op=op, M=M, V=V, K=K, dtype=rng.choice(["bf16", "bf16", "f16"]),
                pad=rng.choice([0, 0, 8, 256]))
    if op != "greedy":
        case.update(ignored=rng.choice([0.0, 0.05, 0.5]), reduction=rng.choice(["mean", "mean", "sum", "none"]))
    return case


def _ignored_rows(case):
    return min(case["M"] - 1, round(case["M"] * case.get("ignored", 0.0)))


def _padded_tokens(case):
    return min(case["T"] - 1, round(case["T"] * case["padded"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    dt = TYPES[case["dtype"]]
    if case["op"] == "moe":
        T, E, k = case["T"], case["E"], case["k"]
        # router logits with some experts ahead of the others, and the router's own choice
        logits = (normal(T, E) + 0.7 * normal(E)).to(dt)
        experts = logits.float().topk(k, dim=1).indices.contiguous()
        out = torch.randperm(T, device="cuda", generator=gen)[:_padded_tokens(case)]
        experts[out] = -1
        return dict(case=case, logits=logits, experts=experts)
    M, V, K = case["M"], case["V"], case["K"]
    # normalised hidden states; unit-length weight rows up to chance, so that logits spread by about one;
    # each state leans to one token, by a margin that is anything from none to certain (fwd, train) or
    # clear (greedy, where the answer is that token)
    weight = (normal(V, K) / math.sqrt(K)).to(dt)
    lean = torch.randint(0, V, (M,), device="cuda", generator=gen)
    lo, hi = (10.0, 20.0) if case["op"] == "greedy" else (0.0, 15.0)
    z = lo + (hi - lo) * torch.rand(M, 1, device="cuda", generator=gen)
    w = weight[lean].float()
    hidden = normal(M, K)
    hidden += z * w / w.square().sum(1, keepdim=True).clamp_min(1e-6)
    buf = torch.empty(M, K + case["pad"], device="cuda", dtype=dt)
    state = dict(case=case, hidden=buf[:, :K], weight=weight)
    state["hidden"].copy_(hidden)
    if case["op"] == "greedy":
        return state
    lean[torch.randperm(M, device="cuda", generator=gen)[:_ignored_rows(case)]] = IGNORE
    state["targets"] = lean
    # the gradient that comes from the rest of the program: one number, or one for each row
    g = torch.rand(M if case["reduction"] == "none" else 1, device="cuda", generator=gen)
    state["grad"] = (0.5 + g).float()
    return state


# --- the plain forms -------------------------------------------------------------------------------


def _plain_head(s, train):
    case, t = s["case"], s["targets"]
    h, w = s["hidden"].float(), s["weight"].float()
    x = h @ w.T
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    d = e.sum(1, keepdim=True)
    lse = (m + torch.log(d)).squeeze(1)
    keep = t != IGNORE
    at = torch.where(keep, t, 0)
    row = torch.where(keep, lse - x.gather(1, at[:, None]).squeeze(1), 0.0)
    n = keep.sum().float()
    loss = None
    if case["reduction"] != "none":
        loss = (row.double().sum() / (n if case["reduction"] == "mean" else 1.0)).float()
    out = {"loss": loss, "row_loss": row, "lse": torch.where(keep, lse, 0.0)}
    if not train:
        return out
    g = e.div_(d)
    g.scatter_add_(1, at[:, None], torch.full_like(d, -1.0))
    scale = keep * s["grad"]
    if case["reduction"] == "mean":
        scale = scale / n
    g.mul_(scale[:, None])
    dt = s["weight"].dtype
    return {"loss": loss, "row_loss": row, "d_hidden": (g @ w).to(dt), "d_weight": (g.T @ h).to(dt)}


def _plain_greedy(s):
    x = s["hidden"].float() @ s["weight"].float().T
    m = x.amax(1, keepdim=True)
    ids = torch.arange(x.shape[1], device=x.device)
    token = torch.where(x == m, ids, x.shape[1]).amin(1)  # the lowest index of equal ones
    return {"token": token, "logprob": -torch.log(torch.exp(x - m).sum(1))}


def _plain_moe(s):
    logits, ex = s["logits"], s["experts"]
    E, k = logits.shape[1], ex.shape[1]
    keep = (ex >= 0).any(1)
    n = keep.sum().double()
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ex.device)
    flat = torch.where(ex >= 0, ex, E).reshape(-1)
    counts = counts.scatter_add(0, flat, torch.ones_like(flat))[:E]
    x = logits.float()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    d = e.sum(1, keepdim=True)
    lse = (m + torch.log(d)).squeeze(1)
    p = e / d
    kept = keep.float()
    mean = (p * kept[:, None]).double().sum(0) / n
    f = counts.double()
    loss = BALANCE * E / (k * n) * (f * mean).sum() + ZLOSS * (kept * lse).double().square().sum() / n
    # f - sum p f is a small difference of large counts: formed about their mean
    c = (f - f.mean()).float()
    grad = p * (c - (p * c).sum(1, keepdim=True)) * (BALANCE * E / (k * n * n)).float()
    grad = grad + p * (2 * ZLOSS / n * lse.double()).float()[:, None]
    return {"loss": loss.float(), "counts": counts, "grad": (grad * kept[:, None]).to(logits.dtype)}


def _own(s):
    import cross_entropy_loss_ce_gb300 as gbce
    case = s["case"]
    if case["op"] == "moe":
        loss, counts, grad = gbce.moe_balance(s["logits"], s["experts"], BALANCE, ZLOSS)
        return {"loss": loss, "counts": counts, "grad": grad}
    if case["op"] == "greedy":
        token, logprob = gbce.linear_greedy(s["hidden"], s["weight"])
        return {"token": token, "logprob": logprob}
    loss, row, lse = gbce.linear_ce_fwd(s["hidden"], s["weight"], s["targets"], IGNORE, case["reduction"])
    if case["op"] == "fwd":
        return {"loss": loss, "row_loss": row, "lse": lse}
    dh, dw = gbce.linear_ce_bwd(s["hidden"], s["weight"], s["targets"], lse, s["grad"], IGNORE,
                                case["reduction"], row_loss=row)
    return {"loss": loss, "row_loss": row, "d_hidden": dh, "d_weight": dw}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "moe":
        return _plain_moe(state)
    if op == "greedy":
        return _plain_greedy(state)
    return _plain_head(state, op == "train")


# --- the definitions in 64 bits --------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        x = s["logits"].double().requires_grad_()
        E, k = case["E"], case["k"]
        live = s["experts"][(s["experts"] >= 0).any(1)]
        xs = x[(s["experts"] >= 0).any(1)]
        n = xs.shape[0]
        counts = torch.bincount(live[live >= 0], minlength=E)
        share = counts.double() / (k * n)
        loss = BALANCE * E * (share * torch.softmax(xs, 1).mean(0)).sum()
        loss = loss + ZLOSS * torch.logsumexp(xs, 1).square().mean()
        (grad,) = torch.autograd.grad(loss, x)
        return {"loss": loss.detach(), "counts": counts, "grad": grad}
    flops = 2.0 * case["M"] * case["V"] * case["K"] * (3 if case["op"] == "train" else 1)
    if flops > 3e12:
        return None  # the card's 64-bit rate is about 1e12 a second
    h, w = s["hidden"].double(), s["weight"].double()
    if case["op"] == "greedy":
        lp = torch.log_softmax(h @ w.T, 1)
        best = lp.max(1, keepdim=True).values
        ids = torch.arange(lp.shape[1], device=lp.device).expand_as(lp)
        return {"token": ids.masked_fill(lp < best, lp.shape[1]).amin(1), "logprob": best.squeeze(1)}
    h.requires_grad_()
    w.requires_grad_()
    x = torch.nn.functional.linear(h, w)
    t = s["targets"]
    red = case["reduction"]
    row = torch.nn.functional.cross_entropy(x, t, ignore_index=IGNORE, reduction="none")
    loss = None if red == "none" else torch.nn.functional.cross_entropy(x, t, ignore_index=IGNORE, reduction=red)
    if case["op"] == "fwd":
        lse = torch.logsumexp(x, 1).masked_fill(t == IGNORE, 0.0)
        return {"loss": None if loss is None else loss.detach(), "row_loss": row.detach(), "lse": lse.detach()}
    up = s["grad"].double()
    dh, dw = torch.autograd.grad((row if red == "none" else loss.reshape(1)), (h, w), up)
    return {"loss": None if loss is None else loss.detach(), "row_loss": row.detach(), "d_hidden": dh, "d_weight": dw}


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "moe":
        T, E, k = case["T"], case["E"], case["k"]
        n = T - _padded_tokens(case)
        # read the counted tokens' logits and every choice, write the gradient and the counts
        return {"bytes": n * E * es + T * E * es + T * k * 8 + E * 8 + 4, "flops": 10.0 * n * E}
    M, V, K = case["M"], case["V"], case["K"]
    n = M - (_ignored_rows(case) if case["op"] != "greedy" else 0)
    # one product of the counted rows with the weights forward; training needs two more (a form that
    # does not keep the logits pays a fourth, which is not counted here)
    product = 2.0 * n * V * K
    reads = (n * K + V * K) * es + M * 8
    if case["op"] == "train":
        return {"bytes": reads + (M * K + V * K) * es + M * 4, "flops": 3 * product}
    return {"bytes": reads + M * 12, "flops": product}
