"""64-bit plain forms of the output-layer and router operators, and their tolerances.

Tolerances, from the arithmetic (u = half a step of the stored type: bf16 2^-8, fp16 2^-11):
  logits      products of 16-bit values are exact in fp32; K of them are added in fp32, 16 or more at a
              time, each addition off by at most one step (2^-23, truncation included):
                D = (K / 16 + 8) 2^-23 max_v sum_k |h_k w_vk|   per row.
  lse         a mean of the logits' errors, so D, and a few fp32 roundings: D + 2^-20 (1 + |lse|).
  row loss    lse - x_y: 2 D + 2^-20 (1 + |lse| + |x_y|).
  gradients   G = (p - onehot) k is rounded once to the stored type (u), its p carries 2 D and a few
              fp32 roundings; R terms are added in fp32 and the result is rounded once (u):
                |err| <= (u + 2 D + 2^-19 + (R / 16 + 8) 2^-23) sum |G'| |W| + u |result|,
              with |G'| = (p + onehot) |k|, since p - 1 keeps p's absolute error.  A row's k is formed
              relative to the largest: fp16 entries below 2^-24 / 2^14 of that may be flushed.
              fp16 results below 2^-14 are off by at most half their spacing, 2^-25.
              Every p, product and result below 2^-126, fp32's smallest normal number, may be flushed
              to 0: each of the R terms is off by 2^-126 max(|k|, 1) |W| more, the result by 2^-126.
"""
import torch

U = {torch.float64: 2.0 ** -53, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


class HeadRef:
    """Everything of linear_ce in float64 on the operands' device."""

    def __init__(self, hidden, weight, targets=None, ignore_index=-100, reduction="mean", grad=None):
        h, w = hidden.double(), weight.double()
        self.x = x = h @ w.T
        M, V = x.shape
        K = h.shape[1]
        self.lse = torch.logsumexp(x, 1)
        reach = (h.abs() @ w.abs().T).amax(1) if M else x.new_zeros(0)
        self.D = (K / 16 + 8) * 2.0 ** -23 * reach
        top = x.amax(1, keepdim=True)
        ids = torch.arange(V, device=x.device)
        self.token = torch.where(x == top, ids, V).amin(1) if M else ids[:0]
        self.logprob = top.squeeze(1) - self.lse
        if targets is None:
            return
        keep = targets != ignore_index
        good = keep & (targets >= 0) & (targets < V)
        at = torch.where(good, targets, 0)
        xy = x.gather(1, at[:, None]).squeeze(1)
        nan = float("nan")
        self.row_loss = torch.where(good, self.lse - xy, torch.where(keep, nan, 0.0).to(x))
        self.lse_out = torch.where(good, self.lse, torch.where(keep, nan, 0.0).to(x))
        self.row_tol = 2 * self.D + 2.0 ** -20 * (1 + self.lse.abs() + xy.abs())
        self.lse_tol = self.D + 2.0 ** -20 * (1 + self.lse.abs())
        n = int(keep.sum())
        if reduction == "none":
            self.loss = self.loss_tol = None
        else:
            div = n if reduction == "mean" else 1
            total = self.row_loss.sum()
            self.loss = total / div if div else x.new_tensor(nan)
            self.loss_tol = (self.row_tol * good).sum() / max(div, 1) + 2.0 ** -22 * self.row_loss.abs().nansum() / max(div, 1)
        k = torch.ones(M, dtype=torch.float64, device=x.device)
        if grad is not None:
            k = k * grad.double().to(x.device)
        k = k / max(n, 1) if reduction == "mean" else k
        k = torch.where(good, k, 0.0)
        p = torch.exp(x - self.lse[:, None])
        hot = torch.zeros_like(p).scatter_(1, at[:, None], 1.0)
        G = (p - hot) * k[:, None]
        A = (p + hot) * k.abs()[:, None]
        u = U[hidden.dtype]
        self.d_hidden, self.d_weight = G @ w, G.T @ h
        kmax = float(k.abs().max()) if M else 0.0
        flush = 2.0 ** -126 * max(kmax, 1.0) + (2.0 ** -38 * kmax if hidden.dtype == torch.float16 else 0.0)
        spacing = 2.0 ** -25 if hidden.dtype == torch.float16 else 2.0 ** -126
        rel = u + 2 * self.D[:, None] + 2.0 ** -19
        self.dh_tol = (rel + (V / 16 + 8) * 2.0 ** -23) * (A @ w.abs()) + u * self.d_hidden.abs() \
            + flush * w.abs().sum(0) + spacing
        self.dw_tol = ((A * (rel + (M / 16 + 8) * 2.0 ** -23)).T @ h.abs()) + u * self.d_weight.abs() \
            + flush * h.abs().sum(0) + spacing


def near(got, want, tol, what):
    got, want = got.double(), want.double()
    tol = tol.to(want) if torch.is_tensor(tol) else torch.full_like(want, tol)
    same_nan = torch.isnan(got) == torch.isnan(want)
    assert bool(same_nan.all()), f"{what}: NaN in other places"
    bad = ~torch.isnan(want) & ((got - want).abs() > tol)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; at {i} got {got[i]:.9g} "
                             f"want {want[i]:.9g} tol {tol[i]:.3g}")


def make_head(M, K, V, dtype, seed=0, ignored=0.0, device="cuda", pad=0, shift=0, spread=1.0):
    """(hidden, weight, targets): rows with `pad` spare columns, starting `shift` elements in."""
    g = torch.Generator().manual_seed(1000 * seed + M + 3 * K + 7 * V)
    buf_h = torch.full((M, K + pad + shift), 7.0).to(dtype)
    buf_w = torch.full((V, K + pad + shift), -5.0).to(dtype)
    buf_h[:, shift:shift + K] = (torch.randn(M, K, generator=g) * spread).to(dtype)
    buf_w[:, shift:shift + K] = (torch.randn(V, K, generator=g) / K ** 0.5).to(dtype)
    t = torch.randint(0, V, (M,), generator=g)
    t[torch.rand(M, generator=g) < ignored] = -100
    buf_h, buf_w = buf_h.to(device), buf_w.to(device)
    return buf_h[:, shift:shift + K], buf_w[:, shift:shift + K], t.to(device)


class MoeRef:
    """moe_balance in float64.

    The loss is a mean of products of fp32 numbers, each a few roundings (2^-24) off: 2^-19 of the
    terms' sizes.  A gradient entry p (a E / (k n^2) (f - sum p f) + 2 b / n lse) carries a few fp32
    roundings of each term, f about its mean: 2^-19 of their sizes, then one rounding to its type."""

    def __init__(self, logits, experts, a, b, scale=1.0):
        E, k = logits.shape[1], experts.shape[1]
        good = ((experts >= -1) & (experts < E)).all(1)
        live = good & (experts >= 0).any(1)
        n = int(live.sum())
        ids = experts[live]
        self.counts = torch.bincount(ids[ids >= 0], minlength=E)
        x = logits.double()
        p = torch.softmax(x, 1)
        lse = torch.logsumexp(x, 1)
        f = self.counts.double()
        c = f - f.mean()
        div = max(n, 1)
        ka = a * E / (k * div)
        row = ka * (p @ f) + b * lse * lse
        size = ka * (f.mean() + p @ c.abs()) + b * lse * lse
        self.loss = (row * live).sum() / n if n else x.new_tensor(float("nan"))
        if not bool(good.all()):
            self.loss = x.new_tensor(float("nan"))
        self.loss_tol = 2.0 ** -19 * (size.abs() * live).sum() / div
        dot = p @ c
        term = (scale * ka / div, scale * 2 * b / div)
        g = p * (term[0] * (c - dot[:, None]) + term[1] * lse[:, None])
        s = p * (abs(term[0]) * (c.abs() + (p @ c.abs())[:, None]) + abs(term[1]) * (1 + lse.abs()[:, None]))
        self.grad = torch.where(live[:, None], g, 0.0)
        dt = logits.dtype
        tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -126
        self.grad_tol = 2.0 ** -19 * s + U[dt] * g.abs() + tiny
