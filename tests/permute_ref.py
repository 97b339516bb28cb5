"""64-bit plain forms of the expert permutation and of the norm of many tensors, and their tolerances.

Tolerances, from the arithmetic (u = half a step of the stored type: bf16 2^-8, fp16 2^-11, fp32 2^-24;
one fp32 rounding is 2^-24):
  dispatch   copies bits: equal.
  combine    k products are added in fp32, one rounding each, and the sum is rounded to its type:
               (k + 1) 2^-24 sum_j |w_j y_j| + u |out|.
  d_y        a product in fp32, rounded to its type: (2^-24 + u) |w d_out|.
  d_weights  H products added in fp32: a lane adds one of 32 of them (or fewer), then 5 and at most 8
             sums are joined: (H / 32 + 16) 2^-24 sum_h |d_out_h y_h| + u |d_w|.
  norms      64 + 1 terms are added in fp32, each at most 2^-24 off; sums of those carry their errors
             (2^-24 once more) and end in fp64.  Sums are relatively 68 2^-24 off, their root half of
             that, rounded once; the maximum is exact.
  clipped    f carries the norm's error, f and the product are rounded to fp32, the result to its type.
fp32 results below 2^-126 may be flushed to 0, each term and the result; fp16 results below 2^-14 are off
by at most half their spacing, 2^-25.
"""
import torch

from head_ref import U, near  # noqa: F401

FLUSH = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float64: 0.0}


class PlanRef:
    """The plan of experts [T, k], an expert at a time."""

    def __init__(self, experts, E, align=1):
        T, k = experts.shape
        flat = experts.reshape(-1).cpu()
        n = flat.numel()
        self.rows = -(-(n + min(E, n) * (align - 1)) // align) * align
        position, source = torch.full_like(flat, -1), torch.full((self.rows,), -1, dtype=torch.int64)
        offsets, counts, at = [0], [], 0
        by = torch.where((flat >= 0) & (flat < E), flat, E)
        slots = torch.argsort(by, stable=True)
        ends = torch.bincount(by, minlength=E + 1).cumsum(0).tolist()
        for e in range(E):
            mine = slots[ends[e - 1] if e else 0:ends[e]]
            c = mine.numel()
            position[mine] = torch.arange(at, at + c)
            source[at:at + c] = mine
            at += -(-c // align) * align
            offsets.append(at)
            counts.append(c)
        self.position = position.reshape(T, k).int().to(experts.device)
        self.source = source.int().to(experts.device)
        self.offsets = torch.tensor(offsets, dtype=torch.int32, device=experts.device)
        self.counts = torch.tensor(counts, dtype=torch.int32, device=experts.device)

    def check(self, plan):
        for name in ("position", "source", "offsets", "counts"):
            got, want = getattr(plan, name), getattr(self, name)
            assert got.dtype == torch.int32 and got.shape == want.shape, name
            assert torch.equal(got, want), f"{name}: {int((got != want).sum())} differ"


def combine_ref(y, position, weights):
    """(out, tolerance): a slot at a time."""
    T, k = position.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
    size = torch.zeros_like(out)
    for j in range(k):
        p = position[:, j].long()
        term = y[p.clamp_min(0)].double() if y.shape[0] else torch.zeros_like(out)
        if weights is not None:
            term = term * weights[:, j].double()[:, None]
        term = torch.where((p >= 0)[:, None], term, 0.0)
        out += term
        size += term.abs()
    return out, (k + 1) * (2.0 ** -24 * size + 2.0 ** -126) + U[y.dtype] * out.abs() + FLUSH[y.dtype]


def combine_bwd_ref(d_out, y, position, weights):
    """((d_y, tolerance), (d_weights, tolerance))."""
    T, k = position.shape
    H = y.shape[1]
    d_y = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    d_w = torch.zeros(T, k, dtype=torch.float64, device=y.device)
    size = torch.zeros_like(d_w)
    g = d_out.double()
    for j in range(k):
        p = position[:, j].long()
        t = (p >= 0).nonzero().squeeze(1)
        d_y[p[t]] = weights[t, j].double()[:, None] * g[t]
        prod = g[t] * y[p[t]].double()
        d_w[t, j] = prod.sum(1)
        size[t, j] = prod.abs().sum(1)
    dt, wt = y.dtype, weights.dtype
    return (d_y, (2.0 ** -24 + U[dt]) * d_y.abs() + FLUSH[dt]), \
        (d_w, (H / 32 + 16) * 2.0 ** -24 * size + U[wt] * d_w.abs() + FLUSH[wt] + H * 2.0 ** -126)


def norm_ref(tensors, kind):
    """(norm, relative tolerance) of tensors as one vector; values below 2^-126 may count as 0."""
    parts = [t.double().abs() for t in tensors if t.numel()]
    if not parts:
        return torch.zeros((), dtype=torch.float64), 0.0
    if kind == float("inf"):
        return torch.stack([p.amax() for p in parts]).amax(), 0.0
    if kind == 2.0:
        parts = [p.square() for p in parts]
    least = 2.0 ** -126 if kind == 1.0 else 2.0 ** -252
    total = torch.stack([p.sum() for p in parts]).sum()
    lost = float(torch.stack([torch.where(p < least, p, 0.0).sum() for p in parts]).sum() / total) if total > 0 else 0.0
    return (total, 70 * 2.0 ** -24 + lost) if kind == 1.0 else (total.sqrt(), 36 * 2.0 ** -24 + lost)


def clip_ref(tensor, norm, rel, max_norm, eps):
    """(clipped, tolerance) of one tensor."""
    f = min(1.0, max_norm / (float(norm) + eps))
    out = tensor.double() * f
    if f == 1.0:
        return out, torch.zeros_like(out)
    return out, (rel + 2 * 2.0 ** -24 + U[tensor.dtype]) * out.abs() + FLUSH[tensor.dtype]
