"""How exact the output-layer gradients are where the 64-bit forms of head_ref allow more than the kernels
should need: tolerances of their own, from the arithmetic that each test states (GPU)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import HeadRef, U, make_head, near

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def half_step(x, dtype):
    """Half the spacing of dtype's values at x (normal ones, and fp16's subnormal ones)."""
    e = torch.floor(torch.log2(x.double().abs().clamp_min(2.0 ** -126)))
    if dtype == F16:
        e = e.clamp_min(-14)
    return torch.exp2(e) * U[dtype]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("reduction,factor", [("sum", 1.37), ("mean", 0.91), ("sum", -0.73)])
@pytest.mark.parametrize("M", [16, 300])
def test_a_factor_of_all_rows_is_not_rounded_with_the_entries(M, reduction, factor, dtype):
    # Logits near 0 over 9000 classes: every p is about 1.1e-4, less than half a step below 1 (2^-9 in bf16,
    # 2^-12 in fp16), so a target's entry p - 1 rounds to -1, off by p.  The factor is applied in fp32 after
    # the products: a weight row that is one row's target is off by p |h| k, half a step of the others'
    # p |h| k, fp32 roundings (2^-18 of the terms) and the last rounding, half a step of the result.
    V, K = 9000, 64
    h, w, t = make_head(M, K, V, dtype, spread=0.1)
    t = torch.arange(M, device="cuda") * 29 + 5
    g = torch.full((1,), factor, device="cuda")
    loss, _, lse = gbce.linear_ce_fwd(h, w, t, reduction=reduction)
    _, dw = gbce.linear_ce_bwd(h, w, t, lse, g, reduction=reduction)
    k = float(g.double()) / (M if reduction == "mean" else 1)
    p = torch.softmax(h.double() @ w.double().T, 1)
    assert float(p.max()) < 2.0 ** -12
    hot = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
    want = k * (p - hot).T @ h.double()
    tol = abs(k) * ((p * hot + U[dtype] * p + 2.0 ** -18 * (p + hot)).T @ h.double().abs()) + 2.0 ** -38 * abs(k)
    near(dw[t], want[t], tol[t] + half_step(want[t].abs() + tol[t], dtype), "weight rows of the targets")


# --- nearly certain targets ----------------------------------------------------------------------


def certain(M, V, dtype, top, losses):
    """Rows whose target's logit is about ``top`` and whose loss is about losses[r % len]: x = base_r for all
    classes but the target (a column of ones in the weights), plus a little noise."""
    g = torch.Generator().manual_seed(M + V)
    n = len(losses)
    h, w = torch.zeros(M, 64), torch.zeros(V, 64)
    w[:, 0] = 1.0
    t = torch.arange(M) % n * 3 + 1
    r = torch.arange(M) % n
    base = top + torch.log(torch.tensor(losses, dtype=torch.float64) / V)[r]
    h[:, 0] = base.float().to(dtype).float()
    h[torch.arange(M), 1 + r] = 1.0
    w[torch.arange(n) * 3 + 1, 1 + torch.arange(n)] = (top - h[:n, 0]).to(dtype).float()
    h[:, 32:] = torch.randn(M, 32, generator=g) * 0.25
    w[:, 32:] = torch.randn(V, 32, generator=g) * 0.25
    return h.to(dtype).cuda(), w.to(dtype).cuda(), t.cuda()


def certain_tolerances(h, w, t, k):
    """The gradients in 64 bits and their tolerances by |p - onehot|: every entry of G is off by half a step
    of its type (fp16 ones below the smallest normal by 2^-25 / 2^14 at most), by the error of a logit
    against its row's lse, 2 (K / 16 + 8) 2^-23 max |h||w| (head_ref), by four roundings of lse's size and a few
    others (2^-19); sums over 60 classes or the rows in fp32, and half a step of the result."""
    a, b = h.double(), w.double()
    x = a @ b.T
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
    entry = torch.where(hot > 0, torch.expm1(x - lse[:, None]), p)
    # p - 1 from the others, where x - lse cancels in 64 bits too
    entry = torch.where(hot > 0, -(p * (1 - hot)).sum(1, keepdim=True), entry)
    D = (h.shape[1] / 16 + 8) * 2.0 ** -23 * (a.abs() @ b.abs().T).amax(1)
    rel = U[h.dtype] + 2 * D + 4 * lse.abs() * 2.0 ** -24 + 2.0 ** -19
    E = entry.abs()
    tiny = 2.0 ** -39 if h.dtype == F16 else 2.0 ** -126
    both = []
    for want, bound, flat, n in ((entry @ b, (rel[:, None] * E) @ b.abs(), b.abs().sum(0), w.shape[0]),
                                 (entry.T @ a, (rel[:, None] * E).T @ a.abs(), a.abs().sum(0), h.shape[0])):
        size = E @ b.abs() if want.shape == h.shape else E.T @ a.abs()
        tol = k * (bound + (n / 16 + 8) * 2.0 ** -23 * size + tiny * flat)
        both.append((k * want, tol + half_step(k * want.abs() + tol, h.dtype)))
    return both


LOSSES = [1e-2, 1e-3, 1e-4, 1e-5, 1e-6]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M", [10, 300])
@pytest.mark.parametrize("top", [20.0, 100.0])
def test_nearly_certain_targets(M, top, dtype):
    h, w, t = certain(M, 60, dtype, top, LOSSES)
    factor = 1024.0  # a loss scale: fp16 results stay normal numbers
    (dh, dh_tol), (dw, dw_tol) = certain_tolerances(h, w, t, factor)
    a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
    rows = gbce.linear_cross_entropy(a, b, t, reduction="none")
    rows = rows.detach()
    assert float(rows.min()) < 4e-6 and float(rows.max()) < 4e-2
    loss = gbce.linear_cross_entropy(a, b, t, reduction="sum")
    (loss * factor).backward()
    near(a.grad, dh, dh_tol, "d_hidden")
    near(b.grad, dw, dw_tol, "d_weight")
    _, row, lse = gbce.linear_ce_fwd(h, w, t, reduction="sum")
    raw = gbce.linear_ce_bwd(h, w, t, lse, factor, reduction="sum", row_loss=row)
    assert torch.equal(raw[0], a.grad) and torch.equal(raw[1], b.grad)


def test_row_losses_of_another_shape_or_type_are_refused():
    h, w, t = make_head(8, 64, 100, BF)
    _, row, lse = gbce.linear_ce_fwd(h, w, t)
    for wrong in (row[:4], row.double(), row[:, None]):
        with pytest.raises(ValueError, match="row_loss"):
            gbce.linear_ce_bwd(h, w, t, lse, row_loss=wrong)


def test_row_losses_that_a_program_changes_in_place():
    # the rows that linear_cross_entropy returns are the caller's: masking them in place changes no gradient
    h, w, t = make_head(50, 64, 300, BF, ignored=0.2)
    g = torch.rand(50, device="cuda")
    grads = []
    for change in (False, True):
        a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
        rows = gbce.linear_cross_entropy(a, b, t, reduction="none")
        grads.append(torch.autograd.grad((rows.mul_(g) if change else rows * g).sum(), (a, b)))
    assert all(torch.equal(p, q) for p, q in zip(*grads))


# --- long sums -----------------------------------------------------------------------------------
#
# The tensor cores cut every addition (16 products of the axis at a time) toward zero, by one step, 2^-23 of
# the sum or of the largest product, at most (as head_ref has it, whose bounds go by the sum of the products'
# sizes too); N additions lose up to N 2^-23 of that, in one direction, which no rounding to nearest does.


@pytest.mark.parametrize("dtype,K,run", [(F16, 131072, 2048), (BF, 1 << 20, 16384), (F16, 5000, 2048), (F16, 4160, 2048)])
def test_wide_hidden_states(dtype, K, run):
    # logits of about 32 from products of one sign; the tensor cores add up `run` of K at most.  An entry of G:
    # half a step, the error of its logit (run / 16 + 8 additions) against the forward's lse (1024 / 16 + 8).
    M, V = 70, 300
    g = torch.Generator("cuda").manual_seed(K)
    h = (0.5 + torch.rand(M, K, device="cuda", generator=g)).to(dtype)
    size = 32.0 / K * (1 + 0.02 * torch.randn(V, 1, device="cuda", generator=g))
    w = (size * (0.5 + torch.rand(V, K, device="cuda", generator=g))).to(dtype)
    t = torch.arange(M, device="cuda") + 200
    factor = 4096.0 if dtype == F16 else 1.0
    _, _, lse = gbce.linear_ce_fwd(h, w, t, reduction="sum")
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse, factor, reduction="sum")
    a, b = h.double(), w.double()
    x = a @ b.T
    p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    hot = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
    reach = float(x.amax())
    rel = U[dtype] + ((run / 16 + 8) + (1024 / 16 + 8)) * 2.0 ** -23 * reach + 2.0 ** -18
    tiny = factor * 2.0 ** -39 if dtype == F16 else 0.0
    tol = factor * rel * (p + hot).T @ a + tiny * a.sum(0)
    want = factor * (p - hot).T @ a
    near(dw, want, tol + half_step(want.abs() + tol, dtype), "d_weight")
    tol = factor * rel * (p + hot) @ b + tiny * b.sum(0)
    want = factor * (p - hot) @ b
    near(dh, want, tol + half_step(want.abs() + tol, dtype), "d_hidden")


def test_hidden_gradient_of_many_classes():
    # 524288 classes, 76 tiles of two rows of tiles: no tile is cut.  Only the first 64 columns of the hidden
    # states hold anything (cheap logits); the gradient's are all sums over the classes of p W, of one sign.
    # At most 16384 classes are added on the tensor cores: 1024 additions, 2^-13 of the sizes added.  Those are
    # the sum of p W and the target's W (its entry is -1): once that stands in a run's sum, its steps are what
    # the others are cut to.
    M, K, V = 512, 9728, 524288
    g = torch.Generator("cuda").manual_seed(1)
    h = torch.zeros(M, K, device="cuda", dtype=F16)
    h[:, :64] = 0.3 * torch.randn(M, 64, device="cuda", generator=g).to(F16)
    w = torch.empty(V, K, device="cuda", dtype=F16)
    for i in range(0, V, 32768):
        w[i:i + 32768] = 0.5 + torch.rand(32768, K, device="cuda", generator=g).to(F16)
    t = torch.randint(0, V, (M,), device="cuda", generator=g)
    _, _, lse = gbce.linear_ce_fwd(h, w, t, reduction="sum")
    dh, _ = gbce.linear_ce_bwd(h, w, t, lse, None, reduction="sum", want_weight=False)
    rows = torch.arange(0, M, 64, device="cuda")
    x = h[rows, :64].double() @ w[:, :64].double().T
    p = torch.softmax(x, 1)
    sums = torch.zeros(len(rows), K, device="cuda", dtype=torch.float64)
    for i in range(0, V, 32768):
        sums += p[:, i:i + 32768] @ w[i:i + 32768].double()
    target = w[t[rows]].double()
    off = (dh[rows].double() - (sums - target)) / (sums + target)
    assert abs(float(off.mean())) <= 2.0 ** -13
    assert float(off.abs().max()) <= 1024 * 2.0 ** -23 + 2 * U[F16]


def test_weight_gradient_of_many_rows():
    # the same for the weights of classes that are no target: 262144 rows, 76 tiles; at most 16384 rows are
    # added on the tensor cores
    M, K, V = 262144, 4864, 1024
    g = torch.Generator("cuda").manual_seed(2)
    h = 0.5 + torch.rand(M, K, device="cuda", generator=g).to(F16)
    h[:, :64] = torch.randn(M, 64, device="cuda", generator=g).to(F16)
    w = torch.zeros(V, K, device="cuda", dtype=F16)
    w[:, :64] = 0.125 * torch.randn(V, 64, device="cuda", generator=g).to(F16)
    t = torch.zeros(M, device="cuda", dtype=torch.int64)
    _, _, lse = gbce.linear_ce_fwd(h, w, t, reduction="sum")
    _, dw = gbce.linear_ce_bwd(h, w, t, lse, None, reduction="sum", want_hidden=False)
    p = torch.softmax(h[:, :64].double() @ w[:, :64].double().T, 1)
    some = slice(100, 164)
    want = p[:, some].T @ h[:, 4000:4512].double()
    off = (dw[some, 4000:4512].double() - want) / want
    assert abs(float(off.mean())) <= 2.0 ** -13
    assert float(off.abs().max()) <= 1024 * 2.0 ** -23 + 2 * U[F16] + 2.0 ** -18


@pytest.mark.parametrize("dtype", [BF, F16])
def test_an_infinite_factor_stays_in_its_row(dtype):
    h, w, t = make_head(70, 64, 300, dtype)
    g = torch.full((70,), 100.0, device="cuda")
    g[7], g[9] = float("inf"), float("nan")
    ref = HeadRef(h, w, t, reduction="none", grad=torch.where(torch.isfinite(g), g, 1.0))
    _, _, lse = gbce.linear_ce_fwd(h, w, t, reduction="none")
    dh, _ = gbce.linear_ce_bwd(h, w, t, lse, g, reduction="none")
    ok = torch.isfinite(g)
    near(dh[ok], ref.d_hidden[ok], ref.dh_tol[ok], "rows of finite factors")
    assert not bool(torch.isfinite(dh[~ok]).any())


def test_factors_at_the_top_of_fp32():
    # 1.2e38 lies between 2^126 and 2^127
    h, w, t = make_head(70, 64, 300, BF, spread=0.1)
    g = torch.full((70,), 1.2e38, device="cuda")
    w.mul_(0.25)
    ref = HeadRef(h, w, t, reduction="none", grad=g)
    _, _, lse = gbce.linear_ce_fwd(h, w, t, reduction="none")
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse, g, reduction="none")
    near(dh, ref.d_hidden, ref.dh_tol, "d_hidden")
    near(dw, ref.d_weight, ref.dw_tol, "d_weight")


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("factor", [float("nan"), float("inf")])
def test_no_counted_row_leaves_zeros_whatever_the_factor(M, factor):
    # the mean of no row is NaN, and so may be what comes back
    h, w, t = make_head(M, 64, 300, BF)
    t.fill_(-100)
    for reduction in ("mean", "sum", "none"):
        _, row, lse = gbce.linear_ce_fwd(h, w, t, reduction=reduction)
        dh, dw = gbce.linear_ce_bwd(h, w, t, lse, factor, reduction=reduction, row_loss=row)
        assert not bool(dh.any()) and not bool(dw.any())
