"""How exact the output-layer gradients are where the 64-bit forms of head_ref allow more than the kernels
should need: tolerances of their own, from the arithmetic that each test states (GPU)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import U, make_head, near

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
