"""Errors of the norm that all parts of a sum share, which no number of values averages out (GPU).

A square of an 8- or 11-bit number is short, so the last bits of long fp32 chains of them are not spread evenly
and round down more often than up.  What one call rounds last, the norm to fp32, is off by less than 2^-24 of it
either way, uniformly over norms of all sizes: the mean of N such errors has a standard deviation of at most
2^-24 / sqrt(3 N), 0.018 2^-24 for N = 1024.  Chains of one 16-byte vector, whose errors are not carried, may leave
0.13 2^-24 (fp16, by simulation of the additions; 0.06 for bf16, nothing for fp32).  0.13 and four deviations: 0.2."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [2.0, 1.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_errors_have_no_common_sign(dtype, kind):
    N, n = 1024, 2 ** 18
    g = torch.Generator("cuda").manual_seed(11)
    sizes = torch.rand(N, 1, device="cuda", generator=g) + 0.5  # norms of all significands
    x = (torch.randn(N, n, device="cuda", generator=g) * sizes).to(dtype)
    got = torch.stack([gbce.grad_norm([t], kind) for t in x]).double()
    want = torch.cat([torch.linalg.vector_norm(p.double(), kind, dim=1) for p in x.split(64)])
    mean = float(((got - want) / want).mean()) * 2 ** 24
    assert abs(mean) <= 0.2, mean
