"""Hidden states wider than 1024, whose products the forward and the arg max add up in several runs, against
the 64-bit plain forms of head_ref (tolerances derived there; GPU)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import HeadRef, make_head, near
from test_gpu_linear import run_all

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


# K above 1024 is added up in runs on the tensor cores: an odd and an even number of runs, a last run of one
# 64-wide step, one that is no whole step, odd widths; classes enough for several tiles of a CTA pair (or, up
# to 64 rows, of a CTA)
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("K", [1025, 1032, 1088, 2048, 2056, 3080])
@pytest.mark.parametrize("M,V", [(5, 40000), (40, 40000), (65, 40001), (300, 40000), (600, 20011)])
def test_wide_rows_in_several_runs(M, V, K, dtype):
    h, w, t = make_head(M, K, V, dtype, ignored=0.1)
    t[0] = 17
    ref = HeadRef(h, w, t)
    run_all(h, w, t, ref=ref)
    tok, lp = gbce.linear_greedy(h, w)
    near(lp, ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")
    near(ref.x.gather(1, tok[:, None]).squeeze(1), ref.x.amax(1), 2 * ref.D, "the token's logit")
