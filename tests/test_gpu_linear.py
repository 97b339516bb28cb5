"""Cross-entropy and greedy tokens through the output layer's weights, on the GPU, against the 64-bit
plain forms of head_ref (tolerances derived there)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import HeadRef, make_head, near

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16

# (M, K, V): one token and one class; K below, at and across a 64-wide step; V below, at and across a
# 128- and a 256-row tile; M at the borders of the kernels' row tiles (32, 64, 256)
SHAPES = [(1, 8, 1), (1, 64, 17), (7, 64, 1000), (32, 72, 300), (33, 128, 129), (64, 104, 4099),
          (65, 64, 513), (200, 40, 1001), (256, 64, 256), (257, 256, 777), (520, 1000, 2100)]


@pytest.fixture(autouse=True)
def no_flag():
    gbce.last_error()
    yield


def run_all(h, w, t, reduction="mean", grad=None, ignore_index=-100, ref=None):
    ref = ref or HeadRef(h, w, t, ignore_index, reduction, grad)
    loss, row, lse = gbce.linear_ce_fwd(h, w, t, ignore_index, reduction)
    assert (loss is None) == (reduction == "none")
    near(row, ref.row_loss, ref.row_tol, "row loss")
    near(lse, ref.lse_out, ref.lse_tol, "lse")
    if loss is not None:
        near(loss, ref.loss, ref.loss_tol, "loss")
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse, grad, ignore_index, reduction)
    near(dh, ref.d_hidden, ref.dh_tol, "d_hidden")
    near(dw, ref.d_weight, ref.dw_tol, "d_weight")
    return dh, dw


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M,K,V", SHAPES)
def test_shapes(M, K, V, dtype):
    h, w, t = make_head(M, K, V, dtype, ignored=0.0)
    run_all(h, w, t)
    assert gbce.last_error() == gbce.OK


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("M,K,V", [(50, 64, 333), (300, 136, 1500)])
def test_reductions_with_ignored_rows_and_grad(M, K, V, reduction, dtype):
    h, w, t = make_head(M, K, V, dtype, ignored=0.4)
    g = torch.rand(M if reduction == "none" else 1, device="cuda") + 0.25
    dh, _ = run_all(h, w, t, reduction, g)
    assert bool((dh[t == -100] == 0).all())


# columns that are no multiple of 8, rows with spare columns, bases off 16 bytes: the packed forms
@pytest.mark.parametrize("M,K,V,pad,shift", [(40, 33, 300, 0, 0), (300, 129, 700, 0, 0), (40, 64, 300, 8, 0),
                                             (300, 64, 700, 3, 0), (300, 72, 520, 8, 5), (20, 1, 50, 0, 0)])
def test_strides_and_alignment(M, K, V, pad, shift):
    h, w, t = make_head(M, K, V, BF, pad=pad, shift=shift, ignored=0.1)
    run_all(h, w, t)
    tok, lp = gbce.linear_greedy(h, w)
    ref = HeadRef(h, w)
    near(lp, ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")
    near(ref.x.gather(1, tok[:, None]).squeeze(1), ref.x.amax(1), 2 * ref.D, "the token's logit")


def test_strided_gradients_leave_the_rest():
    h, w, t = make_head(70, 72, 300, BF)
    bh = torch.full((70, 90), 3.0, device="cuda", dtype=BF)
    bw = torch.full((301, 80), 4.0, device="cuda", dtype=BF)
    _, _, lse = gbce.linear_ce_fwd(h, w, t)
    ref = HeadRef(h, w, t)
    gbce.linear_ce_bwd(h, w, t, lse, d_hidden=bh[:, 5:77], d_weight=bw[:300, :72])
    near(bh[:, 5:77], ref.d_hidden, ref.dh_tol, "d_hidden")
    near(bw[:300, :72], ref.d_weight, ref.dw_tol, "d_weight")
    assert bool((bh[:, :5] == 3).all() and (bh[:, 77:] == 3).all())
    assert bool((bw[300] == 4).all() and (bw[:, 72:] == 4).all())


def test_only_one_gradient():
    h, w, t = make_head(70, 72, 300, BF)
    _, _, lse = gbce.linear_ce_fwd(h, w, t)
    both = gbce.linear_ce_bwd(h, w, t, lse)
    a = gbce.linear_ce_bwd(h, w, t, lse, want_weight=False)
    b = gbce.linear_ce_bwd(h, w, t, lse, want_hidden=False)
    assert a[1] is None and b[0] is None
    assert torch.equal(a[0], both[0]) and torch.equal(b[1], both[1])


@pytest.mark.parametrize("M", [5, 300])
def test_every_row_ignored(M):
    h, w, t = make_head(M, 64, 300, BF)
    t.fill_(-100)
    loss, row, lse = gbce.linear_ce_fwd(h, w, t)
    assert bool(torch.isnan(loss)) and bool((row == 0).all()) and bool((lse == 0).all())
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse)
    assert bool((dh == 0).all()) and bool((dw == 0).all())
    assert float(gbce.linear_ce_fwd(h, w, t, reduction="sum")[0]) == 0.0


def test_no_rows():
    h, w, t = make_head(0, 64, 300, BF)
    loss, row, lse = gbce.linear_ce_fwd(h, w, t)
    assert bool(torch.isnan(loss)) and row.numel() == 0
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse)
    assert dh.shape == (0, 64) and bool((dw == 0).all())
    assert gbce.linear_greedy(h, w)[0].numel() == 0


@pytest.mark.parametrize("M", [9, 130])
def test_bad_targets(M):
    h, w, t = make_head(M, 64, 300, BF, ignored=0.2)
    t[3], t[4] = 300, -1
    loss, row, lse = gbce.linear_ce_fwd(h, w, t, reduction="sum")
    assert gbce.last_error() == gbce.ERR_BAD_TARGET
    assert bool(torch.isnan(loss)) and bool(torch.isnan(row[3:5]).all())
    ref = HeadRef(h, w, t, reduction="sum")
    near(row, ref.row_loss, ref.row_tol, "row loss")
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse, reduction="sum")
    assert gbce.last_error() == gbce.ERR_BAD_TARGET
    near(dh, ref.d_hidden, ref.dh_tol, "d_hidden")
    near(dw, ref.d_weight, ref.dw_tol, "d_weight")


def test_ignore_index_as_a_class():
    h, w, t = make_head(100, 64, 300, BF)
    t[::3] = 7
    run_all(h, w, t, ignore_index=7)


@pytest.mark.parametrize("M", [20, 300])
def test_large_and_very_negative_logits(M):
    h, w, t = make_head(M, 64, 500, BF, spread=300.0)
    run_all(h, w, t)
    h2 = torch.full_like(h, 100.0)
    w2 = torch.full_like(w, -100.0)  # every logit -640000: the sum starts from an empty part
    run_all(h2, w2, t)


@pytest.mark.parametrize("M", [20, 300])
def test_nan_and_infinity_stay_in_their_rows(M):
    h, w, t = make_head(M, 64, 500, BF)
    h[2, 5] = float("nan")
    h[4, 6] = float("inf")
    _, row, _ = gbce.linear_ce_fwd(h, w, t)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[2] = bad[4] = True
    assert bool((torch.isnan(row) == bad).all())
    tok, lp = gbce.linear_greedy(h, w)
    assert bool((torch.isnan(lp) == bad).all()) and bool(((tok >= 0) & (tok < 500)).all())


def test_fp16_factors_far_apart_and_far_from_one():
    h, w, t = make_head(200, 64, 300, F16)
    g = torch.ones(200, device="cuda")
    g[::2] = 2.0 ** -12
    run_all(h, w, t, "none", g)
    run_all(h, w, t, "mean", torch.full((1,), 1024.0, device="cuda"))
    run_all(h, w, t, "mean", torch.full((1,), -3.0, device="cuda"))
    run_all(h, w, t, "sum", torch.zeros(1, device="cuda"))


@pytest.mark.parametrize("M,V,K", [(8192, 40000, 72), (2000, 140000, 64)])
def test_several_pieces_of_the_vocabulary(M, V, K):
    # 512 MB of logit gradients hold 32768 and 131072 classes of these rows
    h, w, t = make_head(M, K, V, BF, ignored=0.05)
    run_all(h, w, t)


def test_many_rows_and_a_full_head():
    M, K, V = 1024, 512, 32000
    h, w, t = make_head(M, K, V, BF, ignored=0.02, spread=2.0)
    run_all(h, w, t)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M,K,V", [(1, 8, 1), (1, 64, 5000), (3, 200, 129), (32, 64, 40000), (33, 72, 2433),
                                   (64, 64, 1000), (65, 64, 1000), (300, 136, 1500)])
def test_greedy(M, K, V, dtype):
    h, w, t = make_head(M, K, V, dtype)
    with torch.no_grad():  # each state leans clearly to one token
        h += (8.0 * w[t.clamp_min(0)].float() / w[t.clamp_min(0)].float().square().sum(1, keepdim=True)).to(dtype)
    ref = HeadRef(h, w)
    tok, lp = gbce.linear_greedy(h, w)
    two = ref.x.topk(min(2, V), 1).values
    clear = torch.ones(M, dtype=torch.bool, device="cuda") if V == 1 else two[:, 0] - two[:, 1] > 4 * ref.D
    assert bool((tok == ref.token)[clear].all())
    near(lp, ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")


@pytest.mark.parametrize("M", [2, 40, 300])
def test_greedy_takes_the_lowest_of_equal_tokens(M):
    h, w, t = make_head(M, 64, 3000, BF)
    w[1500:] = w[:1500]  # every logit twice
    w[700] = w[20]
    tok, _ = gbce.linear_greedy(h, w)
    assert bool((tok < 1500).all()) and not bool((tok == 700).any())
    w.zero_()
    assert bool((gbce.linear_greedy(h, w)[0] == 0).all())


def test_gradients_against_differences():
    h, w, t = make_head(60, 64, 200, BF, ignored=0.2)
    _, _, lse = gbce.linear_ce_fwd(h, w, t)
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse)

    def loss(a, b):
        return HeadRef(a, b, t).loss

    g = torch.Generator(device="cuda").manual_seed(5)
    for d, base, other in ((dh, h, "h"), (dw, w, "w")):
        v = torch.randn(base.shape, generator=g, device="cuda", dtype=torch.float64)
        b64, e = base.double(), 1e-4
        if other == "h":
            diff = (F64Loss(b64 + e * v, w, t) - F64Loss(b64 - e * v, w, t)) / (2 * e)
        else:
            diff = (F64Loss(h, b64 + e * v, t) - F64Loss(h, b64 - e * v, t)) / (2 * e)
        ref = HeadRef(h, w, t)
        tol = ((ref.dh_tol if other == "h" else ref.dw_tol) * v.abs()).sum() + 1e-6
        assert abs(float((d.double() * v).sum() - diff)) <= float(tol)


def F64Loss(a, b, t):
    x = a.double() @ b.double().T
    keep = t != -100
    row = torch.logsumexp(x, 1) - x.gather(1, torch.where(keep, t, 0)[:, None]).squeeze(1)
    return (row * keep).sum() / keep.sum()


def test_autograd_form():
    h, w, t = make_head(120, 64, 300, BF, ignored=0.1)
    hidden = h.reshape(4, 30, 64).clone().requires_grad_()
    weight = w.clone().requires_grad_()
    loss = gbce.linear_cross_entropy(hidden, weight, t.reshape(4, 30))
    (loss * 3.0).backward(retain_graph=True)
    ref = HeadRef(h, w, t, grad=torch.tensor([3.0]))
    near(hidden.grad.reshape(120, 64), ref.d_hidden, ref.dh_tol, "d_hidden")
    near(weight.grad, ref.d_weight, ref.dw_tol, "d_weight")
    first = weight.grad.clone()
    weight.grad = None
    (loss * 3.0).backward()
    assert torch.equal(weight.grad, first)  # nothing was consumed
    rows = gbce.LinearCrossEntropyLoss(reduction="none")(hidden, weight, t.reshape(4, 30))
    assert rows.shape == (4, 30)
    near(rows.reshape(-1), ref.row_loss, ref.row_tol, "row loss")


def test_autograd_of_expanded_and_transposed_operands():
    h, w, t = make_head(40, 64, 300, BF)
    one = h[:1].clone().requires_grad_()
    wt = w.T.contiguous().requires_grad_()
    gbce.linear_cross_entropy(one.expand(40, 64), wt.T, t).backward()
    ref = HeadRef(h[:1].expand(40, 64), w, t)
    # the 40 rows' gradients, each rounded, are added in bf16 by autograd
    near(one.grad, ref.d_hidden.sum(0, keepdim=True), ref.dh_tol.sum(0, keepdim=True) +
         2.0 ** -8 * 2 * ref.d_hidden.abs().sum(0, keepdim=True), "gradient of the shared row")
    near(wt.grad.T, ref.d_weight, ref.dw_tol, "d_weight")


def test_same_bits_every_time_and_on_two_streams():
    cases = [make_head(M, 136, 1500, BF, ignored=0.2) for M in (20, 300)]
    want = []
    for h, w, t in cases:
        _, row, lse = gbce.linear_ce_fwd(h, w, t)
        want.append((row, lse, *gbce.linear_ce_bwd(h, w, t, lse), *gbce.linear_greedy(h, w)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s, (h, w, t) in zip(streams, cases):
            _, row, lse = gbce.linear_ce_fwd(h, w, t, stream=s)
            with torch.cuda.stream(s):
                got.append((row, lse, *gbce.linear_ce_bwd(h, w, t, lse), *gbce.linear_greedy(h, w)))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


def test_captured_and_replayed_with_new_values():
    h, w, t = make_head(300, 136, 1500, BF, ignored=0.2)
    h2, w2, t2 = make_head(300, 136, 1500, BF, seed=1, ignored=0.5)
    out = {}

    def step():
        out["fwd"] = gbce.linear_ce_fwd(h, w, t)
        out["bwd"] = gbce.linear_ce_bwd(h, w, t, out["fwd"][2])
        out["tok"] = gbce.linear_greedy(h, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    h.copy_(h2)
    w.copy_(w2)
    t.copy_(t2)
    graph.replay()
    torch.cuda.synchronize()
    ref = HeadRef(h, w, t)
    near(out["fwd"][1], ref.row_loss, ref.row_tol, "row loss")
    near(out["bwd"][0], ref.d_hidden, ref.dh_tol, "d_hidden")
    near(out["bwd"][1], ref.d_weight, ref.dw_tol, "d_weight")
    near(out["tok"][1], ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")


def test_greedy_rows_of_longer_sequences():
    full = torch.randn(6, 9, 64, device="cuda").to(BF)
    w = (torch.randn(900, 64, device="cuda") / 8).to(BF)
    last = full[:, -1]
    assert torch.equal(gbce.linear_greedy(last, w)[0], gbce.linear_greedy(last.contiguous(), w)[0])


@pytest.mark.parametrize("K", [9, 17, 129, 203, 1001])
@pytest.mark.parametrize("M,V", [(20, 333), (300, 515)])
def test_odd_widths_at_every_offset(M, V, K):
    # rows that start at every even offset of 16 bytes, packed and written unaligned
    h, w, t = make_head(M, K, V, BF, shift=1, pad=2, ignored=0.2)
    dh = torch.full((M, K + 2), 3.0, device="cuda", dtype=BF)
    dw = torch.full((V, K + 4), 5.0, device="cuda", dtype=BF)
    _, _, lse = gbce.linear_ce_fwd(h, w, t)
    gbce.linear_ce_bwd(h, w, t, lse, d_hidden=dh[:, 1:K + 1], d_weight=dw[:, 3:K + 3])
    ref = HeadRef(h, w, t)
    near(dh[:, 1:K + 1], ref.d_hidden, ref.dh_tol, "d_hidden")
    near(dw[:, 3:K + 3], ref.d_weight, ref.dw_tol, "d_weight")
    assert bool((dh[:, 0] == 3).all() and (dh[:, K + 1] == 3).all())
    assert bool((dw[:, :3] == 5).all() and (dw[:, K + 3:] == 5).all())


@pytest.mark.parametrize("n", [1, 255, 256, 257])
def test_counted_rows_at_the_borders_of_a_tile(n):
    # a padded batch of 600 rows of which n count
    h, w, t = make_head(600, 72, 700, BF)
    keep = torch.randperm(600, generator=torch.Generator().manual_seed(n))[:n].cuda()
    targets = torch.full_like(t, -100)
    targets[keep] = t[keep]
    run_all(h, w, targets)


@pytest.mark.parametrize("M", [1024, 1025, 2000])
def test_the_two_ways_of_listing_rows(M):
    # up to 1024 rows every CTA lists them, above one CTA does
    h, w, t = make_head(M, 64, 300, BF, ignored=0.5)
    run_all(h, w, t, "none", torch.rand(M, device="cuda"))


def test_split_tiles_of_both_gradients():
    # few output tiles and a long axis: both products are cut along K and added up
    h, w, t = make_head(2100, 264, 9000, BF, ignored=0.1)
    run_all(h, w, t)
    h, w, t = make_head(300, 520, 20000, F16, ignored=0.1)
    run_all(h, w, t, "sum")


def test_matches_the_loss_from_stored_logits():
    # the library's ce_fwd_bwd on fp32 logits formed in 64 bits: the same losses
    h, w, t = make_head(200, 136, 1500, BF, ignored=0.2)
    logits = (h.double() @ w.double().T).float()
    loss, rows = gbce.ce_fwd_bwd_ex(logits, t, want_row_loss=True)
    ref = HeadRef(h, w, t)
    got, row, _ = gbce.linear_ce_fwd(h, w, t)
    near(row, rows, ref.row_tol + 1e-5 * rows.abs(), "row loss")
    near(got, loss, ref.loss_tol + 1e-5 * loss.abs(), "loss")


@pytest.mark.parametrize("M", [20, 64, 300, 1100])
def test_rows_that_do_not_count_may_hold_anything(M):
    h, w, t = make_head(M, 64, 500, BF, ignored=0.4)
    clean = h.clone()
    h[t == -100] = float("nan")
    h[(t == -100) & (torch.arange(M, device="cuda") % 2 == 0)] = float("inf")
    run_all(h, w, t, ref=HeadRef(torch.where((t == -100)[:, None], torch.zeros_like(clean), clean), w, t))


@pytest.mark.parametrize("n", list(range(29, 65, 5)) + [64])
def test_few_rows_shared_out_among_the_groups(n):
    h, w, t = make_head(n, 72, 1111, F16, ignored=0.1)
    run_all(h, w, t)
    tok, lp = gbce.linear_greedy(h, w)
    ref = HeadRef(h, w)
    near(lp, ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")
    near(ref.x.gather(1, tok[:, None]).squeeze(1), ref.x.amax(1), 2 * ref.D, "the token's logit")


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("M,K,V,pad,shift", [(1, 64, 700, 0, 0), (31, 72, 1000, 8, 0), (64, 200, 3001, 0, 0),
                                             (40, 201, 900, 0, 0), (33, 64, 900, 0, 3)])
def test_few_rows_as_they_stand_and_packed(M, K, V, pad, shift, reduction):
    # up to 64 rows are read where they lie if a tensor map can (whole 16-byte rows), with ignored and
    # bad targets among them; odd weights are copied first
    h, w, t = make_head(M, K, V, BF, pad=pad, shift=shift, ignored=0.3)
    if M > 5:
        t[2], t[4] = V + 5, -7
    ref = HeadRef(h, w, t, reduction=reduction)
    gbce.last_error()
    loss, row, lse = gbce.linear_ce_fwd(h, w, t, reduction=reduction)
    assert gbce.last_error() == (gbce.ERR_BAD_TARGET if M > 5 else gbce.OK)
    near(row, ref.row_loss, ref.row_tol, "row loss")
    near(lse, ref.lse_out, ref.lse_tol, "lse")
    if loss is not None:
        near(loss, ref.loss, ref.loss_tol, "loss")
