"""Outputs that share memory with a call's operands are refused, columns of one buffer are not (the check
itself on the CPU, the calls on the GPU)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce


def refused(out, t):
    try:
        gbce._apart("grad", out, ("logits", t))
    except ValueError as e:
        assert str(e) == "grad shares memory with logits"
        return True
    return False


def views():
    flat = torch.zeros(400)
    wide = flat[:320].view(16, 20)
    return flat, wide


def test_every_overlap_is_seen():
    # all pairs of views of one buffer, against the elements that they hold
    flat, _ = views()
    base = torch.arange(400)
    kinds = [(r, c, s, o) for r in (1, 2, 5) for c in (1, 4, 9) for s in (9, 20) for o in (0, 3, 9, 10, 11, 20, 45)
             if s >= c and o + (r - 1) * s + c <= 400]
    for r, c, s, o in kinds:
        a = flat.as_strided((r, c), (s, 1), o)
        mine = set(base.as_strided((r, c), (s, 1), o).flatten().tolist())
        for r2, c2, s2, o2 in kinds:
            b = flat.as_strided((r2, c2), (s2, 1), o2)
            shares = bool(mine & set(base.as_strided((r2, c2), (s2, 1), o2).flatten().tolist()))
            if shares:
                assert refused(a, b), (r, c, s, o, r2, c2, s2, o2)
            elif s == s2 and r > 1 and r2 > 1 and (o2 - o) % s >= c and (o2 - o) % s + c2 <= s:
                assert not refused(a, b)  # side by side


def test_columns_of_one_buffer_and_other_types():
    _, wide = views()
    assert not refused(wide[:, :10], wide[:, 10:]) and not refused(wide[:, 10:], wide[2:, :10])
    assert refused(wide[:, :11], wide[:, 10:]) and refused(wide[1:], wide[:-1]) and refused(wide, wide)
    ints = torch.zeros(16, 10, dtype=torch.int64)  # rows of 80 bytes, as 20 floats
    assert not refused(ints.view(torch.float32)[:, :16], ints[:, 8:])
    assert refused(ints.view(torch.float32)[:, :17], ints[:, 8:])
    gbce._apart("grad", wide, ("experts", None))


gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("T", [40, 600])
def test_router_gradients_beside_and_over_their_logits(T):
    g = torch.Generator("cuda").manual_seed(T)
    buf = torch.randn(T + 1, 32, device="cuda", generator=g)
    x = buf[:T, :16]
    ex = x.topk(2, 1).indices.contiguous()
    want = gbce.moe_balance(x, ex, 0.1, 0.01)
    for grad in (buf[1:, :16], buf[:T, 8:24], buf.view(-1)[:T * 16].view(T, 16), buf.view(-1)[1:1 + T * 32].view(T, 32)[:, :16]):
        with pytest.raises(ValueError, match="grad shares memory with logits"):
            gbce.moe_balance(x, ex, 0.1, 0.01, grad=grad)
    ids = torch.empty(T, 8, device="cuda", dtype=torch.int64)
    ids[:, :2] = ex
    with pytest.raises(ValueError, match="grad shares memory with experts"):
        gbce.moe_balance(x, ids[:, :2], 0.1, 0.01, grad=ids.view(torch.float32))
    scale = buf[T, 31:].fill_(1.0)
    with pytest.raises(ValueError, match="grad shares memory with grad_scale"):
        gbce.moe_balance(buf[1:, :16].clone(), ex, 0.1, 0.01, grad_scale=scale, grad=buf[1:, 16:])
    beside = gbce.moe_balance(x, ex, 0.1, 0.01, grad=buf[:T, 16:])
    assert all(torch.equal(a, b) for a, b in zip(beside, want))
    over = gbce.moe_balance(x, ex, 0.1, 0.01, grad=x)
    assert torch.equal(over[2], want[2]) and torch.equal(over[0], want[0])


@gpu
def test_hidden_gradients_beside_and_over_the_operands():
    g = torch.Generator("cuda").manual_seed(3)
    buf = torch.randn(70, 128, device="cuda", generator=g).bfloat16()
    h, w = buf[:, :64], (torch.randn(300, 64, device="cuda", generator=g) / 8).bfloat16()
    t = torch.randint(0, 300, (70,), device="cuda", generator=g)
    _, row, lse = gbce.linear_ce_fwd(h, w, t)
    want = gbce.linear_ce_bwd(h, w, t, lse, row_loss=row)
    with pytest.raises(ValueError, match="d_hidden shares memory with hidden"):
        gbce.linear_ce_bwd(h, w, t, lse, d_hidden=buf[:, 32:96])
    flat = torch.empty(300 * 32, device="cuda")
    flat[:70] = lse
    with pytest.raises(ValueError, match="d_weight shares memory with lse"):
        gbce.linear_ce_bwd(h, w, t, flat[:70], d_weight=flat.view(torch.bfloat16).view(300, 64))
    got = gbce.linear_ce_bwd(h, w, t, lse, row_loss=row, d_hidden=buf[:, 64:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
