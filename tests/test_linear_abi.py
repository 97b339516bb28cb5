"""Refusals of the output-layer and router calls, on the host before anything is launched (CPU)."""
import ctypes

import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from cross_entropy_loss_ce_gb300 import build as gbuild

FAKE = 0x10000  # never dereferenced
NULL, SIZE, DTYPE, ALIGN, REDUCTION = 1, 2, 3, 4, 9


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gbce.load_library()


def fwd(**kw):
    a = dict(h=FAKE, hs=64, w=FAKE, ws=64, t=FAKE, loss=FAKE, row=FAKE, lse=FAKE, M=4, K=64, V=100, ii=-100,
             dtype=1, red=0)
    a.update(kw)
    return [a[k] for k in ("h", "hs", "w", "ws", "t", "loss", "row", "lse", "M", "K", "V", "ii", "dtype", "red")] + [None]


def bwd(**kw):
    a = dict(h=FAKE, hs=64, w=FAKE, ws=64, t=FAKE, lse=FAKE, g=None, dh=FAKE, dhs=64, dw=FAKE, dws=64, M=4, K=64,
             V=100, ii=-100, dtype=1, red=0)
    a.update(kw)
    return [a[k] for k in ("h", "hs", "w", "ws", "t", "lse", "g", "dh", "dhs", "dw", "dws", "M", "K", "V", "ii",
                           "dtype", "red")] + [None]


def greedy(**kw):
    a = dict(h=FAKE, hs=64, w=FAKE, ws=64, tok=FAKE, lp=FAKE, M=4, K=64, V=100, dtype=1)
    a.update(kw)
    return [a[k] for k in ("h", "hs", "w", "ws", "tok", "lp", "M", "K", "V", "dtype")] + [None]


def moe(**kw):
    a = dict(x=FAKE, xs=16, e=FAKE, es=2, c=FAKE, loss=FAKE, g=FAKE, gs=16, sc=None, T=4, E=16, k=2, a=0.1, b=0.1,
             dtype=0)
    a.update(kw)
    return [a[k] for k in ("x", "xs", "e", "es", "c", "loss", "g", "gs", "sc", "T", "E", "k", "a", "b", "dtype")] + [None]


HEAD = [(dict(h=None), NULL), (dict(w=None), NULL), (dict(hs=63), SIZE), (dict(ws=63), SIZE), (dict(M=-1), SIZE),
        (dict(M=2 ** 27), SIZE), (dict(K=0), SIZE), (dict(K=2 ** 24 + 1, hs=2 ** 25, ws=2 ** 25), SIZE),
        (dict(V=0), SIZE), (dict(V=2 ** 31 - 1024), SIZE), (dict(hs=2 ** 46 + 1), SIZE),
        (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(h=FAKE + 1), ALIGN), (dict(w=FAKE + 1), ALIGN)]


@pytest.mark.parametrize("kw,code", HEAD + [(dict(t=None), NULL), (dict(loss=None), NULL), (dict(row=None), NULL),
                                            (dict(t=FAKE + 4), ALIGN), (dict(loss=FAKE + 2), ALIGN),
                                            (dict(row=FAKE + 4), ALIGN), (dict(lse=FAKE + 2), ALIGN),
                                            (dict(red=3), REDUCTION)])
def test_linear_ce_fwd_refuses(lib, kw, code):
    assert lib.linear_ce_fwd(*fwd(**kw)) == code


@pytest.mark.parametrize("kw,code", HEAD + [(dict(t=None), NULL), (dict(lse=None), NULL), (dict(dh=None, dw=None), NULL),
                                            (dict(dhs=63), SIZE), (dict(dws=63), SIZE), (dict(dh=FAKE + 1), ALIGN),
                                            (dict(dw=FAKE + 1), ALIGN), (dict(lse=FAKE + 1), ALIGN),
                                            (dict(g=FAKE + 2), ALIGN), (dict(red=-1), REDUCTION)])
def test_linear_ce_bwd_refuses(lib, kw, code):
    assert lib.linear_ce_bwd(*bwd(**kw)) == code


@pytest.mark.parametrize("kw,code", HEAD + [(dict(tok=None), NULL), (dict(lp=None), NULL), (dict(tok=FAKE + 4), ALIGN),
                                            (dict(lp=FAKE + 2), ALIGN)])
def test_linear_greedy_refuses(lib, kw, code):
    assert lib.linear_greedy(*greedy(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(e=None), NULL), (dict(c=None), NULL), (dict(loss=None, g=None), NULL),
    (dict(xs=15), SIZE), (dict(gs=15), SIZE), (dict(es=1), SIZE), (dict(T=-1), SIZE), (dict(T=2 ** 27), SIZE),
    (dict(E=0), SIZE), (dict(E=1025, xs=2048, gs=2048), SIZE), (dict(k=0), SIZE), (dict(k=65, es=65), SIZE),
    (dict(dtype=3), DTYPE), (dict(x=FAKE + 2), ALIGN), (dict(g=FAKE + 2), ALIGN), (dict(e=FAKE + 4), ALIGN),
    (dict(c=FAKE + 4), ALIGN), (dict(loss=FAKE + 2), ALIGN), (dict(sc=FAKE + 2), ALIGN)])
def test_moe_balance_refuses(lib, kw, code):
    assert lib.moe_balance(*moe(**kw)) == code


def test_nothing_to_do_needs_no_device(lib):
    assert lib.linear_greedy(*greedy(M=0)) == gbce.OK
    assert lib.linear_ce_bwd(*bwd(M=0, dw=None)) == gbce.OK


def test_binding_refuses_before_any_launch():
    h, w, t = torch.zeros(4, 8).bfloat16(), torch.zeros(6, 8).bfloat16(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        gbce.linear_ce_fwd(h, w, t)
    with pytest.raises(ValueError, match="CUDA"):
        gbce.linear_greedy(h, w)
    with pytest.raises(ValueError, match="CUDA"):
        gbce.moe_balance(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64), 0.1)
    with pytest.raises(ValueError, match="rows"):
        gbce.linear_cross_entropy(h, w, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="tokens"):
        gbce.moe_balance_loss(torch.zeros(4, 8), torch.zeros(3, 2, dtype=torch.int64), 0.1)
    with pytest.raises(ValueError, match="reduction"):
        gbce.LinearCrossEntropyLoss(reduction="median")


def test_shared_memory_of_outputs_is_seen():
    x = torch.zeros(8, 8)
    with pytest.raises(ValueError, match="shares memory with hidden"):
        gbce._apart("d_hidden", x[:4], ("hidden", x[3:]))
    gbce._apart("d_hidden", x[:4], ("hidden", x[4:]))
    gbce._apart("d_hidden", x[:0], ("hidden", x))
