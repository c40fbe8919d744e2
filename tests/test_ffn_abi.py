"""The feed-forward operators' argument checks, without a GPU: every refusal
comes before the device is touched."""
from __future__ import annotations

import pytest
import torch

import fp32_sgemm_02_amd as sg

P = 0x10000   # never dereferenced


def linear(**kw):
    a = dict(dtype=1, M=4, N=6, K=8, X=P, ldx=8, W=P, ldw=8, bias=P, R=P, ldr=6, act=2, Y=P, ldy=6,
             Z=P, ldz=6)
    a.update(kw)
    return sg.sgemm_linear(**a)


@pytest.mark.parametrize("i,kw", [
    (1, dict(dtype=3)), (1, dict(dtype=-1)), (2, dict(M=-1)), (3, dict(N=-1)), (4, dict(K=-1)),
    (5, dict(X=None)), (5, dict(X=P + 1)), (5, dict(dtype=0, X=P + 2)), (6, dict(ldx=7)),
    (7, dict(W=None)), (7, dict(W=P + 1)), (8, dict(ldw=7)), (9, dict(bias=P + 1)),
    (10, dict(R=P + 1)), (11, dict(ldr=5)), (12, dict(act=5)), (12, dict(act=-1)),
    (13, dict(Y=None)), (13, dict(Y=P + 1)), (14, dict(ldy=5)), (15, dict(Z=P + 1)),
    (16, dict(ldz=5)),
])
def test_linear_refusals(i, kw):
    st = linear(**kw)
    assert st == -(100 + i)
    assert sg.status_string(st) == f"invalid argument {i}"


def test_linear_empty_calls():
    assert linear(M=0, X=None, Y=None, W=None) == 0
    assert linear(N=0, W=None, Y=None, ldy=1) == 0
    assert linear(R=None, ldr=0, Z=None, ldz=0, bias=None, M=0) == 0


def backward(**kw):
    a = dict(dtype=2, M=4, N=6, K=8, dY=P, lddy=6, Z=P, ldz=6, act=1, X=P, ldx=8, W=P, ldw=8, dX=P,
             lddx=8, dW=P, lddw=8, db=P)
    a.update(kw)
    return sg.sgemm_linear_backward(**a)


@pytest.mark.parametrize("i,kw", [
    (1, dict(dtype=7)), (2, dict(M=-1)), (3, dict(N=-2)), (4, dict(K=-1)), (5, dict(dY=None)),
    (5, dict(dY=P + 1)), (6, dict(lddy=5)), (7, dict(Z=None)), (7, dict(Z=P + 1)), (8, dict(ldz=5)),
    (9, dict(act=9)), (10, dict(X=None)), (10, dict(X=P + 1)), (11, dict(ldx=7)), (12, dict(W=None)),
    (13, dict(ldw=7)), (14, dict(dX=P + 1)), (15, dict(lddx=7)), (16, dict(dW=P + 1)),
    (17, dict(lddw=7)), (18, dict(db=P + 1)),
])
def test_backward_refusals(i, kw):
    assert backward(**kw) == -(100 + i)


def moe(**kw):
    a = dict(dtype=1, T=4, D=16, F=24, E=8, top_k=2, gated=1, renormalize=1, act=2, X=P, ldx=16, Wr=P,
             ldr=16, W1=P, ld1=16, stride1=768, W2=P, ld2=24, stride2=384, Y=P, ldy=16)
    a.update(kw)
    return sg.sgemm_moe(**a)


@pytest.mark.parametrize("i,kw", [
    (1, dict(dtype=4)), (2, dict(T=-1)), (2, dict(T=65)), (3, dict(D=0)), (3, dict(D=64513, ldx=70000)),
    (4, dict(F=0)), (4, dict(F=(1 << 20) + 1)), (5, dict(E=0)), (5, dict(E=513)), (6, dict(top_k=0)),
    (6, dict(top_k=9)), (6, dict(E=64, top_k=17)), (7, dict(gated=2)), (8, dict(renormalize=-1)),
    (9, dict(act=5)), (10, dict(X=None)), (10, dict(X=P + 1)), (11, dict(ldx=15)), (12, dict(Wr=None)),
    (13, dict(ldr=15)), (14, dict(W1=None)), (15, dict(ld1=15)), (16, dict(stride1=-1)),
    (17, dict(W2=P + 1)), (18, dict(ld2=23)), (19, dict(stride2=-1)), (20, dict(Y=None)),
    (21, dict(ldy=15)), (22, dict(ids=P + 2)), (23, dict(weights=P + 2)),
])
def test_moe_refusals(i, kw):
    assert moe(**kw) == -(100 + i)


def test_moe_no_tokens():
    assert moe(T=0, X=None, Wr=None, W1=None, W2=None, Y=None) == 0


def test_status_strings():
    for i in range(1, 24):
        assert sg.status_string(-(100 + i)) == f"invalid argument {i}"
    assert sg.status_string(-124) == "unknown status" and sg.status_string(-100) == "unknown status"


def test_bindings_refuse_host_tensors_and_types():
    x, w = torch.zeros(2, 4), torch.zeros(3, 4)
    with pytest.raises(ValueError, match="GPU"):
        sg.linear(x, w)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        sg.linear(x.double(), w.double())
    with pytest.raises(ValueError, match="2-D"):
        sg.linear(x[0], w)
    with pytest.raises(ValueError, match="GPU"):
        sg.linear_backward(torch.zeros(2, 3), x, w)
    with pytest.raises(ValueError, match="GPU"):
        sg.moe(x, torch.zeros(2, 4), torch.zeros(2, 6, 4), torch.zeros(2, 4, 3), 1)
