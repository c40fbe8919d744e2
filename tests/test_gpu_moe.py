"""The mixture-of-experts layer against its definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import fp32_sgemm_02_amd as sg
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def padded(shape, dtype, pad, off, g, scale):
    """A stack of row-major matrices with NaN between rows, matrices and before."""
    *lead, cols = shape
    n = 1
    for s in lead:
        n *= s
    buf = torch.full((n * (cols + pad) + off + 8,), float("nan"), device=DEV, dtype=dtype)
    v = buf[off:off + n * (cols + pad)].view(*lead, cols + pad)[..., :cols]
    v.copy_((torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype))
    return v


def problem(T, D, F, E, dtype, gated, seed, pad=0, off=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (padded((T, D), dtype, pad, off, g, 1.0),
            padded((E, D), dtype, pad, off, g, 1.5 * D ** -0.5),
            padded((E, 2 * F if gated else F, D), dtype, pad, off, g, D ** -0.5),
            padded((E, D, F), dtype, pad, off, g, F ** -0.5))


def check(args, k, name, renorm, dtype):
    X, Wr, W1, W2 = args
    gated = W1.shape[1] == 2 * W2.shape[2]
    Y, ids, w = sg.moe(X, Wr, W1, W2, k, act=ref.ACTS[name], renormalize=renorm, return_routing=True)
    y, i, p, bound = ref.moe(X, Wr, W1, W2, k, name, gated, renorm)
    assert torch.equal(ids.long(), i)
    assert bool(((w.double() - p).abs() <= ref.rounding(p, torch.float32) + 1e-12).all())
    assert bool(((Y.double() - y).abs() <= bound + ref.rounding(y.abs() + bound, dtype)).all())
    return Y


CASES = [  # T, D, F, E, k
    (1, 1, 1, 1, 1), (1, 64, 48, 4, 2), (1, 515, 333, 9, 3), (2, 100, 17, 5, 5), (5, 256, 512, 8, 2),
    (16, 128, 40, 64, 8), (17, 72, 65, 4, 1), (31, 200, 64, 3, 2), (33, 96, 128, 6, 4),
    (64, 136, 72, 16, 8), (64, 32, 16, 2, 2), (7, 1024, 96, 512, 16), (64, 64, 33, 130, 16),
]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,D,F,E,k", CASES)
def test_moe(T, D, F, E, k, gated, t):
    name = list(ref.ACTS)[(T + D + F) % 5]
    check(problem(T, D, F, E, TYPES[t], gated, T * D + F), k, name, bool((T + k) % 2), TYPES[t])


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 1), (1, 5)])
def test_moe_strides(pad, off, t):
    for T in (1, 20, 40):
        check(problem(T, 136, 72, 6, TYPES[t], True, T, pad, off), 3, "silu", True, TYPES[t])


def test_moe_result_rows_are_padded():
    args = problem(4, 40, 24, 4, torch.float32, True, 1)
    buf = torch.full((4, 48), 7.0, device=DEV)
    Y = sg.moe(*args, 2, out=buf[:, :40])
    assert torch.equal(Y, sg.moe(*args, 2)) and bool((buf[:, 40:] == 7.0).all())


@pytest.mark.parametrize("T", [1, 16, 64])
def test_moe_ties_take_the_lowest_index(T):
    X, Wr, W1, W2 = problem(T, 64, 32, 12, torch.bfloat16, True, 4)
    Wr[5] = Wr[2]
    Wr[9] = Wr[2]
    Wr[2:] *= 0.0
    _, ids, w = sg.moe(X, Wr, W1, W2, 4, return_routing=True)
    assert torch.equal(ids.long(), ref.moe(X, Wr, W1, W2, 4, "silu", True, True)[1])
    check((X, Wr, W1, W2), 4, "silu", True, torch.bfloat16)


@pytest.mark.parametrize("T", [16, 33, 64])
def test_moe_one_expert_takes_all(T):
    """Every token chooses the same expert first: 64 rows for one, and experts
    that nobody chooses hold NaN."""
    X, Wr, W1, W2 = problem(T, 96, 80, 8, torch.bfloat16, True, 5)
    X[:, 0] = 8.0
    Wr[:, 0] = torch.tensor([9.0, -9, -9, 5, -9, -9, -9, -9], device=DEV)
    for e in (1, 2, 4, 5, 6, 7):
        W1[e] = float("nan")
        W2[e] = float("nan")
    check((X, Wr, W1, W2), 2, "gelu_tanh", False, torch.bfloat16)


def test_moe_nan_token_keeps_to_itself():
    X, Wr, W1, W2 = problem(5, 64, 48, 6, torch.float32, True, 6)
    clean = sg.moe(X, Wr, W1, W2, 2)
    X[3, 7] = float("nan")
    Y, ids, w = sg.moe(X, Wr, W1, W2, 2, return_routing=True)
    keep = [0, 1, 2, 4]
    assert torch.equal(Y[keep], clean[keep])
    assert bool(torch.isnan(Y[3]).all()) and bool(torch.isnan(w[3]).all())
    assert torch.equal(ids[3].cpu(), torch.tensor([0, 1], dtype=torch.int32))


def test_moe_repeatable_and_no_tokens():
    for T in (1, 24, 64):
        args = problem(T, 520, 264, 16, torch.bfloat16, True, T)
        Y = sg.moe(*args, 4)
        for _ in range(3):
            assert torch.equal(sg.moe(*args, 4), Y)
    X, Wr, W1, W2 = problem(1, 64, 48, 6, torch.float32, True, 6)
    assert sg.moe(X[:0], Wr, W1, W2, 2).shape == (0, 64)
