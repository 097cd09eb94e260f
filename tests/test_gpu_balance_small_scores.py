"""Sigmoid scores whose sigmoids are near or under fp32's range: p is a quotient of them, and as well defined as any other."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import balance_oracle as bo
from test_gpu_balance import DEV, case, check, f64

pytestmark = pytest.mark.gpu


def one_hot_index(S, T, E, seed):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, E, (S, T, 1)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("S,T,E", [(1, 5, 2), (1, 7, 40), (2, 300, 61), (1, 900, 700)])
@pytest.mark.parametrize("shift", [-40.0, -44.4, -64.0, -87.0, -103.0, -600.0])
def test_rows_of_small_sigmoids(shift, S, T, E, dtype):
    """All logits far down, some rows further than others.  The oracle's sigmoids are those of float64, good to -700."""
    z, _ = case(S, T, E, 1, dtype, 21, 2.0)
    z = (z.float() + shift + torch.arange(T)[None, :, None] % 7 - 3).to(z.dtype)
    index = one_hot_index(S, T, E, 22)
    check(mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, "sigmoid", grad=True), z, index, 1.0, "sigmoid", dtype)


def test_further_down_than_any_sigmoid():
    """Past -745 the sigmoids are 0 in float64 too; there p is the softmax, to 1 part in e^700."""
    z, _ = case(1, 500, 30, 1, "f32", 23, 3.0)
    index = one_hot_index(1, 500, 30, 24)
    for shift in (-2000.0, -1e6):
        y = z + shift
        check(mu.expert_balance(y.to(DEV), index.to(DEV), 1.0, "sigmoid", grad=True), y, index, 1.0, "softmax", "f32")


def test_small_and_other_rows_together():
    """Rows of either kind, experts that a row may not choose, rows without any expert, and a row with one large logit."""
    z, _ = case(3, 400, 20, 1, "f32", 25)
    rng = np.random.default_rng(26)
    z = z + torch.from_numpy(np.where(rng.random((3, 400, 1)) < 0.5, -90.0, 0.0).astype(np.float32))
    z[torch.from_numpy(rng.random((3, 400, 20)) < 0.3)] = float("-inf")
    z[0, 3] = float("-inf")
    z[1, 5], z[1, 5, 7] = -95.0, 4.0
    mask = torch.from_numpy(rng.random((3, 400)) < 0.9)
    index = one_hot_index(3, 400, 20, 27)
    clean = z.clone()
    z[~mask] = float("nan")
    got = mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, "sigmoid", mask.to(DEV), grad=True)
    check(got, clean, index, 1.0, "sigmoid", "f32", mask)
    assert not got[2][0, 3].any()


def test_gradient_against_differences():
    z, _ = case(1, 6, 5, 1, "f32", 28)
    z = z - 88.0
    index = one_hot_index(1, 6, 5, 29)
    g = f64(mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, "sigmoid", grad=True)[2])
    z64, h = f64(z), 1e-4
    for at in np.ndindex(z64.shape):
        up, down = z64.copy(), z64.copy()
        up[at] += h
        down[at] -= h
        d = (bo.balance(up, index.numpy(), 1.0, "sigmoid")[0] - bo.balance(down, index.numpy(), 1.0, "sigmoid")[0]) / (2 * h)
        # third derivatives of p are under 1, f under E: h^2 E / 6; the loss is good to 2^-50 of E; the gradient to 1e-6
        assert abs(g[at] - d) <= h * h * 5 / 6 + 5 * 2.0 ** -50 / h + 1e-6
