"""NaN and infinities on their way from a matrix through its 8-bit code (all zero codes beside scale byte 255) and every
kind of product of it: exactly the elements of C that the marked blocks enter are NaN, for either type of C and format of A
and for the block in either operand."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BAD = [float("nan"), float("inf"), float("-inf")]


def matrix(*shape, seed=0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).to(DEV)


def only_rows(C, rows):
    """Whether the rows of C are NaN, all of them, and nothing else."""
    want = torch.zeros(C.shape[0], 1, dtype=torch.bool, device=DEV)
    want[rows] = True
    return torch.equal(torch.isnan(C), want.expand_as(C)) and bool(torch.isfinite(C[~want[:, 0]]).all())


# few rows (8 and 16 waves), 64 x 128 tiles, those split along k, 128 x 128, 256 x 256
SHAPES = [(1, 300, 500), (7, 40, 8300), (40, 300, 500), (300, 130, 257), (40, 300, 5000), (1030, 3001, 400), (4090, 3999, 2300)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, fmt, dtype):
    for i, bad in enumerate(BAD):
        print(m, n, k, fmt, dtype, bad, flush=True)
        X, W = matrix(m, k, seed=1), matrix(n, k, seed=2)
        a, b = mu.fp8_quantize([X], format=fmt), mu.fp8_quantize([W])
        X[m - 1, (k // 2, 0, k - 1)[i]] = bad
        W[n // 2, (0, k - 1, k // 3)[i]] = bad
        bad_a, bad_b = mu.fp8_quantize([X], format=fmt), mu.fp8_quantize([W])
        for q, p, rows, cols in ((bad_a, b, [m - 1], []), (a, bad_b, [], [n // 2])):
            C = mu.fp8_matmul(q, p, DT[dtype])[0]
            assert only_rows(C, rows) if rows else only_rows(C.t(), cols)
            D = [torch.ones(m, n, dtype=DT[dtype], device=DEV)]
            mu.fp8_matmul(q, p, out=D, accumulate=True)
            assert torch.equal(torch.isnan(D[0]), torch.isnan(C))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,n,k", [([5, 0, 3, 30], 70, 300), ([200, 0, 128, 129], 333, 200), ([2563, 0, 4900], 2040, 1900)])
def test_grouped_product(counts, n, k, fmt, dtype):
    rows, last = sum(counts), len(counts) - 1
    start = rows - counts[last]
    for i, bad in enumerate(BAD):
        print(counts, n, k, fmt, dtype, bad, flush=True)
        X, W = matrix(rows, k, seed=3), [matrix(n, k, seed=4 + e) for e in range(len(counts))]
        c = torch.tensor(counts, dtype=torch.int32, device=DEV)
        a, b = mu.fp8_quantize([X], format=fmt), mu.fp8_quantize(W, "tile")
        X[counts[0] - 1, (0, k // 2, k - 1)[i]] = bad
        W[last][n - 1, 0] = bad
        C = mu.fp8_grouped_matmul(mu.fp8_quantize([X], format=fmt), b, c, DT[dtype])[0]
        assert only_rows(C, [counts[0] - 1])
        C = mu.fp8_grouped_matmul(a, mu.fp8_quantize(W, "row"), c, DT[dtype])[0]
        assert bool(torch.isfinite(C[:start]).all()) and only_rows(C[start:].t(), [n - 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,m,n", [([5, 0, 130, 2], 70, 150), ([700, 0, 130, 1], 4100, 4099)])
def test_grouped_weight_gradient(counts, m, n, fmt, dtype):
    """In 128 x 128 tiles; in 256 x 256 ones, for fp32 by blocks that stay for tile after tile."""
    rows = sum(counts)
    for i, bad in enumerate(BAD):
        print(counts, m, n, fmt, dtype, bad, flush=True)
        dY, X = matrix(rows, m, seed=8), matrix(rows, n, seed=9)
        c = torch.tensor(counts, dtype=torch.int32, device=DEV)
        code = lambda x, f: mu.fp8_quantize([x], transpose=True, counts=c, format=f)  # noqa: E731
        a, b = code(dY, fmt), code(X, "e4m3")
        dY[counts[0] + 129, m - 1] = bad  # the second unit of group 2
        X[(0, 1, 4)[i], n // 2] = bad     # group 0
        G = mu.fp8_grouped_weight_grad(code(dY, fmt), b, c, DT[dtype])
        assert only_rows(G[2], [m - 1]) and all(bool(torch.isfinite(G[e]).all()) for e in (0, 1, 3))
        G = mu.fp8_grouped_weight_grad(a, code(X, "e4m3"), c, DT[dtype])
        assert only_rows(G[0].t(), [n // 2]) and all(bool(torch.isfinite(g).all()) for g in G[1:])
        assert not G[1].any()
