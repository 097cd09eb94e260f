"""The 8-bit products where only one scale, or one type of C, was met before: the larger tiles of groups with scales that
differ by row and block, group starts off 16 and either format; far-out scales with bf16 C; and the fp32 sums that the 8-bit
matrix instruction makes, against what its definition allows it to lose."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from test_gpu_fp8 import DEV, DT, check, check_product, device_counts, f64, groups_of, random_code, skewed, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,rows,n,k", [(skewed(1097, 9, 5), 1100, 520, 640), ([301, 0, 396], 700, 300, 400),
                                             (skewed(9997, 4, 5), 10000, 1100, 200), ([2563, 0, 4900], 7600, 2040, 1900)])
def test_grouped_product(counts, rows, n, k, fmt, dtype):
    """128 x 128 and (the last) 256 x 256 tiles."""
    print(counts, rows, n, k, fmt, dtype, flush=True)
    A, B = random_code(1, rows, k, 71, fmt=fmt), random_code(len(counts), n, k, 72)
    a, b = values(A)[0], values(B)
    C0 = torch.randn(rows, n, device=DEV).to(DT[dtype]) * 1000
    C, D = mu.fp8_grouped_matmul(A, B, device_counts(counts), DT[dtype])[0], [C0.clone()]
    mu.fp8_grouped_matmul(A, B, device_counts(counts), out=D, accumulate=True)
    for e, i, j in groups_of(counts, rows):
        check(C[i:j], a[i:j], b[e], dtype)
        check(D[0][i:j], a[i:j], b[e], dtype, C0[i:j])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m,n,counts", [(2300, 2100, [700, 0, 130, 1]), (4100, 4099, [700, 0, 130, 1]),
                                        (1030, 515, [129, 3, 0, 256, 300, 128] * 12), (2100, 2100, [1] * 12 + [0])])
def test_grouped_weight_gradient(m, n, counts, fmt, dtype):
    """128 x 128 and 256 x 256 tiles, and blocks that stay: the scales of a tile's first unit are loaded in the tile before."""
    print(m, n, counts[:6], fmt, dtype, flush=True)
    G, rows = len(counts), sum(counts)
    A, B = random_code(1, m, rows, 73, fmt=fmt, groups=G), random_code(1, n, rows, 74, groups=G)
    C0 = [torch.randn(m, n, device=DEV).to(DT[dtype]) * 1000 for _ in counts]
    C, D = mu.fp8_grouped_weight_grad(A, B, device_counts(counts), DT[dtype]), [c.clone() for c in C0]
    mu.fp8_grouped_weight_grad(A, B, device_counts(counts), out=D, accumulate=True)
    whole = lambda q: values(mu.FP8(q.codes, q.scales, q.codes[0].shape[0] * 64))[0]  # noqa: E731
    a, b, at = whole(A), whole(B), 0
    for e, c in enumerate(counts):
        part = slice(at * 128, (at + -(-c // 128)) * 128)
        if c:
            check(C[e], a[:, part], b[:, part], dtype)
            check(D[e], a[:, part], b[:, part], dtype, C0[e])
        else:
            assert not C[e].any() and torch.equal(D[e], C0[e])
        at += -(-c // 128)


@pytest.mark.parametrize("m", [3, 40, 300])
def test_far_out_scales_with_bf16_results(m):
    """Scale bytes 0 and 240 in one product, results far up; a product of the smallest scales is 0.  Dense and in groups."""
    A, B = random_code(1, m, 256, 75, 0, 3), random_code(1, 50, 256, 76, 237, 240)
    check_product(mu.fp8_matmul(A, B), A, B, "bf16")
    check(mu.fp8_grouped_matmul(A, B, device_counts([m]))[0], values(A)[0], values(B)[0], "bf16")
    Z = random_code(1, 50, 256, 77, 0, 3)
    assert not mu.fp8_matmul(A, Z)[0].any() and not mu.fp8_grouped_matmul(A, Z, device_counts([m]))[0].any()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_fp32_sums_of_the_8_bit_instruction(fmt):
    """A product of bf16 C that is split along k leaves its pieces' fp32 sums in the workspace, here 10 of 4 units each.

    What the instruction may lose: of eight neighbouring products, those that are no multiple of 2^-13 of the power of two
    at or under the largest of them lose less than that each.  Each of the 64 sums of eight, and the few additions that join
    an instruction's, round the fp32 sum by at most a step, 2^-23 of the magnitudes."""
    m, n, k = 40, 60, 40 * 128
    rng = np.random.default_rng(78)
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV)  # noqa: E731
    A, B = mu.fp8_quantize([normal(m, k)], format=fmt), mu.fp8_quantize([normal(n, k)])
    need = mu.fp8_workspace_size(1, m, n, k)
    assert need // (4 * m * n) == 10
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    C = mu.fp8_matmul(A, B, workspace=ws)
    check_product(C, A, B, "bf16")
    got = f64(ws.view(torch.float32)[:10 * m * n].view(10, m, n))
    a, b = values(A)[0].reshape(m, 10, 512), values(B)[0].reshape(n, 10, 512)
    error, total = 0.0, 0.0
    for q in range(10):
        p = (a[:, None, q] * b[None, :, q]).reshape(m, n, 64, 8)
        top = np.abs(p).max(-1, keepdims=True)
        cut = np.where(top > 0, 2.0 ** (np.floor(np.log2(np.where(top > 0, top, 1.0))) - 13), 0.0)
        lost = np.where(p != np.trunc(p / np.where(cut > 0, cut, 1.0)) * cut, cut, 0.0).sum((-1, -2))
        size = np.abs(p).sum((-1, -2))
        diff, want = np.abs(got[q] - p.sum((-1, -2))), p.sum((-1, -2))
        assert np.all(diff <= lost + 72 * 2.0 ** -23 * size), f"piece {q}: {np.max(diff / (lost + 72 * 2.0 ** -23 * size))}"
        error, total = error + (diff ** 2).sum(), total + (want ** 2).sum()
    print(f"{fmt}: rms error 2^{np.log2(np.sqrt(error / total)):.2f} of the sums")
