"""8-bit code with a scale for each block of 128 and its products on the device against the fp64 oracle.  The code is exact
arithmetic and has to agree bit for bit."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import fp8_oracle as fo
from synth import inputs as syn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
f64 = syn.to_f64


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def matrices(batch, rows, cols, dtype, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(batch):
        x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * spread)
        x[rng.random((rows, cols)) < 0.02] = 0.0
        out.append(torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).to(DEV))
    return out


def same_code(q, X, fmt="e4m3", tile=False):
    for c, s, x in zip(q.codes, q.scales, X):
        wc, ws = fo.quantize(x, fmt, tile)
        assert c.dtype == F8[fmt] and s.shape[1] == fo.pitch(x.shape[0])
        assert np.array_equal(s.cpu().numpy()[:, :x.shape[0]], ws), "scales"
        assert np.array_equal(bytes_of(c), wc), "codes"


def values(q):
    fmt = "e4m3" if q.codes[0].dtype == F8["e4m3"] else "e5m2"
    return [fo.decode(bytes_of(c), s.cpu().numpy(), q.cols, fmt) for c, s in zip(q.codes, q.scales)]


SIZES = [(1, 1, 1), (2, 1, 33), (1, 31, 32), (1, 5, 128), (3, 64, 129), (1, 127, 257), (1, 130, 1000), (2, 257, 63),
         (1, 300, 640), (1, 33, 4104)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch,rows,cols", SIZES)
def test_code_bit_for_bit(dtype, fmt, batch, rows, cols):
    print(dtype, fmt, batch, rows, cols, flush=True)
    X = matrices(batch, rows, cols, dtype, 1)
    x64 = [f64(x) for x in X]
    for block in ("row", "tile"):
        tile = block == "tile"
        a = mu.fp8_quantize(X, block, format=fmt)
        t = mu.fp8_quantize(X, block, transpose=True, format=fmt)
        b, bt = mu.fp8_quantize(X, block, transpose="both", format=fmt)
        assert (a.rows, a.cols, t.rows, t.cols) == (rows, cols, cols, rows)
        for q in (a, b):
            same_code(q, x64, fmt, tile)
        for q in (t, bt):
            same_code(q, [x.T for x in x64], fmt, tile)
        for q, shape in ((a, (rows, cols)), (t, (cols, rows))):
            for dt in (torch.float32, torch.bfloat16):
                for y, want in zip(mu.fp8_dequantize(q, dt), values(q)):
                    assert tuple(y.shape) == shape and y.dtype == dt
                    assert np.array_equal(f64(y), want)
        if tile:  # both orientations hold the same values
            for y, z in zip(values(a), values(t)):
                assert np.array_equal(y, z.T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [2, 3, 4, 5, 6, 7, 32, 125, 130, 131, 253])
def test_code_of_edge_tiles(dtype, cols):
    """Every number of columns over a thread's four, rows that end anywhere in a tile, and a NaN and an infinity in the
    last row and column, which belong to their own blocks only."""
    for rows in (1, 17, 95, 129, 161):
        X = matrices(1, rows, cols, dtype, 6)
        for bad in (None, float("nan"), float("-inf")):
            if bad is not None:
                X[0][-1, -1] = bad
            for block in ("row", "tile"):
                q, t = mu.fp8_quantize(X, block, transpose="both")
                same_code(q, [f64(X[0])], tile=block == "tile")
                same_code(t, [f64(X[0]).T], tile=block == "tile")
                same_code(mu.fp8_quantize(X, block), [f64(X[0])], tile=block == "tile")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_code_of_every_bf16_value(fmt):
    """All finite bf16 values in blocks whose largest magnitude is near theirs: every rounding border, and subnormal
    inputs, in both orientations."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    vals = bits[torch.isfinite(bits.float())].float().sort().values
    for shift in (0, 61):  # other neighbours in a block
        v = torch.zeros(513 * 128)
        v[shift:shift + len(vals)] = vals
        X = v.view(513, 128).to(torch.bfloat16).to(DEV)
        same_code(mu.fp8_quantize([X], format=fmt), [f64(X)], fmt)
        same_code(mu.fp8_quantize([X.t().contiguous()], transpose=True, format=fmt), [f64(X)], fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_code_ties_borders_and_signs(fmt):
    """Halves between codes and their fp32 neighbours, subnormal codes, signed zeros; largest magnitudes at, just under and
    just over the format's largest value times a power of two."""
    table = fo.magnitudes(fmt)
    mids = (table[1:] + table[:-1]) / 2
    rows = []
    for e in (-140, -127, -126, -30, 0, 30, 100):
        for top in (table[-1], np.nextafter(np.float32(table[-1]), np.float32(0)), np.nextafter(np.float32(table[-1]), np.float32(1e9))):
            for at in range(0, len(mids), 40):
                r = np.zeros(128, np.float32)
                m = mids[at:at + 40].astype(np.float32)
                y = np.concatenate((m, np.nextafter(m, np.float32(0)), -np.nextafter(m, np.float32(1e9))))
                r[:len(y)] = np.ldexp(y, e)
                r[120:122] = (0.0, -0.0)
                r[127] = np.ldexp(np.float32(top), e)
                rows.append(r)
    X = torch.from_numpy(np.stack(rows)).to(DEV)
    assert torch.isfinite(X).all()
    same_code(mu.fp8_quantize([X], format=fmt), [f64(X)], fmt)
    same_code(mu.fp8_quantize([X.t().contiguous()], transpose=True, format=fmt), [f64(X)], fmt)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_mark_their_block(bad):
    X = torch.randn(140, 300, device=DEV)
    X[3, 140] = bad
    q, t = mu.fp8_quantize([X], transpose="both")
    same_code(q, [f64(X)])
    same_code(t, [f64(X).T])
    y = mu.fp8_dequantize(q)[0]
    assert torch.isnan(y[3, 128:256]).all() and int(torch.isnan(y).sum()) == 128
    y = mu.fp8_dequantize(t)[0]
    assert torch.isnan(y[140, 0:128]).all() and int(torch.isnan(y).sum()) == 128
    y = mu.fp8_dequantize(mu.fp8_quantize([X], "tile"))[0]
    assert torch.isnan(y[:128, 128:256]).all() and int(torch.isnan(y).sum()) == 128 * 128


def test_values_of_every_code_and_scale():
    """All codes with all scale bytes: fp32 holds every product (infinite over its range), bf16 those from 2^-133 on."""
    for fmt in F8:
        codes = torch.arange(256, dtype=torch.uint8).view(2, 1, 128).expand(2, 256, 128)
        codes = torch.where(torch.from_numpy(np.isnan(np.concatenate([fo.magnitudes(fmt), np.full(128 - len(fo.magnitudes(fmt)), np.nan)] * 2)))
                            .view(2, 1, 128), torch.zeros((), dtype=torch.uint8), codes)
        codes = codes.reshape(2, 256, 2, 64).permute(0, 2, 1, 3).reshape(4, 256, 64).contiguous()
        scales = torch.arange(256, dtype=torch.uint8).view(1, 256).expand(2, 256).contiguous()
        q = mu.FP8([codes.to(DEV).view(F8[fmt])], [scales.to(DEV)], 256)
        want = values(q)[0]
        want[np.abs(want) >= 2.0 ** 128] = np.inf * np.sign(want[np.abs(want) >= 2.0 ** 128])
        assert np.array_equal(want, f64(mu.fp8_dequantize(q)[0]), equal_nan=True)
        got = mu.fp8_dequantize(q, torch.bfloat16)[0]
        rounded = f64(torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16))
        assert np.array_equal(rounded, f64(got), equal_nan=True)


def test_quantize_into_given_buffers_touches_nothing_else():
    X = matrices(2, 37, 150, "f32", 3)
    q = mu.FP8.empty(2, 37, 150, DEV)
    guard = [torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV) for n in (4 * 37 * 64, 4 * 37 * 64, 2 * 48, 2 * 48)]
    out = mu.FP8([g[32:-32].view(F8["e4m3"]).view(4, 37, 64) for g in guard[:2]], [g[32:-32].view(2, 48) for g in guard[2:]], 150)
    assert mu.fp8_quantize(X, out=out) is out and mu.fp8_quantize(X, out=q) is q
    same_code(out, [f64(x) for x in X])
    for g in guard:
        assert (g[:32] == 0xA5).all() and (g[-32:] == 0xA5).all()
    assert all((s[:, 37:] == 0xA5).all() for s in out.scales)  # behind the last row
    Y = [torch.full((37 * 150 + 40,), 7.0, device=DEV) for _ in range(2)]
    mu.fp8_dequantize(q, out=[y[17:17 + 37 * 150].view(37, 150) for y in Y])
    for y, want in zip(Y, values(q)):
        assert (y[:17] == 7).all() and (y[17 + 37 * 150:] == 7).all()
        assert np.array_equal(f64(y[17:17 + 37 * 150]).reshape(37, 150), want)
    # both orientations, tiles
    t = mu.FP8.empty(2, 150, 37, DEV)
    assert mu.fp8_quantize(X, "tile", "both", out=(q, t)) == (q, t)
    same_code(q, [f64(x) for x in X], tile=True)
    same_code(t, [f64(x).T for x in X], tile=True)


def test_quantize_of_misaligned_matrices():
    for dtype, off in (("bf16", 1), ("bf16", 4), ("f32", 1), ("f16", 3)):
        x = matrices(1, 66, 264, dtype, 4)[0]
        buf = torch.zeros(66 * 264 + 8, dtype=DT[dtype], device=DEV)
        v = buf[off:off + 66 * 264].view(66, 264)
        v.copy_(x)
        q, t = mu.fp8_quantize([v], transpose="both")
        same_code(q, [f64(x)])
        same_code(t, [f64(x).T])
        same_code(mu.fp8_quantize([v]), [f64(x)])


def test_code_of_more_matrices_than_one_launch_takes():
    X = matrices(35, 9, 70, "bf16", 25)
    q, t = mu.fp8_quantize(X, transpose="both")
    same_code(q, [f64(x) for x in X])
    same_code(t, [f64(x).T for x in X])
    for y, want in zip(mu.fp8_dequantize(q), values(q)):
        assert np.array_equal(f64(y), want)


# --- product -------------------------------------------------------------------------------------------------------
def random_code(batch, rows, k, seed, low=120, high=132, fmt="e4m3", whole=False, groups=0):
    """Arbitrary finite codes (whole: integers up to 8 only) and scale bytes in [low, high], zeros behind the last element."""
    rng = np.random.default_rng(seed)
    units = mu.binding._fp8_units(k, groups)
    table = fo.magnitudes(fmt)
    allowed = np.flatnonzero((table <= 8) & (table == np.floor(table))) if whole else np.arange(len(table))
    codes = rng.choice(allowed, (batch, rows, units * 128)) | (rng.integers(0, 2, (batch, rows, units * 128)) << 7)
    if not groups:
        codes[..., k:] = 0
    codes = codes.astype(np.uint8).reshape(batch, rows, 2 * units, 64).transpose(0, 2, 1, 3)
    scales = rng.integers(low, high + 1, (batch, units, fo.pitch(rows))).astype(np.uint8)
    dev = lambda a: [torch.from_numpy(x.copy()).to(DEV) for x in a]  # noqa: E731
    return mu.FP8([c.view(F8[fmt]) for c in dev(codes)], dev(scales), k, groups)


def check(got, a, b, dtype, C0=None, exact=False):
    want, bound = fo.matmul(a, b, eights=dtype == "bf16")
    if C0 is not None:
        want = want + f64(C0)
        bound = bound + 2.0 ** -24 * np.abs(want)
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)  # half a step, relative to the value
        if exact:
            want = f64(torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16))
    got = f64(got)
    if exact:
        assert np.array_equal(got, want), f"{np.sum(got != want)} of {got.size} differ"
    else:
        assert np.all(np.abs(got - want) <= bound), f"{np.sum(~(np.abs(got - want) <= bound))} out of bounds"


def check_product(C, A, B, dtype, C0=None, exact=False):
    for i, (c, a, b) in enumerate(zip(C, values(A), values(B))):
        check(c, a, b, dtype, None if C0 is None else C0[i], exact)


SHAPES = [(1, 1, 1, 1), (1, 5, 7, 33), (2, 31, 65, 127), (1, 64, 64, 128), (1, 65, 129, 129), (3, 130, 70, 257),
          (1, 257, 300, 1000), (1, 1, 4096, 7001), (1, 3, 300, 640), (2, 16, 513, 2050), (1, 300, 1, 640),
          (1, 17, 1000, 31), (1, 512, 512, 512), (1, 129, 2049, 384), (1, 33, 40, 9000), (4, 20, 96, 1200),
          (1, 700, 520, 1153), (1, 5, 700, 8300), (19, 3, 40, 300), (17, 20, 50, 600),
          (1, 1030, 3001, 400), (2, 700, 2100, 150), (1, 4100, 2900, 300), (1, 3333, 4003, 129)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n,k", SHAPES)
def test_product_exact(dtype, batch, m, n, k):
    """Whole numbers up to 8 and one scale: sums of up to 2^24 / 64 = 262144 products are exact in fp32 in any order, and
    the result has to be equal."""
    print(dtype, batch, m, n, k, flush=True)
    A, B = random_code(batch, m, k, 5, 127, 127, whole=True), random_code(batch, n, k, 6, 127, 127, whole=True)
    check_product(mu.fp8_matmul(A, B, DT[dtype]), A, B, dtype, exact=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(4090, 3999, 2300), (4000, 4095, 2750)])
def test_product_in_the_largest_tiles(m, n, k, dtype):
    """A whole round of 256 x 256 tiles and k long enough for them (18 and 22 units), exact and with scales."""
    print(dtype, m, n, k, flush=True)
    A, B = random_code(1, m, k, 15, 127, 127, whole=True), random_code(1, n, k, 16, 127, 127, whole=True)
    check_product(mu.fp8_matmul(A, B, DT[dtype]), A, B, dtype, exact=True)
    A, B = random_code(1, m, k, 17, fmt="e5m2"), random_code(1, n, k, 18)
    C0 = [torch.randn(m, n, device=DEV).to(DT[dtype])]
    C = [C0[0].clone()]
    mu.fp8_matmul(A, B, out=C, accumulate=True)
    check_product(C, A, B, dtype, C0)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("batch,m,n,k", SHAPES)
def test_product_with_scales(fmt, batch, m, n, k):
    """All codes, scales that differ from block to block and row to row; also added to C."""
    print(fmt, batch, m, n, k, flush=True)
    A, B = random_code(batch, m, k, 7, fmt=fmt), random_code(batch, n, k, 8)
    for dtype in ("f32", "bf16"):
        check_product(mu.fp8_matmul(A, B, DT[dtype]), A, B, dtype)
        C0 = [torch.randn(m, n, device=DEV).to(DT[dtype]) * 1000 for _ in range(batch)]
        C = [c.clone() for c in C0]
        assert mu.fp8_matmul(A, B, out=C, accumulate=True) is C
        check_product(C, A, B, dtype, C0)


@pytest.mark.parametrize("m,n", [(40, 300), (1, 300), (300, 300)])
def test_product_nan_scale_marks_its_row(m, n):
    A, B = random_code(1, m, 500, 12), random_code(1, n, 500, 13)
    A.scales[0][2, m - 1] = 255
    A.scales[0][:, m:] = 255  # bytes behind the last row are not used
    C = mu.fp8_matmul(A, B, torch.float32)[0]
    assert torch.isnan(C[m - 1]).all() and not torch.isnan(C[:m - 1]).any()
    D = mu.fp8_matmul(B, A, torch.float32)[0]
    assert torch.isnan(D[:, m - 1]).all() and not torch.isnan(D[:, :m - 1]).any()


def test_product_extreme_scales():
    """Scale bytes 0 and 240 in one product, results far up; a product of the smallest scales is 0."""
    A, B = random_code(1, 40, 256, 9, 0, 3), random_code(1, 50, 256, 10, 237, 240)
    check_product(mu.fp8_matmul(A, B, torch.float32), A, B, "f32")
    Z = random_code(1, 50, 256, 11, 0, 3)
    assert not mu.fp8_matmul(A, Z, torch.float32)[0].any()


@pytest.mark.parametrize("m,n,k", [(1, 300, 900), (70, 130, 300), (300, 270, 700)])
def test_product_writes_nothing_else(m, n, k):
    A, B = random_code(1, m, k, 14), random_code(1, n, k, 15)
    for dt in (torch.float32, torch.bfloat16):
        for off in (64, 33):
            buf = torch.full((m * n + 2 * 64,), -3.0, dtype=dt, device=DEV)
            C = buf[off:off + m * n].view(m, n)
            mu.fp8_matmul(A, B, out=[C])
            assert torch.equal(C, mu.fp8_matmul(A, B, dt)[0])
            assert (buf[:off] == -3).all() and (buf[off + m * n:] == -3).all()


def test_product_of_a_matrix_with_itself():
    A = random_code(1, 200, 300, 16)
    C = mu.fp8_matmul(A, A, torch.float32)
    check_product(C, A, A, "f32")
    assert torch.equal(C[0], C[0].t())


def test_product_is_reproducible_with_a_given_workspace():
    A, B = random_code(1, 300, 5000, 17), random_code(1, 260, 5000, 18)
    need = mu.fp8_workspace_size(1, 300, 260, 5000)
    assert need > 256  # split along k
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # contents on entry are ignored
    a = mu.fp8_matmul(A, B, torch.float32, workspace=ws)[0]
    b = mu.fp8_matmul(A, B, torch.float32)[0]
    c = mu.fp8_matmul(A, B, torch.float32, workspace=ws)[0]
    assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(mu.MuonError):
        mu.fp8_matmul(A, B, torch.float32, workspace=ws[:need - 1])


# --- groups --------------------------------------------------------------------------------------------------------
def device_counts(counts):
    return torch.tensor(counts, dtype=torch.int32, device=DEV)


def skewed(rows, groups, seed):
    rng = np.random.default_rng(seed)
    share = rng.random(groups) ** 3 * (rng.random(groups) > 0.2) + 1e-9
    return rng.multinomial(rows, share / share.sum()).tolist()


COUNTS = [([1], 1), ([0, 1, 0], 1), ([5, 0, 0, 128, 129], 262), ([300], 300), ([0, 0, 40], 40), ([1] * 30, 30),
          ([2, 256, 0, 255, 257, 1], 771), ([130, 7], 200), ([0, 0], 9), (skewed(900, 150, 1), 900),
          (skewed(1500, 7, 2), 1530), ([16] * 129 + [5], 2069)]


def groups_of(counts, rows):
    at = 0
    for e, c in enumerate(counts):
        yield e, at, at + c
        at += c
    assert at <= rows


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,rows", COUNTS)
def test_grouped_product(counts, rows, fmt):
    """Groups of any size, without rows, more of them than a launch takes, rows behind the last one."""
    for n, k, dtype in ((70, 200, "f32"), (333, 130, "bf16")):
        print(counts[:8], rows, n, k, dtype, flush=True)
        A, B = random_code(1, rows, k, 31, fmt=fmt), random_code(len(counts), n, k, 32)
        a, b = values(A)[0], values(B)
        C = mu.fp8_grouped_matmul(A, B, device_counts(counts), DT[dtype])
        assert len(C) == 1
        C0 = torch.randn(rows, n, device=DEV).to(DT[dtype])
        D = [C0.clone()]
        assert mu.fp8_grouped_matmul(A, B, device_counts(counts), out=D, accumulate=True) is D
        F = [C0.clone()]
        mu.fp8_grouped_matmul(A, B, device_counts(counts), out=F)
        for e, i, j in groups_of(counts, rows):
            check(C[0][i:j], a[i:j], b[e], dtype)
            check(D[0][i:j], a[i:j], b[e], dtype, C0[i:j])
        total = sum(counts)
        assert torch.equal(F[0][:total], C[0][:total])
        assert not C[0][total:].any() and torch.equal(D[0][total:], C0[total:]) and torch.equal(F[0][total:], C0[total:])


@pytest.mark.parametrize("rows,groups,n,k", [(10000, 4, 1100, 200), (1100, 9, 520, 640), (700, 2, 300, 400)])
def test_grouped_product_in_larger_tiles(rows, groups, n, k):
    """256 x 256 tiles and 128 x 128 ones, exact."""
    counts = skewed(rows - 3, groups, 5)
    A, B = random_code(1, rows, k, 33, 127, 127, whole=True), random_code(groups, n, k, 34, 127, 127, whole=True)
    a, b = values(A)[0], values(B)
    for dtype in ("f32", "bf16"):
        C = mu.fp8_grouped_matmul(A, B, device_counts(counts), DT[dtype])[0]
        for e, i, j in groups_of(counts, rows):
            check(C[i:j], a[i:j], b[e], dtype, exact=True)
        assert not C[-3:].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_product_in_the_largest_tiles(dtype):
    """256 x 256 tiles, which need a long k, with an empty group and rows behind the last one: exact, and added to C."""
    rows, n, k, counts = 7600, 2040, 1900, [2563, 0, 4900]
    A, B = random_code(1, rows, k, 36, 127, 127, whole=True), random_code(3, n, k, 37, 127, 127, whole=True)
    a, b = values(A)[0], values(B)
    C0 = torch.randint(-8, 8, (rows, n), device=DEV).to(DT[dtype])
    C, D = mu.fp8_grouped_matmul(A, B, device_counts(counts), DT[dtype])[0], [C0.clone()]
    mu.fp8_grouped_matmul(A, B, device_counts(counts), out=D, accumulate=True)
    for e, i, j in groups_of(counts, rows):
        want = a[i:j] @ b[e].T  # whole numbers under 2^24, as what C holds
        for got, w in ((C[i:j], want), (D[0][i:j], want + f64(C0[i:j]))):
            assert np.array_equal(f64(got), f64(torch.from_numpy(w.astype(np.float32)).to(DT[dtype])))
    assert not C[-137:].any() and torch.equal(D[0][-137:], C0[-137:])


def test_grouped_product_with_counts_that_do_not_fit():
    """Counts under 0 are 0, and groups end with the last row."""
    A, B = random_code(1, 100, 256, 35, 127, 127, whole=True), random_code(4, 50, 256, 36, 127, 127, whole=True)
    a, b = values(A)[0], values(B)
    for counts in ([30, -5, 2 ** 31 - 1, 40], [-2 ** 31, 200, 1, 1], [2 ** 31 - 1] * 4):
        fits, at = [], 0
        for c in counts:
            c = max(0, min(c, 100 - at))
            fits.append(c)
            at += c
        C = mu.fp8_grouped_matmul(A, B, device_counts(counts), torch.float32)[0]
        for e, i, j in groups_of(fits, 100):
            assert np.array_equal(f64(C[i:j]), a[i:j] @ b[e].T)
        q = mu.fp8_quantize([torch.ones(100, 40, device=DEV)], transpose=True, counts=device_counts(counts))
        used = sum(-(-c // 128) for c in fits)
        wc, ws = fo.quantize_columns(np.ones((100, 40)), fits)
        assert np.array_equal(bytes_of(q.codes[0])[:2 * used], wc) and np.array_equal(q.scales[0].cpu().numpy()[:used, :40], ws)
        G = mu.fp8_grouped_weight_grad(q, q, device_counts(counts))
        assert [float(g[0, 0]) for g in G] == [float(c) for c in fits]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,rows", COUNTS)
def test_code_of_columns_in_groups(counts, rows, dtype):
    X = matrices(1, rows, 133, dtype, 41)
    used = sum(-(-c // 128) for c in counts)
    wc, ws = fo.quantize_columns(f64(X[0]), counts)
    t = mu.fp8_quantize(X, transpose=True, counts=device_counts(counts))
    q, bt = mu.fp8_quantize(X, transpose="both", counts=device_counts(counts))
    same_code(q, [f64(X[0])])  # all rows, also those behind the last group
    given = mu.FP8.empty(1, 133, rows, DEV, groups=len(counts))
    given.codes[0].view(torch.uint8).fill_(0xA5)
    given.scales[0].fill_(0xA5)
    mu.fp8_quantize(X, transpose=True, counts=device_counts(counts), out=given)
    for x in (t, bt, given):
        assert (x.rows, x.cols, x.groups) == (133, rows, len(counts))
        assert np.array_equal(bytes_of(x.codes[0])[:2 * used], wc)
        assert np.array_equal(x.scales[0].cpu().numpy()[:used, :133], ws)
    assert (bytes_of(given.codes[0])[2 * used:] == 0xA5).all() and (given.scales[0][used:] == 0xA5).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,rows", COUNTS)
def test_grouped_weight_gradient(counts, rows, fmt):
    for m, n, dtype in ((70, 200, "f32"), (300, 129, "bf16")):
        if len(counts) > 20 and m > 100:
            continue
        print(counts[:8], rows, m, n, dtype, flush=True)
        G = len(counts)
        A, B = random_code(1, m, rows, 51, fmt=fmt, groups=G), random_code(1, n, rows, 52, groups=G)
        C = mu.fp8_grouped_weight_grad(A, B, device_counts(counts), DT[dtype])
        C0 = [torch.randn(m, n, device=DEV).to(DT[dtype]) for _ in counts]
        D = [c.clone() for c in C0]
        assert mu.fp8_grouped_weight_grad(A, B, device_counts(counts), out=D, accumulate=True) is D
        at = 0
        whole = lambda q: values(mu.FP8(q.codes, q.scales, q.codes[0].shape[0] * 64))[0]  # noqa: E731
        a, b = whole(A), whole(B)
        for e, c in enumerate(counts):
            u = -(-c // 128)
            part = slice(at * 128, (at + u) * 128)
            check(C[e], a[:, part], b[:, part], dtype)
            check(D[e], a[:, part], b[:, part], dtype, C0[e])
            if c == 0:
                assert not C[e].any() and torch.equal(D[e], C0[e])
            at += u


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,counts", [(4100, 4099, [700, 0, 130, 1]), (2300, 2100, [700, 0, 130, 1]),
                                        (1030, 515, [129, 3, 0, 256, 300, 128] * 12),
                                        (2100, 2100, [1] * 12 + [0])])  # no room behind the last group's units
def test_grouped_weight_gradient_in_large_tiles(m, n, counts, dtype):
    """Every size of tiles, blocks that stay for tile after tile (odd and even numbers of units, groups without rows, tiles
    that are not full), exact; also added to C."""
    G, rows = len(counts), sum(counts)
    A = random_code(1, m, rows, 53, 127, 127, whole=True, groups=G)
    B = random_code(1, n, rows, 54, 127, 127, whole=True, groups=G)
    C = mu.fp8_grouped_weight_grad(A, B, device_counts(counts), DT[dtype])
    D = [torch.ones(m, n, dtype=DT[dtype], device=DEV) for _ in counts]
    mu.fp8_grouped_weight_grad(A, B, device_counts(counts), out=D, accumulate=True)
    whole = lambda q: torch.from_numpy(values(mu.FP8(q.codes, q.scales, q.codes[0].shape[0] * 64))[0]).to(DEV)  # noqa: E731
    a, b, at = whole(A), whole(B), 0
    for c, g, d in zip(counts, C, D):
        part = slice(at * 128, (at + -(-c // 128)) * 128)
        want = a[:, part] @ b[:, part].t().contiguous()
        assert torch.equal(g, want.to(g.dtype)) and torch.equal(d, (want + 1).to(g.dtype))
        at += -(-c // 128)


# --- refusals, graphs, streams, sizes ---------------------------------------------------------------------------------
def test_refusals_on_the_device():
    A, B = random_code(1, 4, 100, 19), random_code(1, 5, 100, 20)
    X, n2 = torch.zeros(4, 100, device=DEV), device_counts([2, 2])
    for match, call in [
            ("row length", lambda: mu.fp8_matmul(A, random_code(1, 5, 101, 20))),
            ("batch", lambda: mu.fp8_matmul(A, random_code(2, 5, 100, 20))),
            ("accumulate", lambda: mu.fp8_matmul(A, B, accumulate=True)),
            ("e4m3", lambda: mu.fp8_matmul(A, random_code(1, 5, 100, 20, fmt="e5m2"))),
            ("out", lambda: mu.fp8_matmul(A, B, out=[torch.zeros(5, 4, device=DEV)])),
            ("transpose", lambda: mu.fp8_quantize([X], transpose="rows")),
            ("block", lambda: mu.fp8_quantize([X], block="cell")),
            ("format", lambda: mu.fp8_quantize([X], format="e3m4")),
            ("out", lambda: mu.fp8_quantize([X], out=random_code(1, 4, 101, 1))),
            ("out", lambda: mu.fp8_quantize([X], out=A, format="e5m2")),
            ("contiguous", lambda: mu.fp8_quantize([torch.zeros(3, 4, device=DEV).t()])),
            ("empty", lambda: mu.fp8_quantize([torch.zeros(0, 5, device=DEV)])),
            ("counts", lambda: mu.fp8_quantize([X], counts=n2)),
            ("counts", lambda: mu.fp8_quantize([X], "tile", True, counts=n2)),
            ("counts", lambda: mu.fp8_quantize([X, X + 1], transpose=True, counts=n2)),
            ("counts", lambda: mu.fp8_quantize([X], transpose=True, counts=n2.long())),
            ("counts", lambda: mu.fp8_quantize([X], transpose=True, counts=[2, 2])),
            ("counts", lambda: mu.fp8_grouped_matmul(A, B, n2)),
            ("counts", lambda: mu.fp8_grouped_matmul(A, B, n2.view(1, 2))),
            ("out", lambda: mu.fp8_grouped_matmul(A, random_code(2, 5, 100, 3), n2, out=[torch.zeros(5, 5, device=DEV)])),
            ("groups", lambda: mu.fp8_matmul(mu.fp8_quantize([X], transpose=True, counts=n2), random_code(1, 5, 4, 20))),
            ("groups", lambda: mu.fp8_dequantize(mu.fp8_quantize([X], transpose=True, counts=n2))),
            ("counts", lambda: mu.fp8_grouped_weight_grad(A, A, n2)),
            ("units", lambda: mu.fp8_matmul(mu.FP8(A.codes, A.scales, 300), B)),
            ("rows rounded", lambda: mu.fp8_matmul(mu.FP8(A.codes, [A.scales[0][:, :4]], 100), B)),
            ("float8", lambda: mu.fp8_matmul(mu.FP8([A.codes[0].view(torch.uint8)], A.scales, 100), B)),
            ("overlaps", lambda: mu.fp8_matmul(random_code(2, 4, 100, 19), random_code(2, 5, 100, 20),
                                               out=[torch.zeros(4, 5, device=DEV)] * 2)),
            ("stream", lambda: mu.fp8_matmul(A, B, stream=type("S", (), {"cuda_stream": 0, "device": torch.device("cuda:1")})()))]:
        with pytest.raises(ValueError, match=match):
            call()
    codes = torch.zeros(2 * 4 * 64 + 8, dtype=torch.uint8, device=DEV)[8:].view(F8["e4m3"]).view(2, 4, 64)
    with pytest.raises(ValueError, match="aligned"):
        mu.fp8_matmul(mu.FP8([codes], A.scales, 100), B)
    for call in (lambda: mu.fp8_matmul(A, B, torch.float16), lambda: mu.fp8_dequantize(A, torch.float16),
                 lambda: mu.fp8_grouped_matmul(A, random_code(2, 5, 100, 3), n2, torch.float16)):
        with pytest.raises(mu.MuonError):
            call()


def test_captured_layer_replays_like_eager():
    """Codes, products (the split over k among them), the experts' three products and accumulation in one graph; new data
    and new counts between the replays; two graphs replayed side by side."""
    sets = []
    for seed in range(2):
        gen = torch.Generator().manual_seed(seed)
        X, dY = torch.randn(300, 2000, generator=gen).to(DEV).bfloat16(), torch.randn(300, 200, generator=gen).to(DEV)
        W = random_code(1, 200, 2000, 21 + seed)
        E, Et = random_code(3, 200, 2000, 23 + seed), random_code(3, 2000, 200, 25 + seed)
        counts = device_counts([100, 150, 50])
        C, S = [torch.zeros(300, 200, device=DEV)], [torch.zeros(300, 200, device=DEV)]
        Y, dX, dW = [torch.zeros(300, 200, device=DEV)], [torch.zeros(300, 2000, device=DEV)], \
            [torch.zeros(200, 2000, device=DEV) for _ in range(3)]

        def layer(X=X, dY=dY, W=W, E=E, Et=Et, counts=counts, C=C, S=S, Y=Y, dX=dX, dW=dW):
            q, qt = mu.fp8_quantize([X], transpose="both", counts=counts)
            mu.fp8_matmul(q, W, out=C)
            mu.fp8_matmul(q, W, out=S, accumulate=True)
            mu.fp8_grouped_matmul(q, E, counts, out=Y)
            d, dt = mu.fp8_quantize([dY], transpose="both", counts=counts)
            mu.fp8_grouped_matmul(d, Et, counts, out=dX)
            mu.fp8_grouped_weight_grad(dt, qt, counts, out=dW)

        layer()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer()
        sets.append((graph, torch.cuda.Stream(), layer, X, counts, (C, Y, dX, dW), S, S[0].clone()))
    for i, new in enumerate(([100, 150, 50], [0, 300, 0], [1, 2, 3], [299, 0, 1])):
        for _, _, _, X, counts, *_ in sets:
            X.copy_(torch.randn(300, 2000, generator=torch.Generator().manual_seed(i)))
            counts.copy_(torch.tensor(new, dtype=torch.int32))
        torch.cuda.synchronize()
        for graph, s, *_ in sets:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, layer, _, _, outs, S, total in sets:
            got = [x.clone() for o in outs for x in o]
            total += got[0]
            assert torch.equal(S[0], total), i
            layer()
            S[0].copy_(total)
            assert all(torch.equal(a, b) for a, b in zip(got, [x for o in outs for x in o])), i


def test_two_products_at_once_on_two_streams():
    A, B = random_code(1, 260, 6000, 22), random_code(1, 300, 6000, 23)
    want = mu.fp8_matmul(A, B, torch.float32)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[mu.fp8_matmul(A, B, torch.float32, stream=s)[0] for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for pair in got for x in pair)


def test_given_outputs_raise_their_version_and_launches_are_traced():
    X = matrices(1, 40, 200, "f32", 61)
    counts = device_counts([40])
    q, t = mu.fp8_quantize(X, transpose="both", counts=counts)
    Y, C, G = [torch.zeros(40, 200, device=DEV)], [torch.zeros(40, 40, device=DEV)], [torch.zeros(200, 200, device=DEV)]
    ws = torch.zeros(mu.fp8_workspace_size(1, 40, 40, 200), dtype=torch.uint8, device=DEV)
    written = q.codes + q.scales + t.codes + t.scales + Y + C + G + [ws]
    before, held = [x._version for x in written], (X[0]._version, counts._version)
    mu.trace_enable(True)
    mu.fp8_quantize(X, transpose="both", counts=counts, out=(q, t))
    codes = [x._version for x in q.codes + q.scales]
    mu.fp8_dequantize(q, out=Y)
    mu.fp8_matmul(q, q, out=C, workspace=ws)
    mu.fp8_grouped_matmul(q, q, counts, out=C)
    mu.fp8_grouped_weight_grad(t, t, counts, out=G)
    recs = mu.trace_collect()
    mu.trace_enable(False)
    assert all(x._version > b for x, b in zip(written, before))
    assert (X[0]._version, counts._version) == held and [x._version for x in q.codes + q.scales] == codes
    assert [r["role"] for r in recs] == ["fp8_quantize", "fp8_dequantize", "fp8_matmul", "fp8_grouped_matmul", "fp8_weight_grad"]
    assert recs[2]["flops"] == 2.0 * 40 * 40 * 200


def test_code_and_product_past_2_31_bytes():
    """66000 x 32768: 2.16e9 elements of X and as many code bytes; the last rows' codes in both orientations, and a product
    whose A ends behind 2^31 bytes."""
    rows, cols = 66000, 32768
    X = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    X[-300:] = torch.randn(300, cols, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(torch.bfloat16)
    q, t = mu.fp8_quantize([X], transpose="both")
    wc, ws = fo.quantize(f64(X[-80:]))
    assert np.array_equal(bytes_of(q.codes[0][:, -80:].contiguous()), wc)
    assert np.array_equal(q.scales[0][:, rows - 80:rows].cpu().numpy(), ws)
    wc, ws = fo.quantize(f64(X[65920:]).T)  # the last unit starts at row 515 * 128
    assert np.array_equal(bytes_of(t.codes[0][2 * 515:]), wc) and np.array_equal(t.scales[0][515:].cpu().numpy(), ws)
    assert not bytes_of(t.codes[0][:2 * 513, :4].contiguous()).any()
    only = mu.fp8_quantize([X])
    assert torch.equal(only.codes[0].view(torch.uint8), q.codes[0].view(torch.uint8))
    del only, t
    Y = mu.fp8_dequantize(q, torch.bfloat16)[0]
    want = fo.decode(bytes_of(q.codes[0][:, -80:].contiguous()), q.scales[0][:, rows - 80:rows].cpu().numpy(), cols)
    assert np.array_equal(f64(Y[-80:]), want)
    del Y, X
    B = random_code(1, 40, cols, 3)
    for dt in (torch.float32, torch.bfloat16):
        C = mu.fp8_matmul(q, B, dt)[0]
        check(C[-80:], want, values(B)[0], "f32" if dt == torch.float32 else "bf16")
        assert not C[:65000].any()
    # the same rows as the last of two groups
    C = mu.fp8_grouped_matmul(q, mu.FP8([B.codes[0].clone(), B.codes[0]], [B.scales[0].clone(), B.scales[0]], cols),
                              device_counts([65900, 100]), torch.float32)[0]
    check(C[-80:], want, values(B)[0], "f32")


def test_product_past_2_31_elements():
    """50000 x 50000 results (2.5e9): rows at the start, in the middle and at the end."""
    A = random_code(1, 50000, 100, 26, 127, 127, whole=True)
    B = random_code(1, 50000, 100, 27, 127, 127, whole=True)
    b64, a64 = values(B)[0], values(A)[0]
    C = mu.fp8_matmul(A, B, torch.bfloat16)[0]
    for i in (0, 1, 255, 256, 42949, 42950, 49997, 49999):
        assert np.array_equal(f64(C[i]), f64(torch.from_numpy((a64[i] @ b64.T).astype(np.float32)).to(torch.bfloat16))), i
