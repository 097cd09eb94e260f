"""Microscaled 4-bit code and product on the device against the fp64 oracle.  The code is exact arithmetic and has to
agree bit for bit."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import mx4_oracle as xo
from synth import inputs as syn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
f64 = syn.to_f64


def matrices(batch, rows, cols, dtype, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(batch):
        x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * spread)
        x[rng.random((rows, cols)) < 0.02] = 0.0
        out.append(torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).to(DEV))
    return out


def same_code(q, X):
    for c, s, x in zip(q.codes, q.scales, X):
        wc, ws = xo.quantize(x)
        assert np.array_equal(s.cpu().numpy(), ws), "scales"
        assert np.array_equal(c.cpu().numpy(), wc), "codes"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (2, 1, 33), (1, 31, 32), (1, 5, 128), (3, 64, 129), (1, 127, 257),
                                             (1, 130, 1000), (2, 257, 63), (1, 300, 640), (1, 33, 4104)])
def test_code_bit_for_bit(dtype, batch, rows, cols):
    print(dtype, batch, rows, cols, flush=True)
    X = matrices(batch, rows, cols, dtype, 1)
    x64 = [f64(x) for x in X]
    a = mu.mx4_quantize(X)
    t = mu.mx4_quantize(X, transpose=True)
    b, bt = mu.mx4_quantize(X, transpose="both")
    assert (a.rows, a.cols, t.rows, t.cols) == (rows, cols, cols, rows)
    for q in (a, b):
        same_code(q, x64)
    for q in (t, bt):
        same_code(q, [x.T for x in x64])
    for q, shape in ((a, (rows, cols)), (t, (cols, rows))):
        for dt in (torch.float32, torch.bfloat16):
            for y, c, s in zip(mu.mx4_dequantize(q, dt), q.codes, q.scales):
                assert tuple(y.shape) == shape and y.dtype == dt
                assert np.array_equal(f64(y), xo.decode(c.cpu().numpy(), s.cpu().numpy(), shape[1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [2, 3, 4, 5, 6, 7, 32, 125, 130, 131, 253])
def test_code_of_edge_tiles(dtype, cols):
    """Every number of columns over a thread's four, rows that end anywhere in a tile, and a NaN and an infinity in the
    last row and column, which belong to their own blocks only."""
    for rows in (1, 33, 95, 129, 161):
        X = matrices(1, rows, cols, dtype, 6)
        for bad in (None, float("nan"), float("-inf")):
            if bad is not None:
                X[0][-1, -1] = bad
            q, t = mu.mx4_quantize(X, transpose="both")
            same_code(q, [f64(X[0])])
            same_code(t, [f64(X[0]).T])
            same_code(mu.mx4_quantize(X, transpose=True), [f64(X[0]).T])


def test_code_of_every_bf16_value():
    """All finite bf16 values as elements of blocks whose largest magnitude is 7.9375 2^e: every rounding border and
    subnormal input, in both orientations."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    vals = bits[torch.isfinite(bits.float())].to(DEV)
    vals = vals[vals.abs().float() < 2.0 ** 127]
    n = vals.numel() // 31 * 31
    X = torch.zeros(n // 31, 32, dtype=torch.bfloat16, device=DEV)
    X[:, :31] = vals.float().sort().values[:n].to(torch.bfloat16).view(-1, 31)
    X[:, 31] = (2.0 ** torch.floor(torch.log2(X[:, :31].float().abs().amax(1).clamp(min=2.0 ** -120))) * 1.984375).to(torch.bfloat16)
    same_code(mu.mx4_quantize([X]), [f64(X)])
    same_code(mu.mx4_quantize([X.t().contiguous()], transpose=True), [f64(X)])


def test_code_ties_saturation_and_signs():
    """Halves between codes at every magnitude, both signs, signed zeros, values over 6 of the scale, fp32 subnormals."""
    y = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.999, 0.2499999, 0.7500001, 1.2499999, 2.5000002, -0.25,
                  -0.75, -5.0, -7.5, 0.0, -0.0], dtype=np.float32)
    rows = []
    for e in (-140, -127, -126, -30, 0, 30, 125):
        r = np.zeros(64, dtype=np.float32)
        r[:19] = np.ldexp(y, e)
        r[31] = np.ldexp(np.float32(7.9), e)
        r[40:59] = r[:19]
        r[63] = np.ldexp(np.float32(4.0), e)
        rows.append(r)
    X = torch.from_numpy(np.stack(rows)).to(DEV)
    same_code(mu.mx4_quantize([X]), [f64(X)])
    same_code(mu.mx4_quantize([X.t().contiguous()], transpose=True), [f64(X)])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_mark_their_block(bad):
    X = torch.randn(40, 200, device=DEV)
    X[3, 40] = bad
    q, t = mu.mx4_quantize([X], transpose="both")
    same_code(q, [f64(X)])
    same_code(t, [f64(X).T])
    y = mu.mx4_dequantize(q)[0]
    assert torch.isnan(y[3, 32:64]).all() and int(torch.isnan(y).sum()) == 32
    y = mu.mx4_dequantize(t)[0]
    assert torch.isnan(y[40, 0:32]).all() and int(torch.isnan(y).sum()) == 32


def test_quantize_into_given_buffers_touches_nothing_else():
    X = matrices(2, 37, 150, "f32", 3)
    q = mu.MX4.empty(2, 37, 150, DEV)
    guard = [torch.full((2 * 37 * n + 64,), 0xA5, dtype=torch.uint8, device=DEV) for n in (64, 64, 4, 4)]
    out = mu.MX4([g[32:-32].view(2, 37, 64) for g in guard[:2]], [g[32:-32].view(2, 37, 4) for g in guard[2:]], 150)
    assert mu.mx4_quantize(X, out=out) is out and mu.mx4_quantize(X, out=q) is q
    same_code(out, [f64(x) for x in X])
    assert all(torch.equal(a, b) for a, b in zip(out.codes + out.scales, q.codes + q.scales))
    for g in guard:
        assert (g[:32] == 0xA5).all() and (g[-32:] == 0xA5).all()
    Y = [torch.full((37 * 150 + 40,), 7.0, device=DEV) for _ in range(2)]
    mu.mx4_dequantize(q, out=[y[17:17 + 37 * 150].view(37, 150) for y in Y])
    for y, c, s in zip(Y, q.codes, q.scales):
        assert (y[:17] == 7).all() and (y[17 + 37 * 150:] == 7).all()
        assert np.array_equal(f64(y[17:17 + 37 * 150]).reshape(37, 150), xo.decode(c.cpu().numpy(), s.cpu().numpy(), 150))


def test_quantize_of_misaligned_matrices():
    for dtype, off in (("bf16", 1), ("bf16", 4), ("f32", 1), ("f16", 3)):
        x = matrices(1, 66, 264, dtype, 4)[0]
        buf = torch.zeros(66 * 264 + 8, dtype=DT[dtype], device=DEV)
        v = buf[off:off + 66 * 264].view(66, 264)
        v.copy_(x)
        q, t = mu.mx4_quantize([v], transpose="both")
        same_code(q, [f64(x)])
        same_code(t, [f64(x).T])


# --- product -------------------------------------------------------------------------------------------------------
def random_code(batch, rows, k, seed, low=120, high=132):
    """Arbitrary codes and scale bytes in [low, high], with the padding the quantiser leaves."""
    rng = np.random.default_rng(seed)
    units = -(-k // 128)
    codes = rng.integers(0, 256, (batch, units, rows, 64)).astype(np.uint8)
    scales = rng.integers(low, high + 1, (batch, units, rows, 4)).astype(np.uint8)
    last = k - (units - 1) * 128
    nib = np.stack((codes[:, -1] & 15, codes[:, -1] >> 4), -1).reshape(batch, rows, 128)
    nib[..., last:] = 0
    codes[:, -1] = nib[..., 0::2] | (nib[..., 1::2] << 4)
    scales[:, -1, :, -(-last // 32):] = 0
    dev = lambda a: [torch.from_numpy(x.copy()).to(DEV) for x in a]  # noqa: E731
    return mu.MX4(dev(codes), dev(scales), k)


def decoded(q):
    return [xo.decode(c.cpu().numpy(), s.cpu().numpy(), q.cols) for c, s in zip(q.codes, q.scales)]


def check_product(C, A, B, dtype, C0=None, exact=False):
    for c, a, b, i in zip(C, decoded(A), decoded(B), range(len(C))):
        want, bound = xo.matmul(a, b)
        if C0 is not None:
            want = want + f64(C0[i])
            bound = bound + 2.0 ** -24 * np.abs(want)
        if dtype == "bf16":
            bound = bound + 2.0 ** -8 * np.abs(want)  # half a step, relative to the value
            if exact:
                want = f64(torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16))
        got = f64(c)
        if exact:
            assert np.array_equal(got, want), f"matrix {i}: {np.sum(got != want)} of {got.size} differ"
        else:
            assert np.all(np.abs(got - want) <= bound), f"matrix {i}: {np.sum(np.abs(got - want) > bound)} out of bounds"


SHAPES = [(1, 1, 1, 1), (1, 5, 7, 33), (2, 31, 65, 127), (1, 64, 64, 128), (1, 65, 129, 129), (3, 130, 70, 257),
          (1, 257, 300, 1000), (1, 1, 4096, 7001), (1, 3, 300, 640), (2, 16, 513, 2050), (1, 300, 1, 640),
          (1, 17, 1000, 31), (1, 512, 512, 512), (1, 129, 2049, 384), (1, 33, 40, 9000), (4, 20, 96, 1200),
          (1, 700, 520, 1153),
          (1, 5, 700, 8300), (19, 3, 40, 300), (17, 20, 50, 600),  # 16 waves a block; more matrices than one launch takes
          (1, 1030, 3001, 400), (2, 700, 2100, 150),               # 128 x 128 tiles, ragged
          (1, 4100, 2900, 300), (1, 3333, 4003, 129)]              # 256 x 256 tiles, ragged


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n,k", SHAPES)
def test_product_exact(dtype, batch, m, n, k):
    """One scale for all blocks: every product is a multiple of 1/4 of at most 36, so sums of up to 116000 of them are
    exact in fp32 in any order and the result has to be equal."""
    print(dtype, batch, m, n, k, flush=True)
    A, B = random_code(batch, m, k, 5, 127, 127), random_code(batch, n, k, 6, 127, 127)
    check_product(mu.mx4_matmul(A, B, DT[dtype]), A, B, dtype, exact=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n,k", SHAPES)
def test_product_with_scales(dtype, batch, m, n, k):
    """Scales that differ from block to block and row to row; also added to C."""
    print(dtype, batch, m, n, k, flush=True)
    A, B = random_code(batch, m, k, 7), random_code(batch, n, k, 8)
    check_product(mu.mx4_matmul(A, B, DT[dtype]), A, B, dtype)
    C0 = [torch.randn(m, n, device=DEV).to(DT[dtype]) * 1000 for _ in range(batch)]
    C = [c.clone() for c in C0]
    assert mu.mx4_matmul(A, B, out=C, accumulate=True) is C
    check_product(C, A, B, dtype, C0)


def test_product_extreme_scales():
    """Scale bytes 0 and 254 in one product, results far up; a product of the smallest scales is 0."""
    A, B = random_code(1, 40, 256, 9, 0, 3), random_code(1, 50, 256, 10, 251, 254)
    check_product(mu.mx4_matmul(A, B, torch.float32), A, B, "f32")
    Z = random_code(1, 50, 256, 11, 0, 3)
    assert not mu.mx4_matmul(A, Z, torch.float32)[0].any()


@pytest.mark.parametrize("m,n", [(40, 300), (1, 300), (300, 300)])
def test_product_nan_scale_marks_its_row(m, n):
    A, B = random_code(1, m, 500, 12), random_code(1, n, 500, 13)
    A.scales[0][2, m - 1, 1] = 255
    C = mu.mx4_matmul(A, B, torch.float32)[0]
    assert torch.isnan(C[m - 1]).all() and not torch.isnan(C[:m - 1]).any()
    D = mu.mx4_matmul(B, A, torch.float32)[0]
    assert torch.isnan(D[:, m - 1]).all() and not torch.isnan(D[:, :m - 1]).any()


@pytest.mark.parametrize("m,n,k", [(1, 300, 900), (70, 130, 300), (300, 270, 700)])
def test_product_writes_nothing_else(m, n, k):
    A, B = random_code(1, m, k, 14), random_code(1, n, k, 15)
    for dt in (torch.float32, torch.bfloat16):
        for off in (64, 33):
            buf = torch.full((m * n + 2 * 64,), -3.0, dtype=dt, device=DEV)
            C = buf[off:off + m * n].view(m, n)
            mu.mx4_matmul(A, B, out=[C])
            assert torch.equal(C, mu.mx4_matmul(A, B, dt)[0])
            assert (buf[:off] == -3).all() and (buf[off + m * n:] == -3).all()


def test_product_of_a_matrix_with_itself():
    A = random_code(1, 200, 300, 16)
    C = mu.mx4_matmul(A, A, torch.float32)
    check_product(C, A, A, "f32")
    assert torch.equal(C[0], C[0].t())


def test_product_is_reproducible_with_a_given_workspace():
    A, B = random_code(1, 300, 5000, 17), random_code(1, 260, 5000, 18)
    need = mu.mx4_workspace_size(1, 300, 260, 5000)
    assert need > 256  # split along k
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # contents on entry are ignored
    a = mu.mx4_matmul(A, B, torch.float32, workspace=ws)[0]
    b = mu.mx4_matmul(A, B, torch.float32)[0]
    c = mu.mx4_matmul(A, B, torch.float32, workspace=ws)[0]
    assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(mu.MuonError):
        mu.mx4_matmul(A, B, torch.float32, workspace=ws[:need - 1])


def test_mx4_refusals_on_the_device():
    A, B = random_code(1, 4, 100, 19), random_code(1, 5, 100, 20)
    with pytest.raises(ValueError, match="row length"):
        mu.mx4_matmul(A, random_code(1, 5, 101, 20))
    with pytest.raises(ValueError, match="batch"):
        mu.mx4_matmul(A, random_code(2, 5, 100, 20))
    with pytest.raises(ValueError, match="accumulate"):
        mu.mx4_matmul(A, B, accumulate=True)
    with pytest.raises(ValueError, match="out"):
        mu.mx4_matmul(A, B, out=[torch.zeros(5, 4, device=DEV)])
    with pytest.raises(mu.MuonError):
        mu.mx4_matmul(A, B, torch.float16)
    with pytest.raises(mu.MuonError):
        mu.mx4_dequantize(A, torch.float16)
    with pytest.raises(ValueError, match="transpose"):
        mu.mx4_quantize([torch.zeros(3, 3, device=DEV)], transpose="rows")
    with pytest.raises(ValueError, match="out"):
        mu.mx4_quantize([torch.zeros(3, 3, device=DEV)], out=A)
    with pytest.raises(ValueError, match="contiguous"):
        mu.mx4_quantize([torch.zeros(3, 4, device=DEV).t()])
    codes = torch.zeros(1 * 4 * 64 + 8, dtype=torch.uint8, device=DEV)[8:].view(1, 4, 64)
    with pytest.raises(ValueError, match="aligned"):
        mu.mx4_matmul(mu.MX4([codes], A.scales, 100), B)
    two, twoB = random_code(2, 4, 100, 19), random_code(2, 5, 100, 20)
    C = torch.zeros(4, 5, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        mu.mx4_matmul(two, twoB, out=[C, C])
    with pytest.raises(ValueError, match="overlaps"):
        q = mu.MX4.empty(1, 4, 100, DEV)
        mu.mx4_quantize([torch.zeros(4, 100, device=DEV)] * 2, out=mu.MX4(q.codes * 2, q.scales * 2, 100))
    with pytest.raises(ValueError, match="stream"):
        mu.mx4_matmul(A, B, stream=type("S", (), {"cuda_stream": 0, "device": torch.device("cuda:1")})())
    with pytest.raises(ValueError, match="empty"):
        mu.mx4_quantize([torch.zeros(0, 5, device=DEV)])


# --- graphs, streams -----------------------------------------------------------------------------------------------
def test_captured_layer_replays_like_eager():
    """Code, product (the split over k among them) and accumulation in one graph; new data between the replays."""
    X = torch.randn(300, 2000, device=DEV).to(torch.bfloat16)
    W = random_code(1, 200, 2000, 21)
    q = mu.MX4.empty(1, 300, 2000, DEV)
    C, S = [torch.zeros(300, 200, device=DEV)], [torch.zeros(300, 200, device=DEV)]

    def layer():
        mu.mx4_quantize([X], out=q)
        mu.mx4_matmul(q, W, out=C)
        mu.mx4_matmul(q, W, out=S, accumulate=True)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    total = S[0].clone()
    for i in range(4):
        X.copy_(torch.randn(300, 2000, device=DEV, generator=torch.Generator(DEV).manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        want = mu.mx4_matmul(mu.mx4_quantize([X]), W, torch.float32)[0]
        assert torch.equal(C[0], want), i
        total = total + want
        assert torch.equal(S[0], total), i


def test_two_products_at_once_on_two_streams():
    A, B = random_code(1, 260, 6000, 22), random_code(1, 300, 6000, 23)
    want = mu.mx4_matmul(A, B, torch.float32)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[mu.mx4_matmul(A, B, torch.float32, stream=s)[0] for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for pair in got for x in pair)


def test_two_captured_products_replayed_at_once():
    """Two graphs of products that are split along k, each with its own scratch, replayed side by side."""
    sets = []
    for i in range(2):
        A, B = random_code(1, 260, 6000, 30 + i), random_code(1, 300, 6000, 40 + i)
        C = [torch.zeros(260, 300, device=DEV)]
        mu.mx4_matmul(A, B, out=C)
        want = C[0].clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mu.mx4_matmul(A, B, out=C)
        sets.append((g, C, want, torch.cuda.Stream(), A, B))
    for _ in range(4):
        for g, C, *_ in sets:
            C[0].zero_()
        torch.cuda.synchronize()
        for g, C, want, s, A, B in sets:
            with torch.cuda.stream(s):
                g.replay()
        mu.mx4_matmul(sets[0][4], sets[0][5], torch.float32)  # eager work beside them
        torch.cuda.synchronize()
        for g, C, want, *_ in sets:
            assert torch.equal(C[0], want)


def test_code_of_more_matrices_than_one_launch_takes():
    X = matrices(35, 9, 70, "bf16", 25)
    q, t = mu.mx4_quantize(X, transpose="both")
    same_code(q, [f64(x) for x in X])
    same_code(t, [f64(x).T for x in X])
    for y, c, s in zip(mu.mx4_dequantize(q), q.codes, q.scales):
        assert np.array_equal(f64(y), xo.decode(c.cpu().numpy(), s.cpu().numpy(), 70))


def test_code_and_values_past_2_31_elements():
    """66000 x 32768 bf16 (2.16e9 elements): the last rows' codes in both orientations, and their values."""
    rows, cols = 66000, 32768
    X = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    X[-300:] = torch.randn(300, cols, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(torch.bfloat16)
    q, t = mu.mx4_quantize([X], transpose="both")
    # the last whole unit of 128 rows and what follows start at row 515 * 128 = 65920 of 66000
    tail = mu.MX4([q.codes[0][:, -80:].contiguous()], [q.scales[0][:, -80:].contiguous()], cols)
    same_code(tail, [f64(X[-80:])])
    wc, ws = xo.quantize(f64(X[65920:]).T)
    assert np.array_equal(t.codes[0][515:].cpu().numpy(), wc) and np.array_equal(t.scales[0][515:].cpu().numpy(), ws)
    assert not q.codes[0][:, :65700].any() and not t.codes[0][:513].any()
    only = mu.mx4_quantize([X])
    assert torch.equal(only.codes[0], q.codes[0]) and torch.equal(only.scales[0], q.scales[0])
    del only, t
    Y = mu.mx4_dequantize(q, torch.bfloat16)[0]
    assert np.array_equal(f64(Y[-80:]), xo.decode(tail.codes[0].cpu().numpy(), tail.scales[0].cpu().numpy(), cols))
    assert not Y[:65700].any()


def test_product_past_2_31_elements():
    """50000 x 50000 results (2.5e9): rows at the start, in the middle and at the end."""
    A, B = random_code(1, 50000, 100, 26, 127, 127), random_code(1, 50000, 100, 27, 127, 127)
    b64 = decoded(B)[0]
    C = mu.mx4_matmul(A, B, torch.bfloat16)[0]
    a64 = decoded(A)[0]
    for i in (0, 1, 255, 256, 42949, 42950, 49997, 49999):
        want = f64(torch.from_numpy((a64[i] @ b64.T).astype(np.float32)).to(torch.bfloat16))
        assert np.array_equal(f64(C[i]), want), i


def test_mx4_launches_are_traced():
    X = matrices(1, 64, 128, "f32", 24)
    mu.trace_enable(True)
    q = mu.mx4_quantize(X)
    mu.mx4_dequantize(q)
    mu.mx4_matmul(q, q)
    recs = mu.trace_collect()
    mu.trace_enable(False)
    assert [r["role"] for r in recs] == ["mx4_quantize", "mx4_dequantize", "mx4_matmul"]
    assert recs[2]["flops"] == 2.0 * 64 * 64 * 128


def test_values_of_every_scale_byte():
    """All scale bytes with all codes: fp32 holds every product exactly up to byte 252 (6 times 2^125)."""
    units, rows = 2, 256
    scales = torch.arange(256, dtype=torch.uint8).view(1, 256, 1).expand(units, rows, 4).contiguous()
    codes = torch.arange(64, dtype=torch.uint8).mul(37).view(1, 1, 64).expand(units, rows, 64).contiguous()
    codes[..., :16] = torch.arange(16, dtype=torch.uint8) * 17
    q = mu.MX4([codes.to(DEV)], [scales.to(DEV)], 256)
    want = xo.decode(codes.numpy(), scales.numpy(), 256)
    big = np.abs(want) >= 2.0 ** 128  # over fp32's largest value (bytes 253 and 254): infinite
    want[big] = np.sign(want[big]) * np.inf
    for dt in (torch.float32, torch.bfloat16):
        assert np.array_equal(want, f64(mu.mx4_dequantize(q, dt)[0]), equal_nan=True)


def test_given_outputs_raise_their_version():
    """Writing into out= is seen by autograd, as any in-place operation is."""
    X = matrices(1, 40, 200, "f32", 61)
    q, t = mu.mx4_quantize(X, transpose="both")
    Y, C = [torch.zeros(40, 200, device=DEV)], [torch.zeros(40, 40, device=DEV)]
    ws = torch.zeros(mu.mx4_workspace_size(1, 40, 40, 200), dtype=torch.uint8, device=DEV)
    written = q.codes + q.scales + t.codes + t.scales + Y + C + [ws]
    before = [x._version for x in written]
    held = X[0]._version
    mu.mx4_quantize(X, transpose="both", out=(q, t))
    codes = [x._version for x in q.codes + q.scales]
    mu.mx4_dequantize(q, out=Y)
    mu.mx4_matmul(q, q, out=C, workspace=ws)
    assert all(x._version > b for x, b in zip(written, before))
    assert X[0]._version == held and [x._version for x in q.codes + q.scales] == codes
    p = torch.nn.Parameter(Y[0])
    loss = (p * p).sum()
    mu.mx4_dequantize(q, out=[p])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
