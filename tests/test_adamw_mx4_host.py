"""CPU checks of the AdamW step and the microscaled 4-bit code: the oracles against independent statements of the same
definitions, and the refusals of the C ABI and of the binding (no device work)."""
import ctypes

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from matrix_orthogonalizing_optimizer_step_amd import binding as bd
from oracle import adamw_oracle as ao
from oracle import mx4_oracle as xo


# --- oracles -------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_adamw_oracle_against_torch(wd):
    """torch.optim.AdamW in float64: W <- (1 - lr wd) W - lr m_hat / (sqrt(v_hat) + eps), the same step."""
    rng = np.random.default_rng(1)
    W = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(W.copy()))
    opt = torch.optim.AdamW([p], lr=0.02, betas=(0.9, 0.99), eps=1e-6, weight_decay=wd)
    m = v = np.zeros(50)
    for t in range(1, 6):
        G = rng.standard_normal(50)
        p.grad = torch.from_numpy(G.copy())
        opt.step()
        W, m, v = ao.adamw(W, m, v, G, t, 0.02, 0.9, 0.99, 1e-6, wd)
        assert np.allclose(W, p.detach().numpy(), rtol=0, atol=64 * 2.0 ** -53 * t)


def test_e4m3_table_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ao.decode_e4m3(codes.numpy()), want, equal_nan=True)


def test_root_rounding_keeps_the_expected_square():
    """Over all u the share of roundings up is (x^2 - lo^2) / (hi^2 - lo^2), so the mean square is x^2."""
    table = ao.e4m3_values()
    x = np.array([0.3, 1.03, 200.5, 447.0, 2.0 ** -8 * 1.5])
    j = np.searchsorted(table, x, side="right")
    lo, hi = table[j - 1], table[j]
    share = (x * x - lo * lo) / (hi * hi - lo * lo)
    assert np.allclose(share * hi * hi + (1 - share) * lo * lo, x * x, rtol=1e-12)
    u = ao.chances(1 << 20, 7, 3, 0)
    assert abs(u.mean() - 0.5) < 5 * np.sqrt(1 / 12 / u.size)          # five standard deviations
    assert abs(np.corrcoef(u[:-1], u[1:])[0, 1]) < 5 / np.sqrt(u.size)
    assert abs((u < 0.006).mean() - 0.006) < 5 * np.sqrt(0.006 / u.size) + 1 / 65536


@pytest.mark.parametrize("values,byte,codes", [
    ([0.0] * 32, 0, [0] * 32),
    ([4.0, -1.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.2], 127, [6, 10, 0, 2, 2, 4, 4, 6, 6, 7, 8]),
    ([1.0], 125, [6]),                                     # 2^0: two binades under is 2^-2, code of 4
    ([2.0 ** -126], 0, [4]),                               # the scale stops at 2^-127: 2^-126 is 2 of it
    ([float("inf"), 1.0], 255, [0, 0]),
    ([1.0, float("nan")], 255, [0, 0]),
    ([3.4028234663852886e38], 252, [7]),                   # largest fp32: 2^125 times 6 (saturated)
])
def test_mx4_oracle_by_hand(values, byte, codes):
    X = np.zeros((1, 32))
    X[0, :len(values)] = values
    c, s = xo.quantize(X)
    assert s[0, 0, 0] == byte
    nib = np.stack((c[0, 0] & 15, c[0, 0] >> 4), -1).reshape(-1)
    assert nib[:len(codes)].tolist() == codes
    assert np.all(s[0, 0, 1:] == 0) and np.all(c[0, 0, 16:] == 0)


def test_mx4_oracle_error_bound():
    """Without saturation a value is off by at most half a step of its binade: 1/4 of the scale below 2, 1/2 below 4, 1
    up to 6; above 6 by less than 2."""
    rng = np.random.default_rng(5)
    X = rng.standard_normal((7, 300)) * np.exp(rng.standard_normal((7, 1)) * 5)
    c, s = xo.quantize(X)
    Y = xo.decode(c, s, 300)
    P = np.zeros((7, 384))
    P[:, :300] = X
    scale = np.repeat(np.ldexp(1.0, xo.scale_bytes(P.reshape(7, 12, 32)).astype(int) - 127), 32, axis=1)[:, :300]
    a = np.abs(X) / scale
    bound = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a <= 6, 1.0, 2.0))) * scale
    assert np.all(np.abs(Y - X) <= bound)


# --- refusals ------------------------------------------------------------------------------------------------------
_keep = []


def ptrs(*values):
    """The address of a new host array of (bogus, never used) device pointers."""
    a = (ctypes.c_void_p * len(values))(*values)
    _keep.append(a)
    return ctypes.addressof(a)


P = [ptrs(*[4096 * (i + 1)] * 3) for i in range(8)]


def _adamw(lib, tensors=1, sizes=(4,), W=P[0], wdt=0, M=P[1], V=P[2], G=P[3], gdt=0, null_cfg=False, **cfg):
    c = bd._AdamWConfig()
    lib.muon_adamw_config_init(ctypes.byref(c))
    for k, v in cfg.items():
        setattr(c, k, v)
    arr = (ctypes.c_int64 * len(sizes))(*sizes) if sizes is not None else None
    p = None if null_cfg else ctypes.byref(c)
    a = lib.muon_adamw_step(tensors, arr, W, wdt, M, V, G, gdt, p, None)
    st = bd._AdamW8State(M, V, P[4], P[5])
    b = lib.muon_adamw8_step(tensors, arr, W, wdt, ctypes.byref(st), G, gdt, p, None)
    return a, b


def test_adamw_refusals_before_any_device_work():
    lib = mu.load_library()
    nan, inf = float("nan"), float("inf")
    for kw, code in [(dict(tensors=0), 1), (dict(tensors=-1), 1), (dict(sizes=None), 1), (dict(sizes=(-1,)), 1),
                     (dict(sizes=(1 << 50,)), 1), (dict(W=None), 1), (dict(M=None), 1), (dict(V=None), 1),
                     (dict(G=None), 1), (dict(M=P[0]), 1), (dict(G=P[0]), 1), (dict(V=P[1]), 1), (dict(null_cfg=True), 1),
                     (dict(W=ptrs(None)), 1), (dict(tensors=2, sizes=(0, 4), G=ptrs(None, None)), 1),
                     (dict(wdt=7), 1), (dict(gdt=9), 1), (dict(wdt=2), 2), (dict(lr=nan), 1), (dict(lr=inf), 1),
                     (dict(lr=1e39), 1), (dict(weight_decay=nan), 1), (dict(eps=0.0), 1), (dict(eps=-1e-8), 1),
                     (dict(eps=1e-60), 1), (dict(beta1=1.0), 1), (dict(beta1=-0.1), 1), (dict(beta2=1.0), 1),
                     (dict(beta2=nan), 1), (dict(step=0), 1), (dict(step=-3), 1)]:
        assert _adamw(lib, **kw) == (code, code), kw
    full = (ctypes.c_int64 * 1)(4)
    c = bd._AdamWConfig()
    lib.muon_adamw_config_init(ctypes.byref(c))
    assert (c.lr, c.beta1, c.beta2, c.eps, c.weight_decay, c.step) == (1e-3, 0.9, 0.999, 1e-8, 0.0, 1)
    assert lib.muon_adamw8_step(1, full, P[0], 0, None, P[3], 0, ctypes.byref(c), None) == 1
    for missing in range(4):
        st = bd._AdamW8State(*[None if i == missing else P[4 + i] for i in range(4)])
        assert lib.muon_adamw8_step(1, full, P[0], 0, ctypes.byref(st), P[3], 0, ctypes.byref(c), None) == 1
    lib.muon_adamw_config_init(None)  # no-op


def test_empty_tensors_need_no_device():
    """A list of empty tensors has nothing to launch."""
    none = [ptrs(None, None, None) for _ in range(4)]
    assert _adamw(mu.load_library(), tensors=3, sizes=(0, 0, 0), W=none[0], M=none[1], V=none[2], G=none[3]) == (0, 0)


def test_adamw8_refuses_what_its_quotients_cannot_hold():
    """The 8-bit step works with lr / (1 - beta1^t) and 1 / (c2 root + eps) in fp32: values whose quotients overflow (at
    t = 1, the largest) or fall under the normal range are refused there; the 32-bit step has neither quotient."""
    lib = mu.load_library()
    none = [ptrs(None, None, None) for _ in range(4)]
    empty = dict(tensors=1, sizes=(0,), W=none[0], M=none[1], V=none[2], G=none[3])
    for kw in (dict(lr=1e38), dict(lr=3.4e38), dict(lr=-1e38), dict(lr=1e30, beta1=1 - 2.0 ** -40), dict(eps=1e38),
               dict(eps=2.0 ** 126 * 1.001)):
        assert _adamw(lib, **empty, **kw) == (0, 1), kw
    for kw in (dict(lr=3e37), dict(lr=3.4e38, beta1=0.0), dict(lr=1e20, beta1=1 - 2.0 ** -40), dict(eps=2.0 ** 126)):
        assert _adamw(lib, **empty, **kw) == (0, 0), kw


def test_adamw_binding_refusals():
    z = torch.zeros(4)
    with pytest.raises(ValueError, match="empty list"):
        mu.adamw_step([], [], [], [], 1, 1e-3)
    with pytest.raises(ValueError, match="device tensors"):
        mu.adamw_step([z], [z], [z], [z], 1, 1e-3)
    with pytest.raises(ValueError, match="list of tensors"):
        mu.adamw_step(z, z, z, z, 1, 1e-3)
    with pytest.raises(ValueError, match="list of tensors"):
        mu.adamw_step([1.0], [z], [z], [z], 1, 1e-3)


def test_mx4_refusals_before_any_device_work():
    lib = mu.load_library()
    q = lambda b=1, r=4, c=4, X=P[0], dt=0, codes=P[1], scales=P[2], ct=P[3], st=P[4]: (  # noqa: E731
        lib.muon_mx4_quantize(b, r, c, X, dt, codes, scales, ct, st, None))
    for kw in [dict(b=0), dict(r=0), dict(c=0), dict(r=(1 << 20) + 1), dict(c=(1 << 20) + 1), dict(X=None),
               dict(dt=5), dict(codes=None), dict(scales=None), dict(ct=None), dict(st=None),
               dict(codes=None, scales=None, ct=None, st=None), dict(codes=P[0]), dict(st=P[2]),
               dict(X=ptrs(None)), dict(b=2, ct=ptrs(64, None))]:
        assert q(**kw) == 1, kw
    d = lambda b=1, r=4, c=4, codes=P[0], scales=P[1], Y=P[2], dt=0: (  # noqa: E731
        lib.muon_mx4_dequantize(b, r, c, codes, scales, Y, dt, None))
    for kw, code in [(dict(b=0), 1), (dict(r=0), 1), (dict(c=-1), 1), (dict(codes=None), 1), (dict(scales=None), 1),
                     (dict(Y=None), 1), (dict(dt=9), 1), (dict(Y=P[0]), 1), (dict(scales=P[0]), 1), (dict(dt=2), 2),
                     (dict(Y=ptrs(None)), 1)]:
        assert d(**kw) == code, kw
    assert lib.muon_mx4_workspace_size(1, 4, 4, 4) > 0
    for args in [(0, 4, 4, 4), (1, 0, 4, 4), (1, 4, 0, 4), (1, 4, 4, 0), (1, 1 << 17, 4, 1 << 15),
                 (1, 4, 1 << 20, 1 << 12)]:
        assert lib.muon_mx4_workspace_size(*args) == 0, args
    assert lib.muon_mx4_workspace_size(1, (1 << 16) - 1, 4, 1 << 16) > 0
    g = lambda b=1, m=4, n=4, k=4, A=P[0], As=P[1], B=P[2], Bs=P[3], C=P[4], dt=0, acc=0, ws=256, wsb=1 << 40: (  # noqa: E731
        lib.muon_mx4_matmul(b, m, n, k, A, As, B, Bs, C, dt, acc, ws, wsb, None))
    for kw, code in [(dict(b=0), 1), (dict(m=0), 1), (dict(k=0), 1), (dict(A=None), 1), (dict(As=None), 1),
                     (dict(B=None), 1), (dict(Bs=None), 1), (dict(C=None), 1), (dict(C=P[0]), 1), (dict(C=P[3]), 1), (dict(C=ptrs(None)), 1),
                     (dict(dt=4), 1), (dict(acc=2), 1), (dict(dt=2), 2), (dict(ws=None), 3), (dict(wsb=0), 3),
                     (dict(ws=272), 3), (dict(m=1 << 17, k=1 << 15), 1)]:
        assert g(**kw) == code, kw


def test_mx4_codes_off_their_alignment_are_refused():
    """Codes need 16 bytes (they are read and written 16 at a time), scales 4; in any matrix of the batch."""
    lib = mu.load_library()
    ok = ptrs(1 << 20, 1 << 21)
    for off in (1, 4, 8, 12):
        for at in (0, 1):
            codes = ptrs(*[(1 << 22) + (off if i == at else 0) for i in range(2)])
            scales = ptrs(*[(1 << 23) + (off % 4 or 2 if i == at else 0) for i in range(2)])
            for bad in (0, 1):
                c, s = (codes, ptrs(1 << 24, 1 << 25)) if bad == 0 else (ptrs(1 << 24, 1 << 25), scales)
                assert lib.muon_mx4_quantize(2, 4, 4, ok, 0, c, s, None, None, None) == 1
                assert lib.muon_mx4_quantize(2, 4, 4, ok, 0, None, None, c, s, None) == 1
                assert lib.muon_mx4_dequantize(2, 4, 4, c, s, ok, 0, None) == 1
                fine = (ptrs(1 << 26, 1 << 27), ptrs(1 << 28, 1 << 29))
                assert lib.muon_mx4_matmul(2, 4, 4, 4, c, s, *fine, ok, 0, 0, 256, 1 << 40, None) == 1
                assert lib.muon_mx4_matmul(2, 4, 4, 4, *fine, c, s, ok, 0, 0, 256, 1 << 40, None) == 1

def test_mx4_binding_refusals():
    u8 = torch.uint8
    good = mu.MX4([torch.zeros(2, 5, 64, dtype=u8)], [torch.zeros(2, 5, 4, dtype=u8)], 200)
    assert good.rows == 5
    with pytest.raises(ValueError, match="device tensors"):
        mu.mx4_dequantize(good)
    for bad in [mu.MX4([], [], 200), mu.MX4(good.codes, [], 200), mu.MX4(good.codes, good.scales, 300),
                mu.MX4([torch.zeros(2, 5, 32, dtype=u8)], good.scales, 200), mu.MX4(good.codes, good.scales, 0)]:
        with pytest.raises(ValueError):
            mu.mx4_matmul(bad, good)
    with pytest.raises(ValueError):
        mu.mx4_quantize([torch.zeros(3, 3)])
