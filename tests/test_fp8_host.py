"""CPU checks of the 8-bit code, its products and the experts' balance: the oracles against independent statements of the same
definitions, and the refusals of the C ABI and of the binding (no device work)."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import balance_oracle as bo
from oracle import fp8_oracle as fo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# --- oracles -------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_tables_and_rounding_against_torch(fmt, dtype):
    table = fo.magnitudes(fmt)
    assert np.array_equal(torch.arange(len(table), dtype=torch.uint8).view(dtype).double().numpy(), table)
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 256)) * np.exp(rng.standard_normal((40, 256)) * 3)).astype(np.float32)
    codes, scales = fo.quantize(x.astype(np.float64), fmt)
    power = np.repeat(np.ldexp(1.0, scales.T.astype(int) - 127), 128, 1)
    want = torch.from_numpy((x / power).astype(np.float32)).to(dtype).view(torch.uint8).numpy()
    assert np.array_equal(codes.transpose(1, 0, 2).reshape(40, 256), want)


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("e5m2", 57344.0)])
def test_scale_is_the_smallest_that_holds_the_block(fmt, top):
    for value, byte in [(top, 127), (np.nextafter(top, 1e9), 128), (np.nextafter(top, 0), 127), (top / 2, 126),
                        (0.0, 0), (2.0 ** -149, 0), (np.inf, 255), (np.nan, 255), (3.4028234663852886e38, None)]:
        X = np.zeros((1, 128))
        X[0, 5] = -value
        codes, scales = fo.quantize(X, fmt)
        if byte is not None:
            assert scales[0, 0] == byte, value
        if np.isfinite(value):
            y = fo.decode(codes, scales, 128, fmt)[0, 5]
            assert abs(-value - y) <= max(abs(value) * (2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3), 2.0 ** -127)
            if scales[0, 0] > 0:
                assert abs(value) > top * 2.0 ** (int(scales[0, 0]) - 128)  # the next smaller one would not do
        else:
            assert not codes.any()


def test_tile_codes_are_the_same_in_both_orientations():
    X = np.random.default_rng(2).standard_normal((300, 200)) * np.exp(np.random.default_rng(3).standard_normal((300, 1)) * 4)
    a, b = fo.quantize(X, tile=True), fo.quantize(X.T.copy(), tile=True)
    assert np.array_equal(fo.decode(*a, 200), fo.decode(*b, 300).T)
    assert len(set(a[1][0, :128])) == 1 and len(set(a[1][1, 256:])) == 1


def test_column_code_of_groups_by_hand():
    X = np.arange(1, 7.0)[:, None] * np.ones((1, 2))
    codes, scales = fo.quantize_columns(X, [2, 0, 4])
    assert codes.shape == (4, 2, 64) and scales.shape == (2, 2)
    y = fo.decode(codes, scales, 256)
    assert y[0, :2].tolist() == [1, 2] and y[1, 128:132].tolist() == [3, 4, 5, 6] and not y[:, 2:128].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_oracle_against_autograd(score):
    rng = np.random.default_rng(4)
    S, T, E, K = 3, 11, 7, 2
    z = torch.from_numpy(rng.standard_normal((S, T, E)) * 2).requires_grad_()
    index = rng.integers(-1, E + 1, (S, T, K))
    mask = rng.random((S, T)) < 0.7
    mask[2] = False
    loss = 0.0
    for s in range(S):
        rows = z[s][torch.from_numpy(mask[s])]
        if len(rows) == 0:
            continue
        p = torch.softmax(rows, -1) if score == "softmax" else torch.sigmoid(rows) / torch.sigmoid(rows).sum(-1, keepdim=True)
        f = torch.zeros(E, dtype=torch.float64)
        for e in range(E):
            f[e] = E * np.sum(index[s][mask[s]] == e) / (K * len(rows))
        loss = loss + 0.3 * (f * p.mean(0)).sum() / S
    loss.backward()
    wl, wc, wg = bo.balance(z.detach().numpy(), index, 0.3, score, mask)
    assert abs(wl - float(loss.detach())) < 1e-14 and np.allclose(wg, z.grad.numpy(), rtol=0, atol=1e-15)
    assert wc.tolist() == [int(np.sum(index[mask] == e)) for e in range(E)]


def test_perfect_balance_has_loss_one():
    """With every expert chosen equally often f = 1, and the loss is alpha sum_e mean p_e = alpha."""
    z, index = np.random.default_rng(5).standard_normal((1, 8, 4)), np.arange(8)[None, :, None] % 4
    loss, counts, grad = bo.balance(z, index, 0.25)
    assert abs(loss - 0.25) < 1e-15 and counts.tolist() == [2] * 4 and np.abs(grad).max() < 1e-16


# --- refusals ------------------------------------------------------------------------------------------------------
_keep = []


def ptrs(*values):
    """The address of a new host array of (bogus, never used) device pointers."""
    a = (ctypes.c_void_p * len(values))(*values)
    _keep.append(a)
    return ctypes.addressof(a)


P = [ptrs(*[4096 * (i + 1)] * 3) for i in range(8)]


def test_code_refusals_before_any_device_work():
    lib = mu.load_library()
    mu.binding._require_list_calls(lib, mu.binding._FP8_CALLS)

    def q(b=1, r=4, c=4, X=P[0], dt=0, tile=0, f=0, counts=None, g=0, codes=P[1], scales=P[2], ct=P[3], st=P[4]):
        return lib.muon_fp8_quantize(b, r, c, X, dt, tile, f, counts, g, codes, scales, ct, st, None)

    for kw in [dict(b=0), dict(r=0), dict(c=0), dict(r=(1 << 20) + 1), dict(c=(1 << 20) + 1), dict(X=None), dict(dt=5),
               dict(tile=2), dict(f=2), dict(codes=None), dict(scales=None), dict(ct=None), dict(st=None),
               dict(codes=None, scales=None, ct=None, st=None), dict(codes=P[0]), dict(st=P[2]), dict(X=ptrs(None)),
               dict(b=2, ct=ptrs(64, None)), dict(g=1), dict(counts=4096), dict(counts=4096, g=-1), dict(counts=4098, g=2),
               dict(counts=4096, g=2, b=2), dict(counts=4096, g=2, tile=1), dict(counts=4096, g=2, ct=None, st=None),
               dict(counts=4096, g=1 << 20, r=1 << 11), dict(counts=4096, g=65535)]:
        assert q(**kw) == 1, kw
    for off in (1, 4, 8):
        for name in ("codes", "scales", "ct", "st"):
            assert q(**{name: ptrs((1 << 20) + off)}) == 1
    d = lambda b=1, r=4, c=4, codes=P[0], scales=P[1], f=0, Y=P[2], dt=0: (  # noqa: E731
        lib.muon_fp8_dequantize(b, r, c, codes, scales, f, Y, dt, None))
    for kw, code in [(dict(b=0), 1), (dict(r=0), 1), (dict(c=-1), 1), (dict(codes=None), 1), (dict(scales=None), 1),
                     (dict(f=3), 1), (dict(Y=None), 1), (dict(dt=9), 1), (dict(Y=P[0]), 1), (dict(scales=P[0]), 1),
                     (dict(dt=2), 2), (dict(Y=ptrs(None)), 1), (dict(codes=ptrs(8)), 1)]:
        assert d(**kw) == code, kw


def test_product_refusals_before_any_device_work():
    lib = mu.load_library()
    assert lib.muon_fp8_workspace_size(1, 4, 4, 4) > 0
    for args in [(0, 4, 4, 4), (1, 0, 4, 4), (1, 4, 0, 4), (1, 4, 4, 0), (1, (1 << 20) + 1, 4, 4), (16, 1 << 20, 1 << 20, 4)]:
        assert lib.muon_fp8_workspace_size(*args) == 0, args
    g = lambda b=1, m=4, n=4, k=4, A=P[0], As=P[1], f=0, B=P[2], Bs=P[3], C=P[4], dt=0, acc=0, ws=256, wsb=1 << 40: (  # noqa: E731
        lib.muon_fp8_matmul(b, m, n, k, A, As, f, B, Bs, C, dt, acc, ws, wsb, None))
    for kw, code in [(dict(b=0), 1), (dict(m=0), 1), (dict(k=0), 1), (dict(A=None), 1), (dict(As=None), 1), (dict(f=2), 1),
                     (dict(B=None), 1), (dict(Bs=None), 1), (dict(C=None), 1), (dict(C=P[0]), 1), (dict(C=P[3]), 1),
                     (dict(C=ptrs(None)), 1), (dict(dt=4), 1), (dict(acc=2), 1), (dict(dt=2), 2), (dict(ws=None), 3),
                     (dict(wsb=0), 3), (dict(ws=272), 3), (dict(A=ptrs(24)), 1), (dict(Bs=ptrs(4)), 1)]:
        assert g(**kw) == code, kw
    m = lambda e=2, r=4, n=4, k=4, c=4096, A=4096, As=8192, f=0, B=P[2], Bs=P[3], C=64, dt=0, acc=0, cl=0: (  # noqa: E731
        lib.muon_fp8_grouped_matmul(e, r, n, k, c, A, As, f, B, Bs, C, dt, acc, cl, None))
    for kw, code in [(dict(e=0), 1), (dict(r=0), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(c=None), 1), (dict(c=4098), 1),
                     (dict(A=None), 1), (dict(As=8), 1), (dict(f=-1), 1), (dict(B=None), 1), (dict(Bs=ptrs(16, None)), 1),
                     (dict(C=None), 1), (dict(C=4096, A=4096), 1), (dict(dt=3), 1), (dict(acc=2), 1), (dict(cl=2), 1),
                     (dict(dt=2), 2),
                     (dict(e=1 << 12, r=1 << 20, B=ptrs(*[16] * 4096), Bs=ptrs(*[16] * 4096)), 1)]:
        assert m(**kw) == code, kw
    w = lambda e=2, r=4, m=4, n=4, c=4096, A=4096, As=8192, f=0, B=64, Bs=128, C=P[4], dt=0, acc=0: (  # noqa: E731
        lib.muon_fp8_grouped_weight_grad(e, r, m, n, c, A, As, f, B, Bs, C, dt, acc, None))
    for kw, code in [(dict(e=0), 1), (dict(r=0), 1), (dict(m=0), 1), (dict(n=0), 1), (dict(c=None), 1), (dict(A=None), 1),
                     (dict(As=4), 1), (dict(B=None), 1), (dict(Bs=None), 1), (dict(f=7), 1), (dict(C=None), 1),
                     (dict(C=ptrs(8, None)), 1), (dict(dt=3), 1), (dict(acc=-1), 1), (dict(dt=2), 2)]:
        assert w(**kw) == code, kw


def test_balance_refusals_before_any_device_work():
    lib = mu.load_library()
    assert lib.muon_expert_balance_workspace_size(1, 4, 4, 2) > 0
    for args in [(0, 4, 4, 2), (1, 0, 4, 2), (1, 4, 0, 2), (1, 4, 4, 0), (1, 4, 1025, 2), (65536, 4, 4, 2),
                 (4, 1 << 29, 4, 1), (1, 1 << 30, 4, 2)]:
        assert lib.muon_expert_balance_workspace_size(*args) == 0, args
    nan, inf = float("nan"), float("inf")

    def b(S=1, T=4, E=4, K=2, z=4096, dt=0, stride=4, i=8192, bits=64, mask=None, score=0, a=0.1, gs=None, loss=64, counts=128,
          grad=256, acc=0, ws=512, wsb=1 << 30):
        return lib.muon_expert_balance(S, T, E, K, z, dt, stride, i, bits, mask, score, a, gs, loss, counts, grad, acc, ws, wsb,
                                       None)

    for kw, code in [(dict(S=0), 1), (dict(T=0), 1), (dict(E=0), 1), (dict(E=2000), 1), (dict(K=0), 1), (dict(z=None), 1),
                     (dict(dt=3), 1), (dict(stride=-1), 1), (dict(i=None), 1), (dict(bits=16), 1), (dict(score=2), 1),
                     (dict(a=nan), 1), (dict(a=inf), 1), (dict(a=1e39), 1), (dict(loss=None), 1), (dict(counts=None), 1),
                     (dict(grad=None, acc=1), 1), (dict(acc=2), 1), (dict(grad=4096), 1), (dict(ws=None), 3),
                     (dict(wsb=0), 3), (dict(ws=520), 3)]:
        assert b(**kw) == code, kw


def test_binding_refusals():
    u8, f8 = torch.uint8, torch.float8_e4m3fn
    good = mu.FP8([torch.zeros(4, 5, 64, dtype=u8).view(f8)], [torch.zeros(2, 16, dtype=u8)], 200)
    assert good.rows == 5
    with pytest.raises(ValueError, match="device tensors"):
        mu.fp8_dequantize(good)
    for bad in [mu.FP8([], [], 200), mu.FP8(good.codes, [], 200), mu.FP8(good.codes, good.scales, 300),
                mu.FP8([torch.zeros(4, 5, 32, dtype=u8).view(f8)], good.scales, 200), mu.FP8(good.codes, good.scales, 0),
                mu.FP8(good.codes, good.scales, 200, -1), mu.FP8(good.codes, good.scales, 200, 2)]:
        with pytest.raises(ValueError):
            mu.fp8_matmul(bad, good)
    with pytest.raises(ValueError):
        mu.fp8_quantize([torch.zeros(3, 3)])
    with pytest.raises(ValueError, match="device tensor"):
        mu.expert_balance(torch.zeros(3, 3), torch.zeros(3, 1, dtype=torch.int64), 1.0)
    with pytest.raises(ValueError, match="format"):
        mu.FP8.empty(1, 2, 2, "cpu", format="e8m0")
    e = mu.FP8.empty(2, 17, 130, "cpu", "e5m2", groups=3)
    assert e.codes[0].shape == (2 * ((130 + 127 * 3) // 128), 17, 64) and e.scales[1].shape == ((130 + 127 * 3) // 128, 32)


PROBE = """
import torch
import matrix_orthogonalizing_optimizer_step_amd as mu
try:
    mu.adamw_step([], [], [], [], 1, 1e-3)
except ValueError as e:
    print("adamw:", e)
for call in (lambda: mu.fp8_quantize([torch.zeros(2, 2)]), lambda: mu.fp8_workspace_size(1, 2, 2, 2),
             lambda: mu.expert_balance(torch.zeros(2, 2), torch.zeros(2, 1, dtype=torch.int64), 1.0)):
    try:
        call()
    except ImportError as e:
        print("refused:", e)
"""


def test_other_calls_need_no_newer_entry_points(tmp_path):
    """A library with the calls on lists of an earlier build and without these (a stand-in with the other functions only)."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "muon.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)) - {"sizeof"})
    old = [n for n in names if "fp8" not in n and "balance" not in n]
    assert len(names) - len(old) == 8
    source = tmp_path / "old.c"
    source.write_text("\n".join(f"unsigned long {n}(void) {{ return 6; }}" for n in old))
    lib = tmp_path / "libold.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(source)], check=True)
    out = subprocess.run([sys.executable, "-c", PROBE], cwd=ROOT, env=dict(os.environ, MUON_LIBRARY=str(lib)),
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    lines = out.stdout.splitlines()
    assert lines[0].startswith("adamw:") and "empty list" in lines[0]
    assert len(lines) == 4 and all("older build of the library" in r for r in lines[1:])
