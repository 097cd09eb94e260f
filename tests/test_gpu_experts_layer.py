"""The operators together, as training steps of a mixture of experts use them: the router's balance loss with counts and
gradient, the tokens' code sorted by expert, the experts' three products with the counts, the Muon step on the experts'
weights and AdamW on the router's, and the updated weights coded again.  Each stage is checked against the oracles on the
values that went into it."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import adamw_oracle as ao
from oracle import balance_oracle as bo
from oracle import fp8_oracle as fo
from oracle import muon_oracle as orc
from synth import inputs as syn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
f64 = syn.to_f64


def coded(x, fmt="e4m3", tile=False):
    return fo.decode(*fo.quantize(x, fmt, tile), x.shape[1], fmt)


def within(got, want, bound, what):
    bad = ~(np.abs(f64(got) - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}"


@pytest.mark.parametrize("tokens,experts,top,n_in,n_out,fmt", [(1, 4, 2, 130, 96, "e4m3"), (150, 6, 2, 200, 136, "e4m3"),
                                                               (333, 3, 1, 256, 70, "e5m2")])
def test_training_steps_of_a_mixture(tokens, experts, top, n_in, n_out, fmt):
    rng = np.random.default_rng(7)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV)  # noqa: E731
    W = [dev(rng.standard_normal((n_out, n_in)) * 0.1) for _ in range(experts)]
    M = [torch.zeros_like(w) for w in W]
    R, Rm, Rv = [dev(rng.standard_normal((experts, n_in)) * 0.05)], [torch.zeros(experts, n_in, device=DEV)], \
        [torch.zeros(experts, n_in, device=DEV)]
    w_code, w_code_t = mu.fp8_quantize(W, "tile", transpose="both")
    for t in (1, 2):
        X = dev(rng.standard_normal((tokens, n_in)))
        G = dev(rng.standard_normal((tokens, top, n_out)))  # the gradient that comes back for every choice
        # router
        z = (X @ R[0].t()).contiguous()
        index = torch.topk(z, top, -1).indices
        loss, counts, dz = mu.expert_balance(z, index, 0.05, grad=True)
        wl, wc, wg = bo.balance(f64(z)[None], index.cpu().numpy()[None], 0.05)
        bl, bg = bo.tolerance(f64(z)[None], index.cpu().numpy()[None], 0.05)
        assert abs(float(loss) - wl) <= bl + 2.0 ** -24 * wl and np.array_equal(counts.cpu().numpy(), wc)
        within(dz, wg[0], bg[0] + 2.0 ** -24 * np.abs(wg[0]), "router gradient")
        # tokens sorted by expert, their code in both orientations
        order = torch.argsort(index.flatten(), stable=True)
        rows = X[order // top].contiguous()
        dH = [G.flatten(0, 1)[order].contiguous()]
        x, xt = mu.fp8_quantize([rows], transpose="both", counts=counts)
        d, dt = mu.fp8_quantize(dH, transpose="both", counts=counts, format=fmt)
        H = mu.fp8_grouped_matmul(x, w_code, counts, torch.float32)[0]
        dX = mu.fp8_grouped_matmul(d, w_code_t, counts, torch.float32)[0]
        dW = mu.fp8_grouped_weight_grad(dt, xt, counts)
        at = 0
        for e, c in enumerate(wc):
            part = slice(at, at + c)
            w64, x64, d64 = f64(W[e]), f64(rows[part]), f64(dH[0][part])
            if c:
                within(H[part], *fo.matmul(coded(x64), coded(w64, tile=True)), "H")
                within(dX[part], *fo.matmul(coded(d64, fmt), coded(w64, tile=True).T), "dX")
                within(dW[e], *fo.matmul(coded(d64.T.copy(), fmt), coded(x64.T.copy())), "dW")
            else:
                assert not dW[e].any()
            at += c
        # steps
        W0, M0 = [f64(w) for w in W], [f64(m) for m in M]
        O = [torch.empty_like(w) for w in W]
        mu.muon_step(W, M, dW, 0.95, 0.02, 0.0, "standard", mu.NSConfig(compute="f32"), O_out=O)
        for e in range(experts):
            _, Mr, Or = orc.muon_step(W0[e], M0[e], f64(dW[e]), float(np.float32(0.95)), float(np.float32(0.02)), 0.0,
                                      "standard", state_dtype="f32", w_dtype="f64")
            assert np.array_equal(f64(M[e]), Mr)
            if Mr.any():
                assert orc.relative_frobenius(f64(O[e]), Or) < 1e-4
        dR = [(dz.t() @ X).contiguous()]
        args = (f64(R[0]), f64(Rm[0]), f64(Rv[0]), f64(dR[0]), t, 1e-3, 0.9, 0.99, 1e-8, 0.0)
        mu.adamw_step(R, Rm, Rv, dR, t, 1e-3, 0.9, 0.99)
        within(R[0], ao.adamw(*args)[0], ao.adamw_tolerance(*args)[0], "router weights")
        # the updated weights, coded for the next step into the same buffers
        mu.fp8_quantize(W, "tile", transpose="both", out=(w_code, w_code_t))
        for q, w in zip(mu.fp8_dequantize(w_code), W):
            assert np.array_equal(f64(q), coded(f64(w), tile=True))


def test_gradients_of_the_products_against_differences():
    """Operands that the code holds exactly (whole numbers), a loss linear in the experts' outputs: differences over one step
    of a weight or an input are the gradients, in every digit."""
    rng = np.random.default_rng(8)
    counts_list, n_in, n_out = [5, 0, 130, 2], 9, 6
    counts = torch.tensor(counts_list, dtype=torch.int32, device=DEV)
    rows = sum(counts_list)
    whole = lambda *s: torch.from_numpy(rng.integers(-4, 5, s).astype(np.float32)).to(DEV)  # noqa: E731
    X, G, W = whole(rows, n_in), whole(rows, n_out), [whole(n_out, n_in) for _ in counts_list]

    def loss(X, W):
        h = mu.fp8_grouped_matmul(mu.fp8_quantize([X]), mu.fp8_quantize(W, "tile"), counts, torch.float32)[0]
        return float((h.double() * G.double()).sum())

    x, xt = mu.fp8_quantize([X], transpose="both", counts=counts)
    d, dt = mu.fp8_quantize([G], transpose="both", counts=counts)
    dW = mu.fp8_grouped_weight_grad(dt, xt, counts)
    dX = mu.fp8_grouped_matmul(d, mu.fp8_quantize(W, "tile", transpose=True), counts, torch.float32)[0]
    for e in range(len(W)):
        for i, j in ((0, 0), (3, 7), (n_out - 1, n_in - 1)):
            up, down = [w.clone() for w in W], [w.clone() for w in W]
            up[e][i, j] += 1
            down[e][i, j] -= 1
            assert (loss(X, up) - loss(X, down)) / 2 == float(dW[e][i, j])
    for i, j in ((0, 0), (4, 8), (5, 3), (134, 1), (rows - 1, n_in - 1)):
        up, down = X.clone(), X.clone()
        up[i, j] += 1
        down[i, j] -= 1
        assert (loss(up, W) - loss(down, W)) / 2 == float(dX[i, j])


def test_a_step_on_another_stream_and_from_a_padded_batch():
    """A whole forward on a stream of its own; rows behind the counted ones (padding that goes to no expert) stay 0."""
    torch.manual_seed(0)
    T, E, n, k = 64, 4, 48, 160
    z = torch.randn(T, E, device=DEV)
    mask = torch.arange(T, device=DEV) < 50
    index = torch.topk(z, 1, -1).indices
    W = mu.fp8_quantize([torch.randn(n, k, device=DEV) for _ in range(E)], "tile")
    X = torch.randn(T, k, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss, counts, _ = mu.expert_balance(z, index, 1.0, mask=mask)
        order = torch.argsort(torch.where(mask, index[:, 0], E), stable=True)
        Y = mu.fp8_grouped_matmul(mu.fp8_quantize([X[order].contiguous()]), W, counts, torch.float32)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert int(counts.sum()) == 50 and not Y[50:].any()
    w = mu.fp8_dequantize(W)
    x = mu.fp8_dequantize(mu.fp8_quantize([X]))[0]
    for r, t in enumerate(order[:50].tolist()):
        want = f64(x[t]) @ f64(w[int(index[t, 0])]).T
        assert np.all(np.abs(f64(Y[r]) - want) <= (k + 2) * 2.0 ** -23 * (np.abs(f64(x[t])) @ np.abs(f64(w[int(index[t, 0])])).T))
