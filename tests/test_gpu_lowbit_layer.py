"""The operators together, as one training step of a low-bit linear layer with its neighbours uses them: the layer's
three products on coded operands, the Muon step on its weight, AdamW on its bias and (8-bit) on an embedding, and the
updated weight coded again.  Each stage is checked against the oracles on the values that went into it."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import adamw_oracle as ao
from oracle import muon_oracle as orc
from oracle import mx4_oracle as xo
from synth import inputs as syn

DEV = "cuda:0"
f64 = syn.to_f64


def coded(x):
    c, s = xo.quantize(x)
    return xo.decode(c, s, x.shape[1])


def within(got, want, bound, what):
    bad = np.abs(f64(got) - want) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}"


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,n_in,n_out", [(1, 256, 384), (77, 200, 136)])
def test_training_steps_of_a_low_bit_layer(tokens, n_in, n_out):
    vocab, lr, mom = 50, 0.02, 0.95
    rng = np.random.default_rng(3)
    dev = lambda a, dt=torch.float32: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV).to(dt)  # noqa: E731
    W = [dev(rng.standard_normal((n_out, n_in)) * 0.1)]
    M = [torch.zeros_like(W[0])]
    bias, bias_m, bias_v = [dev(np.zeros(n_out))], [dev(np.zeros(n_out))], [dev(np.zeros(n_out))]
    E = [dev(rng.standard_normal((vocab, n_in)), torch.bfloat16)]
    e_state = mu.AdamW8State.zeros(E)
    hyper = dict(lr=lr, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01)
    w_code, w_code_t = mu.mx4_quantize(W, transpose="both")
    for t in (1, 2):
        ids = torch.from_numpy(rng.integers(0, vocab, tokens)).to(DEV)
        target = dev(rng.standard_normal((tokens, n_out)))
        # forward
        X = [E[0][ids].contiguous()]
        x_code, x_code_t = mu.mx4_quantize(X, transpose="both")
        Y = mu.mx4_matmul(x_code, w_code, torch.float32)
        want, bound = xo.matmul(coded(f64(X[0])), coded(f64(W[0])))
        within(Y[0], want, bound, "Y")
        # backward of 1/2 |Y + bias - target|^2
        dY = [(Y[0] + bias[0] - target).contiguous()]
        d_code, d_code_t = mu.mx4_quantize(dY, transpose="both")
        dX = mu.mx4_matmul(d_code, w_code_t, torch.float32)
        dW = mu.mx4_matmul(d_code_t, x_code_t, torch.float32)
        d64 = f64(dY[0])
        within(dX[0], *xo.matmul(coded(d64), coded(f64(W[0]).T)), "dX")
        within(dW[0], *xo.matmul(coded(d64.T), coded(f64(X[0]).T)), "dW")
        dE = torch.zeros(vocab, n_in, device=DEV).index_add_(0, ids, dX[0])
        # steps
        W0, M0 = f64(W[0]), f64(M[0])
        O = [torch.empty_like(W[0])]
        mu.muon_step(W, M, dW, mom, lr, 0.0, "standard", mu.NSConfig(compute="f32"), O_out=O)
        Wr, Mr, Or = orc.muon_step(W0, M0, f64(dW[0]), float(np.float32(mom)), float(np.float32(lr)), 0.0, "standard",
                                   state_dtype="f32", w_dtype="f64")
        assert np.array_equal(f64(M[0]), Mr)
        assert orc.relative_frobenius(f64(O[0]), Or) < 1e-4
        db = [dY[0].sum(0)]
        args = (f64(bias[0]), f64(bias_m[0]), f64(bias_v[0]), f64(db[0]), t, lr, 0.9, 0.99, 1e-8, 0.01)
        mu.adamw_step(bias, bias_m, bias_v, db, t, **hyper)
        for got, want, bound in zip((bias[0], bias_m[0], bias_v[0]), ao.adamw(*args), ao.adamw_tolerance(*args)):
            within(got, want, bound, "bias")
        m_old, v_old = (f64(x[0]) for x in e_state.values())
        args = (f64(E[0]), m_old, v_old, f64(dE), t, lr, 0.9, 0.99, 1e-8, 0.01)
        mu.adamw8_step(E, e_state, [dE], t, seed=4, **hyper)
        within(E[0], ao.adamw(*args)[0], 21.5 / 17 * ao.adamw_tolerance(*args, w_half=2.0 ** -8)[0], "embedding")
        # the updated weight, coded in both orientations for the next step, into the same buffers
        mu.mx4_quantize(W, transpose="both", out=(w_code, w_code_t))
        assert np.array_equal(f64(mu.mx4_dequantize(w_code)[0]), coded(f64(W[0])))
        assert np.array_equal(f64(mu.mx4_dequantize(w_code_t)[0]), coded(f64(W[0]).T))


def exact_gradient(X, W, D):
    """The formulas of the layer's gradients on uncoded operands: dX = D W, dW = D^T X."""
    return D @ W, D.T @ X


def test_layer_gradients_against_differences():
    """dX = dY W and dW = dY^T X of 1/2 |X W^T - T|^2 against central differences (fp64, CPU): the three products that
    the library's operand orders stand for."""
    rng = np.random.default_rng(0)
    X, W, T = rng.standard_normal((3, 5)), rng.standard_normal((4, 5)), rng.standard_normal((3, 4))
    loss = lambda X, W: 0.5 * np.sum((X @ W.T - T) ** 2)  # noqa: E731
    dX, dW = exact_gradient(X, W, X @ W.T - T)
    for P, dP, f in ((X, dX, lambda P: loss(P, W)), (W, dW, lambda P: loss(X, P))):
        for i in np.ndindex(P.shape):
            e = np.zeros_like(P)
            e[i] = 1e-5
            assert abs((f(P + e) - f(P - e)) / 2e-5 - dP[i]) < 1e-7 * (1 + abs(dP[i]))


def loss64(X, W, T):
    return 0.5 * np.sum((X @ W.T - T) ** 2)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,n_in,n_out", [(3, 5, 4), (20, 33, 18), (1, 130, 7)])
def test_products_give_the_gradients_that_differences_give(tokens, n_in, n_out):
    """The layer's products through the library, on operands the code holds exactly, against central differences of
    1/2 |X W^T - T|^2 in fp64: dX = dY W and dW = dY^T X, the latter also added to a gradient that is there.

    X, W and dY hold small multiples of 1/2 with a 6 in every block, so coding changes nothing and all sums are exact in
    fp32.  The loss is quadratic, so the differences' only error is rounding: at most a few 2^-53 of the loss over 2 e."""
    rng = np.random.default_rng(47)
    values = np.array([-3.0, -2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 2.0, 3.0])

    def exact(rows, cols):
        a = rng.choice(values, (rows, cols))
        a[::32, :] = 6.0  # every block along rows or columns has its largest magnitude at 6: scale 1
        a[:, ::32] = 6.0
        return a

    X, W, D = exact(tokens, n_in), exact(n_out, n_in), exact(tokens, n_out)
    T = X @ W.T - D
    dev = lambda a: [torch.from_numpy(a.astype(np.float32)).to(DEV)]  # noqa: E731
    x, x_t = mu.mx4_quantize(dev(X), transpose="both")
    w, w_t = mu.mx4_quantize(dev(W), transpose="both")
    Y = mu.mx4_matmul(x, w, torch.float32)
    dY = [(Y[0] - dev(T)[0]).contiguous()]
    assert np.array_equal(f64(dY[0]), D)
    d, d_t = mu.mx4_quantize(dY, transpose="both")
    dX = f64(mu.mx4_matmul(d, w_t, torch.float32)[0])
    G = dev(np.full((n_out, n_in), 0.25))
    mu.mx4_matmul(d_t, x_t, out=G, accumulate=True)
    dW = f64(G[0]) - 0.25
    e = 0.5  # a power of two; the difference quotient of a quadratic is its derivative for every e
    bound = 64 * 2.0 ** -53 * (loss64(X, W, T) + np.abs(D).sum() * 100 + 1e4) / (2 * e)
    for P, dP, f in ((X, dX, lambda P: loss64(P, W, T)), (W, dW, lambda P: loss64(X, P, T))):
        for i in np.ndindex(P.shape):
            up, down = P.copy(), P.copy()
            up[i] += e
            down[i] -= e
            assert abs((f(up) - f(down)) / (2 * e) - dP[i]) <= bound, i
