"""The experts' balance loss, counts and gradient on the device against the fp64 oracle."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import balance_oracle as bo
from synth import inputs as syn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half a step of the smallest numbers
f64 = syn.to_f64


def case(S, T, E, K, dtype="f32", seed=0, spread=1.0):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy((rng.standard_normal((S, T, E)) * spread + rng.standard_normal(E)).astype(np.float32)).to(DT[dtype])
    index = torch.from_numpy(np.argsort(-rng.random((S, T, E)) ** np.exp(rng.standard_normal(E)), -1)[..., :K].copy())
    return z, index


def check(got, z, index, alpha, score, dtype, mask=None, G0=None, scale=1.0):
    loss, counts, grad = got
    z64, i64 = f64(z), index.numpy()
    m = None if mask is None else mask.cpu().numpy()
    wl, wc, wg = bo.balance(z64, i64, alpha, score, m)
    bl, bg = bo.tolerance(z64, i64, alpha, score, m)
    assert loss.dtype == torch.float32 and loss.dim() == 0 and counts.dtype == torch.int32
    assert np.array_equal(counts.cpu().numpy(), wc), "counts"
    assert abs(float(loss) - wl) <= bl + 2.0 ** -24 * abs(wl), (float(loss), wl, bl)
    if grad is not None:
        want, bound = wg * scale, bg * abs(scale) + 2 * 2.0 ** -24 * np.abs(wg * scale)
        if G0 is not None:
            want = want + f64(G0)
            bound = bound + 2.0 ** -24 * np.abs(want)
        bound = bound + HALF_STEP[dtype] * (np.abs(want) + bound) + LEAST[dtype]
        g = f64(grad).reshape(want.shape)
        assert np.all(np.abs(g - want) <= bound), f"{np.sum(~(np.abs(g - want) <= bound))} of {g.size} gradients"


SIZES = [(1, 1, 1, 1), (1, 1, 8, 2), (1, 7, 8, 2), (1, 300, 5, 3), (1, 33, 64, 6), (2, 100, 61, 6), (3, 257, 16, 1),
         (1, 4099, 256, 8), (5, 640, 130, 4), (1, 50, 1000, 10), (1, 2000, 512, 8), (1, 700, 1024, 2), (300, 3, 9, 2),
         (1, 20000, 3, 2), (7, 1, 32, 4), (1, 70000, 8, 4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("S,T,E,K", SIZES)
def test_balance(S, T, E, K, dtype):
    for score in ("softmax", "sigmoid"):
        print(S, T, E, K, dtype, score, flush=True)
        z, index = case(S, T, E, K, dtype, S + T + E)
        wide = score == "softmax"
        got = mu.expert_balance(z.to(DEV), (index if wide else index.int()).to(DEV), 0.02, score, grad=True)
        check(got, z, index, 0.02, score, dtype)
        again = mu.expert_balance(z.to(DEV), index.to(DEV), 0.02, score)
        assert again[2] is None and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
        if S == 1:  # without the dimension of sequences
            flat = mu.expert_balance(z[0].to(DEV), index[0].to(DEV), 0.02, score, grad=True)
            assert flat[2].shape == (T, E) and torch.equal(flat[2], got[2][0]) and torch.equal(flat[0], got[0])


@pytest.mark.parametrize("S,T,E,K", [(1, 6, 8, 2), (4, 200, 61, 3), (1, 5000, 64, 6), (40, 100, 20, 2)])
def test_masks_and_rows_that_do_not_count(S, T, E, K):
    """Padded sequences, one without any token, whose logits hold NaN and infinities and whose indices are anything;
    experts that a row may not choose, rows without any expert, choices that are not counted."""
    for score in ("softmax", "sigmoid"):
        z, index = case(S, T, E, K, "f32", 3)
        rng = np.random.default_rng(4)
        mask = torch.from_numpy(np.arange(T)[None] < rng.integers(1, T + 1, (S, 1)))
        mask[-1] = S == 1
        mask[0, 0] = True
        z[torch.from_numpy(rng.random((S, T, E)) < 0.1)] = float("-inf")
        z[0, 0] = float("-inf")
        index[torch.from_numpy(rng.random((S, T, K)) < 0.1)] = -1
        clean_z, clean_i = z.clone(), index.clone()
        z[~mask] = float("nan")
        index[~mask] = 2 ** 40
        G0 = torch.randn(S, T, E)
        for m in (mask, mask.to(torch.uint8) * 7):
            got = mu.expert_balance(z.to(DEV), index.to(DEV), 0.5, score, m.to(DEV), grad=True)
            check(got, clean_z, clean_i, 0.5, score, "f32", mask)
            assert not got[2][~mask.to(DEV)].any() and not got[2][0, 0].any()
        G = G0.to(DEV)
        s = torch.tensor([-3.0], device=DEV)
        got = mu.expert_balance(z.to(DEV), index.to(DEV), 0.5, score, mask.to(DEV), grad=G, accumulate=True, grad_scale=s)
        assert got[2] is G
        check(got, clean_z, clean_i, 0.5, score, "f32", mask, G0, -3.0)
        assert torch.equal(G[~mask.to(DEV)].cpu(), G0[~mask])


@pytest.mark.parametrize("S,T,E", [(1, 5, 8), (1, 1, 1), (3, 300, 61), (1, 3000, 520), (2, 4100, 3)])
def test_all_experts_alike(S, T, E):
    """As many tokens for every expert: f is the same for all, so the gradient is 0, whatever the logits, and the loss 1."""
    z, _ = case(S, T, E, 1, "f32", 12, 5.0)
    index = torch.arange(E).expand(S, T, E).contiguous()
    for score in ("softmax", "sigmoid"):
        loss, counts, grad = mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, score, grad=True)
        assert abs(float(loss) - 1.0) <= (T + 8) * 2.0 ** -24 and (counts == S * T).all() and not grad.any()


def test_nothing_counts():
    z, index = case(3, 50, 16, 2)
    for T in (2, 50):
        got = mu.expert_balance(z[:, :T].contiguous().to(DEV), index[:, :T].contiguous().to(DEV), 1.0,
                                mask=torch.zeros(3, T, dtype=torch.bool, device=DEV), grad=True)
        assert float(got[0]) == 0.0 and not got[1].any() and not got[2].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """Central differences of the oracle's loss (f does not change: the choices are given)."""
    z, index = case(2, 6, 7, 2, "f32", 9)
    g = f64(mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, score, grad=True)[2])
    z64, h = f64(z), 1e-4
    for at in np.ndindex(z64.shape):
        up, down = z64.copy(), z64.copy()
        up[at] += h
        down[at] -= h
        d = (bo.balance(up, index.numpy(), 1.0, score)[0] - bo.balance(down, index.numpy(), 1.0, score)[0]) / (2 * h)
        # third derivatives of p are under 1, f under E: h^2 E / 6; the loss is good to 2^-50 of E; the gradient to 1e-6
        assert abs(g[at] - d) <= h * h * 7 / 6 + 7 * 2.0 ** -50 / h + 1e-6


def test_extreme_logits():
    """Logits far apart: softmax of 1e4 and -1e4, sigmoids that are all tiny or all 1."""
    for scale in (50.0, 1e4):
        z, index = case(1, 200, 32, 4, "f32", 5, scale)
        check(mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, grad=True), z, index, 1.0, "softmax", "f32")
    z, index = case(1, 100, 32, 4, "f32", 5)
    z[..., :16] = -3.4e38  # the lowest numbers in place of -infinity
    z[0, 7] = 3.4e38
    check(mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, grad=True), z, index, 1.0, "softmax", "f32")
    for shift in (-60.0, 60.0):
        z, index = case(1, 200, 32, 4, "f32", 6)
        z = z + shift
        check(mu.expert_balance(z.to(DEV), index.to(DEV), 1.0, "sigmoid", grad=True), z, index, 1.0, "sigmoid", "f32")


def test_nan_and_infinite_logits_propagate():
    for T in (3, 3000):
        z, index = case(1, T, 20, 2, "f32", 7)
        for score in ("softmax", "sigmoid"):
            for bad in (float("nan"), float("inf")):
                y = z.clone()
                y[0, 2, 5] = bad
                loss, counts, grad = mu.expert_balance(y.to(DEV), index.to(DEV), 1.0, score, grad=True)
                if score == "sigmoid" and bad == float("inf"):  # a sigmoid of 1
                    check((loss, counts, grad), y, index, 1.0, score, "f32")
                else:
                    assert torch.isnan(loss) and torch.isnan(grad[0, 2]).all() and not torch.isnan(grad[0, :2]).any()


def test_strided_logits_and_odd_places():
    """Rows further apart than they are long, and rows that start at any element."""
    for dtype in DT:
        z, index = case(1, 777, 30, 3, dtype, 8)
        wide = torch.full((777, 41), float("nan"), dtype=DT[dtype], device=DEV)
        for off in (0, 1, 5):
            wide[:, off:off + 30] = z[0].to(DEV)
            check(mu.expert_balance(wide[:, off:off + 30], index[0].to(DEV), 0.1, grad=True), z, index, 0.1, "softmax", dtype)
        same = z[0, :1].to(DEV).expand(777, 30)  # one row for all tokens
        check(mu.expert_balance(same, index[0].to(DEV), 0.1, grad=True), z[:, :1].expand(1, 777, 30), index, 0.1, "softmax", dtype)


def test_writes_nothing_else():
    z, index = case(1, 901, 13, 3, "bf16", 10)
    buf = torch.full((901 * 13 + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
    for off in (32, 31):
        g = buf[off:off + 901 * 13].view(901, 13)
        got = mu.expert_balance(z[0].to(DEV), index[0].to(DEV), 0.1, grad=g)
        check(got, z, index, 0.1, "softmax", "bf16")
        assert (buf[:off] == 3).all() and (buf[off + 901 * 13:] == 3).all()
        buf.fill_(3.0)


def test_given_workspace_and_reproducibility():
    z, index = case(2, 3000, 64, 6, "bf16", 11)
    z, index = z.to(DEV), index.to(DEV)
    need = mu.expert_balance_workspace_size(2, 3000, 64, 6)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # contents on entry are ignored
    want = mu.expert_balance(z, index, 0.1, grad=True)
    for _ in range(5):
        got = mu.expert_balance(z, index, 0.1, grad=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(mu.MuonError):
        mu.expert_balance(z, index, 0.1, workspace=ws[:need - 1])


def test_captured_calls_replay_like_eager():
    """Small and large calls in one graph, new logits and choices between the replays; two graphs at once."""
    graphs = []
    for seed in range(2):
        small, large = case(1, 9, 8, 2, "f32", seed), case(2, 4000, 64, 6, "bf16", seed)
        static = [t.to(DEV) for t in (*small, *large)]
        grads = [torch.zeros_like(static[0]), torch.zeros_like(static[2])]

        def step(static=static, grads=grads):
            a = mu.expert_balance(static[0], static[1], 0.1, grad=grads[0])
            b = mu.expert_balance(static[2], static[3], 0.1, "sigmoid", grad=grads[1])
            return a[:2] + b[:2]

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, static, grads, out, torch.cuda.Stream()))
    for i in range(4):
        for _, static, *_ in graphs:
            static[0].copy_(torch.randn(1, 9, 8, generator=torch.Generator().manual_seed(i)))
            static[2].copy_(torch.randn(2, 4000, 64, generator=torch.Generator().manual_seed(i + 50)))
            static[3].copy_(torch.randint(0, 64, (2, 4000, 6), generator=torch.Generator().manual_seed(i)))
        torch.cuda.synchronize()
        for g, *_, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, static, grads, out, _ in graphs:
            a = mu.expert_balance(static[0], static[1], 0.1, grad=True)
            b = mu.expert_balance(static[2], static[3], 0.1, "sigmoid", grad=True)
            for x, y in zip((*out, *grads), (*a[:2], *b[:2], a[2], b[2])):
                assert torch.equal(x, y), i


def test_refusals_on_the_device():
    z, index = (t.to(DEV) for t in case(1, 10, 8, 2))
    z, index, wide = z[0], index[0], torch.zeros(10, 20, device=DEV)
    for match, call in [
            ("score", lambda: mu.expert_balance(z, index, 1.0, "argmax")),
            ("logits must be", lambda: mu.expert_balance(z[0], index, 1.0)),
            ("logits must not", lambda: mu.expert_balance(z[:0], index[:0], 1.0)),
            ("behind one another", lambda: mu.expert_balance(z.t().contiguous().t(), index, 1.0)),
            ("index must", lambda: mu.expert_balance(z, index.float(), 1.0)),
            ("one row for each", lambda: mu.expert_balance(z, index[:5], 1.0)),
            ("index must", lambda: mu.expert_balance(z, index[:, :0], 1.0)),
            ("mask must", lambda: mu.expert_balance(z, index, 1.0, mask=torch.ones(10, device=DEV))),
            ("mask must", lambda: mu.expert_balance(z, index, 1.0, mask=torch.ones(9, dtype=torch.bool, device=DEV))),
            ("grad must", lambda: mu.expert_balance(z, index, 1.0, grad=torch.zeros(10, 8, device=DEV, dtype=torch.half))),
            ("accumulate", lambda: mu.expert_balance(z, index, 1.0, accumulate=True)),
            ("accumulate", lambda: mu.expert_balance(z, index, 1.0, grad=True, accumulate=True)),
            ("grad_scale", lambda: mu.expert_balance(z, index, 1.0, grad_scale=torch.ones(2, device=DEV))),
            ("overlaps", lambda: mu.expert_balance(z, index, 1.0, grad=z)),
            ("overlaps", lambda: mu.expert_balance(wide[:, :8], index, 1.0, grad=wide.flatten()[90:170].view(10, 8))),
            ("dtype", lambda: mu.expert_balance(z.double(), index, 1.0))]:
        with pytest.raises(ValueError, match=match):
            call()
    for coefficient in (float("nan"), float("inf"), 1e39):
        with pytest.raises(mu.MuonError):
            mu.expert_balance(z, index, coefficient)
    with pytest.raises(mu.MuonError):
        mu.expert_balance(torch.zeros(4, 1025, device=DEV), index[:4].contiguous(), 1.0)


def test_given_outputs_raise_their_version_and_launches_are_traced():
    z, index = (t.to(DEV) for t in case(1, 3000, 64, 2))
    g, ws = torch.zeros_like(z), torch.zeros(mu.expert_balance_workspace_size(1, 3000, 64, 2), dtype=torch.uint8, device=DEV)
    before = (z._version, g._version, ws._version)
    mu.trace_enable(True)
    mu.expert_balance(z, index, 1.0, grad=g, workspace=ws)
    recs = mu.trace_collect()
    mu.trace_enable(False)
    assert [r["role"] for r in recs] == ["expert_counts", "expert_balance"]
    assert (z._version, g._version > before[1], ws._version > before[2]) == (before[0], True, True)
