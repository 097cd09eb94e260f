"""AdamW steps (32-bit and 8-bit moments) on the device against the fp64 oracle."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import adamw_oracle as ao
from synth import inputs as syn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step relative to the value
f64 = syn.to_f64


def make(sizes, w, g, seed, offset=0, first=False, zero_every=0):
    """Lists W, M, V, G on the device; ``offset`` elements in front make the views misaligned."""
    rng = np.random.default_rng(seed)

    def put(a, dt):
        buf = torch.zeros(a.size + offset + 3, dtype=dt, device=DEV)
        buf[offset:offset + a.size] = torch.from_numpy(a).to(DEV).to(dt)
        return buf[offset:offset + a.size]

    W, M, V, G = [], [], [], []
    for j, n in enumerate(sizes):
        gr = rng.standard_normal(n).astype(np.float32) * 1e-2
        if zero_every:
            gr[(np.arange(n) // zero_every) % 2 == 0] = 0.0
        W.append(put(rng.standard_normal(n).astype(np.float32) * 0.1, DT[w]))
        M.append(put((0 if first else 1) * rng.standard_normal(n).astype(np.float32) * 3e-3, torch.float32))
        V.append(put((0 if first else 1) * np.square(rng.standard_normal(n).astype(np.float32) * 1e-2), torch.float32))
        G.append(put(gr, DT[g]))
    return W, M, V, G


def compare32(W, M, V, G, W0, M0, V0, t, w, **kw):
    for k in range(len(W)):
        args = (f64(W0[k]), f64(M0[k]), f64(V0[k]), f64(G[k]), t, kw["lr"], kw["beta1"], kw["beta2"], kw["eps"],
                kw["weight_decay"], kw.get("scale", 1.0))
        want = ao.adamw(*args)
        tol = ao.adamw_tolerance(*args, w_half=HALF[w])
        for name, got, ref, bound in zip("WMV", (W[k], M[k], V[k]), want, tol):
            bad = np.abs(f64(got) - ref) > bound
            assert not bad.any(), f"tensor {k} {name}: {bad.sum()} of {bad.size} out of bounds"


HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.05)


@pytest.mark.parametrize("w", ["f32", "bf16"])
@pytest.mark.parametrize("g", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes,offset", [((1,), 0), ((3, 0, 4096, 5), 0), ((4097, 2, 12345), 0), ((4099, 257), 1),
                                          ((8192 + 3, 1, 1, 64), 4)])
def test_adamw_against_oracle(w, g, sizes, offset):
    print(w, g, sizes, offset, flush=True)
    W, M, V, G = make(sizes, w, g, 11, offset)
    W0, M0, V0 = ([x.clone() for x in L] for L in (W, M, V))
    G0 = [x.clone() for x in G]
    mu.adamw_step(W, M, V, G, 7, **HYPER)
    torch.cuda.synchronize()
    compare32(W, M, V, G, W0, M0, V0, 7, w, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(G, G0))
    for L in (W, M, V):  # nothing in front of or behind a tensor is touched
        for x in L:
            whole = torch.as_strided(x, (x.numel() + offset + 3,), (1,), 0)
            assert not whole[:offset].any() and not whole[offset + x.numel():].any()


@pytest.mark.parametrize("count", [255, 256, 257, 700])
def test_adamw_many_tensors(count):
    """Lists over the number of tensors of one launch, sizes 0 among them."""
    sizes = [(37 * i) % 311 for i in range(count)]
    W, M, V, G = make(sizes, "f32", "f32", 12)
    W0, M0, V0 = ([x.clone() for x in L] for L in (W, M, V))
    mu.adamw_step(W, M, V, G, 2, **HYPER)
    compare32(W, M, V, G, W0, M0, V0, 2, "f32", **HYPER)


def test_adamw_first_steps_and_shapes():
    """From zero moments, three steps on tensors of several dimensions."""
    W = [torch.randn(s, device=DEV, generator=torch.Generator(DEV).manual_seed(i)) for i, s in enumerate([(3, 5, 7), (64,), (33, 65)])]
    M, V = [torch.zeros_like(x) for x in W], [torch.zeros_like(x) for x in W]
    for t in (1, 2, 3):
        G = [torch.randn(x.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(100 * t + i)) for i, x in enumerate(W)]
        W0, M0, V0 = ([x.clone() for x in L] for L in (W, M, V))
        mu.adamw_step(W, M, V, G, t, **HYPER)
        compare32(W, M, V, G, W0, M0, V0, t, "f32", **HYPER)


@pytest.mark.parametrize("beta1,beta2,t", [(0.0, 0.0, 1), (0.0, 0.99, 3), (0.9, 0.999, 10 ** 6), (0.95, 0.9999, 1)])
def test_adamw_betas_and_steps(beta1, beta2, t):
    hyper = dict(HYPER, beta1=beta1, beta2=beta2)
    W, M, V, G = make((5000,), "f32", "f32", 13)
    W0, M0, V0 = ([x.clone() for x in L] for L in (W, M, V))
    mu.adamw_step(W, M, V, G, t, **hyper)
    compare32(W, M, V, G, W0, M0, V0, t, "f32", **hyper)


def test_adamw_step_and_scale_on_the_device():
    """step and grad_scale read from device memory give what the host's values give, up to the constants' rounding."""
    scale = torch.tensor([0.25], device=DEV)
    for t in (1, 5, 12345):
        W, M, V, G = make((4100, 9), "f32", "bf16", 14)
        W0, M0, V0 = ([x.clone() for x in L] for L in (W, M, V))
        mu.adamw_step(W, M, V, G, torch.tensor([t], device=DEV), grad_scale=scale, **HYPER)
        compare32(W, M, V, G, W0, M0, V0, t, "f32", scale=0.25, **HYPER)
    W, M, V, G = make((300,), "f32", "f32", 14)
    W1, M1, V1, _ = make((300,), "f32", "f32", 14)
    mu.adamw_step(W, M, V, G, torch.tensor([-4], device=DEV), **HYPER)  # under 1 counts as 1
    mu.adamw_step(W1, M1, V1, G, torch.tensor([1], device=DEV), **HYPER)
    assert torch.equal(W[0], W1[0])


def test_adamw_non_finite_gradients_stay_in_their_elements():
    W, M, V, G = make((5000,), "f32", "f32", 15)
    W0, M0, V0 = ([x.clone() for x in L] for L in (W, M, V))
    G[0][17], G[0][4999], G[0][2] = float("nan"), float("inf"), float("-inf")
    mu.adamw_step(W, M, V, G, 4, **HYPER)
    bad = torch.zeros(5000, dtype=torch.bool, device=DEV)
    bad[[17, 4999, 2]] = True
    assert torch.isnan(W[0][bad]).all() and not torch.isfinite(M[0][bad]).any() and not torch.isfinite(V[0][bad]).any()
    keep = [x[~bad] for x in (W[0], M[0], V[0], G[0], W0[0], M0[0], V0[0])]
    compare32(*[[x] for x in keep], 4, "f32", **HYPER)


def test_adamw_zero_gradient_and_state():
    W, M, V, G = make((300,), "f32", "f32", 16, first=True)
    G[0].zero_()
    W0 = W[0].clone()
    mu.adamw_step(W, M, V, G, 1, lr=0.1)
    assert torch.equal(W[0], W0) and not M[0].any() and not V[0].any()


def test_adamw_refuses_a_tensor_twice():
    a, b = torch.zeros(8, device=DEV), torch.zeros(8, device=DEV)
    z = lambda: torch.zeros(8, device=DEV)  # noqa: E731
    with pytest.raises(ValueError, match="overlaps"):
        mu.adamw_step([a, a], [z(), z()], [z(), z()], [z(), z()], 1, 1e-3)
    with pytest.raises(ValueError, match="overlaps"):
        mu.adamw_step([a], [b], [b], [z()], 1, 1e-3)
    with pytest.raises(ValueError, match="overlaps"):
        mu.adamw_step([a], [z()], [z()], [a], 1, 1e-3)
    with pytest.raises(ValueError, match="step"):
        mu.adamw_step([a], [z()], [z()], [z()], torch.ones(2, dtype=torch.int64, device=DEV), 1e-3)
    with pytest.raises(ValueError, match="grad_scale"):
        mu.adamw_step([a], [z()], [z()], [z()], 1, 1e-3, grad_scale=torch.ones(1))
    with pytest.raises(mu.MuonError):
        mu.adamw_step([a], [z()], [z()], [z()], 0, 1e-3)
    assert not a.any()


def test_adamw_checks_every_list():
    z = lambda n=8, dt=torch.float32: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
    call = lambda W=None, M=None, V=None, G=None: mu.adamw_step(  # noqa: E731
        W or [z(), z(5)], M or [z(), z(5)], V or [z(), z(5)], G or [z(), z(5)], 1, 1e-3)
    call()
    for kw, what in [(dict(G=[z()]), "one tensor per tensor"), (dict(M=[z()]), "one tensor per tensor"),
                     (dict(W=[z(), z(5, torch.bfloat16)]), "dtype"), (dict(G=[z(), z(5, torch.float16)]), "dtype"),
                     (dict(M=[z(8, torch.bfloat16), z(5, torch.bfloat16)]), "dtype"),
                     (dict(W=[z(8, torch.float16), z(5, torch.float16)]), "dtype"),
                     (dict(G=[z(8, torch.float64), z(5, torch.float64)]), "dtype"), (dict(V=[z(), z(6)]), "number"),
                     (dict(G=[z(), torch.zeros(5)]), "device of W"), (dict(G=[z(), z(10)[::2]]), "contiguous")]:
        with pytest.raises(ValueError, match=what):
            call(**kw)
    both = z(16)
    with pytest.raises(ValueError, match="overlaps"):  # views that share elements
        call(W=[both[:8], both[7:12]])
    G = [z(), z(5)]
    call(W=[both[:8], both[8:13]], G=G)                # neighbours, and gradients read only
    same = z()
    mu.adamw_step([z(), z()], [z(), z()], [z(), z()], [same, same], 1, 1e-3)
    s = mu.AdamW8State.zeros([z(), z(300)])
    s.m_scales[1] = z(2)
    with pytest.raises(ValueError, match="number"):
        mu.adamw8_step([z(), z(300)], s, [z(), z(300)], 1, 1e-3)


@pytest.mark.parametrize("order", ["ascending", "descending", "shuffled", "interleaved"])
def test_adamw_finds_an_overlap_in_any_order(order):
    """One element shared by two of 90 neighbouring views, in lists whose addresses run in any order."""
    n, size = 90, 33
    at = list(range(n))
    if order == "descending":
        at = at[::-1]
    elif order == "shuffled":
        np.random.default_rng(48).shuffle(at)
    elif order == "interleaved":
        at = at[::2] + at[1::2]
    flat = [torch.zeros(n * size, device=DEV) for _ in range(4)]
    lists = [[f[i * size:(i + 1) * size] for i in at] for f in flat]
    mu.adamw_step(*lists, 1, 1e-3)  # neighbours do not overlap
    for which in range(3):
        for j in (0, 41, n - 1):
            i = at[j]
            bad = list(lists[which])
            bad[j] = flat[which][i * size + 1:(i + 1) * size + 1] if i < n - 1 else flat[which][i * size - 1:(i + 1) * size - 1]
            with pytest.raises(ValueError, match="overlaps"):
                mu.adamw_step(*(bad if k == which else L for k, L in enumerate(lists)), 1, 1e-3)

@pytest.mark.parametrize("eight", [False, True])
def test_adamw_refuses_a_scale_or_step_inside_what_it_writes(eight):
    """The step number and the gradient scale are read by every block while others write."""
    z = lambda n=8, dt=torch.float32: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
    W, M, V, G, state = [z()], [z()], [z()], [z()], mu.AdamW8State.zeros([z()])

    def call(step=1, **kw):
        if eight:
            mu.adamw8_step(W, state, G, step, 1e-3, **kw)
        else:
            mu.adamw_step(W, M, V, G, step, 1e-3, **kw)

    other = state.m_scales[0] if eight else M[0]
    for t in (W[0], other):
        with pytest.raises(ValueError, match="overlaps"):
            call(grad_scale=t[:1])
        if t.numel() > 1:
            with pytest.raises(ValueError, match="overlaps"):
                call(step=t[2:4].view(torch.int64))
    call(grad_scale=G[0][:1])  # gradients are read only
    both = torch.ones(2, dtype=torch.int64, device=DEV)
    call(step=both[:1], grad_scale=both[1:].view(torch.float32)[:1])


@pytest.mark.parametrize("eight", [False, True])
def test_adamw_step_numbers_of_other_types(eight):
    z = lambda: torch.zeros(8, device=DEV)  # noqa: E731
    W, M, V, G, state = [z()], [z()], [z()], [z()], mu.AdamW8State.zeros([z()])
    call = lambda step: (mu.adamw8_step(W, state, G, step, 1e-3) if eight  # noqa: E731
                         else mu.adamw_step(W, M, V, G, step, 1e-3))
    for bad in (1.0, 2.5, None, "3", 1 << 63, -(1 << 63) - 1, [1]):
        with pytest.raises(ValueError, match="step"):
            call(bad)
    for bad in (torch.tensor([1]), torch.tensor([1.0], device=DEV), torch.ones(2, dtype=torch.int64, device=DEV)):
        with pytest.raises(ValueError, match="step"):
            call(bad)
    for good in (1, np.int64(2), np.int32(3), (1 << 63) - 1):
        call(good)
    for bad in (0, -1):
        with pytest.raises(mu.MuonError):
            call(bad)
    assert not W[0].any()


# --- 8-bit moments -------------------------------------------------------------------------------------------------
# m and v before they are coded are fp32 values with the relative errors of adamw_tolerance, on top of the decoded
# moments (one product each, h; v's square 2 h more): at most 10 h of the magnitudes of their terms, so x = sqrt(v) / s
# is off by at most 12 h and x^2 - lo^2 by 24 h x^2; hi^2 - lo^2 is at least x^2 / 4.6 in the normal range (lo = 15/8
# binade steps: (16^2 - 15^2) / 15^2 = 0.138 x^2), so the share is off by at most 24 h / 0.138 < 2^-16 < 1e-4.
SLACK = 1e-4


def state_of(M, V, offset=0):
    """8-bit state coding the given moments (by the oracle's scales, torch's nearest rounding)."""
    def view(x):
        buf = torch.zeros(x.numel() + offset + 3, dtype=x.dtype, device=DEV)
        buf[offset:offset + x.numel()] = x
        return buf[offset:offset + x.numel()]

    out = mu.AdamW8State([], [], [], [])
    for codes, scales, values in ((out.m_codes, out.m_scales, M), (out.r_codes, out.r_scales, [v.sqrt() for v in V])):
        for x in values:
            each, s = ao.group_scales(f64(x))
            y = np.divide(f64(x), each, out=np.zeros(x.numel()), where=each > 0)
            codes.append(view(torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).to(DEV)))
            scales.append(view(torch.from_numpy(s).float().to(DEV)))
    return out


def bytes_of(x):
    return x.view(torch.uint8).cpu().numpy()


def step8(W, state, G, t, seed, w, hyper, scale=1.0):
    """Runs adamw8_step and checks W, codes and scales of every tensor."""
    W0 = [f64(x) for x in W]
    old = [[f64(c.float()) * np.repeat(f64(s), 128)[:c.numel()] for c, s in zip(cs, ss)]
           for cs, ss in ((state.m_codes, state.m_scales), (state.r_codes, state.r_scales))]
    kw = {} if scale == 1.0 else dict(grad_scale=torch.tensor([scale], device=DEV))
    mu.adamw8_step(W, state, G, t, seed=seed, **kw, **hyper)
    torch.cuda.synchronize()
    for k in range(len(W)):
        n = W0[k].size
        if n == 0:
            continue
        args = (W0[k], old[0][k], old[1][k] ** 2, f64(G[k]), t, hyper["lr"], hyper["beta1"], hyper["beta2"],
                hyper["eps"], hyper["weight_decay"], scale)
        w_new, m, v = ao.adamw(*args)
        tol = ao.adamw_tolerance(*args, w_half=HALF[w])[0]
        # decoding adds h to m and 3 h to v, so 2.5 h to the step's 17 h; the reciprocal (2 h, and the product with it h)
        # in the place of the quotient's h adds 2 h: 21.5 h in all
        assert np.all(np.abs(f64(W[k]) - w_new) <= tol * 21.5 / 17), f"tensor {k}: W"
        bad = ao.check_moment_codes(bytes_of(state.m_codes[k]), f64(state.m_scales[k]), m, SLACK)
        assert bad == 0, f"tensor {k}: {bad} codes of m"
        bad = ao.check_root_codes(bytes_of(state.r_codes[k]), f64(state.r_scales[k]), v,
                                  ao.chances(n, seed, t, k), SLACK)
        assert bad == 0, f"tensor {k}: {bad} codes of the root of v"


@pytest.mark.parametrize("w,g", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f16"), ("f32", "f16"),
                                 ("bf16", "f32")])
@pytest.mark.parametrize("sizes,offset", [((1,), 0), ((5, 0, 2048, 127, 128, 129), 0), ((12345,), 0), ((3001, 2), 1)])
def test_adamw8_against_oracle(w, g, sizes, offset):
    print(w, g, sizes, offset, flush=True)
    W, M, V, G = make(sizes, w, g, 21, offset)
    state = state_of(M, V, offset)
    step8(W, state, G, 9, 3, w, HYPER)
    for L in (W, state.m_codes, state.r_codes, state.m_scales, state.r_scales):
        for x in L:
            whole = torch.as_strided(x, (x.numel() + offset + 3,), (1,), 0).view(torch.uint8)
            e = x.element_size()
            assert not whole[:offset * e].any() and not whole[(offset + x.numel()) * e:].any()


def test_adamw8_many_tensors():
    """A list over several launches: the roundings go by the place in the whole list."""
    sizes = [(53 * i) % 397 for i in range(150)]
    W, M, V, G = make(sizes, "f32", "f32", 25)
    step8(W, state_of(M, V), G, 6, 12, "f32", HYPER)


@pytest.mark.parametrize("eight", [False, True])
def test_adamw_past_2_31_elements(eight):
    """One tensor of 2^31 + 1003 elements: both ends are stepped, what has no gradient and no decay stays."""
    n = 2 ** 31 + 1003
    W = [torch.ones(n, dtype=torch.bfloat16, device=DEV)]
    G = [torch.zeros(n, dtype=torch.bfloat16, device=DEV)]
    ends = torch.cat((torch.arange(3000), torch.arange(n - 3000, n))).to(DEV)
    G[0][ends] = torch.randn(6000, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16)
    hyper = dict(lr=0.03, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    if eight:
        state = mu.AdamW8State.zeros(W)
        mu.adamw8_step(W, state, G, 1, **hyper)
    else:
        M, V = [torch.zeros(n, device=DEV)], [torch.zeros(n, device=DEV)]
        mu.adamw_step(W, M, V, G, 1, **hyper)
    g = f64(G[0][ends])
    one, zero = np.ones(6000), np.zeros(6000)
    args = (one, zero, zero, g, 1, 0.03, 0.9, 0.999, 1e-8, 0.0)
    w, m, v = ao.adamw(*args)
    tol = ao.adamw_tolerance(*args, w_half=2.0 ** -8)
    assert np.all(np.abs(f64(W[0][ends]) - w) <= tol[0] * 21.5 / 17)
    if not eight:
        assert np.all(np.abs(f64(M[0][ends]) - m) <= tol[1]) and np.all(np.abs(f64(V[0][ends]) - v) <= tol[2])
    for part in (slice(3000, 2 ** 30), slice(2 ** 30, n - 3000)):
        assert bool((W[0][part] == 1).all())
        if eight:
            assert not state.m_codes[0][part].view(torch.uint8).any() and not state.r_codes[0][part].view(torch.uint8).any()
        else:
            assert not M[0][part].any() and not V[0][part].any()


def test_adamw8_tiny_gradients():
    """Gradients down to fp32's subnormal squares: no division by zero, no NaN, W within the bounds of eps."""
    n = 512
    W = [torch.ones(n, device=DEV)]
    G = [torch.logspace(-44, 0, n, device=DEV, dtype=torch.float64).float()]
    state = mu.AdamW8State.zeros(W)
    for t in (1, 2, 3):
        mu.adamw8_step(W, state, G, t, 0.01)
    m, v = state.values()
    assert torch.isfinite(W[0]).all() and torch.isfinite(m[0]).all() and torch.isfinite(v[0]).all()
    # For a constant gradient m_hat / sqrt(v_hat) is at most 1 before rounding.  Coding m changes it by a factor of at most
    # 2 (the smallest magnitude that is not stored as 0 is half the smallest code), coding the root divides it by at most
    # 2 (it goes to its lower neighbour, and never to 0), so a step's quotient grows by at most 4: 1, 4 and 16 times lr.
    assert ((1 - W[0]).abs() <= 0.01 * (1 + 4 + 16)).all()
    # Over 2^-6 of its group's code range (1e-3 of the last group's largest gradient is 0.448 of 448) m loses at most
    # 1/16 and the root gains at most 1/8 a step: at least 1, 0.83 and 0.69 times lr.
    big = G[0] > 1e-3
    assert ((1 - W[0])[big] > 0.01 * (1 + 0.83 + 0.69)).all()


def test_adamw8_codes_of_tiny_second_moments():
    """Groups whose second moments are subnormal, as a whole or beside large ones, and around the largest root of 2^-33
    from which on the kernel takes its short root: codes of exactly the fp32 moments."""
    rng = np.random.default_rng(31)
    spread = [(-20.5, -17.6), (-19.0, -18.9), (-20.0, -12.0), (-20.0, -3.0), (-9.0, -8.3), (-10.0, -8.43), (-18.0, -8.42),
              (-3.0, 0.0)]
    mag = np.concatenate([10.0 ** rng.uniform(lo, hi, 128) for lo, hi in spread])
    mag[::11] = 0.0
    g = (mag * rng.choice([-1.0, 1.0], mag.size)).astype(np.float32)
    W, G = [torch.ones(g.size, device=DEV)], [torch.from_numpy(g).to(DEV)]
    state = mu.AdamW8State.zeros(W)
    mu.adamw8_step(W, state, G, 1, 0.01, seed=77)
    m = np.float32(1 - 0.9) * g
    v = (np.float32(1 - 0.999) * g) * g
    assert v.dtype == np.float32 and (v[:256] < 2.0 ** -126).all() and v[:256].any()
    assert ao.check_moment_codes(bytes_of(state.m_codes[0]), f64(state.m_scales[0]), m.astype(np.float64), SLACK) == 0
    bad = ao.check_root_codes(bytes_of(state.r_codes[0]), f64(state.r_scales[0]), v.astype(np.float64),
                              ao.chances(g.size, 77, 1, 0), SLACK)
    assert bad == 0, f"{bad} codes of the root of v"


def moments32(s, g, t):
    """The fp32 moments of a step as the library rounds them (one rounding for each product and sum), subnormals
    kept."""
    b1, b2, o1, o2 = (np.float32(x) for x in (s["beta1"], s["beta2"], 1 - s["beta1"], 1 - s["beta2"]))
    m, v = b1 * s["m"] + o1 * g, b2 * s["v"] + (o2 * g) * g
    assert m.dtype == np.float32 and v.dtype == np.float32
    return m, v


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-20, 1e-15, 1e-10, 1e-8])
def test_adamw_weights_of_tiny_second_moments(eight, beta2, eps):
    """Second moments that are subnormal, alone in their group or beside large ones, with every kind of eps: W is the
    step on exactly the fp32 moments.

    Half a step is h = 2^-24.  Of the step's quotient: c1 and its product 2 h; of the denominator the root 1.5 h (nearest
    from 2^-102 on and wherever eps lets it be seen; otherwise another 2^-25 of the denominator), c2 and its product 2 h,
    eps and the sum 2 h; the quotient by v_rcp_f32 2 h and its product h (nearest: h); lr and its product 2 h: at most
    13 h.  Decay: wd, lr and their products with the sum 5 h.  The result's own rounding h."""
    rng = np.random.default_rng(33)
    spread = [(-23.0, -17.0), (-22.5, -19.0), (-21.0, -3.0), (-24.0, 0.0), (-18.5, -15.0), (-3.0, 0.0)]
    mag = np.concatenate([10.0 ** rng.uniform(lo, hi, 256) for lo, hi in spread])
    mag[::13] = 0.0
    mag[5::128][::2] = 1.0  # every second group has a large neighbour
    lr, wd = 0.01, 0.1
    hyper = dict(lr=lr, beta1=0.9, beta2=beta2, eps=eps, weight_decay=wd)
    w0 = np.where(np.arange(mag.size) % 2 == 0, 0.0, rng.standard_normal(mag.size)).astype(np.float32)
    W = [torch.from_numpy(w0).to(DEV)]
    zero = np.zeros(mag.size, dtype=np.float32)
    M, V, state = [torch.zeros_like(W[0])], [torch.zeros_like(W[0])], mu.AdamW8State.zeros(W)
    s = dict(beta1=0.9, beta2=beta2, m=zero, v=zero)
    h = 2.0 ** -24
    for t in (1, 2, 3):
        g = (mag * rng.choice([-1.0, 1.0], mag.size) * rng.uniform(0.5, 2.0, mag.size)).astype(np.float32)
        G, w_old = [torch.from_numpy(g).to(DEV)], f64(W[0])
        m, v = moments32(s, g, t)
        if eight:
            mu.adamw8_step(W, state, G, t, seed=5, **hyper)
        else:
            mu.adamw_step(W, M, V, G, t, **hyper)
            assert np.array_equal(M[0].cpu().numpy(), m) and np.array_equal(V[0].cpu().numpy(), v)
        assert t > 1 or ((v > 0) & (v < 2.0 ** -126)).sum() > 100
        step = lr * (m / (1 - 0.9 ** t)) / (np.sqrt(v.astype(np.float64)) / np.sqrt(1 - beta2 ** t) + eps)
        want = w_old - step - lr * wd * w_old
        bound = 13 * h * np.abs(step) + 5 * h * lr * wd * np.abs(w_old) + 2 * h * np.abs(want) + 2.0 ** -149
        off = np.abs(f64(W[0]) - want)
        assert np.all(off <= bound), f"t = {t}: {np.sum(off > bound)} weights, worst {np.max(off / bound):.3g} bounds"
        if eight:
            assert ao.check_moment_codes(bytes_of(state.m_codes[0]), f64(state.m_scales[0]), m.astype(np.float64), SLACK) == 0
            assert ao.check_root_codes(bytes_of(state.r_codes[0]), f64(state.r_scales[0]), v.astype(np.float64),
                                       ao.chances(g.size, 5, t, 0), SLACK) == 0
            codes = [c[0].float().cpu().numpy() * np.repeat(x[0].cpu().numpy(), 128)
                     for c, x in ((state.m_codes, state.m_scales), (state.r_codes, state.r_scales))]
            s.update(m=codes[0], v=codes[1] * codes[1])
        else:
            s.update(m=m, v=v)


@pytest.mark.parametrize("w", ["f32", "bf16"])
@pytest.mark.parametrize("g", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("eight", [False, True])
def test_adamw_large_calls_compute_the_same(w, g, eight):
    """A tensor beside a large one: bit for bit what it is in a call of its own."""
    W, M, V, G = make((70001, 4096), w, g, 32)
    n = 100_000_000

    def run(extra):
        P, Q = [x.clone() for x in W], list(G)
        if extra:
            P.append(torch.zeros(n, dtype=DT[w], device=DEV))
            Q.append(torch.zeros(n, dtype=DT[g], device=DEV))
        if eight:
            s = state_of(M, V)
            big = mu.AdamW8State.zeros(P[2:])
            for a in ("m_codes", "m_scales", "r_codes", "r_scales"):
                setattr(s, a, list(getattr(s, a)) + list(getattr(big, a)))
            mu.adamw8_step(P, s, Q, 5, seed=4, **HYPER)
            out = P[:2] + s.m_codes[:2] + s.m_scales[:2] + s.r_codes[:2] + s.r_scales[:2]
        else:
            A, B = [x.clone() for x in M], [x.clone() for x in V]
            if extra:
                A.append(torch.zeros(n, device=DEV))
                B.append(torch.zeros(n, device=DEV))
            mu.adamw_step(P, A, B, Q, 5, **HYPER)
            out = P[:2] + A[:2] + B[:2]
        assert not extra or not P[2].any()
        return [x.view(torch.uint8).cpu() for x in out]

    assert all(torch.equal(a, b) for a, b in zip(run(False), run(True)))


def test_adamw8_several_steps_from_zero():
    W, _, _, _ = make((4096 + 77, 300), "f32", "f32", 22)
    state = mu.AdamW8State.zeros(W)
    for t in range(1, 5):
        _, _, _, G = make((4096 + 77, 300), "f32", "bf16", 100 + t, zero_every=512)
        step8(W, state, G, t, 99, "f32", HYPER, scale=0.5 if t == 3 else 1.0)
    m, v = state.values()
    assert [x.shape for x in m] == [x.shape for x in W] and all((x >= 0).all() for x in v)


def test_adamw8_is_reproducible_and_depends_on_seed_and_step():
    def run(seed, t):
        W, M, V, G = make((6000,), "f32", "f32", 23)
        s = state_of(M, V)
        mu.adamw8_step(W, s, G, t, 1e-3, seed=seed)
        return bytes_of(s.r_codes[0]), W[0].cpu()

    a, wa = run(1, 5)
    b, wb = run(1, 5)
    assert np.array_equal(a, b) and torch.equal(wa, wb)
    c, wc = run(2, 5)
    assert not np.array_equal(a, c) and torch.equal(wa, wc)
    assert not np.array_equal(a, run(1, 6)[0])


def test_adamw8_non_finite_gradient_poisons_its_group_only():
    W, M, V, G = make((1000,), "f32", "f32", 24)
    s, clean = state_of(M, V), state_of(M, V)
    W2 = [W[0].clone()]
    mu.adamw8_step(W2, clean, G, 3, 1e-3)
    G[0][130] = float("nan")
    G[0][900] = float("inf")
    mu.adamw8_step(W, s, G, 3, 1e-3)
    bad = torch.zeros(1000, dtype=torch.bool)
    bad[128:256] = bad[896:1000] = True
    m, v = s.values()
    assert torch.equal(~torch.isfinite(m[0].cpu()), bad) and torch.equal(~torch.isfinite(v[0].cpu()), bad)
    assert not s.m_codes[0].float().cpu()[bad].any() and not s.r_codes[0].float().cpu()[bad].any()
    assert torch.equal(m[0].cpu()[~bad], clean.values()[0][0].cpu()[~bad])
    wrong = (W[0] != W2[0]).cpu()
    assert wrong.sum() <= 2 and wrong[130]  # W sees the gradient's own element only


def test_adamw8_follows_a_second_moment_that_changes_slowly():
    """Constant |g| = 2 after a state of 1: v has to approach 4 as 1 - 0.999^t does, which rounding to nearest would
    not do at all.  4096 elements, 400 steps: mean v = 4 - 3 * 0.999^400 = 1.990.  The mean over 4096 independent
    elements has a standard deviation of at most (v's spread, under one code step of v, 25 %) * 2 / 64 < 1 %."""
    n = 4096
    W = [torch.zeros(n, device=DEV)]
    one = torch.ones(n, device=DEV)
    one[::128] = 4.0  # a larger neighbour in every group keeps the scale away from the others
    state = state_of([one * 0], [one * one])
    G = [torch.where(one > 1, 4.0, 2.0)]
    for t in range(1, 401):
        mu.adamw8_step(W, state, G, t, 0.0, seed=8)
    v = state.values()[1][0][one == 1]
    want = 4 - 3 * 0.999 ** 400
    assert abs(v.double().mean().item() - want) < 0.05 * want


@pytest.mark.parametrize("count", [7, 8, 9, 86, 87, 88, 174, 175])
def test_adamw_lists_around_the_length_of_a_launch(count):
    """Short lists of at most 8 tensors, 87 tensors a launch, and one more or less; empty ones among them."""
    sizes = [(37 * i + 5) % 311 if i % 7 != 3 else 0 for i in range(count)]
    W, M, V, G = make(sizes, "f32", "bf16", 44)
    W0, M0, V0 = ([x.clone() for x in L] for L in (W, M, V))
    mu.trace_enable(True)
    mu.adamw_step(W, M, V, G, 2, **HYPER)
    launches = len(mu.trace_collect())
    mu.trace_enable(False)
    assert launches == sum(any(sizes[a:a + 87]) for a in range(0, count, 87))  # none for empty tensors alone
    compare32(W, M, V, G, W0, M0, V0, 2, "f32", **HYPER)


@pytest.mark.parametrize("count", [7, 8, 9, 63, 64, 65, 128, 129])
def test_adamw8_lists_around_the_length_of_a_launch(count):
    """As above with 64 tensors a launch; the roundings go by the place in the whole list."""
    sizes = [(53 * i + 5) % 397 if i % 7 != 3 else 0 for i in range(count)]
    W, M, V, G = make(sizes, "f32", "bf16", 45)
    state = state_of(M, V)
    mu.trace_enable(True)
    step8(W, state, G, 6, 12, "f32", HYPER)
    launches = len(mu.trace_collect())
    mu.trace_enable(False)
    assert launches == sum(any(sizes[a:a + 64]) for a in range(0, count, 64))


def code_bytes32(x, u32, v):
    """Codes of m (nearest) or, with chances, of the root of v, from fp32 values x = value / scale: every operation in
    fp32 with one rounding, as the definitions in include/muon.h are computed."""
    f = np.float32
    if u32 is None:
        return torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    binade = np.maximum(x.view(np.uint32) & np.uint32(0x7F800000), np.uint32(121 << 23))
    y = x * (np.uint32(257 << 23) - binade).view(f)
    lo = np.floor(y)
    bar = u32 * ((2 * lo + 1) * f(2.0 ** -32))
    up = ((y - lo) * (y + lo) > bar) | ((lo == 0) & (v > 0))
    step = (binade - np.uint32(3 << 23)).view(f)
    value = np.where(up, lo + f(1), lo) * step
    return torch.from_numpy(value.astype(f)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


@pytest.mark.parametrize("low,high", [(-40, 40), (-62, -20), (0, 1)])
def test_adamw8_codes_and_scales_bit_for_bit(low, high):
    """One step from zero over 2^14 groups with scales of any binade and any mantissa: the moments' fp32 sums, the root
    rounded to nearest, the scales, their reciprocals rounded to nearest and the codes are exactly those of single fp32
    operations, so they cannot depend on which approximations or fused operations a kernel uses."""
    f = np.float32
    groups = 1 << 14
    rng = np.random.default_rng(46)
    top = np.exp2(rng.uniform(low, high, (groups, 1)))
    g = top * rng.standard_normal((groups, 128)) * np.exp2(-rng.exponential(3.0, (groups, 128)))
    g[:, 7] = top[:, 0] * rng.uniform(4, 8, groups)
    g = g.astype(f).reshape(-1)
    W, G = [torch.zeros(g.size, device=DEV)], [torch.from_numpy(g).to(DEV)]
    state = mu.AdamW8State.zeros(W)
    mu.adamw8_step(W, state, G, 1, 0.01, seed=9)
    m, v = f(1 - 0.9) * g, (f(1 - 0.999) * g) * g
    u32 = (ao.chances(g.size, 9, 1, 0) * 2.0 ** 32).astype(f)
    for x, codes, scales, chance in ((m, state.m_codes, state.m_scales, None), (np.sqrt(v), state.r_codes, state.r_scales, u32)):
        assert x.dtype == f
        s = np.abs(x).reshape(groups, 128).max(1) * (f(1) / f(448))
        assert (s >= 2.0 ** -126).all()
        assert np.array_equal(scales[0].cpu().numpy(), s)
        y = x * np.repeat(f(1) / s, 128)
        want = code_bytes32(np.clip(y, f(-448), f(448)), chance, v)
        got = bytes_of(codes[0])
        assert np.array_equal(got, want), f"{np.sum(got != want)} of {got.size} codes differ"


def chances_from(first, count, seed, t, tensor):
    """ao.chances of the elements from ``first`` on."""
    key = ao.mix(np.uint64(seed) + ao.mix(np.uint64(t) + ao.mix(np.uint64(tensor))))
    i = np.arange(first, first + count, dtype=np.uint64)
    h = ao.mix((i >> np.uint64(1)) + key)
    return (np.where(i & np.uint64(1), h >> np.uint64(16), h & np.uint64(0xFFFF)).astype(np.float64) + 0.5) / 65536.0


def test_adamw8_codes_past_2_31_elements():
    """Both ends of one tensor of 2^31 + 1003 elements: codes, scales and chances of the last groups too."""
    n = 2 ** 31 + 1003
    W, G = [torch.ones(n, dtype=torch.bfloat16, device=DEV)], [torch.zeros(n, dtype=torch.bfloat16, device=DEV)]
    count = n - 2 ** 31 + 4096  # whole groups, and the short one at the end
    gen = torch.Generator(DEV).manual_seed(2)
    for part in (slice(0, 4096), slice(n - count, n)):
        G[0][part] = torch.randn(part.stop - part.start, device=DEV, generator=gen).to(torch.bfloat16)
    state = mu.AdamW8State.zeros(W)
    mu.adamw8_step(W, state, G, 1, 0.03, seed=6)
    u = np.concatenate((ao.chances(4096, 6, 1, 0), chances_from(n - count, count, 6, 1, 0)))
    at = 0
    for part in (slice(0, 4096), slice(n - count, n)):
        g = f64(G[0][part])
        groups = slice(part.start // 128, (part.stop + 127) // 128)
        m, v = (1 - 0.9) * g, (1 - 0.999) * g * g
        bad = ao.check_moment_codes(bytes_of(state.m_codes[0][part]), f64(state.m_scales[0][groups]), m, SLACK)
        assert bad == 0, f"{bad} codes of m"
        bad = ao.check_root_codes(bytes_of(state.r_codes[0][part]), f64(state.r_scales[0][groups]), v, u[at:at + g.size], SLACK)
        assert bad == 0, f"{bad} codes of the root of v"
        at += g.size
    middle = slice(4096 // 128, (n - count) // 128)
    assert not state.m_scales[0][middle].any() and not state.r_scales[0][middle].any()


# --- graphs, streams -----------------------------------------------------------------------------------------------
def test_adamw_captured_with_a_step_on_the_device():
    """Replays of one captured step of both kinds equal eager steps, with eager work in between."""
    sizes = (5000, 33)
    W, M, V, G = make(sizes, "f32", "bf16", 31)
    W8, M8, V8, _ = make(sizes, "f32", "bf16", 32)
    s8 = state_of(M8, V8)
    t = torch.tensor([4], device=DEV)
    copy = lambda L: [x.clone() for x in L]  # noqa: E731
    eW, eM, eV, eW8 = copy(W), copy(M), copy(V), copy(W8)
    e8 = mu.AdamW8State(*(copy(L) for L in (s8.m_codes, s8.m_scales, s8.r_codes, s8.r_scales)))

    def both(W, M, V, W8, s8, t):
        mu.adamw_step(W, M, V, G, t, **HYPER)
        mu.adamw8_step(W8, s8, G, t, seed=1, **HYPER)

    keep = [copy(L) for L in (W, M, V, W8, s8.m_codes, s8.m_scales, s8.r_codes, s8.r_scales)]
    both(W, M, V, W8, s8, t)  # builds the pointer arrays
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        t += 1
        both(W, M, V, W8, s8, t)
    for L, K in zip((W, M, V, W8, s8.m_codes, s8.m_scales, s8.r_codes, s8.r_scales), keep):
        for x, k in zip(L, K):
            x.copy_(k)
    for i in range(4):
        graph.replay()
        both(eW, eM, eV, eW8, e8, torch.tensor([5 + i], device=DEV))
        torch.cuda.synchronize()
        for a, b in zip([*W, *M, *V, *W8, *s8.m_scales, *s8.r_scales], [*eW, *eM, *eV, *eW8, *e8.m_scales, *e8.r_scales]):
            assert torch.equal(a, b), i
        for a, b in zip([*s8.m_codes, *s8.r_codes], [*e8.m_codes, *e8.r_codes]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
    assert t.item() == 8


def test_adamw_on_side_streams():
    """Two calls at once on two streams, on tensors made there."""
    ref = make((70000,), "f32", "f32", 41)
    mu.adamw_step(*ref, 3, **HYPER)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for s in streams:
        with torch.cuda.stream(s):
            sets.append(make((70000,), "f32", "f32", 41))
    torch.cuda.synchronize()
    for s, x in zip(streams, sets):
        mu.adamw_step(*x, 3, stream=s, **HYPER)
    torch.cuda.synchronize()
    for x in sets:
        assert all(torch.equal(a[0], b[0]) for a, b in zip(x, ref))


def test_adamw_launches_are_traced():
    W, M, V, G = make((5000,), "f32", "bf16", 42)
    mu.trace_enable(True)
    mu.adamw_step(W, M, V, G, 1, 1e-3)
    mu.adamw8_step(W, mu.AdamW8State.zeros(W), G, 1, 1e-3)
    recs = mu.trace_collect()
    mu.trace_enable(False)
    assert [r["role"] for r in recs] == ["adamw", "adamw8"]


@pytest.mark.parametrize("eight", [False, True])
def test_adamw_raises_the_version_of_what_it_writes(eight):
    """A step between forward and backward is seen: autograd refuses the old graph's saved weights."""
    W, M, V, G = make((300, 5), "f32", "f32", 43)
    lists = (W, M, V)
    if eight:
        state = state_of(M, V)
        lists = (W, state.m_codes, state.m_scales, state.r_codes, state.r_scales)
    step = lambda: mu.adamw8_step(W, state, G, 1, 1e-3) if eight else mu.adamw_step(W, M, V, G, 1, 1e-3)  # noqa: E731
    before = [[x._version for x in L] for L in lists]
    held = [x._version for x in G]
    step()
    assert all(x._version > b for L, B in zip(lists, before) for x, b in zip(L, B))
    assert [x._version for x in G] == held
    p = torch.nn.Parameter(W[0].clone())
    W[0] = p
    loss = (p * p).sum()
    step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with pytest.raises(ValueError):
        mu.adamw_step([p], [V[0]], [V[0]], [G[0]], 1, 1e-3)
    now = p._version
    with pytest.raises(mu.MuonError):
        mu.adamw_step([p], [M[0]], [V[0]], [G[0]], 0, 1e-3)
    assert p._version == now  # a refused call has written nothing
    with torch.inference_mode():  # tensors without a version
        Z = [torch.zeros(9, device=DEV) for _ in range(4)]
        mu.adamw_step(*[[z] for z in Z], 1, 1e-3)
