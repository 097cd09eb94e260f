"""fp64 reference of the AdamW step and of its 8-bit moments (numpy, no code shared with the library).

Definitions as in include/muon.h: muon_adamw_step, muon_adamw8_step."""
import numpy as np

GROUP = 128
TOP = 448.0


def adamw(W, m, v, G, t, lr, beta1, beta2, eps, wd, grad_scale=1.0):
    """(W, m, v) after step t; float64 in and out."""
    g = grad_scale * G
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    m_hat = m / (1.0 - beta1 ** t)
    v_hat = v / (1.0 - beta2 ** t)
    return W - lr * (m_hat / (np.sqrt(v_hat) + eps) + wd * W), m, v


def adamw_tolerance(W, m, v, G, t, lr, beta1, beta2, eps, wd, grad_scale=1.0, w_half=2.0 ** -24):
    """Largest fp32 rounding error of (W, m, v), elementwise.  h = 2^-24 is half a step relative to the value.

    m: the constants b1, 1 - b1 (h each), the scaled gradient (h), two products and the sum (h each): at most 4 h of
    b1 |m| + (1 - b1) |g|.  v: constant, two factors g (h each), two products, sum: at most 6 h of its (non-negative)
    terms.  The step: m (4 h) times c1 (h, product h) over d, with d's relative error half of v's (3 h), the root, c2
    (h, product h), eps and the sum (h each): 8 h; the quotient, lr and their product (h each): 17 h of
    lr |m|-terms c1 / d.  Decay: wd, lr and two products, the sum with the step: 5 h.  W: one rounding of the result
    to W's type (w_half) and one of the fp32 difference."""
    h = 2.0 ** -24
    g = np.abs(grad_scale * G)
    am = beta1 * np.abs(m) + (1 - beta1) * g
    av = beta2 * v + (1 - beta2) * g * g
    d = np.sqrt(av / (1 - beta2 ** t)) + eps
    ref = adamw(W, m, v, G, t, lr, beta1, beta2, eps, wd, grad_scale)[0]
    tw = 17 * h * lr * am / (1 - beta1 ** t) / d + 5 * h * lr * wd * np.abs(W) + (w_half + h) * np.abs(ref)
    tiny = 2.0 ** -149  # below the normal range one rounding is half of this at most
    return tw + tiny, 4 * h * am + 4 * tiny, 6 * h * av + 4 * tiny


def e4m3_values():
    """The 127 non-negative finite e4m3 values in code order."""
    return np.array([j * 2.0 ** -9 if j < 8 else (8 + j % 8) * 2.0 ** (j // 8 - 10) for j in range(127)])


def decode_e4m3(codes):
    """float64 values of uint8 e4m3 codes."""
    table = np.append(e4m3_values(), np.nan)
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 128, -1.0, 1.0) * table[c & 127]


def mix(x):
    mask = np.uint64(0xFFFFFFFF)
    x = np.asarray(x, dtype=np.uint64) & mask
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x9E3779B1)) & mask
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xB7E15163)) & mask
    return x ^ (x >> np.uint64(16))


def chances(n, seed, t, tensor):
    """u of every element of a tensor of n elements."""
    key = mix(np.uint64(seed) + mix(np.uint64(t) + mix(np.uint64(tensor))))
    i = np.arange(n, dtype=np.uint64)
    h = mix((i >> np.uint64(1)) + key)
    half = np.where(i & np.uint64(1), h >> np.uint64(16), h & np.uint64(0xFFFF))
    return (half.astype(np.float64) + 0.5) / 65536.0


def group_scales(x):
    """The scale of each group of 128 elements of a flat array, spread over the elements, and by group."""
    n = x.size
    groups = (n + GROUP - 1) // GROUP
    padded = np.zeros(groups * GROUP)
    padded[:n] = np.abs(x)
    s = padded.reshape(groups, GROUP).max(1) / TOP
    s = np.where(s < 2.0 ** -126, 0.0, s)
    return np.repeat(s, GROUP)[:n], s


def check_moment_codes(codes, scales, m, slack):
    """Whether codes/scales are the nearest e4m3 code of m (flat, float64) up to the fp32 error ``slack`` of m / s in
    units of a code step.  Returns the number of wrong elements."""
    each, s = group_scales(m)
    if not np.allclose(scales, s, rtol=8 * 2.0 ** -24, atol=0):
        return m.size
    x = np.divide(np.abs(m), each, out=np.zeros_like(m), where=each > 0)
    got = decode_e4m3(codes)
    step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(x, 2.0 ** -6))) - 3), 2.0 ** -9)
    ok = np.abs(np.abs(got) - x) <= step * (0.5 + slack)
    ok &= (got == 0) | (np.sign(got) == np.sign(m))
    return int(np.sum(~ok))


def check_root_codes(codes, scales, v, u, slack):
    """Whether codes/scales are the randomly rounded e4m3 code of sqrt(v) for the chances u; where the decision is
    closer than ``slack`` to the threshold, or x within ``slack`` of a code, either neighbour passes."""
    root = np.sqrt(v)
    each, s = group_scales(root)
    if not np.allclose(scales, s, rtol=8 * 2.0 ** -24, atol=0):
        return v.size
    x = np.minimum(np.divide(root, each, out=np.zeros_like(v), where=each > 0), TOP)
    table = e4m3_values()
    j = np.clip(np.searchsorted(table, x, side="right"), 1, 126)
    lo, hi = table[j - 1], table[j]
    share = (x * x - lo * lo) / (hi * hi - lo * lo)
    want = np.where(share > u, j, j - 1)
    want = np.where((want == 0) & (v > 0) & (each > 0), 1, want)
    got = np.asarray(codes, dtype=np.int64)
    wrong = got != want
    at_threshold = np.abs(share - u) <= slack
    at_code = np.minimum(share, 1 - share) <= slack
    near = np.abs(decode_e4m3(got) - x) <= 2 * (hi - lo)  # x on a code: either side's neighbours
    return int(np.sum(wrong & ~((at_threshold | at_code) & near)))
