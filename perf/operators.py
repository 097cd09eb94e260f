"""Cases for the operators that stand beside the Muon step: the AdamW step over many tensors (states in 32 bits or in
8), the microscaled 4-bit code, and the product that reads it.

``run`` computes an operator in elementary torch operations, or, where ``own`` is set, through this package's entry
points; ``exact`` computes the same from the definitions in float64.

Definitions
  adamw   g = s G, m <- b1 m + (1-b1) g, v <- b2 v + (1-b2) g^2,
          W <- W - lr (m/(1-b1^t) / (sqrt(v)/sqrt(1-b2^t) + eps) + wd W)
  adamw8  the same with m = c_m s_m and sqrt(v) = c_r s_r, c in e4m3, one fp32 scale (largest magnitude / 448) for each
          128 consecutive elements of a tensor.  c_m is rounded to nearest; c_r goes to the lower or the upper
          neighbour so that the expected square is kept, by 16 bits of a hash of (seed, t, tensor, element), and a
          positive v never gets c_r = 0.
  mx4     blocks of 32 along a row; scale byte = max(exponent field of the block's largest magnitude - 2, 0) (E8M0,
          255 where the block holds a NaN or an infinity), elements e2m1 of x / scale, nearest even, at most 6; two
          elements a byte, the even one in the low half; rows padded with zeros to whole units of 128.  A unit is 64
          code bytes and 4 scale bytes; codes lie as (unit, row, 64), scales as (unit, row, 4).
  product C = A B^T of two operands coded along k.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LR, BETA1, BETA2, EPS, WD = 1e-3, 0.9, 0.999, 1e-8, 0.01
GROUP, BLOCK, UNIT, TOP = 128, 32, 128, 448.0


def listed():
    return [
        # one norm weight of a 3584-wide model: the smallest call, latency only
        {"name": "adamw-one-norm", "op": "adamw", "sizes": "3584", "w": "f32", "g": "f32", "t": 1},
        # norms, biases and small heads of a 22-layer model, ragged sizes, bf16 gradients
        {"name": "adamw-many-ragged", "op": "adamw", "sizes": "45*2048,44*5632,22*333,7,1,1000003,65537", "w": "f32",
         "g": "bf16", "t": 1000},
        # embedding of 65536 tokens at width 3584, bf16 weights and gradients, most rows without a gradient
        {"name": "adamw-embedding", "op": "adamw", "sizes": "234881024", "w": "bf16", "g": "bf16", "t": 20},
        # one small odd tensor with 8-bit states
        {"name": "adamw8-one-odd", "op": "adamw8", "sizes": "5001", "w": "f32", "g": "f32", "t": 3},
        # a small model's remaining parameters with 8-bit states: an embedding of 32768 at 768 and its norms
        {"name": "adamw8-small-model", "op": "adamw8", "sizes": "25165824,25*768,12*2048,131", "w": "f32", "g": "bf16",
         "t": 100},
        # embedding and head of 32768 tokens at width 3584, bf16 weights and gradients
        {"name": "adamw8-embedding-head", "op": "adamw8", "sizes": "117440512,117440512", "w": "bf16", "g": "bf16",
         "t": 20},
        # the activations of a few tokens coded and read back
        {"name": "mx4-code-tokens", "op": "mx4code", "batch": 1, "rows": 5, "cols": 3584, "x": "bf16", "both": False},
        # three MLP weights after their update, coded along rows and along columns, and read back
        {"name": "mx4-code-weights", "op": "mx4code", "batch": 3, "rows": 3584, "cols": 18944, "x": "f32", "both": True},
        # one token through an MLP weight: the weight's codes are what has to be read
        {"name": "mx4-one-token", "op": "mx4mm", "batch": 1, "m": 1, "n": 18944, "k": 3584, "x": "bf16", "c": "bf16"},
        # forward of 4096 tokens: activations coded, then the product
        {"name": "mx4-forward", "op": "mx4mm", "batch": 1, "m": 4096, "n": 3584, "k": 18944, "x": "bf16", "c": "bf16"},
        # eight experts with a ragged number of tokens and an odd k
        {"name": "mx4-experts-odd", "op": "mx4mm", "batch": 8, "m": 77, "n": 2048, "k": 7001, "x": "bf16", "c": "f32"},
        # backward of a linear layer: the output gradient coded both ways, input gradient and weight gradient
        {"name": "mx4-backward", "op": "mx4grad", "batch": 1, "m": 8192, "n": 3584, "k": 7168, "x": "bf16", "c": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw8", "mx4code", "mx4mm", "mx4mm", "mx4grad"])
    if op in ("adamw", "adamw8"):
        count, total = _log(rng, 1, 120), _log(rng, 300, 40_000_000)
        parts = [rng.random() ** 3 + 1e-6 for _ in range(count)]
        sizes = [max(1, int(total * p / sum(parts))) for p in parts]
        return {"op": op, "sizes": ",".join(map(str, sizes)), "w": rng.choice(["f32", "bf16"]),
                "g": rng.choice(["f32", "bf16", "f16"]), "t": _log(rng, 1, 100_000)}
    if op == "mx4code":
        return {"op": op, "batch": rng.randint(1, 3), "rows": _log(rng, 1, 8000), "cols": _log(rng, 1, 8000),
                "x": rng.choice(["f32", "bf16", "f16"]), "both": rng.random() < 0.5}
    if op == "mx4mm":
        return {"op": op, "batch": rng.randint(1, 4), "m": _log(rng, 1, 2048), "n": _log(rng, 8, 4096),
                "k": _log(rng, 16, 8192), "x": rng.choice(["f32", "bf16"]), "c": rng.choice(["f32", "bf16"])}
    return {"op": op, "batch": 1, "m": _log(rng, 40, 4096), "n": _log(rng, 40, 4096), "k": _log(rng, 40, 4096),
            "x": "bf16", "c": rng.choice(["f32", "bf16"])}


def _sizes(case):
    parts = [p.split("*") for p in case["sizes"].split(",")]
    return [int(p[-1]) for p in parts for _ in range(int(p[0]) if len(p) == 2 else 1)]


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _pad_groups(x, group):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % group)).unflatten(-1, (-1, group))


def _pack_mx4(x):
    """Codes and scales of a 2-D fp32 matrix along its rows (used to make inputs)."""
    b = _pad_groups(x, UNIT).flatten(-2).unflatten(-1, (-1, BLOCK))
    field = b.abs().amax(-1).view(torch.int32) >> 23
    byte = (field - 2).clamp(min=0)
    y = (b / _power(byte)[..., None]).abs()
    level = sum((y > e).to(torch.uint8) if i % 2 == 0 else (y >= e).to(torch.uint8)
                for i, e in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    code = (level | (torch.signbit(b).to(torch.uint8) << 3)).flatten(-2)
    by_unit = lambda t, width: t.unflatten(-1, (-1, width)).transpose(0, 1).contiguous()  # noqa: E731
    return by_unit(code[..., 0::2] | (code[..., 1::2] << 4), UNIT // 2), by_unit(byte.to(torch.uint8), UNIT // BLOCK)


def _views(sizes, dtype, device="cuda"):
    """Tensors of the given sizes in one zeroed buffer, at multiples of 64 elements, and the buffer."""
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + (n + 63) // 64 * 64)
    flat = torch.zeros(starts[-1], dtype=dtype, device=device)
    return [flat[a:a + n] for a, n in zip(starts, sizes)], flat


def _flats(s):
    return {key: s[key] for key in ("w_flat", "m_flat", "v_flat", "m_codes_flat", "m_scales_flat", "r_codes_flat",
                                    "r_scales_flat") if key in s}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)

    def normal(*shape, std=1.0):
        x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
        return x

    state = dict(case)
    if case["op"] in ("adamw", "adamw8"):
        # every list of tensors lies in one buffer, each tensor at a multiple of 64 elements, as a program that keeps
        # flat parameter buffers has them; the buffers are what comes back
        sizes = _sizes(case)
        state["W"], state["w_flat"] = _views(sizes, DTYPES[case["w"]])
        state["G"], _ = _views(sizes, DTYPES[case["g"]])
        M, state["m_flat"] = _views(sizes, torch.float32)
        V, state["v_flat"] = _views(sizes, torch.float32)
        for n, W, G, m, v in zip(sizes, state["W"], state["G"], M, V):
            W.copy_(normal(n, std=0.02))
            # gradients of very different sizes from one stretch of 1024 to the next; a part of the stretches has no
            # gradient, as the rows of tokens that a batch does not hold, and a part never had one
            stretches = (n + 1023) // 1024
            size = torch.exp(normal(stretches)) * 1e-3
            kind = torch.rand(stretches, device="cuda", generator=gen)
            now = (size * (kind > 0.3)).repeat_interleave(1024)[:n]
            ever = (size * (kind > 0.1)).repeat_interleave(1024)[:n]
            G.copy_(normal(n) * now)
            if case["t"] > 1:
                m.copy_(normal(n) * ever * 0.3)
                v.copy_((normal(n) * ever).square() * 0.5 + ever.square() * 0.5)
        state.update(step=int(case["t"]) - 1, M=M, V=V)
        if case["op"] == "adamw8":
            del state["M"], state["V"], state["m_flat"], state["v_flat"]
            for key, values in (("m", M), ("r", [v.sqrt() for v in V])):
                codes, state[key + "_codes_flat"] = _views(sizes, torch.float8_e4m3fn)
                scales, state[key + "_scales_flat"] = _views([(n + GROUP - 1) // GROUP for n in sizes], torch.float32)
                for x, c, s in zip(values, codes, scales):
                    s.copy_(_pad_groups(x, GROUP).abs().amax(-1) / TOP)
                    y = (x / s.clamp(min=1e-30).repeat_interleave(GROUP)[:x.numel()]).clamp(-TOP, TOP)
                    c.copy_((torch.where(x > 0, y.clamp(min=2.0 ** -9), y) if key == "r" else y).to(torch.float8_e4m3fn))
                state[key + "_codes"], state[key + "_scales"] = codes, scales
        return state
    B, dt = case["batch"], DTYPES[case["x"]]
    if case["op"] == "mx4code":
        # the entries of one row in a hundred are fifty times the others, as outlier channels are
        state["X"] = [(normal(case["rows"], case["cols"], std=0.05)
                       * torch.where(torch.rand(case["rows"], 1, device="cuda", generator=gen) < 0.01, 50.0, 1.0)).to(dt)
                      for _ in range(B)]
        return state
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "mx4mm":
        state["X"] = [normal(m, k).to(dt) for _ in range(B)]
        packed = [_pack_mx4(normal(n, k, std=0.02)) for _ in range(B)]
        state.update(w_codes=[c for c, _ in packed], w_scales=[s for _, s in packed])
        return state
    # backward: W is n x k and X is m x k, both coded along their other axis by the forward pass; dY is m x n
    state["dY"] = [normal(m, n, std=1e-3).to(dt) for _ in range(B)]
    wt, xt = ([_pack_mx4(normal(r, c, std=s).t().contiguous()) for _ in range(B)] for r, c, s in ((n, k, 0.02), (m, k, 1.0)))
    state.update(wt_codes=[c for c, _ in wt], wt_scales=[s for _, s in wt], xt_codes=[c for c, _ in xt],
                 xt_scales=[s for _, s in xt])
    return state


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _adamw_values(W, G, m, v, t):
    g = G.float()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    step = m / (1 - BETA1 ** t) / (v.sqrt() / math.sqrt(1 - BETA2 ** t) + EPS)
    w = W.float()
    return w - LR * (step + WD * w), m, v


def _adamw(W, G, M, V, t):
    w, m, v = _adamw_values(W, G, M, V, t)
    W.copy_(w)
    M.copy_(m)
    V.copy_(v)


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xB7E15163) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _chance(n, seed, t, tensor):
    """One number in (0, 1) for each of n elements: half of a 32-bit hash for each of a pair."""
    key = _mix((seed + _mix((t + _mix(tensor)) & 0xFFFFFFFF)) & 0xFFFFFFFF)
    h = _mix((torch.arange((n + 1) // 2, device="cuda") + key) & 0xFFFFFFFF)
    return (torch.stack((h & 0xFFFF, h >> 16), -1).flatten()[:n].float() + 0.5) / 65536


def _scale(x):
    """The scale of each group, its inverse (0 for a group that is stored as zero), and the groups' elements."""
    groups = _pad_groups(x, GROUP)
    s = groups.abs().amax(-1) / TOP
    s = torch.where(s < 2.0 ** -126, 0.0, s)
    return s, torch.where((s > 0) & torch.isfinite(s), 1 / s, 0.0), groups


def _adamw8(i, W, G, mc, ms, rc, rs, t, seed):
    n = W.numel()
    spread = lambda s: s.repeat_interleave(GROUP)[:n]  # noqa: E731
    r = rc.float() * spread(rs)
    w, m, v = _adamw_values(W, G, mc.float() * spread(ms), r * r, t)
    W.copy_(w)
    s, inverse, groups = _scale(m)
    mc.copy_((groups * inverse[:, None]).clamp(-TOP, TOP).flatten()[:n].to(torch.float8_e4m3fn))
    ms.copy_(s)
    s, inverse, groups = _scale(v.sqrt())
    x = (groups * inverse[:, None]).clamp(max=TOP).flatten()[:n]
    small = x < 2.0 ** -6
    lo = torch.where(small, (x * 512).floor() / 512, (x.view(torch.int32) & ~0xFFFFF).view(torch.float32))
    hi = torch.where(small, lo + 2.0 ** -9, ((x.view(torch.int32) & ~0xFFFFF) + 0x100000).view(torch.float32))
    up = ((x - lo) * (x + lo) > _chance(n, seed, t, i) * ((hi - lo) * (hi + lo))) | ((lo == 0) & (v > 0) & (spread(s) > 0))
    rc.copy_(torch.where(up, hi, lo).to(torch.float8_e4m3fn))
    rs.copy_(s)


def _power(byte):
    """2^(byte - 127) of E8M0 scale bytes, 255 standing for NaN."""
    return torch.where(byte == 255, 0x7FC00000, torch.where(byte == 0, 0x400000, byte << 23)).to(torch.int32).view(torch.float32)


def _mx4_values(x):
    """The values that the code along the last axis holds."""
    k = x.shape[-1]
    b = _pad_groups(x.float(), BLOCK)
    field = b.abs().amax(-1).view(torch.int32) >> 23
    byte = torch.where(field == 255, 255, (field - 2).clamp(min=0))
    scale = _power(byte)[..., None]
    y = b / scale
    a = y.abs()
    # e2m1: steps of 1/2 below 2, of 1 below 4, of 2 up to 6; round() takes ties to the even multiple
    q = torch.where(a < 2, (a * 2).round() / 2, torch.where(a < 4, a.round(), ((a / 2).round() * 2).clamp(max=6)))
    return (torch.copysign(q, y) * scale).flatten(-2)[..., :k]


def _mx4_decode(codes, scales, k):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    codes, scales = codes.transpose(0, 1).flatten(1), scales.transpose(0, 1).flatten(1)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    y = table[both & 7] * (1 - 2 * (both >> 3)).float()
    return (y.unflatten(-1, (-1, BLOCK)) * _power(scales.int())[..., None]).flatten(-2)[..., :k]


def _plain(s):
    op = s["op"]
    if op == "adamw":
        s["step"] += 1
        [_adamw(W, G, M, V, s["step"]) for W, G, M, V in zip(s["W"], s["G"], s["M"], s["V"])]
        return _flats(s)
    if op == "adamw8":
        s["step"] += 1
        lists = (s[key] for key in ("W", "G", "m_codes", "m_scales", "r_codes", "r_scales"))
        [_adamw8(i, *x, s["step"], 5) for i, x in enumerate(zip(*lists))]
        return _flats(s)
    if op == "mx4code":
        dt = torch.bfloat16 if s["x"] == "bf16" else torch.float32
        out = {"rows": [_mx4_values(x).to(dt) for x in s["X"]]}
        if s["both"]:
            out["columns"] = [_mx4_values(x.t()).to(dt).contiguous() for x in s["X"]]
        return out
    c = DTYPES[s["c"]]
    if op == "mx4mm":
        return [(_mx4_values(x) @ _mx4_decode(w, e, s["k"]).t()).to(c) for x, w, e in zip(s["X"], s["w_codes"], s["w_scales"])]
    dx = [(_mx4_values(d) @ _mx4_decode(w, e, s["n"]).t()).to(c) for d, w, e in zip(s["dY"], s["wt_codes"], s["wt_scales"])]
    dw = [_mx4_values(d.t()) @ _mx4_decode(x, e, s["m"]).t() for d, x, e in zip(s["dY"], s["xt_codes"], s["xt_scales"])]
    return {"dX": dx, "dW": dw}


# ---------------------------------------------------------------------------------------------------------------------
# through the package
# ---------------------------------------------------------------------------------------------------------------------
def _own(s):
    import matrix_orthogonalizing_optimizer_step_amd as mu
    op = s["op"]
    if op == "adamw":
        s["step"] += 1
        mu.adamw_step(s["W"], s["M"], s["V"], s["G"], s["step"], LR, BETA1, BETA2, EPS, WD)
        return _flats(s)
    if op == "adamw8":
        s["step"] += 1
        state = mu.AdamW8State(s["m_codes"], s["m_scales"], s["r_codes"], s["r_scales"])
        mu.adamw8_step(s["W"], state, s["G"], s["step"], LR, BETA1, BETA2, EPS, WD, seed=5)
        return _flats(s)
    if op == "mx4code":
        dt = torch.bfloat16 if s["x"] == "bf16" else torch.float32
        if not s["both"]:
            return {"rows": mu.mx4_dequantize(mu.mx4_quantize(s["X"]), dt)}
        rows, columns = mu.mx4_quantize(s["X"], transpose="both")
        return {"rows": mu.mx4_dequantize(rows, dt), "columns": mu.mx4_dequantize(columns, dt)}
    c = DTYPES[s["c"]]
    if op == "mx4mm":
        return mu.mx4_matmul(mu.mx4_quantize(s["X"]), mu.MX4(s["w_codes"], s["w_scales"], s["k"]), dtype=c)
    d, dt = mu.mx4_quantize(s["dY"], transpose="both")
    return {"dX": mu.mx4_matmul(d, mu.MX4(s["wt_codes"], s["wt_scales"], s["n"]), dtype=c),
            "dW": mu.mx4_matmul(dt, mu.MX4(s["xt_codes"], s["xt_scales"], s["m"]), dtype=torch.float32)}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    size = lambda d: 4 if case[d] == "f32" else 2  # noqa: E731
    if case["op"] in ("adamw", "adamw8"):
        sizes = _sizes(case)
        n = sum(sizes)
        per = 2 * size("w") + size("g") + (16 if case["op"] == "adamw" else 4)
        scales = 0 if case["op"] == "adamw" else 16 * sum((x + GROUP - 1) // GROUP for x in sizes)
        return {"bytes": n * per + scales, "flops": 16 * n}
    code = lambda r, c: r * ((c + UNIT - 1) // UNIT) * 68  # noqa: E731
    B = case["batch"]
    if case["op"] == "mx4code":
        e = B * case["rows"] * case["cols"]
        out = 2 if case["x"] == "bf16" else 4
        return {"bytes": e * (size("x") + out * (2 if case["both"] else 1)), "flops": 4 * e * (2 if case["both"] else 1)}
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "mx4mm":
        return {"bytes": B * (m * k * size("x") + code(n, k) + m * n * size("c")), "flops": 2 * B * m * n * k}
    return {"bytes": B * (m * n * size("x") + code(k, n) + code(k, m) + m * k * size("c") + n * k * 4),
            "flops": 4 * B * m * n * k}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in float64
# ---------------------------------------------------------------------------------------------------------------------
def _e4m3_positive():
    """All non-negative e4m3 values in order: 8 subnormal steps of 2^-9, then 8 steps in each binade, up to 448."""
    return torch.tensor([j * 2.0 ** -9 if j < 8 else (8 + j % 8) * 2.0 ** (j // 8 - 10) for j in range(127)],
                        dtype=torch.float64, device="cuda")


def _exact_adamw(W, G, m, v, t):
    g = G.double()
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g.square() * (1.0 - BETA2)
    mh, vh = m / (1.0 - BETA1 ** t), v / (1.0 - BETA2 ** t)
    w = W.double()
    return w - LR * mh / (vh.sqrt() + EPS) - LR * WD * w, m, v


def _group_max(x):
    n = x.numel()
    at = torch.arange(n, device="cuda") // GROUP
    top = torch.zeros((n + GROUP - 1) // GROUP, dtype=torch.float64, device="cuda")
    return at, top.scatter_reduce_(0, at, x.abs(), "amax")


def _bits(n, seed, t, tensor):
    u32 = lambda x: np.asarray(x, dtype=np.uint64) & np.uint64(0xFFFFFFFF)  # noqa: E731

    def mix(x):
        x = u32(x)
        x = u32((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B1))
        x = u32((x ^ (x >> np.uint64(15))) * np.uint64(0xB7E15163))
        return x ^ (x >> np.uint64(16))

    key = mix(np.uint64(seed) + mix(np.uint64(t) + mix(np.uint64(tensor))))
    out = np.empty(n, dtype=np.uint16)
    for a in range(0, n, 1 << 23):  # in pieces that stay in the cache and in memory
        i = np.arange(a, min(n, a + (1 << 23)), dtype=np.uint64)
        h = mix((i[::2] >> np.uint64(1)) + key)
        out[a:a + len(i)] = np.stack((h & np.uint64(0xFFFF), h >> np.uint64(16)), 1).reshape(-1)[:len(i)].astype(np.uint16)
    return torch.from_numpy(out.astype(np.int32)).cuda().double()


def _exact_adamw8(i, W, G, mc, ms, rc, rs, t, table):
    n = W.numel()
    at = torch.arange(n, device="cuda") // GROUP
    w, m, v = _exact_adamw(W, G, mc.double() * ms.double()[at], (rc.double() * rs.double()[at]).square(), t)
    at, top = _group_max(m)
    s_m = top / TOP
    y = torch.where(s_m[at] > 0, m / s_m[at].clamp(min=1e-300), 0.0)
    j = torch.searchsorted(table, y.abs()).clamp(1, 126)
    lo, hi = table[j - 1], table[j]
    mid = (lo + hi) / 2
    a = y.abs()
    c_m = torch.where(a > mid, hi, torch.where(a < mid, lo, torch.where(j % 2 == 0, hi, lo))) * y.sign()
    at, top = _group_max(v)
    s_r = top.sqrt() / TOP
    x = torch.where(s_r[at] > 0, v.sqrt() / s_r[at].clamp(min=1e-300), 0.0).clamp(max=TOP)
    j = torch.searchsorted(table, x, right=True).clamp(1, 126)
    lo, hi = table[j - 1], table[j]
    share = (x.square() - lo.square()) / (hi.square() - lo.square())
    c_r = torch.where(share * 65536 > _bits(n, 5, t, i) + 0.5, hi, lo)
    c_r = torch.where((x > 0) & (c_r == 0), 2.0 ** -9, c_r)
    return w, c_m, s_m, c_r, s_r


def _power64(e):
    """2^e exactly (pow() is not exact on every device)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx4(x):
    """Values of the code along the last axis, by distance to the eight magnitudes."""
    r, c = x.shape
    out = torch.empty(r, c, dtype=torch.float64, device="cuda")
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    for a in range(0, r, max(1, (1 << 26) // max(c, 1))):
        b = x[a:a + max(1, (1 << 26) // max(c, 1))].double()
        rows = b.shape[0]
        p = torch.zeros(rows, (c + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device="cuda")
        p[:, :c] = b
        p = p.view(rows, -1, BLOCK)
        e = torch.frexp(p.abs().amax(-1)).exponent - 3  # 2^e: two binades under the largest magnitude's own
        e = torch.where(p.abs().amax(-1) == 0, -127, e).clamp(min=-127)
        scale = _power64(e)[..., None]
        y = (p / scale).abs().clamp(max=6)
        j = torch.searchsorted(table, y).clamp(1, 7)
        lo, hi = table[j - 1], table[j]
        q = torch.where(y - lo < hi - y, lo, torch.where(y - lo > hi - y, hi, torch.where(j % 2 == 0, hi, lo)))
        out[a:a + rows] = (q * p.sign() * scale).view(rows, -1)[:, :c]
    return out


def _exact_decode(codes, scales, k):
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64, device="cuda")
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    table = torch.outer(sign, mag).flatten()
    codes, scales = (x.permute(1, 0, 2).reshape(x.shape[1], -1) for x in (codes, scales))
    v = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device="cuda")
    v[:, 0::2] = table[(codes & 15).long()]
    v[:, 1::2] = table[(codes >> 4).long()]
    return (v * _power64(scales.long() - 127).repeat_interleave(BLOCK, 1))[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("adamw", "adamw8"):
        sizes, groups = _sizes(case), [(n + GROUP - 1) // GROUP for n in _sizes(case)]
        names = ["w_flat", "m_flat", "v_flat"] if op == "adamw" else list(_flats(s))
        lists, flats = zip(*[_views(groups if "scales" in name else sizes, torch.float64) for name in names])
        table = _e4m3_positive()
        for i in range(len(sizes)):
            if op == "adamw":
                got = _exact_adamw(s["W"][i], s["G"][i], s["M"][i].double(), s["V"][i].double(), case["t"])
            else:
                got = _exact_adamw8(i, s["W"][i], s["G"][i], s["m_codes"][i], s["m_scales"][i], s["r_codes"][i],
                                    s["r_scales"][i], case["t"], table)
            for to, x in zip(lists, got):
                to[i].copy_(x)
        return dict(zip(names, flats))
    if op == "mx4code":
        out = {"rows": [_exact_mx4(x) for x in s["X"]]}
        if case["both"]:
            out["columns"] = [_exact_mx4(x.t().contiguous()) for x in s["X"]]
        return out
    if op == "mx4mm":
        return [_exact_mx4(x) @ _exact_decode(w, e, case["k"]).t().contiguous()
                for x, w, e in zip(s["X"], s["w_codes"], s["w_scales"])]
    return {"dX": [_exact_mx4(d) @ _exact_decode(w, e, case["n"]).t().contiguous()
                   for d, w, e in zip(s["dY"], s["wt_codes"], s["wt_scales"])],
            "dW": [_exact_mx4(d.t().contiguous()) @ _exact_decode(x, e, case["m"]).t().contiguous()
                   for d, x, e in zip(s["dY"], s["xt_codes"], s["xt_scales"])]}
