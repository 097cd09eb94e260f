"""Cases for the 8-bit code and its products, dense and over experts, and for the experts' balance loss and counts.

``run`` computes an operator in elementary torch operations, or, where ``own`` is set, through this package's entry
points; ``exact`` computes the same from the definitions in float64.

Definitions
  code     blocks of 128 along a row ("row"), or tiles of 128 x 128 ("tile"), share a power of two (E8M0 byte): the
           smallest one, from 2^-127 on, with largest magnitude <= TOP * scale, TOP = 448 (e4m3) or 57344 (e5m2); 255
           where the block holds a NaN or an infinity.  Elements are the nearest 8-bit floats of x / scale, ties to even.
           Rows are padded with zeros to whole blocks.  Codes lie as (half block, row, 64), scales as (block, row), rows
           rounded up to 16; a tile's scale is repeated for each of its rows.
  product  C = A B^T of two operands coded along k.
  experts  rows of A sorted by expert, counts[e] of them for expert e: C = A B_e^T on each expert's rows; for the weight
           gradients C_e = A_e^T B_e, with A and B coded along their rows, each expert's padded to whole blocks.
  balance  p = softmax(z), or sigmoid(z) / its sum; f_e = E count_e / (K T) over the T tokens that count;
           loss = alpha sum_e f_e mean_t p_te, for a batch of sequences the mean of theirs; with its gradient for z.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn,
          "e5m2": torch.float8_e5m2, "i32": torch.int32, "i64": torch.int64}
BLOCK, PIECE, LINE = 128, 64, 16
FORMATS = {"e4m3": (448.0, 8, -6, 3), "e5m2": (57344.0, 15, -14, 2)}  # largest value, its exponent, least one, bits
ALPHA = 0.01


def listed():
    return [
        # a few tokens of a small mixture's router: the smallest call, latency only
        {"name": "balance-few-tokens", "op": "balance", "seqs": 1, "tokens": 7, "experts": 8, "top": 2, "z": "f32",
         "i": "i64", "score": "softmax", "mask": False},
        # a training batch of 32768 tokens over 256 experts
        {"name": "balance-batch", "op": "balance", "seqs": 1, "tokens": 32768, "experts": 256, "top": 8, "z": "bf16",
         "i": "i64", "score": "softmax", "mask": False},
        # padded sequences, each balanced by itself, an odd number of experts with sigmoid scores
        {"name": "balance-sequences-odd", "op": "balance", "seqs": 16, "tokens": 2049, "experts": 61, "top": 6, "z": "f32",
         "i": "i32", "score": "sigmoid", "mask": True},
        # the activations of a few tokens coded and read back
        {"name": "fp8-code-tokens", "op": "code", "batch": 1, "rows": 5, "cols": 3584, "x": "bf16", "block": "row",
         "both": False, "f": "e4m3"},
        # three MLP weights after their update, coded in tiles for both directions, and read back
        {"name": "fp8-code-weights", "op": "code", "batch": 3, "rows": 3584, "cols": 18944, "x": "f32", "block": "tile",
         "both": True, "f": "e4m3"},
        # one token through an MLP weight: the weight's codes are what has to be read
        {"name": "fp8-one-token", "op": "product", "dir": "forward", "batch": 1, "m": 1, "n": 18944, "k": 3584, "x": "bf16",
         "c": "bf16", "f": "e4m3"},
        # forward of 4096 tokens: activations coded, then the product
        {"name": "fp8-forward", "op": "product", "dir": "forward", "batch": 1, "m": 4096, "n": 3584, "k": 18944,
         "x": "bf16", "c": "bf16", "f": "e4m3"},
        # backward of three odd layers: the output gradient in e5m2 both ways, input and weight gradients
        {"name": "fp8-backward-odd", "op": "product", "dir": "backward", "batch": 3, "m": 1025, "n": 2049, "k": 1367,
         "x": "f32", "c": "f32", "f": "e5m2"},
        # backward of a linear layer on 8192 tokens
        {"name": "fp8-backward", "op": "product", "dir": "backward", "batch": 1, "m": 8192, "n": 3584, "k": 7168,
         "x": "bf16", "c": "bf16", "f": "e4m3"},
        # four tokens, each sent to six of 64 experts: the weights that they meet have to be read
        {"name": "experts-few-tokens", "op": "experts", "dir": "forward", "rows": 24, "experts": 64, "n": 2048, "k": 7168,
         "x": "bf16", "c": "bf16", "f": "e4m3"},
        # 2730 tokens, each sent to six of 64 experts, a few of which get most of them
        {"name": "experts-forward", "op": "experts", "dir": "forward", "rows": 16380, "experts": 64, "n": 2048, "k": 7168,
         "x": "bf16", "c": "bf16", "f": "e4m3"},
        # backward of a part of the experts: input gradients and every expert's weight gradient
        {"name": "experts-backward", "op": "experts", "dir": "backward", "rows": 8190, "experts": 16, "n": 2048, "k": 7168,
         "x": "bf16", "c": "bf16", "f": "e4m3"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance", "code", "product", "product", "experts", "experts"])
    f = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op == "balance":
        seqs = rng.choice([1, 1, rng.randint(2, 24)])
        experts = _log(rng, 2, 512)
        return {"op": op, "seqs": seqs, "tokens": _log(rng, 1, 32768 // seqs), "experts": experts,
                "top": rng.randint(1, min(experts, 10)), "z": rng.choice(["f32", "bf16", "f16"]),
                "i": rng.choice(["i32", "i64"]), "score": rng.choice(["softmax", "sigmoid"]), "mask": rng.random() < 0.4}
    if op == "code":
        return {"op": op, "batch": rng.randint(1, 3), "rows": _log(rng, 1, 8000), "cols": _log(rng, 1, 8000),
                "x": rng.choice(["f32", "bf16", "f16"]), "block": rng.choice(["row", "tile"]), "both": rng.random() < 0.5,
                "f": f}
    if op == "product":
        forward = rng.random() < 0.6
        least = 1 if forward else 40
        return {"op": op, "dir": "forward" if forward else "backward", "batch": rng.randint(1, 3),
                "m": _log(rng, least, 4096), "n": _log(rng, 8, 4096), "k": _log(rng, 16, 8192),
                "x": rng.choice(["f32", "bf16"]), "c": rng.choice(["f32", "bf16"]), "f": f}
    return {"op": op, "dir": rng.choice(["forward", "forward", "backward"]), "rows": _log(rng, 1, 8192),
            "experts": _log(rng, 2, 64), "n": _log(rng, 32, 2048), "k": _log(rng, 32, 4096),
            "x": rng.choice(["f32", "bf16"]), "c": rng.choice(["f32", "bf16"]), "f": f}


def _counts(case):
    """Rows of each expert: uneven, some experts without any; the same for every seed."""
    rng = random.Random("%d %d" % (case["rows"], case["experts"]))
    share = [rng.random() ** 2 * (rng.random() > 0.1) + 1e-9 for _ in range(case["experts"])]
    if case["rows"] < 2 * case["experts"]:  # few tokens: mostly different experts
        share = [1.0] * case["experts"]
    out = [0] * case["experts"]
    for e in rng.choices(range(case["experts"]), share, k=case["rows"]):
        out[e] += 1
    return out


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _up(n, to):
    return (n + to - 1) // to * to


def _pack(x, tile=False):
    """Codes and scales (e4m3) of a 2-D fp32 matrix along its rows, as the library lays them out (to make inputs)."""
    r, k = x.shape
    p = _pad(x, _up(r, BLOCK) if tile else r, _up(k, BLOCK))
    blocks = p.unflatten(1, (-1, BLOCK))
    top = blocks.abs().amax(-1)
    if tile:
        top = top.unflatten(0, (-1, BLOCK)).amax(1).repeat_interleave(BLOCK, 0)
    bits = top.view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=0)
    y = (blocks / _power(byte)[..., None]).clamp(-448, 448).flatten(1)[:r].to(torch.float8_e4m3fn)
    codes = y.view(torch.uint8).unflatten(1, (-1, PIECE)).transpose(0, 1).contiguous().view(torch.float8_e4m3fn)
    return codes, _pad(byte[:r].t().to(torch.uint8), byte.shape[1], _up(r, LINE)).contiguous()


def _pack_experts(x, counts):
    """The code of x^T, each expert's rows of x padded to whole blocks; with room for any other counts of these rows."""
    room = (x.shape[0] + (BLOCK - 1) * len(counts)) // BLOCK
    parts, at = [], 0
    for c in counts:
        if c:
            parts.append(_pad(x[at:at + c].t(), x.shape[1], _up(c, BLOCK)))
        at += c
    return _pack(_pad(torch.cat(parts, 1), x.shape[1], room * BLOCK))


def _power(byte):
    """2^(byte - 127) of E8M0 scale bytes, 255 standing for NaN."""
    return torch.where(byte == 255, 0x7FC00000, torch.where(byte == 0, 0x400000, byte << 23)).to(torch.int32).view(torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 104729 + 17)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=gen)

    state = dict(case)
    if case["op"] == "balance":
        S, L, E, K = case["seqs"], case["tokens"], case["experts"], case["top"]
        # some experts are liked by all tokens, as before balance is reached; choices are made with some noise
        z = normal(S, L, E) + normal(E)
        state["index"] = torch.topk(z + 0.3 * normal(S, L, E), K, -1).indices.to(DTYPES[case["i"]]).contiguous()
        state["logits"] = z.to(DTYPES[case["z"]])
        state["mask"] = None
        if case["mask"]:
            length = (uniform(S, 1) * L).ceil().clamp(min=1)
            state["mask"] = (torch.arange(L, device="cuda")[None] < length).contiguous()
        return state
    dt = DTYPES[case["x"]]
    if case["op"] == "code":
        # the entries of one row in a hundred are fifty times the others, as outlier channels are
        state["X"] = [(normal(case["rows"], case["cols"], std=0.05)
                       * torch.where(uniform(case["rows"], 1) < 0.01, 50.0, 1.0)).to(dt) for _ in range(case["batch"])]
        return state
    n, k = case["n"], case["k"]
    if case["op"] == "product":
        m, B = case["m"], case["batch"]
        if case["dir"] == "forward":
            state["X"] = [normal(m, k).to(dt) for _ in range(B)]
            weights = [_pack(normal(n, k, std=0.02), True) for _ in range(B)]
            state.update(w_codes=[c for c, _ in weights], w_scales=[s for _, s in weights])
            return state
        # backward: W is n x k and X is m x k, both coded along their other axis by the forward pass; dY is m x n
        state["dY"] = [normal(m, n, std=1e-3).to(dt) for _ in range(B)]
        wt = [_pack(normal(n, k, std=0.02).t().contiguous(), True) for _ in range(B)]
        xt = [_pack(normal(m, k).t().contiguous()) for _ in range(B)]
        state.update(wt_codes=[c for c, _ in wt], wt_scales=[s for _, s in wt], xt_codes=[c for c, _ in xt],
                     xt_scales=[s for _, s in xt])
        return state
    sizes = _counts(case)
    state.update(sizes=sizes, counts=torch.tensor(sizes, dtype=torch.int32, device="cuda"))
    if case["dir"] == "forward":
        state["X"] = normal(case["rows"], k).to(dt)
        weights = [_pack(normal(n, k, std=0.02), True) for _ in sizes]
        state.update(w_codes=[c for c, _ in weights], w_scales=[s for _, s in weights])
        return state
    state["dY"] = normal(case["rows"], n, std=1e-3).to(dt)
    wt = [_pack(normal(n, k, std=0.02).t().contiguous(), True) for _ in sizes]
    state.update(wt_codes=[c for c, _ in wt], wt_scales=[s for _, s in wt])
    state["xt_codes"], state["xt_scales"] = _pack_experts(normal(case["rows"], k), sizes)
    return state


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _values(x, f, tile=False):
    """The values that the code along the last axis of a matrix holds."""
    r, k = x.shape
    _, high, low, bits = FORMATS[f]
    blocks = _pad(x.float(), _up(r, BLOCK) if tile else r, _up(k, BLOCK)).unflatten(1, (-1, BLOCK))
    top = blocks.abs().amax(-1)
    if tile:
        top = top.unflatten(0, (-1, BLOCK)).amax(1).repeat_interleave(BLOCK, 0)
    top = top.view(torch.int32)
    byte = ((top >> 23) - high + ((top & 0x7FFFFF) > 0x600000)).clamp(min=0)
    scale = _power(torch.where(top >= 0x7F800000, 255, byte))[..., None]
    y = blocks / scale
    e = ((y.view(torch.int32) >> 23) & 255) - 127
    step = _power(e.clamp(min=low) - bits + 127)
    return ((y / step).round() * step * scale).flatten(1)[:r, :k]  # round() takes ties to even


def _decode(codes, scales, k):
    r = codes.shape[1]
    y = codes.float().transpose(0, 1).flatten(1)
    return (y.unflatten(1, (-1, BLOCK)) * _power(scales[:, :r].t().int())[..., None]).flatten(1)[:, :k]


def _balance(s):
    z, index, mask = s["logits"].float(), s["index"].long(), s["mask"]
    S, L, E = z.shape
    K = index.shape[-1]
    valid = torch.ones(S, L, device="cuda") if mask is None else mask.float()
    hits = valid.long()[..., None].expand(S, L, K)
    counts = torch.zeros(S, E, dtype=torch.long, device="cuda").scatter_add_(1, index.flatten(1), hits.flatten(1))
    tokens = valid.double().sum(1).float().clamp(min=1)
    f = counts.float() * (E / (K * tokens))[:, None]
    if s["score"] == "softmax":
        e = (z - z.amax(-1, keepdim=True)).exp()
        p = e / e.sum(-1, keepdim=True)
        slope = p
    else:
        q = 1 / (1 + (-z).exp())
        total = q.sum(-1, keepdim=True)
        p, slope = q / total, q * (1 - q) / total
    inner = (f[:, None] * p).sum(-1)
    loss = ((inner * valid).double().sum(1).float() / tokens).sum() * (ALPHA / S)
    grad = slope * (f[:, None] - inner[..., None]) * (valid * (ALPHA / S) / tokens[:, None])[..., None]
    return {"loss": loss, "counts": counts.sum(0).int(), "grad": grad.to(s["logits"].dtype)}


def _split(x, sizes):
    return torch.split(x, list(sizes))


def _experts_t(codes, scales, sizes):
    """The values of each expert's part of a code along rows (rows of the matrix x that expert's count)."""
    at, out = 0, []
    for c in sizes:
        blocks = (c + BLOCK - 1) // BLOCK
        out.append(_decode(codes[2 * at:2 * (at + blocks)], scales[at:at + blocks], c))
        at += blocks
    return out


def _plain(s):
    op = s["op"]
    if op == "balance":
        return _balance(s)
    f = s["f"]
    if op == "code":
        dt, tile = torch.bfloat16 if s["x"] == "bf16" else torch.float32, s["block"] == "tile"
        out = {"rows": [_values(x, f, tile).to(dt) for x in s["X"]]}
        if s["both"]:
            out["columns"] = [_values(x.t(), f, tile).to(dt).contiguous() for x in s["X"]]
        return out
    c = DTYPES[s["c"]]
    if op == "product" and s["dir"] == "forward":
        return [(_values(x, f) @ _decode(w, e, s["k"]).t()).to(c) for x, w, e in zip(s["X"], s["w_codes"], s["w_scales"])]
    if op == "product":
        dx = [(_values(d, f) @ _decode(w, e, s["n"]).t()).to(c) for d, w, e in zip(s["dY"], s["wt_codes"], s["wt_scales"])]
        dw = [_values(d.t(), f) @ _decode(x, e, s["m"]).t() for d, x, e in zip(s["dY"], s["xt_codes"], s["xt_scales"])]
        return {"dX": dx, "dW": dw}
    if s["dir"] == "forward":
        return torch.cat([(_values(x, f) @ _decode(w, e, s["k"]).t()).to(c)
                          for x, w, e in zip(_split(s["X"], s["sizes"]), s["w_codes"], s["w_scales"]) if len(x)])
    parts = _split(s["dY"], s["sizes"])
    dx = torch.cat([(_values(d, f) @ _decode(w, e, s["n"]).t()).to(c)
                    for d, w, e in zip(parts, s["wt_codes"], s["wt_scales"]) if len(d)])
    dw = [_values(d.t(), f) @ x.t() if len(d) else torch.zeros(s["n"], s["k"], device="cuda")
          for d, x in zip(parts, _experts_t(s["xt_codes"], s["xt_scales"], s["sizes"]))]
    return {"dX": dx, "dW": dw}


# ---------------------------------------------------------------------------------------------------------------------
# through the package
# ---------------------------------------------------------------------------------------------------------------------
def _own(s):
    import matrix_orthogonalizing_optimizer_step_amd as mu
    op = s["op"]
    if op == "balance":
        loss, counts, grad = mu.expert_balance(s["logits"], s["index"], ALPHA, s["score"], s["mask"], grad=True)
        return {"loss": loss, "counts": counts, "grad": grad}
    f = s["f"]
    if op == "code":
        dt = torch.bfloat16 if s["x"] == "bf16" else torch.float32
        if not s["both"]:
            return {"rows": mu.fp8_dequantize(mu.fp8_quantize(s["X"], block=s["block"], format=f), dt)}
        rows, columns = mu.fp8_quantize(s["X"], block=s["block"], transpose="both", format=f)
        return {"rows": mu.fp8_dequantize(rows, dt), "columns": mu.fp8_dequantize(columns, dt)}
    c = DTYPES[s["c"]]
    if op == "product" and s["dir"] == "forward":
        return mu.fp8_matmul(mu.fp8_quantize(s["X"], format=f), mu.FP8(s["w_codes"], s["w_scales"], s["k"]), dtype=c)
    if op == "product":
        d, dt = mu.fp8_quantize(s["dY"], transpose="both", format=f)
        return {"dX": mu.fp8_matmul(d, mu.FP8(s["wt_codes"], s["wt_scales"], s["n"]), dtype=c),
                "dW": mu.fp8_matmul(dt, mu.FP8(s["xt_codes"], s["xt_scales"], s["m"]), dtype=torch.float32)}
    if s["dir"] == "forward":
        x = mu.fp8_quantize([s["X"]], format=f)
        return mu.fp8_grouped_matmul(x, mu.FP8(s["w_codes"], s["w_scales"], s["k"]), s["counts"], dtype=c)[0]
    d, dt = mu.fp8_quantize([s["dY"]], transpose="both", format=f, counts=s["counts"])
    xt = mu.FP8([s["xt_codes"]], [s["xt_scales"]], s["rows"], groups=s["experts"])
    dx = mu.fp8_grouped_matmul(d, mu.FP8(s["wt_codes"], s["wt_scales"], s["n"]), s["counts"], dtype=c)
    return {"dX": dx[0], "dW": mu.fp8_grouped_weight_grad(dt, xt, s["counts"], dtype=torch.float32)}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    size = lambda d: {"f32": 4, "i32": 4, "i64": 8}.get(case[d], 2)  # noqa: E731
    code = lambda r, c: r * _up(c, BLOCK) * (1 + 1 / BLOCK)  # noqa: E731
    op = case["op"]
    if op == "balance":
        t = case["seqs"] * case["tokens"]
        return {"bytes": t * (case["experts"] * 2 * size("z") + case["top"] * size("i")), "flops": 8 * t * case["experts"]}
    if op == "code":
        e = case["batch"] * case["rows"] * case["cols"]
        out = 2 if case["x"] == "bf16" else 4
        return {"bytes": e * (size("x") + out * (2 if case["both"] else 1)), "flops": 4 * e * (2 if case["both"] else 1)}
    n, k = case["n"], case["k"]
    if op == "product":
        B, m = case["batch"], case["m"]
        if case["dir"] == "forward":
            return {"bytes": B * (m * k * size("x") + code(n, k) + m * n * size("c")), "flops": 2 * B * m * n * k}
        return {"bytes": B * (m * n * size("x") + code(k, n) + code(k, m) + m * k * size("c") + n * k * 4),
                "flops": 4 * B * m * n * k}
    m, met = case["rows"], sum(c > 0 for c in _counts(case))
    if case["dir"] == "forward":
        return {"bytes": m * k * size("x") + met * code(n, k) + m * n * size("c"), "flops": 2 * m * n * k}
    return {"bytes": m * n * size("x") + met * code(k, n) + code(k, m) + m * k * size("c") + case["experts"] * n * k * 4,
            "flops": 4 * m * n * k}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in float64
# ---------------------------------------------------------------------------------------------------------------------
def _table(f):
    """All non-negative finite values of the format in order."""
    top, _, low, bits = FORMATS[f]
    v = [j * 2.0 ** (low - bits) for j in range(1 << bits)]
    e = low
    while v[-1] < top:
        v += [(1 + j / (1 << bits)) * 2.0 ** e for j in range(1 << bits)]
        e += 1
    return torch.tensor([x for x in v if x <= top], dtype=torch.float64, device="cuda")


def _power64(e):
    """2^e exactly (pow() is not exact on every device)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(x, f, tile=False):
    """Values of the code along the last axis, by distance to the format's values."""
    r, k = x.shape
    table, out = _table(f), torch.empty(r, k, dtype=torch.float64, device="cuda")
    step = max(BLOCK, (1 << 25) // max(k, 1) // BLOCK * BLOCK)
    for a in range(0, r, step):
        b = x[a:a + step].double()
        rows = b.shape[0]
        p = torch.zeros(_up(rows, BLOCK), _up(k, BLOCK), dtype=torch.float64, device="cuda")
        p[:rows, :k] = b
        p = p.view(p.shape[0], -1, BLOCK)
        top = p.abs().amax(-1)
        if tile:
            top = top.view(-1, BLOCK, top.shape[1]).amax(1, keepdim=True).expand(-1, BLOCK, -1).reshape(top.shape)
        half, e = torch.frexp(top / FORMATS[f][0])  # half 2^e, half in [1/2, 1): the power of two not below it
        e = torch.where(half == 0.5, e - 1, e)
        scale = _power64(torch.where(top == 0, -127, e).clamp(min=-127))[..., None]
        y = (p / scale).abs()
        j = torch.searchsorted(table, y).clamp(1, len(table) - 1)
        lo, hi = table[j - 1], table[j]
        q = torch.where(y - lo < hi - y, lo, torch.where(y - lo > hi - y, hi, torch.where(j % 2 == 0, hi, lo)))
        out[a:a + rows] = (q * p.sign() * scale).view(p.shape[0], -1)[:rows, :k]
    return out


def _exact_decode(codes, scales, k):
    pieces, r, _ = codes.shape
    v = codes.to(torch.float64).permute(1, 0, 2).reshape(r, pieces * PIECE)
    s = _power64(scales[:, :r].long() - 127)
    return (v * s.repeat_interleave(BLOCK, 0).t())[:, :k]


def _exact_balance(s):
    z, index = s["logits"].double(), s["index"].long()
    S, L, E = z.shape
    K = index.shape[-1]
    grad, counts, loss = torch.zeros_like(z), torch.zeros(E, dtype=torch.int32, device="cuda"), 0.0
    for b in range(S):
        keep = slice(None) if s["mask"] is None else s["mask"][b]
        zb = z[b][keep]
        T = len(zb)
        count = torch.bincount(index[b][keep].flatten(), minlength=E)
        f = count.double() * E / (K * T)
        if s["score"] == "softmax":
            p = torch.softmax(zb, -1)
            d = ALPHA / S / T * (f * p - p * (p @ f)[:, None])
        else:
            q = torch.sigmoid(zb)
            total = q.sum(-1, keepdim=True)
            p = q / total
            # dp_j/dz_e = q_e (1 - q_e) ((j = e) - p_j) / total
            d = ALPHA / S / T * q * (1 - q) / total * (f - (p @ f)[:, None])
        grad[b][keep] = d
        counts += count.int()
        loss = loss + ALPHA / S * (f * p.mean(0)).sum()
    return {"loss": loss, "counts": counts, "grad": grad}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        return _exact_balance(s)
    f = case["f"]
    if op == "code":
        tile = case["block"] == "tile"
        out = {"rows": [_exact_values(x, f, tile) for x in s["X"]]}
        if case["both"]:
            out["columns"] = [_exact_values(x.t().contiguous(), f, tile) for x in s["X"]]
        return out
    k = case["k"]
    if op == "product" and case["dir"] == "forward":
        return [_exact_values(x, f) @ _exact_decode(w, e, k).t().contiguous()
                for x, w, e in zip(s["X"], s["w_codes"], s["w_scales"])]
    if op == "product":
        return {"dX": [_exact_values(d, f) @ _exact_decode(w, e, case["n"]).t().contiguous()
                       for d, w, e in zip(s["dY"], s["wt_codes"], s["wt_scales"])],
                "dW": [_exact_values(d.t().contiguous(), f) @ _exact_decode(x, e, case["m"]).t().contiguous()
                       for d, x, e in zip(s["dY"], s["xt_codes"], s["xt_scales"])]}
    name = "X" if case["dir"] == "forward" else "dY"
    w, e = ("w_codes", "w_scales") if case["dir"] == "forward" else ("wt_codes", "wt_scales")
    along = k if case["dir"] == "forward" else case["n"]
    rows, dw, at, block = [], [], 0, 0
    for g, c in enumerate(s["sizes"]):
        x = s[name][at:at + c]
        if c:
            rows.append(_exact_values(x, f) @ _exact_decode(s[w][g], s[e][g], along).t().contiguous())
        if case["dir"] == "backward":
            blocks = (c + BLOCK - 1) // BLOCK
            if c:
                xt = _exact_decode(s["xt_codes"][2 * block:2 * (block + blocks)], s["xt_scales"][block:block + blocks], c)
                dw.append(_exact_values(x.t().contiguous(), f) @ xt.t().contiguous())
            else:
                dw.append(torch.zeros(case["n"], k, dtype=torch.float64, device="cuda"))
            block += blocks
        at += c
    return torch.cat(rows) if case["dir"] == "forward" else {"dX": torch.cat(rows), "dW": dw}
