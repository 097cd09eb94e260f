"""fp64 reference of the experts' balance loss (numpy, no code shared with the library).

Definition as in include/muon.h: muon_expert_balance."""
import numpy as np


def scores(z, score):
    """p and dp_e / dz_e's factor of the gradient (slope) for rows of float64 logits."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if score == "softmax":
            m = z.max(-1, keepdims=True)
            e = np.exp(z - np.where(np.isneginf(m), 0.0, m))
            total = e.sum(-1, keepdims=True)
            p = np.where(total == 0, 0.0, e / total)
            return p, p
        t = np.exp(-np.abs(z))
        q = np.where(z < 0, t, 1.0) / (1.0 + t)
        total = q.sum(-1, keepdims=True)
        p = np.where(total == 0, 0.0, q / total)
        return p, np.where(total == 0, 0.0, t / (1.0 + t) ** 2 / total)


def balance(z, index, coefficient, score="softmax", mask=None):
    """(loss, counts, gradient) of (sequences, tokens, experts) float64 logits."""
    S, T, E = z.shape
    K = index.shape[-1]
    mask = np.ones((S, T), bool) if mask is None else np.asarray(mask) != 0
    grad, counts, loss = np.zeros_like(z), np.zeros(E, np.int64), 0.0
    for s in range(S):
        rows = z[s][mask[s]]
        if len(rows) == 0:
            continue
        chosen = index[s][mask[s]].ravel()
        count = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
        f = E * count / (K * len(rows))
        p, slope = scores(rows, score)
        inner = p @ f
        loss += coefficient / S * inner.mean()
        grad[s][mask[s]] = coefficient / (S * len(rows)) * slope * (f - inner[:, None])
        counts += count
    return loss, counts, grad


def tolerance(z, index, coefficient, score="softmax", mask=None):
    """Bounds of the rounding of (loss, gradient) computed in fp32 as the definition has it.

    u = 2^-24.  exp of an argument off by half a step of itself, |z - max| u, and a function good to 2 steps: e is off by
    (|z - max| + 4) u of itself (sigmoids: |z| in its place, and 4 u more for the sum and the quotient).  The sum of E terms
    adds E u, quotient and product 3 u: p is off by d = (D + E + 12) u, D the largest such argument of the row, infinite
    ones aside (their exp is exactly 0).  f is off by 3 u.  <f, p> is a sum of E terms that are not negative: (d + (E + 4)
    u) of itself.  The slope of the sigmoid is off by 2 d.  A gradient is slope (f - inner) by with by off by 4 u:
      |g| error <= by slope ((f + inner) (3 u + d + (E + 4) u) + |f - inner| (2 d + 8 u)).
    A block's threads add up to N terms in fp32, N the tokens of a sequence at the most: the loss is off by its parts'
    (d + (N + E + 8) u) of itself."""
    u = 2.0 ** -24
    S, T, E = z.shape
    K = index.shape[-1]
    mask = np.ones((S, T), bool) if mask is None else np.asarray(mask) != 0
    bound, loss_bound = np.zeros_like(z), 0.0
    for s in range(S):
        rows = z[s][mask[s]]
        if len(rows) == 0:
            continue
        chosen = index[s][mask[s]].ravel()
        f = E * np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E) / (K * len(rows))
        p, slope = scores(rows, score)
        with np.errstate(invalid="ignore"):
            far = np.abs(rows - rows.max(-1, keepdims=True)) if score == "softmax" else np.abs(rows)
        far = np.where(np.isfinite(far), far, 0.0).max(-1, keepdims=True)
        d = (far + E + 12) * u
        inner = (p @ f)[:, None]
        by = abs(coefficient) / (S * len(rows))
        # what is under fp32's normal range keeps no relative accuracy: 2^-126 of each p, so sum f 2^-126 of <f, p>
        bound[s][mask[s]] = by * ((slope + 2.0 ** -126) * ((f + inner) * (3 * u + d + (E + 4) * u) +
                                                          np.abs(f - inner) * (2 * d + 8 * u) + f.sum() * 2.0 ** -126) +
                                  2.0 ** -126 * (f + inner)) + 2.0 ** -149
        loss_bound += abs(coefficient) / S * (inner * (d + (len(rows) + E + 8) * u)).mean()
    return loss_bound + 2.0 ** -149, bound
