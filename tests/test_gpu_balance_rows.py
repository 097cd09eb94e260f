"""Every row's share of the experts' balance loss.  Rows that are all one expert (logits 0 and -1000: p is exactly 1 and 0)
add exactly that expert's f, so that the bound is a few roundings, far under what one row adds, and a row that was left
out or taken twice shows at any size."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# (one block; one lane a row; 2 .. 64 lanes; two spans a lane; several sequences; several rows a thread)
@pytest.mark.parametrize("S,T,E", [(1, 9, 8), (3, 5, 2), (1, 70000, 8), (1, 20000, 3), (1, 9001, 16), (1, 5003, 30),
                                   (16, 2049, 61), (1, 7001, 100), (1, 4099, 256), (1, 32768, 256), (1, 2003, 512),
                                   (1, 701, 1024), (300, 7, 9)])
def test_every_row_counts_once(S, T, E):
    rng = np.random.default_rng(S * T + E)
    hot = rng.integers(0, E, (S, T))
    chosen = (hot + (rng.random((S, T)) < 0.3)) % E  # not quite the same: f differs from expert to expert
    z = torch.full((S, T, E), -1000.0, device=DEV)
    z.scatter_(2, torch.from_numpy(hot)[..., None].to(DEV), 0.0)
    index = torch.from_numpy(chosen)[..., None].to(DEV)
    f = np.stack([np.bincount(c, minlength=E) for c in chosen]) * (E / T)
    rows = np.take_along_axis(f, hot, 1)  # what each row adds
    dead = [()] + [(s, t) for s, t in {(0, 0), (0, T // 2), (S // 2, T - 1), (S - 1, 0), (S - 1, T - 1), (S - 1, T // 3)}]
    for where in dead:
        y, keep = z, np.ones((S, T))
        if where:  # a row without any expert: its choice counts, it adds nothing
            y = z.clone()
            y[where] = float("-inf")
            keep[where] = 0.0
        for score in ("softmax", "sigmoid"):
            # f is off by 2 half steps (its unit, the distance times it), so is the least f; their sum and a product by p
            # round once each, up to 8 rows a thread 7 times, the coefficient and the result once each: 15 half steps.
            # (A sigmoid of 0 is 1/2 and its sum 1/2, so p is 1 as well.)
            want = (rows * keep).mean(1).mean()
            got = float(mu.expert_balance(y, index, 1.0, score)[0])
            assert abs(got - want) <= 15 * 2.0 ** -24 * want, (where, score, got, want)
            assert 15 * 2.0 ** -24 * want < rows[rows > 0].min() / (S * T) / 2  # one row is more than that
