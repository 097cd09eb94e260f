"""README's mixture of experts, run as it stands there, on a padded batch with choices that do not count."""
import os
import re

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu
from oracle import fp8_oracle as fo
from synth import inputs as syn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
f64 = syn.to_f64


def mixture():
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), flags=re.S)
    found = [b for b in blocks if "expert_balance" in b]
    assert len(found) == 1
    return found[0]


@pytest.mark.parametrize("T,E,top", [(64, 4, 1), (150, 6, 2), (333, 5, 3)])
@pytest.mark.parametrize("padded", [False, True])
def test_mixture(T, E, top, padded):
    rng = np.random.default_rng(T)
    dev = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV)  # noqa: E731
    n_in, n_out = 160, 48
    logits, X = dev(T, E), dev(T, n_in)
    index = torch.topk(logits, top, -1).indices
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    if padded:
        mask[T - T // 4:] = False
        mask[T // 2] = False
        index[T // 3, 0] = -1  # a choice that was dropped
        index[T // 5, -1] = E
    W, dH, G = [dev(n_out, n_in) for _ in range(E)], dev(T * top, n_out), [torch.zeros(n_out, n_in, device=DEV) for _ in range(E)]
    w, w_t = mu.fp8_quantize(W, "tile", transpose="both")
    names = dict(mu=mu, torch=torch, logits=logits, index=index, mask=mask, X=X, dH=dH, G=G, w=w, w_t=w_t, E=E)
    exec(mixture(), names)
    counts, H, order = names["counts"].tolist(), names["H"], names["order"]
    flat, kept = index.flatten().tolist(), mask.repeat_interleave(top).tolist()
    assert counts == [sum(1 for e, k in zip(flat, kept) if k and e == want) for want in range(E)]
    at = 0
    for e, c in enumerate(counts):
        mine = order[at:at + c].tolist()
        assert all(kept[i] and flat[i] == e for i in mine), "rows of other experts"
        x64, d64, w64 = f64(X)[np.array(mine, int) // top], f64(dH)[at:at + c], f64(W[e])
        code = lambda x, tile=False: fo.decode(*fo.quantize(x, "e4m3", tile), x.shape[1])  # noqa: E731
        if c:
            for got, (want, bound) in ((H[at:at + c], fo.matmul(code(x64), code(w64, True), eights=True)),
                                       (names["dX"][at:at + c], fo.matmul(code(d64), code(w64, True).T, eights=True))):
                assert np.all(np.abs(f64(got) - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound))
            want, bound = fo.matmul(code(d64.T.copy()), code(x64.T.copy()))
            assert np.all(np.abs(f64(G[e]) - want) <= bound)
        else:
            assert not G[e].any()
        at += c
    assert not H[at:].any() and not names["dX"][at:].any()
