"""The roundings that a bf16 training step's G has, read off dX of an identity for W, whose sums are one term each: q as it is
kept (ten significant bits, 2^-10) and G (2^-8), of the given classes G's alone; fp32 calls have none but those of sums."""

import numpy as np
import pytest

from helpers import log
from test_distillation_gpu import Case
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,vocab,scale", [(40, 64, 1.0), (200, 600, 1.0), (333, 1000, 0.5), (70, 2048, 1.0)])
def test_roundings_of_g(dtype, n, vocab, scale):
    import torch
    c = Case(dtype, n, vocab, vocab, top=6, masked=0.1, scale=scale, weights=False)
    c.W = torch.eye(vocab).to(c.W.dtype)
    X = c.X.double().numpy()
    z = scale * X
    q = np.exp(z - z.max(1, keepdims=True))
    q /= q.sum(1, keepdims=True)
    given = (c.ids >= 0) & (c.teacher != -np.inf)
    on = given.any(1)
    t = np.where(given, scale * np.where(given, c.teacher, 0.0).astype(np.float64), -np.inf)
    p = np.exp(t - np.where(on, t.max(1), 0.0)[:, None])
    p = np.where(given, p / np.where(on, p.sum(1), 1.0)[:, None], 0.0)
    G = np.where(on[:, None], q, 0.0)
    at = np.zeros(G.shape, dtype=bool)
    for i in np.where(on)[0]:
        G[i, c.ids[i][given[i]]] -= p[i][given[i]]
        at[i, c.ids[i][given[i]]] = True
    got = c.run()[2].double().cpu().numpy()
    # exponents: z exact, differences, products and exponentials of up to 20 binary orders and sums over the classes
    sums = 400 * U * (q + at)
    kept, rounded = (2.0 ** -10, 2.0 ** -8) if dtype == am.BF16 else (0.0, 8 * U)
    bound = scale * (sums + np.where(at, rounded * np.abs(G), ((1 + kept) * (1 + rounded) - 1) * q))
    off = np.abs(got - scale * G)
    log(f"ROUNDINGS {dtype} {n} {vocab}: {float((off / (bound + 1e-30)).max()):.3f} of the bound, "
        f"others {float((off / (scale * q))[on][~at[on]].max() * 256):.3f} of 2^-8")
    assert (off <= bound).all()
