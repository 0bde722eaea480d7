"""Alternatives of logits that are nearer than their sums in fp32 round, from inputs of any magnitude: their order is that of
products in 64 bits where squares of the inputs, or products of them, leave the range of a float."""

import numpy as np
import pytest

from helpers import log
from oracle import token_logprobs as oracle
from test_learned_neural_amd import atlasmem as am
from test_token_logprobs_gpu import Case

pytestmark = pytest.mark.gpu

SIZES = [(6, 48, 3000, 900), (300, 48, 3000, 500), (1100, 72, 16003, 3000), (90, 300, 70000, 3000)]


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("x,w", [(0, 0), (0, -85), (-85, 0), (-70, -62), (70, -70), (-80, 80), (90, -90), (-100, 40), (-112, 50), (-128, 58), (-128, 100), (120, -128)])
@pytest.mark.parametrize("n,d,vocab,alike", SIZES)
def test_near_logits_of_any_magnitude(dtype, x, w, n, d, vocab, alike):
    import torch
    log(f"CASE {dtype} {n} {d} {vocab} 2^{x} 2^{w}")
    c = Case(dtype, n, d, vocab, top=30, masked=0.0)
    rng = np.random.default_rng(5)
    gen = torch.Generator().manual_seed(1)
    half = (d - 8) // 2
    row = 0.5 + torch.rand(d, generator=gen)
    c.X = 0.5 + torch.rand(n, d, generator=gen)
    c.X[:, :8] *= 2.0 ** -14
    # sums of 20 and more round at 2^-20 before they come back to zero: what tells alike classes apart is 2^-13
    c.X[:, 8 + half:8 + 2 * half], row[8 + half:8 + 2 * half] = c.X[:, 8:8 + half], -row[8:8 + half]
    row[:8], row[8 + 2 * half:] = -4.0, 0.0
    c.W = row.repeat(vocab, 1)
    at = rng.permutation(vocab)[:alike]
    c.W[at, :8] = 0.5 + torch.rand(alike, 8, generator=gen)
    c.X, c.W = c.X * 2.0 ** x, c.W * 2.0 ** w
    c.X, c.W = (t.to(torch.bfloat16 if dtype == am.BF16 else torch.float32) for t in (c.X, c.W))
    got = c.run()
    _, _, ids, logs = oracle.forward(c.X.double().numpy(), c.W.double().numpy(), c.tokens, c.scale, c.top)
    ids_got = got[2].cpu().numpy()
    assert np.array_equal(ids_got, ids), (ids_got != ids).sum()
    # z as it is summed in fp32, and the sum over the classes: 2 d roundings of it and 200 of 2^-24
    size = 1 + float((c.X.double().abs() @ c.W[at[0]].double().abs()).max())
    assert np.abs(got[3].double().cpu().numpy() - logs).max() <= (2 * d + 200) * 2.0 ** -24 * 4 * size


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,vocab", [(20, 2000), (1100, 16003)])
def test_rows_and_classes_of_zeros(dtype, n, vocab):
    """Every logit of a row of zeros is equal, and those of classes of zeros."""
    c = Case(dtype, n, 72, vocab, top=9, masked=0.0)
    c.X[::3] = 0.0
    c.W[::5] = 0.0
    c.W[:, 10:] = 0.0
    c.X[1::3, :10] = -c.X[1::3, :10].abs()
    c.W[:, :10] = c.W[:, :10].abs()  # the largest logits of these rows are the zeros
    got = c.run()
    ids = oracle.forward(c.X.double().numpy(), c.W.double().numpy(), c.tokens, c.scale, c.top)[2]
    assert np.array_equal(got[2].cpu().numpy(), ids)
