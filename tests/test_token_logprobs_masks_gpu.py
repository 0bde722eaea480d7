"""Masks of ordinary finite values, a column of W that holds -1e4 or -1e9 for hidden classes: they cost what the lowest float
costs, and hide as much as they say."""

import numpy as np
import pytest

from helpers import DEV, log
from oracle import token_logprobs as oracle
from test_learned_neural_amd import atlasmem as am
from test_token_logprobs_gpu import Case, check

pytestmark = pytest.mark.gpu


def masked(dtype, n, d, vocab, mask, top=20, share=0.4, rows=None):
    """Classes hidden by column 7, which is one in `rows` (all of them) and zero in the others."""
    import torch
    c = Case(dtype, n, d, vocab, top=top, masked=0.0)
    hidden = np.random.default_rng(1).random(vocab) < share
    c.X[:, 7] = 1.0 if rows is None else torch.from_numpy(rows.astype(np.float32)).to(c.X.dtype)
    c.W[:, 7] = 0.0
    c.W[hidden, 7] = mask
    c.tokens = np.where(~hidden)[0][np.arange(n) % (~hidden).sum()]
    return c


def least_time(c):
    import torch
    t, o, ws = c.tensors(), c.outputs(), c.workspace()
    times = []
    for i in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        c.call(t, o, ws)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times[2:])


@pytest.mark.parametrize("dtype,n,d,vocab", [(am.BF16, 5, 1024, 20011), (am.BF16, 300, 512, 5003), (am.BF16, 1100, 1024, 32003),
                                             (am.F32, 40, 1024, 9001), (am.F32, 500, 512, 9001)])
@pytest.mark.parametrize("some", [False, True])
def test_finite_masks_do_not_widen_the_bounds(dtype, n, d, vocab, some):
    """Classes that are computed in 64 bits cost time: with a mask's magnitude in its neighbours' bounds, nearly all are."""
    rows = np.arange(n) % 2 if some else None
    lowest = float(np.finfo(np.float32).min) if dtype == am.F32 else -3.3e38
    least = least_time(masked(dtype, n, d, vocab, lowest, rows=rows))
    for mask in (-1e4, -1e9, -1e17, 1e18 * -0.99):
        at = least_time(masked(dtype, n, d, vocab, mask, rows=rows))
        log(f"TIME {dtype} {n} {d} {vocab} {mask}: {at * 1e3:.1f} us, the lowest {least * 1e3:.1f}")
        assert at <= 2.0 * least + 0.02


@pytest.mark.parametrize("dtype,n,d,vocab", [(am.BF16, 64, 2048, 20011), (am.BF16, 500, 512, 9001), (am.F32, 40, 1024, 9001)])
def test_classes_of_zeros_cost_nothing(dtype, n, d, vocab):
    """A vocabulary's padding."""
    c = Case(dtype, n, d, vocab, top=20, masked=0.0)
    least = least_time(c)
    c.W[::50] = 0.0
    at = least_time(c)
    log(f"TIME {dtype} {n} {d} {vocab}: {at * 1e3:.1f} us, without {least * 1e3:.1f}")
    assert at <= 1.3 * least + 0.01


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e17, -1e19])
@pytest.mark.parametrize("n,d,vocab", [(6, 40, 900), (90, 130, 2000), (1200, 72, 16003)])
def test_masked_in_some_rows(dtype, mask, n, d, vocab):
    check(masked(dtype, n, d, vocab, mask, top=12, share=0.8, rows=np.arange(n) % 2), plain32=True)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -20, 1024.0])
@pytest.mark.parametrize("n,vocab", [(4, 900), (1100, 9000)])
def test_what_is_a_masked_class(dtype, scale, n, vocab):
    """A product of 1e32 or more below the row's largest is no alternative, one of less is, whatever the scale."""
    import torch
    hidden = np.random.default_rng(1).permutation(vocab)[3:]
    for mask, there in ((-1.5e32, False), (-1e36, False), (-0.7e32, True), (-1e20, True)):
        c = Case(dtype, n, 32, vocab, top=8, masked=0.0, scale=scale)
        c.X[:, 7] = 1.0
        c.W[:, 7] = 0.0
        c.W[hidden, 7] = mask
        c.tokens = np.setdiff1d(np.arange(vocab), hidden)[np.arange(n) % 3]
        o = c.run()
        X, W = c.X.double().numpy(), c.W.double().numpy()
        ids = oracle.forward(X, W, c.tokens, scale, 8)[2]
        assert ((ids >= 0).sum(1) == (8 if there else 3)).all()
        assert np.array_equal(o[2].cpu().numpy(), ids), (mask, (o[2].cpu().numpy() != ids).sum())
        assert torch.isfinite(o[0]).all() and (torch.isneginf(o[3]).sum(1) == (0 if there else 5)).all()


@pytest.mark.parametrize("n", [70, 1100])
def test_rows_without_a_class_beside_others(n):
    """Logits that overflow to minus infinity in every tenth row: the others are what they are without the mask."""
    import torch
    c = Case(am.BF16, n, 24, 2500, top=6, masked=0.1)
    none = torch.arange(n) % 10 == 3
    c.X[:, 7] = 0.0
    c.W[:, 7] = 0.0
    a = c.run()
    c.X[none, 7] = 4.0
    c.W[:, 7] = float(torch.finfo(torch.bfloat16).min)
    b = c.run()
    off = torch.from_numpy(c.tokens < 0)
    keep, none = (~none).to(DEV), (none & ~off).to(DEV)
    assert all(torch.equal(x[keep], y[keep]) for x, y in zip(a, b))
    assert torch.isneginf(b[0][none]).all() and not b[1][none].any()
    assert (b[2][none] == -1).all() and torch.isneginf(b[3][none]).all()
