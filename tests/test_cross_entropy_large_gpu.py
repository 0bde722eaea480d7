"""The forms of a large cross entropy call at sizes as small as they come: a forward that leaves rows out
of its products (from 2e11 operations on), and a bf16 backward over several pieces of the vocabulary."""

import numpy as np
import pytest

from helpers import DEV, log
from test_cross_entropy_gpu import Case, check
from test_learned_neural_amd import atlasmem as am
from xent_bounds import expected, within

pytestmark = pytest.mark.gpu

GATHER = 2e11


def operations(c):
    return 2.0 * c.n * c.d * c.vocab * (1 if c.dtype == am.BF16 else 6)


@pytest.mark.parametrize("dtype,n,d,vocab", [(am.BF16, 2100, 2051, 25000), (am.BF16, 4097, 2048, 12500),
                                             (am.F32, 1100, 769, 20011)])
def test_rows_left_out_of_a_large_forward(dtype, n, d, vocab):
    import torch
    c = Case(dtype, n, d, vocab, masked=0.4)
    assert operations(c) >= GATHER
    left = np.flatnonzero(c.labels < 0)
    c.X[left[::3]] = float("nan")
    c.X[left[1::3]] = float("inf")
    c.labels[left[::2]] = vocab
    log(f"CASE large forward {c.size()}")
    t, o = c.tensors(), c.outputs()
    am.cross_entropy(t[0], t[1], *c.size(), t[2], o[0], o[1], c.workspace(False))
    torch.cuda.synchronize()
    some = np.unique(np.concatenate([np.arange(0, n, 7), np.arange(n - 40, n)]))
    want = expected(c.X.double().numpy()[some], c.W.double().numpy(), c.labels[some], None, dtype == am.BF16)
    for i, name in enumerate(("loss", "lse")):
        within(name, o[i].cpu()[torch.from_numpy(some)], *want[name])
    assert not o[0].cpu()[torch.from_numpy(left)].any() and not o[1].cpu()[torch.from_numpy(left)].any()


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_all_rows_left_out_of_a_large_forward(dtype):
    import torch
    c = Case(dtype, 3000, 1000, 40000, masked=1.1)
    assert operations(c) >= GATHER
    c.X[:] = float("nan")
    t, o = c.tensors(), c.outputs()
    am.cross_entropy(t[0], t[1], *c.size(), t[2], o[0], o[1], c.workspace(False))
    torch.cuda.synchronize()
    assert not o[0].any() and not o[1].any()


@pytest.mark.parametrize("d", [32, 21])
def test_bf16_pieces_of_the_vocabulary(d):
    """A piece of 256 MB of 22000 rows holds 5888 classes: two pieces of 3328 and 3173."""
    c = Case(am.BF16, 22000, d, 6501)
    log(f"CASE bf16 pieces {c.size()}")
    check(c)
