"""The fp64 oracles of token log probabilities and distillation: against torch in fp64 (log-softmax, its entropy, a sort,
KL divergence and autograd), against central differences, and at rows and entries that are left out."""

import numpy as np
import pytest
import torch

from oracle import cross_entropy as ce
from oracle import distillation as ds
from oracle import token_logprobs as tl


def inputs(seed=0, n=9, d=7, vocab=23):
    rng = np.random.default_rng(seed)
    return rng, rng.standard_normal((n, d)), rng.standard_normal((vocab, d))


@pytest.mark.parametrize("scale", [1.0, 0.5, 1.75])
def test_logprobs_against_torch(scale):
    rng, X, W = inputs()
    tokens = rng.integers(0, 23, 9)
    logprob, entropy, ids, logs = tl.forward(X, W, tokens, scale, 6)
    logq = torch.log_softmax(torch.from_numpy(scale * (X @ W.T)), 1)
    want = torch.sort(logq, 1, descending=True)
    assert np.allclose(logprob, logq[torch.arange(9), torch.from_numpy(tokens)], rtol=0, atol=1e-13)
    assert np.allclose(entropy, torch.distributions.Categorical(logits=logq).entropy(), rtol=0, atol=1e-13)
    assert np.array_equal(ids, want.indices[:, :6]) and np.allclose(logs, want.values[:, :6], rtol=0, atol=1e-13)


def test_equal_logits_go_to_the_lowest_index():
    X = np.array([[1.0, 0.0], [0.0, 0.0]])
    W = np.array([[2.0, 1.0], [3.0, 0.0], [2.0, 5.0], [3.0, 1.0]])
    _, _, ids, logs = tl.forward(X, W, None, 1.0, 4)
    assert ids.tolist() == [[1, 3, 0, 2], [0, 1, 2, 3]]
    assert np.allclose(logs[1], -np.log(4.0))


def test_masked_classes_and_rows_left_out():
    X = np.ones((2, 1))
    W = np.array([[-np.inf], [1.0], [-3.4e38], [0.0]])
    logprob, entropy, ids, logs = tl.forward(X, W, np.array([1, -5]), 1.0, 3)
    p = 1.0 / (1.0 + np.exp(-1.0))
    assert ids.tolist() == [[1, 3, -1], [-1, -1, -1]]
    assert np.allclose(logs, [[np.log(p), np.log(1 - p), -np.inf], [0, 0, 0]])
    assert np.allclose(logprob, [np.log(p), 0]) and np.allclose(entropy, [-p * np.log(p) - (1 - p) * np.log(1 - p), 0])


def teacher_of(rng, n=9, top=5, vocab=23):
    ids = np.stack([rng.permutation(vocab)[:top] for _ in range(n)])
    return ids, 3.0 * rng.standard_normal((n, top))


@pytest.mark.parametrize("scale", [1.0, 0.25])
def test_distillation_against_torch_autograd(scale):
    rng, X, W = inputs(1)
    ids, t = teacher_of(rng)
    w = rng.standard_normal(9)
    x, v = torch.from_numpy(X).requires_grad_(), torch.from_numpy(W).requires_grad_()
    target = torch.zeros(9, 23, dtype=torch.float64).scatter_(1, torch.from_numpy(ids),
                                                              torch.softmax(torch.from_numpy(scale * t), 1))
    logq = torch.log_softmax(scale * (x @ v.T), 1)
    loss = torch.nn.functional.kl_div(logq, target, reduction="none").sum(1)
    (loss * torch.from_numpy(w)).sum().backward()
    got, lse = ds.forward(X, W, ids, t, scale)
    assert np.allclose(got, loss.detach(), rtol=0, atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(scale * (x @ v.T), 1).detach(), rtol=0, atol=1e-13)
    dX, dW = ds.backward(X, W, ids, t, scale, w)
    assert np.allclose(dX, x.grad, rtol=0, atol=1e-13) and np.allclose(dW, v.grad, rtol=0, atol=1e-13)


def test_distillation_against_differences():
    rng, X, W = inputs(2, n=4, d=3, vocab=6)
    ids, t = teacher_of(rng, 4, 3, 6)
    ids[1, 2] = ids[1, 0]   # one class twice
    ids[2, 1], t[3, 0] = -1, -np.inf
    w = rng.standard_normal(4)
    dX, dW = ds.backward(X, W, ids, t, 0.7, w)
    h = 1e-6
    for A, got in ((X, dX), (W, dW)):
        want = np.zeros_like(A)
        for i in np.ndindex(A.shape):
            kept = A[i]
            A[i] = kept + h
            up = ds.forward(X, W, ids, t, 0.7)[0] @ w
            A[i] = kept - h
            want[i] = (up - ds.forward(X, W, ids, t, 0.7)[0] @ w) / (2 * h)
            A[i] = kept
        assert np.allclose(got, want, rtol=0, atol=1e-8)


def test_one_sure_class_is_cross_entropy():
    rng, X, W = inputs(3)
    labels = rng.integers(0, 23, 9)
    labels[4] = -100
    ids = np.stack([labels, rng.integers(0, 23, 9)], 1)
    t = np.stack([np.zeros(9), np.full(9, -np.inf)], 1)
    w = rng.standard_normal(9)
    assert np.allclose(ds.forward(X, W, ids, t, 1.0), ce.forward(X, W, labels), rtol=0, atol=1e-13)
    for a, b in zip(ds.backward(X, W, ids, t, 1.0, w), ce.backward(X, W, labels, w)):
        assert np.allclose(a, b, rtol=0, atol=1e-13)


def test_rows_without_an_entry_are_left_out():
    rng, X, W = inputs(4)
    ids, t = teacher_of(rng)
    ids[0], t[1] = -1, -np.inf
    ids[2] = 23
    loss, lse = ds.forward(X, W, ids, t, 1.0)
    dX, dW = ds.backward(X, W, ids, t, 1.0, np.ones(9))
    assert not loss[:3].any() and not lse[:3].any() and not dX[:3].any()
    X[:3] = np.nan
    again = ds.backward(X, W, ids, t, 1.0, np.ones(9))
    assert np.array_equal(again[0], dX) and np.array_equal(again[1], dW)
