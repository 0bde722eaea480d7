"""What token log probabilities and distillation refuse, before any device call, and the sizes of their workspaces."""

import ctypes

import pytest

from test_learned_neural_amd import atlasmem as am

P = [0x1000_0000 * (i + 1) for i in range(10)]  # addresses apart from each other, aligned
N, D, V, K = 12, 16, 40, 4


def logprobs(**kw):
    a = dict(X=P[0], W=P[1], dtype=am.BF16, n=N, d=D, vocab=V, scale=1.0, tokens=P[2], top=K, logprob=P[3], entropy=P[4],
             top_ids=P[5], top_logprobs=P[6], workspace=P[7], bytes=None)
    a.update(kw)
    if a["bytes"] is None:
        a["bytes"] = max(am.token_logprobs_workspace_bytes(a["dtype"], a["n"], a["d"], a["vocab"], a["top"]), 0)
    return am.load().atlasmem_token_logprobs(
        a["X"], a["W"], a["dtype"], a["n"], a["d"], a["vocab"], a["scale"], a["tokens"], a["top"], a["logprob"],
        a["entropy"], a["top_ids"], a["top_logprobs"], a["workspace"], a["bytes"], None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), am.E_INVALID), (dict(d=0), am.E_INVALID), (dict(vocab=0), am.E_INVALID), (dict(dtype=2), am.E_INVALID),
    (dict(scale=0.0), am.E_INVALID), (dict(scale=-1.0), am.E_INVALID), (dict(scale=NAN), am.E_INVALID),
    (dict(scale=INF), am.E_INVALID), (dict(scale=2.0 ** -21), am.E_INVALID), (dict(scale=2.0 ** 21), am.E_INVALID),
    (dict(top=-1), am.E_INVALID), (dict(top=41), am.E_INVALID),
    (dict(vocab=100, top=65), am.E_SHAPE), (dict(d=16385), am.E_SHAPE), (dict(n=(1 << 24) + 1), am.E_SHAPE),
    (dict(n=1 << 20, vocab=1 << 19), am.E_SHAPE),
    (dict(X=None), am.E_INVALID), (dict(W=None), am.E_INVALID), (dict(workspace=None), am.E_INVALID),
    (dict(tokens=None), am.E_INVALID),  # a logprob of no token
    (dict(top_ids=None), am.E_INVALID), (dict(top_logprobs=None), am.E_INVALID),
    (dict(workspace=P[7] + 8), am.E_INVALID), (dict(bytes=100), am.E_INVALID),
    (dict(logprob=P[0] + 8), am.E_INVALID), (dict(entropy=P[3] + 4), am.E_INVALID), (dict(top_ids=P[2]), am.E_INVALID),
    (dict(workspace=P[6] - 32), am.E_INVALID),
    (dict(n=0, X=None, workspace=None), am.OK),
    (dict(logprob=None, entropy=None, top=0), am.OK),
])
def test_logprobs(kw, status):
    assert logprobs(**kw) == status


def distill(**kw):
    a = dict(X=P[0], W=P[1], dtype=am.BF16, n=N, d=D, vocab=V, top=K, ids=P[2], teacher=P[3], scale=1.0, loss=P[4],
             lse=P[5], kept=P[6], kept_bytes=None, workspace=P[7], bytes=None)
    a.update(kw)
    size = (a["dtype"], a["n"], a["d"], a["vocab"], a["top"])
    if a["kept_bytes"] is None:
        a["kept_bytes"] = max(am.distillation_kept_bytes(a["dtype"], a["n"], a["vocab"], a["top"]), 0)
    if a["bytes"] is None:
        a["bytes"] = max(am.distillation_workspace_bytes(*size, a["kept"] is not None), 0)
    return am.load().atlasmem_distillation(a["X"], a["W"], *size, a["ids"], a["teacher"], a["scale"], a["loss"], a["lse"],
                                           a["kept"], a["kept_bytes"], a["workspace"], a["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), am.E_INVALID), (dict(d=0), am.E_INVALID), (dict(vocab=0), am.E_INVALID), (dict(dtype=7), am.E_INVALID),
    (dict(scale=0.0), am.E_INVALID), (dict(scale=NAN), am.E_INVALID), (dict(scale=INF), am.E_INVALID),
    (dict(scale=2.0 ** -21), am.E_INVALID), (dict(scale=2.0 ** 21), am.E_INVALID), (dict(top=0), am.E_INVALID), (dict(top=129), am.E_SHAPE), (dict(vocab=(1 << 21) + 1), am.E_SHAPE),
    (dict(d=16385), am.E_SHAPE),
    (dict(X=None), am.E_INVALID), (dict(ids=None), am.E_INVALID), (dict(teacher=None), am.E_INVALID),
    (dict(loss=None), am.E_INVALID), (dict(lse=None), am.E_INVALID), (dict(workspace=None), am.E_INVALID),
    (dict(kept=P[6] + 4), am.E_INVALID), (dict(kept_bytes=64), am.E_INVALID), (dict(bytes=64), am.E_INVALID),
    (dict(loss=P[5]), am.E_INVALID), (dict(kept=P[0]), am.E_INVALID), (dict(lse=P[3] + 4), am.E_INVALID),
    (dict(n=0, X=None, ids=None, workspace=None), am.OK),
])
def test_distillation(kw, status):
    assert distill(**kw) == status


def backward(**kw):
    a = dict(X=P[0], W=P[1], dtype=am.F32, n=N, d=D, vocab=V, top=K, kept=P[2], kept_bytes=None, dloss=P[3], dX=P[4],
             dW=P[5], workspace=P[6], bytes=None)
    a.update(kw)
    size = (a["dtype"], a["n"], a["d"], a["vocab"], a["top"])
    if a["kept_bytes"] is None:
        a["kept_bytes"] = max(am.distillation_kept_bytes(a["dtype"], a["n"], a["vocab"], a["top"]), 0)
    if a["bytes"] is None:
        a["bytes"] = max(am.distillation_workspace_bytes(*size, True), 0)
    return am.load().atlasmem_distillation_backward(a["X"], a["W"], *size, a["kept"], a["kept_bytes"], a["dloss"], a["dX"],
                                                    a["dW"], a["workspace"], a["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), am.E_INVALID), (dict(top=0), am.E_INVALID), (dict(top=300), am.E_SHAPE), (dict(dtype=5), am.E_INVALID),
    (dict(X=None), am.E_INVALID), (dict(W=None), am.E_INVALID), (dict(kept=None), am.E_INVALID),
    (dict(workspace=None), am.E_INVALID), (dict(kept_bytes=8), am.E_INVALID), (dict(bytes=8), am.E_INVALID),
    (dict(kept=P[2] + 8), am.E_INVALID), (dict(workspace=P[6] + 8), am.E_INVALID),
    (dict(dX=P[0]), am.E_INVALID), (dict(dW=P[1] + 4), am.E_INVALID), (dict(dX=P[5]), am.E_INVALID),
    (dict(dW=P[2] + 16), am.E_INVALID), (dict(dX=P[3]), am.E_INVALID),
    (dict(dX=None, dW=None), am.OK),
    (dict(n=0, X=None, W=None, kept=None, workspace=None, dW=None), am.OK),
])
def test_distillation_backward(kw, status):
    assert backward(**kw) == status


@pytest.mark.parametrize("size", [(9, 1, 1, 1, 1), (am.BF16, -1, 1, 1, 1), (am.BF16, 1, 0, 1, 1), (am.BF16, 1, 1, 0, 0),
                                  (am.F32, 1 << 24, 1, 1 << 24, 1), (am.F32, 4, 4, 200, -1), (am.F32, 4, 4, 200, 129)])
def test_sizes_that_are_refused(size):
    assert am.token_logprobs_workspace_bytes(*size) == -1
    assert am.distillation_workspace_bytes(*size) == -1
    if size[2] > 0:  # d is no size of what is kept
        assert am.distillation_kept_bytes(size[0], size[1], size[3], size[4]) == -1


def test_the_binding_raises():
    x = ctypes.create_string_buffer(4096)
    at = ctypes.addressof(x)
    with pytest.raises(am.AtlasMemError, match="atlasmem_token_logprobs"):
        am.token_logprobs(at, at, am.BF16, 1, 1, 1, None, at, None, None, stream=0)
    with pytest.raises(am.AtlasMemError, match="atlasmem_distillation"):
        am.distillation(at, at, am.BF16, 1, 1, 1, 0, at, at, 1.0, at, at, None, stream=0)
    with pytest.raises(am.AtlasMemError, match="atlasmem_distillation_backward"):
        am.distillation_backward(None, None, am.BF16, 1, 1, 1, 1, None, None, at, None, None, stream=0)


@pytest.mark.parametrize("n,d,vocab", [(1, 1024, 50257), (8192, 2048, 65536), (65536, 1024, 131072)])
def test_workspaces_hold_no_logits(n, d, vocab):
    """Copies of the rows, and for each row and 64 classes (fewer of few rows) their four largest logits, 16 bytes, and
    4 and 2 for the sums and maxima of four such groups."""
    rows = 2 * (n + vocab) * d
    least = 16 if n * vocab < 1 << 22 else 64
    assert am.token_logprobs_workspace_bytes(am.BF16, n, d, vocab, 20) <= \
        rows + n * (vocab // least + 4) * 22 + vocab + 20 * n + (1 << 20)
    # of an entry its log probability and its probability, 4 bytes each
    assert am.distillation_workspace_bytes(am.BF16, n, d, vocab, 32) <= \
        rows + n * (8 * (vocab // (4 * least) + 1) + 8 * 32 + 24) + (1 << 20)
    assert am.distillation_kept_bytes(am.BF16, n, vocab, 32) <= 2 * n * (vocab + 64) + 16 * n + (1 << 20)


def test_largest_calls_keep_large_tiles():
    """Many rows of few classes: 64 x 64 tiles (88 bytes a row and tile) would need 2^33 lanes of a grid that holds 2^32."""
    n, vocab = 1 << 24, 8192
    large = am.token_logprobs_workspace_bytes(am.BF16, n, 8, vocab, 64)
    assert large <= n * (88 * (vocab // 128) + 64) + (1 << 24)
    small = am.token_logprobs_workspace_bytes(am.BF16, n >> 10, 8, vocab, 64)  # 64-wide tiles, as far as they go
    assert small >= (n >> 10) * 88 * (vocab // 64)
