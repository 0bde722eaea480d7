"""What the numbers of one row say together: equal logits have equal log probabilities, a later alternative's is no larger,
and a token that is an alternative has the same as both."""

import numpy as np
import pytest

from helpers import log
from test_learned_neural_amd import atlasmem as am
from test_token_logprobs_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,d,vocab,top", [(7, 40, 300, 20), (150, 300, 5003, 33), (900, 72, 9001, 24), (2500, 48, 4001, 20),
                                           (1200, 72, 16003, 32)])
def test_a_row_has_one_sum(dtype, n, d, vocab, top):
    import torch
    log(f"CASE {dtype} {n} {d} {vocab} {top}")
    c = Case(dtype, n, d, vocab, top=top, masked=0.0, scale=0.75)
    c.W[vocab // 2:2 * (vocab // 2)] = c.W[:vocab // 2]  # each class twice
    c.W[-1] = 0.0
    z = c.X.double() @ c.W.double().T
    c.tokens = z.topk(top, 1).indices.sort(1).values[torch.arange(n), torch.arange(n) % top].numpy()
    logprob, _, ids, logs = (x.cpu() for x in c.run())
    assert (logs[:, 1:] <= logs[:, :-1]).all()
    half, paired = vocab // 2, ids < 2 * (vocab // 2)
    base = torch.where(paired, ids % half, -1 - ids)
    same = base[:, 1:] == base[:, :-1]
    assert same.sum() > n * (top // 2 - 2) and torch.equal(logs[:, 1:][same], logs[:, :-1][same])
    at = ids == torch.from_numpy(c.tokens)[:, None]
    rows = at.any(1)
    assert rows.sum() > n // 2 and torch.equal(logs[at], logprob[rows])
