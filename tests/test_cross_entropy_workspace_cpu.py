"""How much workspace cross entropy asks for: copies of its rows, a pair of numbers for each row and tile of
classes, and pieces of G that are 256 MB or, of many rows, 2048 classes."""

import pytest

from test_learned_neural_amd import atlasmem as am

SPARE = 1 << 20
EL = {am.BF16: 2, am.F32: 4}


@pytest.mark.parametrize("dtype,side", [(am.BF16, 256), (am.F32, 128)])
@pytest.mark.parametrize("n,d,vocab", [(262144, 2048, 131072), (8192, 2048, 65536), (65536, 1024, 50257)])
def test_forward_keeps_a_pair_for_each_row_and_tile(dtype, side, n, d, vocab):
    rows = EL[dtype] * (n + vocab) * d
    got = am.cross_entropy_workspace_bytes(dtype, n, d, vocab, False)
    assert rows + 8 * n * (vocab // side) <= got <= rows + 8 * n * (vocab // side + 1) + 16 * n + SPARE


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,d,vocab", [(262144, 2048, 131072), (8192, 2048, 65536), (30000, 1024, 50257), (1, 64, 1 << 24)])
def test_backward_keeps_pieces_of_g(dtype, n, d, vocab):
    el = EL[dtype]
    rows = el * (n + vocab) * d
    piece = max(256 << 20, 2048 * n * el)
    sums = 4 * n * d * max(1, -(-512 * 128 * 128 // (n * d)))  # dX's, in pieces of the contraction that fill the chip
    assert am.cross_entropy_workspace_bytes(dtype, n, d, vocab, True) <= rows + 2 * piece + 2 * sums + 16 * n + SPARE
