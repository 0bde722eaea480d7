"""Group norm against the fp64 oracle with the roundings of the form that runs: a sum's longest way in the
one-pass form (a lane's values, then the halving of a team of lanes) or in the two-pass form (spans of
positions in a thread, the threads of a channel, the spans of a group), counted from the sizes."""

import pytest

import test_group_norm_gpu as gn_tests
from helpers import log
from test_group_norm_gpu import CASES, Case, check
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu

LANES, VECTORS = 64, 4


def up(a, b):
    return -(-a // b)


def pow2_from(n):
    p = 1
    while p < n and p < LANES:
        p *= 2
    return p


def longest_way(n, L, C, G):
    """(form, roundings): what a channel count allows as vector width, tensors being whole allocations."""
    c = C // G
    V = 8 if c % 8 == 0 else 4 if c % 4 == 0 else 1
    vecs = up(c, V)
    across = pow2_from(vecs)
    if (vecs <= LANES * VECTORS) if L == 1 else (vecs <= LANES and L <= LANES // across * VECTORS):
        team = pow2_from(across * L)
        each = up(vecs, team) if L == 1 else up(L * across, team)
        each = each if each <= 2 else 4
        return "one pass", each * V + team.bit_length() + 2
    s = max(1, min(max(1, 1024 // n), up(L, 16)))
    span = up(L, s)
    splits = up(L, span)
    rows = 1 if C // V >= 256 else 256 // (C // V)
    # a union of two partial sums is six roundings; a thread joins blocks of four positions
    moments = 4 * V + 6 * (up(up(span, rows), 4) + rows + up(splits * c // V, 256) + 6 + 4)
    sums = up(span, rows) + rows + up(splits * c, 1024 if splits * c > 1024 else 128) + 6 + 16
    return "two passes", max(moments, sums) + 2


@pytest.mark.parametrize("kw", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_parity(kw, monkeypatch):
    c = Case(**kw)
    form, r = longest_way(c.n, c.L, c.C, c.G)
    log(f"CASE {form}, {r} roundings")
    monkeypatch.setattr(gn_tests, "ways", lambda n, L, C: r)
    check(c)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,L,C,G,form", [
    (300, 1, 512, 4, "one pass"), (50, 1, 2048, 1, "one pass"), (17, 1, 2048 * 2, 2, "one pass"),
    (33, 31, 64, 8, "one pass"), (5, 256, 16, 2, "one pass"), (5, 257, 16, 2, "two passes"),
    (9, 1, 2056, 1, "two passes"), (2, 20011, 24, 3, "two passes"), (1, 40000, 40, 1, "two passes"),
    (2000, 300, 8, 1, "two passes"),
])
def test_parity_at_the_borders_of_the_forms(dtype, n, L, C, G, form, monkeypatch):
    c = Case(dtype, n, L, C, G, True, seed=L + C)
    got, r = longest_way(n, L, C, G)
    log(f"CASE {form}, {r} roundings")
    assert got == form
    monkeypatch.setattr(gn_tests, "ways", lambda n, L, C: r)
    check(c)
