"""Edges of windowed attention, page weights, eviction and draft verification on the GPU, against the
plain forms of tests/_more.py."""
import math

import numpy as np
import pytest
import torch

import _more as M
import _pages as P
from test_gpu_more import (I32, SCALE, Cache, Tables, a_draft, a_tree, attend_window, check_verify, check_window, i32,
                           normal, pool, run_evict, run_verify)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available()


# ------------------------------------------------------------------ verification
def tiny_rows(V, kind):
    """A row whose values are of the order of the sums' step, 2^-58."""
    v = torch.zeros(V, dtype=torch.float64)
    if kind == "below a step":  # nothing is left of them
        v[:256] = 2.0 ** -59
    elif kind == "between steps":
        v[::3] = 1.75 * 2.0 ** -58
        v[V // 2] = 2.25 * 2.0 ** -57
    elif kind == "at the start":  # behind them the row is empty
        v[:200] = 1.9 * 2.0 ** -58
        v[200] = 0.9 * 2.0 ** -58
    elif kind == "beside one":
        v[1::2] = 1.5 * 2.0 ** -58
        v[5] = 1.0
    return v.float()


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("kind", ["below a step", "between steps", "at the start", "beside one"])
@pytest.mark.parametrize("V", [700, 245760, 245761, 500000])
def test_verify_values_near_a_step_of_the_sums(pool, V, kind, draft):
    """Each value counts in whole steps of 2^-58, in the sums and in the search alike: the result is
    the same integer arithmetic at every length, and next_token is always written."""
    B = 5
    row = tiny_rows(V, kind)
    u0 = torch.tensor([0.0, 0.3, 0.5, 0.99, 1 - 2.0 ** -24])
    if draft:
        # the token of node 1 has no chance: p - q is what is drawn from
        p = row.expand(B, 2, V).clone()
        q = (row * (1 + 2.0 ** -23) * 0.5).expand(B, 1, V).clone()
        token = int((row == 0).nonzero()[-1]) if bool((row == 0).any()) else V - 1
        p[..., token], q[..., token] = 0.0, 0.5
        tokens = torch.full((B, 2), token, dtype=torch.int32)
        u = torch.stack([u0, torch.full((B,), 0.5)], 1)
        x = (tokens.cuda(), p.cuda(), q.cuda(), None, u.cuda())
    else:
        x = (torch.zeros(B, 1, dtype=torch.int32).cuda(), row.expand(B, 1, V).contiguous().cuda(), None, None, u0[:, None].cuda())
    got = run_verify(pool, *x)
    fixed = [M.fixed(v) for v in row.tolist()]
    if draft:
        minus = [M.fixed(v) for v in x[2][0, 0].tolist()]
        fixed = [M.fixed(v) for v in x[1][0, 0].tolist()]
        rest = [max(a - b, 0) for a, b in zip(fixed, minus)]
        fixed = rest if sum(rest) else fixed
    want = [M.draw(fixed, float(v)) for v in u0]
    assert got[1] == [1] * B and got[2] == want
    assert pool.get_error() == (0 if sum(fixed) else pool.hs.HS_DEVERR_INDEX_RANGE)
