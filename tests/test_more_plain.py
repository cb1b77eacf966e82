"""The plain forms of windowed attention, page weights, eviction and verification, checked by
hand and against each other, and the entry points' host-side refusals (no GPU needed)."""
import ctypes as C
import math
from collections import Counter

import pytest
import torch

import _more as M
import _pages as P


def test_window_mask():
    assert M.window_mask(6, 2, None, 0, 3, 0).tolist() == [False, False, True, True, True, False]
    assert M.window_mask(6, 2, None, 1, 3, 1).tolist() == [True, False, False, True, True, True]
    assert M.window_mask(6, 2, None, 0, 100, 0).tolist() == P.seen_mask(6, 2, None, 0).tolist()
    assert M.window_mask(6, 2, None, 0, 1, 0).tolist() == [False] * 4 + [True, False]
    # two nodes after the context's end, neither the other's ancestor: both at position 4
    tree = [1, 2]
    assert M.window_mask(6, 2, tree, 1, 3, 0).tolist() == [False, False, True, True, False, True]
    chain = [1, 3]
    for t in range(2):
        assert M.window_mask(6, 2, chain, t, 2, 1).tolist() == M.window_mask(6, 2, None, t, 2, 1).tolist()
    assert M.window_mask(6, 2, [1, 0], 1, 2, 0).tolist() == [False, False, True, True, False, False]


def test_page_weights_sum_to_the_query_rows():
    g = torch.Generator().manual_seed(1)
    T, H, L = 3, 2, 150
    q, kv = torch.randn(T, H, P.DIM, generator=g).double(), torch.randn(L, P.DIM, generator=g).double()
    seen = torch.stack([P.seen_mask(L, T, None, t) for t in range(T)])
    lse = torch.stack([P.attention(q[t], kv, seen[t], 0.05)[1] for t in range(T)])
    w = M.page_weights(q, lse, kv, seen, 0.05)
    assert w.shape == (3,) and abs(float(w.sum()) - T * H) < 1e-9
    lse[1, 0] = -math.inf
    assert abs(float(M.page_weights(q, lse, kv, seen, 0.05).sum()) - (T * H - 1)) < 1e-9


def test_evict_plain():
    table, saved = [5, 4, -1, 3, 2, 1], [-1, 0, 0, 0, 0, 0]
    w = [0.0, 1.0, 9.0, 1.0, math.nan, -math.inf]
    assert M.evict(table, saved, w, 6 * 64, 2, 0, 0, False) == ([1, 3], [0, 4, 5])
    assert M.evict(table, saved, w, 6 * 64, 2, 1, 1, False) == ([0, 5], [1, 3, 4])
    assert M.evict(table, saved, w, 6 * 64, 0, 1, 2, False) == ([0, 4, 5], [1, 3])
    assert M.evict(table, saved, w, 6 * 64, 2, 0, 0, True) == ([0, 1], [3, 4, 5])
    assert M.evict(table, saved, w, 6 * 64, 4, 0, 0, False) == ([0, 1, 3, 4], [5])  # NaN as -inf: the lower page
    assert M.evict(table, saved, w, 6 * 64, -1, 0, 0, False) == ([0, 1, 3, 4, 5], [])
    assert M.evict(table, saved, w, 0, 3, 1, 1, False) == ([], [])
    assert M.evict(table, saved, w, 65, 1, 0, 0, False) == ([1], [0])


def test_draw_and_accept_by_hand():
    assert [M.draw([1, 0, 2, 1], u) for u in (0.0, 0.24, 0.25, 0.74, 0.75, 0.99)] == [0, 0, 2, 2, 3, 3]
    assert M.draw([0, 0], 0.5) == -1
    p = [[0.5, 0.25, 0.25], [0.125, 0.125, 0.75]]
    q = [[0.25, 0.5, 0.25]]
    assert M.verify([0, 0], p, q, None, [0.5, 0.999]) == ([0, 1], 2)  # p >= q: always
    assert M.verify([0, 1], p, q, None, [0.0, 0.49]) == ([0, 1], 0)
    assert M.verify([0, 1], p, q, None, [0.9, 0.5]) == ([0], 0)  # all that is left of p - q
    assert M.verify([0, -1], p, q, None, [0.8, 0.0]) == ([0], 2)  # no token: p itself
    assert M.verify([0, 1], p, None, None, [0.7, 0.25]) == ([0], 2)  # refused: token 1 is out
    assert M.verify([0, 1], p, None, None, [0.7, 0.24]) == ([0, 1], 2)
    # two children of node 0: the second is held against what the first left
    tree = [1, 3, 5]
    p3 = p + [[0.0, 1.0, 0.0]]
    assert M.verify([0, 1, 0], p3, None, tree, [0.0, 0.5, 0.66]) == ([0, 2], 1)
    assert M.verify([0, 1, 0], p3, None, tree, [0.0, 0.5, 0.67]) == ([0], 2)
    assert M.verify([0, 1, 1], p3, None, tree, [0.0, 0.5, 0.0]) == ([0], 0)  # a token twice
    assert M.verify([0, 1], [[0.0] * 3] * 2, None, None, [0.3, 0.3]) == ([0], -1)


@pytest.mark.parametrize("kind", ["draft", "chain", "tree"])
def test_verification_keeps_the_targets_distribution(kind):
    """Over a grid of random numbers the first token after node 0 is distributed as p."""
    n = 24
    p0 = [0.5, 0.125, 0.25, 0.125]
    count = Counter()
    grid = [(i + 0.5) / n for i in range(n)]
    if kind == "draft":  # the draft's token drawn from q first
        q0 = [0.25, 0.5, 0.25, 0.0]
        for x, w in enumerate(q0):
            for a in grid:
                for b in grid:
                    path, nxt = M.verify([0, x], [p0, p0], [q0], None, [a, b])
                    count[x if len(path) > 1 else nxt] += w / n ** 2
    else:
        tree = [1, 3] if kind == "chain" else [1, 3, 5]
        tok = [0, 1] if kind == "chain" else [0, 1, 2]
        for a in grid:
            for b in grid:
                for c in grid if kind == "tree" else [0.0]:
                    path, nxt = M.verify(tok, [p0] * 3, None, tree, [a, b, c][:len(tok)])
                    count[tok[path[1]] if len(path) > 1 else nxt] += 1 / n ** len(tok)
    for v in range(4):
        # each of three draws on a grid of 24 is off by at most one cell
        assert abs(count[v] - p0[v]) <= 3 / n


def test_entry_points_refuse_a_null_pool():
    import __graft_entry__ as g
    g.build()
    import tiered_sparse_mla_gb300 as hs
    lib = hs.load()
    p = C.cast((C.c_int32 * 64)(), C.c_void_p)
    f = C.c_float(0.1)
    inval = hs.HS_ERR_INVALID_ARG
    assert lib.hs_page_mla_decode_window(None, 1, 1, 16, 64, 4, p, p, None, f, p, p, None, 0, None) == inval
    assert lib.hs_page_weights(None, 1, 1, 16, p, p, p, None, f, f, None, p, None, 0, None) == inval
    assert lib.hs_evict_pages(None, 1, 4, 1, 1, 0, p, p, p, p, p, p, None) == inval
    assert lib.hs_verify_drafts(None, 1, 2, 8, 0, p, 8, p, 8, p, None, p, p, p, p, None) == inval
    assert lib.hs_window_workspace_bytes(None, 1, 1, 16, 64, 4) == 0
    assert lib.hs_weights_workspace_bytes(None, 1, 32, 16) == 0


def test_bindings_take_rows_of_wider_buffers(monkeypatch):
    import tiered_sparse_mla_gb300 as hs

    class OnDevice(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

    monkeypatch.setattr(hs, "_only_device", 0)

    def rows(t, *a):
        return hs._prob_rows("x", t.as_subclass(OnDevice), *a)

    wide = torch.zeros(2, 3, 40)
    assert rows(wide, 2, 3, 40) == (wide.data_ptr(), 40, hs.HS_PROB_F32)
    assert rows(wide[..., 1:38], 2, 3, 37) == (wide.data_ptr() + 4, 40, hs.HS_PROB_F32)
    assert rows(wide[:, :1, :37], 2, 1, 37)[1] == 120
    assert rows(wide.to(torch.bfloat16), 2, 3, 40)[1:] == (40, hs.HS_PROB_BF16)
    assert rows(torch.zeros(2, 0, 40), 2, 0, 40)[:2] == (None, 40)
    for bad in (wide[:, :2], wide.transpose(1, 2), wide[..., ::2], torch.zeros(3, 1).expand(2, 3, 40),
                torch.zeros(1, 1, 40).expand(2, 3, 40), torch.zeros(2, 3, 40, dtype=torch.float64)):
        with pytest.raises(ValueError):
            rows(bad, *(bad.shape if bad.shape[1] == 2 else (2, 3, 40)))
