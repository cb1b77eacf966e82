"""Edges of windowed attention, page weights, eviction and draft verification on the GPU, against the
plain forms of tests/_more.py."""
import math

import numpy as np
import pytest
import torch

import _more as M
import _pages as P
from test_gpu_more import (I32, SCALE, Cache, Tables, a_draft, a_tree, attend_window, check_verify, check_weights, check_window, i32,
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


def test_verify_decides_small_probabilities_exactly(pool):
    """u q < p and u s < p, on both sides of equality, for values whose last bits are below any step of the
    sums and for products below f32's normal numbers."""
    ulp = lambda x: float(np.spacing(np.float32(x)))
    chain, draft = [], []  # (u, p) and (u, q, p)
    for e in (-30, -34, -35, -40, -57, -58, -59, -70, -100, -126, -127, -140, -149):
        for m in (1.0, 1.25, 1.9999):
            x = float(np.float32(m * 2.0 ** e))
            if x == 0:
                continue
            chain += [(x, x), (x, x + ulp(x)), (x + ulp(x), x), (max(x - ulp(x), 0.0), x)]
            for q in (1.0, 0.75, 2.0 ** -20, 1.1 * 2.0 ** -60):
                q = float(np.float32(q))
                y = x / q
                for u in (y, y + ulp(y), y - ulp(y), y + 2 * ulp(y)):
                    u = float(np.float32(u))
                    if 0 <= u < 1:
                        draft += [(u, q, x)]
    for cases in (chain, draft):
        B, V = len(cases), 9
        p = torch.zeros(B, 2, V)
        p[:, :, 0] = 0.5
        p[:, 0, 3] = torch.tensor([c[-1] for c in cases], dtype=torch.float64).float()
        tokens = torch.full((B, 2), 3, dtype=torch.int32)
        u = torch.full((B, 2), 0.25)
        u[:, 1] = torch.tensor([c[0] for c in cases], dtype=torch.float64).float()
        q = None
        if cases is draft:
            q = torch.zeros(B, 1, V)
            q[:, 0, 3] = torch.tensor([c[1] for c in cases], dtype=torch.float64).float()
        x = (tokens.cuda(), p.cuda(), None if q is None else q.cuda(), None, u.cuda())
        got = run_verify(pool, *x)
        assert 0.2 * B < got[1].count(2) < 0.9 * B
        check_verify(got, *x)
    # a tree: what an earlier child had is gone first
    cases = [(w, r) for w in (0.5, 0.75, 0.9375) for r in chain]
    B = len(cases)
    p = torch.zeros(B, 3, V)
    p[:, :, 0] = torch.tensor([c[0] for c in cases])[:, None]
    p[:, 0, 3] = torch.tensor([c[1][1] for c in cases], dtype=torch.float64).float()
    tokens = torch.tensor([0, 0, 3], dtype=torch.int32).expand(B, 3).contiguous()
    u = torch.full((B, 3), 0.99)
    u[:, 2] = torch.tensor([min(c[1][0] / (1 - c[0]), 0.9) for c in cases], dtype=torch.float64).float()
    star = torch.tensor([1, 3, 5]).expand(B, 3).contiguous()
    x = (tokens.cuda(), p.cuda(), None, star.cuda(), u.cuda())
    got = run_verify(pool, *x)
    assert 0.2 * B < got[1].count(2) < 0.9 * B
    check_verify(got, *x)
    assert pool.get_error() == 0


# ------------------------------------------------------------------ window
def signed(x):
    return x - (1 << 64) if x >= 1 << 63 else x


def only_seen_pages(c, L, T, trees, window, n_sink):
    """Takes the blocks of all pages away that no query token sees, and fills their rows with NaN."""
    rows, scales = c.pool.gpu_rows(), c.pool.gpu_scales()
    gone = 0
    for b in range(len(L)):
        seen = torch.zeros(L[b], dtype=torch.bool)
        for t in range(T):
            seen |= M.window_mask(L[b], T, trees[b], t, window, n_sink)
        table = c.table[b].copy()
        for page in range(-(-L[b] // 64)):
            if bool(seen[64 * page:64 * page + 64].any()):
                continue
            gone += 1
            block = int(table[page])
            rows[64 * block:64 * block + 64] = 0xFF
            if scales is not None:
                scales[64 * block:64 * block + 64] = math.nan
            table[page] = -1
        c.pool.page_map_range(b, 0, table, table * 0 - 1)
    return gone


@pytest.mark.parametrize("dtype,units", [("bf16", 1), ("fp8", 1), ("bf16", 3)])
@pytest.mark.parametrize("T,window,n_sink,kind", [(4, 100, 0, "tree"), (7, 100, 5, "tree"), (4, 4, 1, "path"), (4, 64, 0, "path"),
                                                  (5, 70, 3, "star"), (6, 80, 0, "empty"), (6, 80, 0, "low"), (63, 64, 0, "path"),
                                                  (64, 64, 0, "tree"), (40, 50, 64, "high"), (3, 2 ** 31 - 1, 0, "path"),
                                                  (9, 20, 0, "random"), (40, 41, 7, "random")])
def test_window_of_a_tree_needs_no_page_that_it_does_not_see(dtype, units, T, window, n_sink, kind):
    """At every alignment of the context's end; with pages of few nodes, and nodes that nobody sees."""
    L = [200 + T + i for i in range(64)] + [T, T + 1, max(1, T - 2), T + 63]
    # 16 heads and more where units are to be taken one after the other
    H = 16 if units == 1 else -(-152 * 2 * 128 // (len(L) * T))
    c = Cache(dtype, L)
    one = (1 << T) - 1
    if kind in ("tree", "path"):
        tree = a_tree(9, len(L), T) if kind == "tree" else torch.tensor(
            [[signed((2 << t) - 1) for t in range(T)]] * len(L)).cuda()
    elif kind == "star":
        tree = torch.tensor([[1 | 1 << t for t in range(T)]] * len(L)).cuda()
    elif kind == "random":
        g = torch.Generator().manual_seed(18)
        tree = (torch.randint(0, 1 << 62, (len(L), T), generator=g) & torch.randint(0, 1 << 62, (len(L), T), generator=g)).cuda()
    else:  # some see no node, or none sees the last nodes, or none the first ones
        bits = {"empty": [0 if t % 2 else 1 << t for t in range(T)], "low": [1] * T, "high": [(1 << t) & ~7 for t in range(T)]}[kind]
        tree = torch.tensor([[x & one for x in bits]] * len(L)).cuda()
    trees = tree.tolist()
    gone = only_seen_pages(c, L, T, trees, window, n_sink)
    assert gone > 30 or window > 200
    q = normal(6, len(L), T, H, P.DIM)
    out, lse = attend_window(c, q, window, n_sink, tree)
    assert c.pool.get_error() == 0
    check_window(c, q, out, lse, window, n_sink, tree, tokens=sorted({0, T // 2, T - 1}))
    c.close()


@pytest.mark.parametrize("kind", ["empty", "unknown"])
def test_window_units_that_end_with_empty_ones(kind):
    """Units one after the other whose last ones have no step: the sums of the unit before are read before
    the empty one's are written. (A race does not show in every run: the results have to be right, and
    the same each time.)"""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    g = torch.Generator().manual_seed(13)
    ctx = [int(x) for x in torch.randint(1, 300, (2 * pairs,), generator=g)] + [0] * pairs
    c = Cache("bf16", ctx)
    q = normal(14, 3 * pairs, 1, 128, P.DIM)
    req = torch.arange(3 * pairs, **I32)
    if kind == "unknown":
        req[2 * pairs:] = -1
    out, lse = attend_window(c, q, 200, 1, req=req)
    check_window(c, q[:2 * pairs], out[:2 * pairs], lse[:2 * pairs], 200, 1)
    assert not out[2 * pairs:].any() and bool((lse[2 * pairs:] == -math.inf).all())
    for _ in range(50):
        again = attend_window(c, q, 200, 1, req=req)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.close(0 if kind == "empty" else c.hs.HS_DEVERR_BAD_REQUEST)


@pytest.mark.parametrize("B,T,H,window", [(160, 1, 128, 4096), (160, 1, 128, 100), (157, 3, 80, 1500), (10, 500, 16, 4096), (3, 1300, 16, 1000)])
def test_window_units_of_uneven_requests(B, T, H, window):
    """Twice as many units as pairs of CTAs and more, of requests of very different lengths: those taken one
    after the other, and those that get CTAs of their own and of which the last are split."""
    g = torch.Generator().manual_seed(16)
    ctx = [T + int(math.exp(x)) for x in (9 * torch.rand(B, generator=g)).tolist()]
    c = Cache("bf16", ctx)
    q = normal(17, B, T, H, P.DIM)
    out, lse = attend_window(c, q, window, 3)
    check_window(c, q, out, lse, window, 3, tokens=sorted({0, T // 3, T // 2, T - 1}))
    again = attend_window(c, q, window, 3)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.close()


@pytest.mark.parametrize("ctx,T,H,window", [([0, 66, 65, 66, 70, 66, 0, 67, 1, 3], 65, 64, 16),
                                            ([0, 1, 53, 55, 1, 1, 52, 80, 52, 81, 159, 1, 53, 112, 53, 1, 79, 53, 58, 53, 645], 52, 40, 818),
                                            ([0] * 100 + [40] * 60 + [0] * 100 + [100] * 100, 1, 128, 64)])
def test_window_units_without_steps_beside_other_work(ctx, T, H, window):
    """Units without steps before and between others, while another stream keeps the GPU busy: no role of a
    pair of CTAs misses what another says (it would wait until the limit: HS_DEVERR_TIMEOUT)."""
    c = Cache("bf16", ctx)
    q = normal(19, len(ctx), T, H, P.DIM)
    out, lse = attend_window(c, q, window, 0)
    check_window(c, q, out, lse, window, 0, tokens=sorted({0, T // 2, T - 1}))
    side, x = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for k in range(30):
        with torch.cuda.stream(side):
            for _ in range(1 + k % 3):
                torch.mm(x[:256 << (k % 4)], x)
        again = attend_window(c, q, window, 0)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,window,n_sink", [(200, 16, 64), (130, 1, 130), (70, 16, 300)])
def test_window_of_sinks_that_are_query_tokens(dtype, T, window, n_sink):
    """Contexts that begin inside the query tokens (a whole prompt, say): the first positions stay visible to
    the later tokens, those among them that are query tokens themselves too; the same by the plain form of
    the measured cases."""
    from perf import more_operators as plain
    case = {"op": "window", "dtype": dtype, "B": 2, "T": T, "H": 16, "ctx": T + 10, "window": window, "sink": n_sink, "tree": False}
    c = Cache(dtype, [T + 10, T], garbage=False)
    q = normal(15, 2, T, 16, P.DIM)
    out, lse = attend_window(c, q, window, n_sink)
    check_window(c, q, out, lse, window, n_sink)
    L = T + 10
    kv = M.window_mask(L, T, None, T - 1, window, n_sink)
    assert int(kv.sum()) == min(L, n_sink + window)  # the last token: none of the sinks is left out
    rows = c.pool.gpu_rows()
    state = {"case": case, "lens": torch.tensor(c.ctx, **I32), "table": torch.from_numpy(c.table).cuda(), "q": q, "tree": None,
             "rows": rows.view(torch.bfloat16) if dtype == "bf16" else rows.view(torch.float8_e4m3fn),
             "scales": None if dtype == "bf16" else c.pool.gpu_scales()}
    assert plain.SCALE == SCALE
    o2, l2 = plain._window(state)
    check_window(c, q, o2, l2, window, n_sink)
    c.close()


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("saved_only", [False, True])
@pytest.mark.parametrize("pages", [513, 2049, 4097, 5000, 8193, 32769, 270000])
def test_evict_releases_pages_of_long_contexts(pages, saved_only):
    """Requests whose pages are dealt to clusters of 1, 2, 4 and 8, and more than fit in their shared
    memory: the table, the host copies and the lists after the call itself."""
    ctx = [pages * 64, pages * 64 - 64 * 17 - 3, 64 * (pages // 3) + 1]
    c = Tables(ctx, seed=pages)
    g = torch.Generator().manual_seed(23)
    w = torch.rand(c.R, c.P, generator=g)
    w[1] = (w[1] * 50).floor()
    want = c.table.copy()
    for budget in (pages - pages // 3, pages // 5, 7):
        kept, freed, count = run_evict(c, [2, 0, 1], [budget] * 3, w.cuda(), c.P, 2, 3, saved_only)
        for i, r in enumerate((2, 0, 1)):
            stay, gone = M.evict(want[r], c.saved[r], w[r].tolist(), ctx[r], budget, 2, 3, saved_only)
            assert kept[i] == stay + [-1] * (c.P - len(stay))
            assert count[i] == len(gone) and freed[i][:len(gone)] == want[r, gone].tolist()
            assert set(freed[i][len(gone):]) <= {-7}
            want[r, gone] = -1
        now = c.now()
        assert np.array_equal(now[..., 0], want) and np.array_equal(now[..., 1], c.saved)
    c.close()


@pytest.mark.parametrize("max_pages", [512, 513, 3000, 16384])
def test_evict_short_requests_of_long_pools(max_pages):
    """The kernel goes by the pool's pages, not by a request's: the same result in any pool."""
    ctx = [0, 1, 64, 65, 2000, 63 * 64, 64 * 64, 300 * 64 + 7]
    c = Tables(ctx, max_ctx=max_pages * 64, seed=3)
    g = torch.Generator().manual_seed(24)
    w = torch.exp(torch.randn(c.R, c.P, generator=g))
    w[4] = 0.5
    for budget in ([0] * 8, [1, 1, 1, 1, 9, 20, 64, 100], [10 ** 9] * 8):
        for plan in (True, False):
            kept, freed, count = run_evict(c, list(range(8)), budget, w.cuda(), 400, 1, 2, False, plan)
            for r in range(8):
                stay, gone = M.evict(c.table[r], c.saved[r], w[r].tolist(), ctx[r], budget[r], 1, 2, False)
                assert kept[r] == stay + [-1] * (400 - len(stay))
                assert count[r] == len(gone) and freed[r][:len(gone)] == c.table[r, gone].tolist()
                if not plan:
                    c.table[r, gone] = -1
            assert np.array_equal(c.now()[..., 0], c.table)
    c.close()


# ------------------------------------------------------------------ the documents' step
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_the_readme_step_of_drafts(dtype):
    """README.md's step of drafts in a cache that must not grow, as it stands there: a tree whose accepted
    rows do not lie where they were drafted, from a list of pages that an earlier step kept."""
    import os
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        blocks = f.read().split("```")[1::2]
    code, = [b for b in blocks if "verify_drafts" in b]
    B, T, H, V = 3, 8, 16, 300
    ctx = [700, 64 * 10 + 3, 640]  # one has just come to a new page
    c = Cache(dtype, ctx, host=2, garbage=False)
    hs = c.hs
    tokens, probs, _, tree, uniform = a_draft(91, B, T, V, torch.float32, "tree", sharp=2.0)
    new_rows, q = normal(92, B, T, P.DIM), normal(93, B, T, H, P.DIM)
    req_ids = torch.arange(B, **I32)
    pages = [[0, 2, 3, 7, 8, 9, 10], [0, 1, 5, 9, 10], [0, 4, 8, 9]]  # the earlier step's, and new ones behind them
    kept = torch.full((B, c.P), -1, **I32)
    for b in range(B):
        kept[b, :len(pages[b])] = i32(*pages[b])
    weights = torch.rand(c.R, c.P, generator=torch.Generator().manual_seed(94)).cuda()
    for b in range(B):
        weights[b, -(-ctx[b] // 64):] = -7.0
    before = weights.clone()
    space = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    names = dict(
        pool=c.pool, new_rows=new_rows, req_ids=req_ids, q=q, tree_masks=tree, sm_scale=SCALE, tokens=tokens, probs=probs,
        uniform=uniform, kept=kept, weights=weights, budget=i32(4, 4, 4),
        out=torch.empty(B, T, H, 512, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(B, T, H, device="cuda"),
        index=torch.empty(B, T, **I32), count=torch.empty(B, **I32), next_token=torch.empty(B, **I32),
        freed=torch.empty(B, c.P, **I32), n_freed=torch.empty(B, **I32),
        ws1=space(hs.hs_window_workspace_bytes(c.pool.handle, B, T, H, 4096, 4)),
        ws2=space(hs.hs_page_decode_workspace_bytes(B, T, H, c.P)),
        ws3=space(hs.hs_weights_workspace_bytes(c.pool.handle, B, T, H)))
    rows = c.pool.gpu_rows().clone()
    scales = None if dtype == "bf16" else c.pool.gpu_scales().clone()
    exec(code, names)
    torch.cuda.synchronize()
    assert c.pool.get_error() == 0
    moved = 0
    for b in range(B):
        path, token = M.verify(tokens[b].tolist(), probs[b].tolist(), None, tree[b].tolist(), uniform[b].tolist())
        assert names["index"][b].tolist() == path + [-1] * (T - len(path)) and int(names["next_token"][b]) == token
        moved += path != list(range(len(path)))
        stay, gone = M.evict(c.table[b], [-1] * c.P, weights[b].tolist(), ctx[b], 4, 1, 2, False)
        assert [x for x in kept[b].tolist() if x >= 0] == stay and int(names["n_freed"][b]) == len(gone)
    assert moved  # otherwise the order of the calls makes no difference
    # what the attention and the weights saw: the draft's rows where its masks say
    c.pool.gpu_rows().copy_(rows)
    if scales is not None:
        c.pool.gpu_scales().copy_(scales)
    c.pool.append_rows(new_rows, req_ids)
    torch.cuda.synchronize()
    for b in range(B):
        for t in range(T):
            pos = torch.cat([torch.arange(x * 64, min(ctx[b], x * 64 + 64)) for x in pages[b]])
            pos = pos[P.seen_mask(ctx[b], T, tree[b].tolist(), t)[pos]]
            ref = P.attention(q[b, t].double(), c.kv(b, pos), torch.ones(len(pos), dtype=torch.bool, device="cuda"), SCALE)
            P.check_attention(names["out"][b, t], names["lse"][b, t], *ref, what=f"request {b} token {t}")
    check_weights(c, weights, q, names["lse"], tree, prior=before, decay=0.99)
    c.close()
