"""Attention with a sliding window, page weights, eviction by them and verification of drafts on
the GPU, against plain forms (tests/_more.py, which derives the tolerances)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import _more as M
import _pages as P
from test_gpu_pages import Cache, I32, SCALE, i32, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available()


def workspace(n):
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")


def a_tree(seed, B, T):
    g = torch.Generator().manual_seed(seed)
    masks = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            up = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            masks[b, t] = (int(masks[b, up]) if up >= 0 else 0) | (1 << t if t < 63 else -(1 << 63))
    return masks.cuda()


# ------------------------------------------------------------------ window
def attend_window(c, q, window, n_sink, tree=None, req=None, scale=SCALE):
    B, T, H = q.shape[:3]
    out = torch.full((B, T, H, 512), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, H), math.nan, device="cuda")
    ws = workspace(c.hs.hs_window_workspace_bytes(c.pool.handle, B, T, H, window, n_sink))
    req = torch.arange(B, **I32) if req is None else req
    c.pool.page_mla_decode_window(q, req, tree, window, n_sink, scale, out, lse, ws)
    torch.cuda.synchronize()
    return out, lse


def check_window(c, q, out, lse, window, n_sink, tree=None, req=None, tokens=None):
    B, T = q.shape[:2]
    for b in range(B):
        r = b if req is None else req[b]
        L = c.ctx[r]
        masks = None if tree is None else tree[b].tolist()
        for t in range(T) if tokens is None else tokens:
            pos = M.window_mask(L, T, masks, t, window, n_sink).nonzero().squeeze(1)
            kv = c.kv(r, pos)
            ref = P.attention(q[b, t].double(), kv, torch.ones(len(pos), dtype=torch.bool, device="cuda"), SCALE)
            P.check_attention(out[b, t], lse[b, t], *ref, what=f"request {b} token {t}")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (63, 4), (64, 0), (65, 64), (100, 65), (128, 130), (700, 3),
                                           (5000, 0), (2 ** 31 - 1, 2 ** 31 - 1), (10, 2000)])
def test_window_of_one_token(dtype, window, n_sink):
    c = Cache(dtype, [1, 2, 63, 64, 65, 66, 129, 1001, 0])
    q = normal(1, 9, 1, 16, P.DIM)
    out, lse = attend_window(c, q, window, n_sink)
    check_window(c, q, out, lse, window, n_sink)
    assert not out[8].any() and bool((lse[8] == -math.inf).all())
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,window,n_sink", [(2, 128, 70, 4), (4, 24, 300, 0), (7, 16, 64, 1), (33, 8, 20, 70),
                                               (130, 3, 5, 5), (200, 16, 129, 2), (64, 1, 1, 0), (3, 300, 90, 0)])
def test_window_of_several_tokens(dtype, T, H, window, n_sink):
    """Chunks of prompt as well: rows whose windows begin in the same and in other pages."""
    c = Cache(dtype, [T + 400, T, T + 63, max(1, T - 2)])
    q = normal(2, 4, T, H, P.DIM)
    out, lse = attend_window(c, q, window, n_sink)
    check_window(c, q, out, lse, window, n_sink)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,window,n_sink", [(1, 16, 1, 0), (7, 16, 7, 3), (16, 128, 65, 0), (33, 24, 100, 70), (64, 8, 64, 1)])
def test_window_of_a_tree(dtype, T, H, window, n_sink):
    c = Cache(dtype, [T + 300, T, T + 1, T + 130])
    q, tree = normal(3, 4, T, H, P.DIM), a_tree(4, 4, T)
    tree[3, T // 2] = 0  # a query token that sees no node
    out, lse = attend_window(c, q, window, n_sink, tree)
    check_window(c, q, out, lse, window, n_sink, tree)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H,ctx,window", [(3, 1, 16, 20000, 9000), (40, 1, 128, 6000, 4096), (2, 500, 16, 2000, 333),
                                              (90, 1, 64, 700, 300), (1, 4, 16, 60000, 50000)])
def test_window_plans_of_every_kind(dtype, B, T, H, ctx, window):
    """One split, two inside a cluster, more through the workspace, the last round's alone."""
    c = Cache(dtype, [ctx - 7 * b for b in range(B)])
    q = normal(5, B, T, H, P.DIM)
    out, lse = attend_window(c, q, window, 4)
    check_window(c, q, out, lse, window, 4, tokens=sorted({0, 1 % T, T // 2, T - 1}))
    again = attend_window(c, q, window, 4)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_window_reads_nothing_outside(dtype):
    """Rows that no query token sees may hold anything, and pages of such rows need no block."""
    L, T, window, n_sink = 900, 3, 150, 70
    c = Cache(dtype, [L])
    first = L - T - window + 1
    rows, scales = c.pool.gpu_rows(), c.pool.gpu_scales()
    for pos in range(n_sink, first):
        rows[c.row(0, pos)] = 0xFF
        if dtype == "fp8":
            scales[c.row(0, pos)] = math.inf if pos % 2 else math.nan
    table = c.table[0].copy()
    table[2:first // 64] = -1
    c.pool.page_map_range(0, 0, table, table * 0 - 1)
    q = normal(6, 1, T, 16, P.DIM)
    out, lse = attend_window(c, q, window, n_sink)
    check_window(c, q, out, lse, window, n_sink)
    # a page inside the window without a block is skipped and reported
    table[L // 64] = -1
    c.pool.page_map_range(0, 0, table, table * 0 - 1)
    out, lse = attend_window(c, q, window, n_sink)
    assert bool(torch.isfinite(out).all())
    c.close(c.hs.HS_DEVERR_BAD_PAGE)


def test_window_of_unknown_requests():
    c = Cache("bf16", [100, 200])
    q = normal(7, 3, 2, 16, P.DIM)
    out, lse = attend_window(c, q, 50, 1, req=i32(1, 2, -1))
    check_window(c, q[:1], out, lse, 50, 1, req=[1])
    assert not out[1:].any() and bool((lse[1:] == -math.inf).all())
    c.close(c.hs.HS_DEVERR_BAD_REQUEST)


# ------------------------------------------------------------------ weights
def lse_of(c, q, tree=None, scale=SCALE):
    """The lse of attention to every resident page, in 32 bits, as the framework gives it."""
    B, T, H = q.shape[:3]
    out = torch.empty(B, T, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, T, H, device="cuda")
    ws = workspace(c.hs.hs_page_decode_workspace_bytes(B, T, H, c.P))
    c.pool.page_mla_decode(q, None, torch.arange(B, **I32), tree, scale, out, lse, ws)
    torch.cuda.synchronize()
    return lse


def run_weights(c, q, lse, tree=None, prior=None, decay=1.0, req=None, weights=None):
    B, T, H = q.shape[:3]
    w = torch.full((c.R, c.P), -7.0, device="cuda") if weights is None else weights
    ws = workspace(c.hs.hs_weights_workspace_bytes(c.pool.handle, B, T, H))
    req = torch.arange(B, **I32) if req is None else req
    c.pool.page_weights(q, lse, req, tree, SCALE, w, prior, decay, ws)
    torch.cuda.synchronize()
    return w


def check_weights(c, w, q, lse, tree=None, prior=None, decay=1.0, req=None, skip=(), which=None):
    B, T = q.shape[:2]
    done = torch.zeros(c.R, c.P, dtype=torch.bool)
    for b in range(B):
        r = b if req is None else int(req[b])
        if not 0 <= r < c.R:
            continue
        L = c.ctx[r]
        n = -(-L // 64)
        done[r, :n] = True
        if which is not None and b not in which:
            continue
        masks = None if tree is None else tree[b].tolist()
        seen = torch.stack([P.seen_mask(L, T, masks, t) for t in range(T)]).cuda()
        kv = torch.nan_to_num(c.kv(r, range(L)), 0.0, 0.0, 0.0)
        for p in skip:
            seen[:, 64 * p:64 * p + 64] = False
        fine = kv * seen.any(0)[:, None]  # what a hidden row holds does not matter
        want = M.page_weights(q[b].double(), lse[b].double(), fine, seen, SCALE)
        tol = M.weights_tolerance(want, q[b].double(), lse[b].double(), fine, SCALE, c.dtype == "fp8")
        if prior is not None and decay:
            old = decay * prior[r, :n].double()
            want, tol = want + old, tol + 2.0 ** -22 * old.abs()
        d = (w[r, :n].double() - want).abs()
        assert bool((d <= tol).all()), f"request {b}: off by {float((d / tol).max()):.3f} of the tolerance"
    assert bool((w[~done.cuda()] == -7.0).all())  # the others as they were


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (3, 16), (1, 64), (5, 13), (3, 32), (1, 128), (4, 48), (2, 128), (300, 1),
                                 (3, 100), (4, 128), (33, 24)])
def test_weights(dtype, T, H):
    """One and several groups of query rows, whole and broken ones; short, odd and empty contexts."""
    ctx = [T, T + 1, 64 + T, 1000, 0 if T == 1 else T + 63]
    c = Cache(dtype, ctx, max_ctx=max(ctx) + 100)
    q = normal(11, 5, T, H, P.DIM)
    lse = lse_of(c, q)
    check_weights(c, run_weights(c, q, lse), q, lse)
    prior = torch.rand(c.R, c.P, generator=torch.Generator().manual_seed(12)).cuda()
    check_weights(c, run_weights(c, q, lse, prior=prior, decay=0.5), q, lse, prior=prior, decay=0.5)
    both = torch.where(torch.arange(c.P)[None] * 64 < torch.tensor(ctx)[:, None], prior.cpu(), -7.0).cuda()
    old = both.clone()
    check_weights(c, run_weights(c, q, lse, prior=both, weights=both), q, lse, prior=old)  # in place
    prior.fill_(math.nan)
    check_weights(c, run_weights(c, q, lse, prior=prior, decay=0.0), q, lse)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H", [(1, 16), (7, 16), (16, 40), (64, 8)])
def test_weights_of_a_tree(dtype, T, H):
    c = Cache(dtype, [T, T + 64, 500])
    q, tree = normal(13, 3, T, H, P.DIM), a_tree(14, 3, T)
    tree[1, T // 2] = 0
    lse = lse_of(c, q, tree)
    check_weights(c, run_weights(c, q, lse, tree), q, lse, tree)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H,long", [(1, 1, 16, 70000), (3, 2, 128, 30000), (300, 1, 24, 300), (77, 4, 128, 600), (40, 3, 8, 9000)])
def test_weights_of_ranges_across_requests(dtype, B, T, H, long):
    """The tiles of all requests laid end to end: ranges that begin and end inside requests, and
    hold many of them; empty ones between."""
    g = torch.Generator().manual_seed(15)
    ctx = [long] + [int(x) for x in torch.randint(T, max(T + 1, long // 2), (B - 1,), generator=g)]
    for b in range(3, B, 5):
        ctx[b] = 0 if b % 2 else T
    c = Cache(dtype, ctx)
    q = normal(16, B, T, H, P.DIM)
    lse = lse_of(c, q)
    w = run_weights(c, q, lse)
    check_weights(c, w, q, lse, which=sorted({0, 1 % B, B // 2, B - 1, 3 % B, 8 % B}))
    total = torch.where(w == -7.0, 0.0, w).sum(1)
    seen = torch.isfinite(lse).sum((1, 2)).float()
    assert bool(((total - seen).abs() <= 2.0 ** -10 * seen).all())  # every request's weights sum to its rows
    again = run_weights(c, q, lse)
    assert torch.equal(w, again)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [16, 32])
def test_weights_leave_out_what_is_not_finite_or_not_there(dtype, H):
    """Query rows without a finite lse add nothing; a page without a block gets nothing; unknown
    requests are skipped; requests come in any order."""
    c = Cache(dtype, [700, 300, 500])
    table = c.table[0].copy()
    table[[0, 4]] = -1
    c.pool.page_map_range(0, 0, table, table * 0 - 1)
    q = normal(17, 4, 2, H, P.DIM)
    q[0, 0, 3] = math.nan
    q[1, 1, 5, 7] = math.inf
    q[3, 1, 2] = 0
    lse = torch.full((4, 2, H), 6.0, device="cuda")
    lse[0, 0, 3] = math.nan
    lse[1, 1, 5] = math.inf
    lse[3, 1, 2] = -math.inf
    req = i32(0, 2, 5, 1)
    w = run_weights(c, q, lse, req=req)
    for b, skip in ((0, (0, 4)), (1, ()), (3, ())):
        one = torch.full_like(w, -7.0)
        r = int(req[b])
        one[r] = w[r]
        qb = torch.where(torch.isfinite(lse[b:b + 1])[..., None], q[b:b + 1], 0.0)
        check_weights(c, one, qb, lse[b:b + 1], req=[r], skip=skip)
    assert not w[0, [0, 4]].any()
    c.close(c.hs.HS_DEVERR_BAD_REQUEST)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_weights_with_a_key_that_is_not_finite(dtype):
    """Its page's weight is not finite where a query row with a finite lse sees it, and nobody else's."""
    c = Cache(dtype, [400])
    if dtype == "bf16":
        c.pool.gpu_rows()[c.row(0, 100), 3] = 0x7F
        c.pool.gpu_rows()[c.row(0, 100), 2] = 0x80
    else:
        c.pool.gpu_scales()[c.row(0, 100)] = math.inf
    q = normal(18, 1, 1, 40, P.DIM)
    lse = torch.full((1, 1, 40), 6.0, device="cuda")
    w = run_weights(c, q, lse)
    assert bool(torch.isfinite(w[0, [0, 2, 3, 4, 5, 6]]).all()) and not bool(torch.isfinite(w[0, 1]))
    lse.fill_(math.nan)  # what attention gives for it
    w = run_weights(c, q, lse)
    assert not w.any()
    c.close()


@pytest.mark.parametrize("H", [40, 8, 32])
def test_weights_with_a_key_of_no_weight_that_is_not_finite(H):
    """An infinity that every query row meets with a negative value: scores of minus infinity,
    a finite lse, and no weight."""
    c = Cache("bf16", [400])
    q = normal(25, 1, 1, H, P.DIM)
    q[..., 0] = -1 - q[..., 0].abs()
    rows = c.pool.gpu_rows()[c.row(0, 100)].view(torch.bfloat16)
    rows[0] = math.inf
    lse = lse_of(c, q)
    assert bool(torch.isfinite(lse).all())
    w = run_weights(c, q, lse)
    kv = c.kv(0, range(400))
    kv[100] = 0
    seen = torch.ones(1, 400, dtype=torch.bool, device="cuda")
    seen[0, 100] = False
    want = M.page_weights(q[0].double(), lse[0].double(), kv, seen, SCALE)
    tol = M.weights_tolerance(want, q[0].double(), lse[0].double(), kv, SCALE, False)
    assert bool(((w[0].double() - want).abs() <= tol).all())
    c.close()


def test_weights_fp8_scales_of_many_magnitudes():
    c = Cache("fp8", [640])
    g = torch.Generator().manual_seed(19)
    s = c.pool.gpu_scales()
    s.mul_(torch.exp2(torch.randint(-30, 2, s.shape, generator=g).float()).cuda())
    q = normal(20, 1, 3, 16, P.DIM)
    q[0, 1] *= 2.0 ** -100
    q[0, 2, 3] *= 16
    lse = lse_of(c, q)
    check_weights(c, run_weights(c, q, lse), q, lse)
    c.close()


# ------------------------------------------------------------------ eviction
def run_evict(c, req, budget, weights, N, n_first=1, n_last=1, saved_only=False, plan=False):
    n = len(req)
    kept, freed = torch.full((n, N), -7, **I32), torch.full((n, c.P), -7, **I32)
    count = torch.full((n,), -7, **I32)
    c.pool.evict_pages(i32(*req), i32(*budget), weights, kept, freed, count, n_first, n_last, saved_only, plan)
    torch.cuda.synchronize()
    return kept.tolist(), freed.tolist(), count.tolist()


class Tables:
    """A pool whose pages share few blocks: eviction reads the table alone."""

    def __init__(self, ctx, max_ctx=None, seed=0, holes=0.2, unsaved=0.3):
        import tiered_sparse_mla_gb300 as hs
        self.hs, self.ctx, self.R = hs, list(ctx), len(ctx)
        self.max_ctx = max_ctx or max(64, max(ctx))
        self.P = -(-self.max_ctx // 64)
        self.pool = hs.Pool(dtype=hs.HS_FP8_E4M3_ROWSCALE, n_gpu_blocks=97, n_host_blocks=8, max_requests=self.R,
                            max_ctx=self.max_ctx, max_topk=32, hot_rows=64)
        rng = np.random.default_rng(seed)
        self.table = rng.integers(0, 97, (self.R, self.P)).astype(np.int32)
        self.saved = rng.integers(0, 8, (self.R, self.P)).astype(np.int32)
        self.table[rng.random((self.R, self.P)) < holes] = -1
        self.saved[rng.random((self.R, self.P)) < unsaved] = -1
        for r in range(self.R):
            self.pool.page_map_range(r, 0, self.table[r], self.saved[r])
        self.pool.set_ctx_lens(torch.tensor(self.ctx, **I32))

    def now(self):
        return self.pool.tables()["page_table"].cpu().numpy()

    close = Cache.close


@pytest.mark.parametrize("saved_only", [False, True])
@pytest.mark.parametrize("n_first,n_last", [(0, 0), (1, 2), (5, 40)])
def test_evict(n_first, n_last, saved_only):
    """Ties, NaN, infinities and zeros of both signs among the weights; budgets of every kind."""
    ctx = [0, 1, 64, 65, 31 * 64, 32 * 64, 33 * 64 - 5, 3000, 20000, 130000, 130000, 130000]
    c = Tables(ctx)
    g = torch.Generator().manual_seed(21)
    w = torch.exp(2 * torch.randn(c.R, c.P, generator=g))
    w[7] = torch.randint(0, 3, (c.P,), generator=g).float()  # many ties
    w[8, ::3], w[8, 1::7], w[8, 2::11], w[8, 5::13] = 0.0, -0.0, math.nan, math.inf
    w[8, 4::17] = -math.inf
    w[10] = 0.25
    w[11] = 1 + torch.arange(c.P) % 7 * 2.0 ** -23  # the last bits decide
    req = list(range(c.R))[::-1]
    for budget in ([0] * 12, [3] * 12, [700, 500, 333, 100, 20, 10, 16, 17, 0, 1, 1, 1], [10 ** 9] * 12, [-1] * 12):
        kept, freed, count = run_evict(c, req, budget, w.cuda(), c.P, n_first, n_last, saved_only, plan=True)
        for i, r in enumerate(req):
            stay, gone = M.evict(c.table[r], c.saved[r], w[r].tolist(), ctx[r], budget[i], n_first, n_last, saved_only)
            assert kept[i] == stay + [-1] * (c.P - len(stay)), (r, budget[i])
            assert count[i] == len(gone) and freed[i][:len(gone)] == [int(c.table[r, p]) for p in gone], (r, budget[i])
            assert set(freed[i][len(gone):]) <= {-7}  # the rest as it was
        now = c.now()
        assert np.array_equal(now[..., 0], c.table) and np.array_equal(now[..., 1], c.saved)
        assert c.pool.get_error() == (c.hs.HS_DEVERR_BAD_PAGE if budget[0] < 0 else 0)
    # and in earnest
    budget = [50] * 12
    kept, freed, count = run_evict(c, req, budget, w.cuda(), c.P, n_first, n_last, saved_only)
    now, want = c.now(), c.table.copy()
    for i, r in enumerate(req):
        stay, gone = M.evict(c.table[r], c.saved[r], w[r].tolist(), ctx[r], 50, n_first, n_last, saved_only)
        assert [p for p in kept[i] if p >= 0] == stay and freed[i][:count[i]] == [int(c.table[r, p]) for p in gone]
        want[r, gone] = -1
    assert np.array_equal(now[..., 0], want) and np.array_equal(now[..., 1], c.saved)
    # again: nothing more to free, the same pages kept
    k2, _, n2 = run_evict(c, req, budget, w.cuda(), c.P, n_first, n_last, saved_only)
    assert k2 == kept and not any(n2)
    c.close()


@pytest.mark.parametrize("pages", [512, 513, 1024, 2049, 5000, 32769, 70000, 270000])
def test_evict_of_long_contexts(pages):
    """More pages than a scan takes at a time, and than keys fit in shared memory."""
    ctx = [pages * 64, pages * 64 - 64 * 17 - 3]
    c = Tables(ctx, seed=pages)
    g = torch.Generator().manual_seed(22)
    w = torch.rand(c.R, c.P, generator=g)
    w[1] = (w[1] * 50).floor()
    for budget in (5, pages // 3, pages - 10):
        kept, freed, count = run_evict(c, [0, 1], [budget] * 2, w.cuda(), c.P, 2, 3, False, True)
        for r in range(2):
            stay, gone = M.evict(c.table[r], c.saved[r], w[r].tolist(), ctx[r], budget, 2, 3, False)
            assert kept[r] == stay + [-1] * (c.P - len(stay))
            assert count[r] == len(gone) and freed[r][:len(gone)] == c.table[r, gone].tolist()
    c.close()


def test_evict_reports_what_does_not_fit():
    c = Tables([640, 640], holes=0.0)
    w = torch.arange(20).float().view(2, 10).cuda()
    hs = c.hs
    kept, freed, count = run_evict(c, [0, 1], [6, 2], w, 4, 0, 0)
    assert kept == [[4, 5, 6, 7], [8, 9, -1, -1]] and count == [4, 8]
    assert c.pool.get_error() == hs.HS_DEVERR_CAPACITY
    assert (c.now()[0, :, 0] >= 0).tolist() == [False] * 4 + [True] * 6
    kept, freed, count = run_evict(c, [2, -1], [1, 1], w, 4)
    assert kept == [[-1] * 4] * 2 and count == [0, 0] and freed[0] == [-7] * 10
    assert c.pool.get_error() == hs.HS_DEVERR_BAD_REQUEST
    c.pool.set_ctx_lens(i32(5000, 640))
    kept, _, count = run_evict(c, [0], [3], w, 4, 0, 0)
    assert kept == [[7, 8, 9, -1]] and count == [3]
    c.close(hs.HS_DEVERR_INDEX_RANGE)


# ------------------------------------------------------------------ verification
def run_verify(pool, tokens, p, q, tree, u):
    B, T = tokens.shape
    index, count, nxt = torch.full((B, T), -7, **I32), torch.full((B,), -7, **I32), torch.full((B,), -7, **I32)
    pool.verify_drafts(tokens, p, q, tree, u, index, count, nxt)
    torch.cuda.synchronize()
    return index.tolist(), count.tolist(), nxt.tolist()


@pytest.fixture
def pool():
    import tiered_sparse_mla_gb300 as hs
    p = hs.Pool(dtype=hs.HS_BF16, n_gpu_blocks=1, n_host_blocks=0, max_requests=1, max_ctx=64, max_topk=32)
    p.hs = hs
    yield p
    p.close()


def check_verify(got, tokens, p, q, tree, u):
    B, T = tokens.shape
    pl, ql = p.double().tolist(), None if q is None else q.double().tolist()
    ul = u.double().tolist()
    for b in range(B):
        path, nxt = M.verify(tokens[b].tolist(), pl[b], None if q is None else ql[b], None if tree is None else tree[b].tolist(),
                             ul[b])
        assert got[0][b] == path + [-1] * (T - len(path)), b
        assert got[1][b] == len(path) and got[2][b] == nxt, b


def a_draft(seed, B, T, V, dtype, kind, sharp=3.0, wide=0):
    """Probabilities, draft, tokens and random numbers whose drafts are often accepted."""
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, T, V, generator=g)
    tree = None
    if kind == "tree":
        tree = a_tree(seed, B, T).cpu()
        tree = tree | 1  # everything hangs on node 0 in the end
    par = torch.tensor([M.parents(T, None if tree is None else [x & ((1 << 64) - 1) for x in tree[b].tolist()]) for b in range(B)])
    rows = logits.gather(1, par.clamp(min=0)[..., None].expand(B, T, V))
    race = -torch.log(-torch.log(torch.rand(B, T, V, generator=g).clamp(1e-9, 1 - 1e-6)))
    guess = rows + 0.3 * torch.randn(B, T, V, generator=g)
    tokens = (guess + race).argmax(-1).to(torch.int32)
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(guess, -1)[:, 1:].to(dtype) if kind == "draft" else None
    u = torch.rand(B, T, generator=g)
    if kind != "draft":
        u[:, 1:] *= 0.5

    def wider(x):
        if not wide or x is None:
            return None if x is None else x.cuda()
        buf = torch.full((*x.shape[:2], V + wide), math.nan, dtype=dtype, device="cuda")
        buf[..., 1:V + 1] = x.cuda()
        return buf[..., 1:V + 1]

    return tokens.cuda(), wider(p), wider(q), None if tree is None else tree.cuda(), u.cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["draft", "chain", "tree"])
@pytest.mark.parametrize("B,T,V,wide", [(3, 1, 100, 0), (5, 2, 1, 0), (20, 4, 257, 3), (7, 16, 1000, 0), (4, 33, 4097, 7),
                                        (2, 64, 300, 0), (2, 5, 40001, 2), (1, 3, 200000, 0)])
def test_verify(pool, dtype, kind, B, T, V, wide):
    x = a_draft(31 + B, B, T, V, dtype, kind, wide=wide)
    check_verify(run_verify(pool, *x), *x)
    assert pool.get_error() == 0


@pytest.mark.parametrize("kind", ["draft", "chain", "tree"])
def test_verify_many(pool, kind):
    """Each way that a draft can end, often enough to be met."""
    x = a_draft(77, 400, 6, 37, torch.float32, kind, sharp=2.0)
    got = run_verify(pool, *x)
    check_verify(got, *x)
    assert len(set(got[1])) >= 4
    assert pool.get_error() == 0


def test_verify_on_the_borders(pool):
    """Probabilities that are multiples of 1/8 and random numbers that are too: a border belongs
    to the next token, and u q = p refuses."""
    n = 8
    p = torch.full((n, 2, n), 1 / n, device="cuda")
    tokens = torch.zeros(n, 2, **I32)
    u = torch.stack([torch.arange(n) / n, torch.full((n,), 1 / n)], 1).cuda()
    index, count, nxt = run_verify(pool, tokens, p, None, None, u)  # u = p: refused, token 0 goes
    assert count == [1] * n
    assert nxt == [M.draw([0] + [1] * 7, k / n) for k in range(n)]
    u[:, 1] = 1 / n - 2.0 ** -27
    index, count, nxt = run_verify(pool, tokens, p, None, None, u)
    assert count == [2] * n and nxt == list(range(n))
    p[:, 0, 0] = 0.25
    q = torch.full((n, 1, n), 0.5, device="cuda")
    u[:, 1] = 0.5
    assert run_verify(pool, tokens, p, q, None, u)[1] == [1] * n
    u[:, 1] = 0.5 - 2.0 ** -25
    assert run_verify(pool, tokens, p, q, None, u)[1] == [2] * n
    assert pool.get_error() == 0


def test_verify_degenerate_rows(pool):
    """Rows that leave nothing, hold NaN, or sum to far more than one; random numbers out of range."""
    hs, V = pool.hs, 700
    g = torch.Generator().manual_seed(41)
    p = torch.softmax(torch.randn(9, 2, V, generator=g), -1)
    q = p[:, :1].clone()  # nothing is left of p - q: by p itself
    p[1] = 0
    p[2, 0] = math.nan
    p[3, 0, 5:] = math.nan
    p[4, 0] = 1.0
    p[5, 0] = 2.0 ** -70  # below the sums' steps
    p[6, 0] = -0.5
    p[7, 0] = 1e30
    q[7] = 0
    q[0, 0, 3] *= 1.5
    tokens = torch.full((9, 2), 3, dtype=torch.int32)
    u = torch.rand(9, 2, generator=g)
    u[:, 1] = 0.9999
    u[8] = torch.tensor([1.5, -3.0])
    x = (tokens.cuda(), p.cuda(), q.cuda(), None, u.cuda())
    got = run_verify(pool, *x)
    check_verify(got, *x)
    assert got[2][1] == -1 and got[2][5] == -1 and 0 <= got[2][0] < V
    assert pool.get_error() == hs.HS_DEVERR_INDEX_RANGE
    u[:] = math.nan
    x = (tokens.cuda(), p.cuda(), None, None, u.cuda())
    check_verify(run_verify(pool, *x), *x)
    pool.get_error()


@pytest.mark.parametrize("kind", ["draft", "chain", "tree"])
def test_verify_ragged_drafts(pool, kind):
    """-1 ends a chain or leaves a node out, and no probability goes with it; tokens out of range
    too, and are reported."""
    tokens, p, q, tree, u = a_draft(51, 60, 7, 50, torch.float32, kind, sharp=2.0)
    g = torch.Generator().manual_seed(52)
    drop = torch.rand(60, 7, generator=g).cuda() < 0.3
    tokens[drop] = -1
    check_verify(run_verify(pool, tokens, p, q, tree, u), tokens, p, q, tree, u)
    assert pool.get_error() == 0
    tokens[:, 0] = 12345  # not looked at
    check_verify(run_verify(pool, tokens, p, q, tree, u), tokens, p, q, tree, u)
    assert pool.get_error() == 0
    tokens[::2, 2] = 50
    tokens[1::2, 3] = -2
    check_verify(run_verify(pool, tokens, p, q, tree, u), tokens, p, q, tree, u)
    assert pool.get_error() == pool.hs.HS_DEVERR_INDEX_RANGE


def test_verify_trees_of_every_shape(pool):
    """Brothers with the same token, nodes off node 0's tree, masks with bits above their own."""
    B, T, V = 200, 12, 6
    g = torch.Generator().manual_seed(61)
    tokens = torch.randint(0, V, (B, T), generator=g).to(torch.int32).cuda()
    p = torch.softmax(torch.randn(B, T, V, generator=g), -1).cuda()
    tree = torch.randint(0, 1 << T, (B, T), generator=g).cuda()
    u = (0.4 * torch.rand(B, T, generator=g)).cuda()
    check_verify(run_verify(pool, tokens, p, None, tree, u), tokens, p, None, tree, u)
    star = torch.ones(B, T, dtype=torch.int64).cuda() | (1 << torch.arange(T).cuda())
    check_verify(run_verify(pool, tokens, p, None, star, u), tokens, p, None, star, u)
    assert pool.get_error() == 0


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_step_of_drafts_in_a_cache_that_must_not_grow(dtype):
    """A tree's rows in, windowed attention, verification, the accepted rows in their places, the
    weights that pages have got, eviction, and attention to the pages that are left; the same
    from a captured graph, replayed, on another stream."""
    B, T, H, V, window, n_sink = 3, 6, 16, 500, 200, 4
    ctx = [700, 901, 640]
    c = Cache(dtype, ctx, host=2, garbage=False)
    hs = c.hs
    tokens, p, _, tree, u = a_draft(71, B, T, V, torch.float32, "tree", sharp=2.0)
    rows, q = normal(72, B, T, P.DIM), normal(73, B, T, H, P.DIM)
    req = torch.arange(B, **I32)
    index, count, nxt = torch.zeros(B, T, **I32), torch.zeros(B, **I32), torch.zeros(B, **I32)
    out, lse = torch.zeros(B, T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, T, H, device="cuda")
    full, flse = out.clone(), lse.clone()
    weights, before = torch.full((c.R, c.P), -7.0, device="cuda"), torch.rand(c.R, c.P, generator=torch.Generator().manual_seed(74)).cuda()
    budget = i32(6, 9, 100)
    kept, freed, n_freed = torch.zeros(B, c.P, **I32), torch.full((B, c.P), -7, **I32), torch.zeros(B, **I32)
    left, llse = out.clone(), lse.clone()
    ws = [workspace(hs.hs_window_workspace_bytes(c.pool.handle, B, T, H, window, n_sink)),
          workspace(hs.hs_page_decode_workspace_bytes(B, T, H, c.P)), workspace(hs.hs_weights_workspace_bytes(c.pool.handle, B, T, H))]
    start = c.pool.gpu_rows().clone()
    scales = None if dtype == "bf16" else c.pool.gpu_scales().clone()
    table = c.pool.tables()["page_table"]
    full_table = table.clone()

    def step():
        c.pool.append_rows(rows, req)
        c.pool.page_mla_decode_window(q, req, tree, window, n_sink, SCALE, out, lse, ws[0])
        c.pool.page_mla_decode(q, None, req, tree, SCALE, full, flse, ws[1])
        c.pool.page_weights(q, flse, req, tree, SCALE, weights, before, 0.5, ws[2])
        c.pool.verify_drafts(tokens, p, None, tree, u, index, count, nxt)
        c.pool.append_rows(rows, req, None, index)
        c.pool.evict_pages(req, budget, weights, kept, freed, n_freed, n_first=1, n_last=2)
        c.pool.page_mla_decode(q, kept, req, tree, SCALE, left, llse, ws[1])

    results = (out, lse, full, flse, weights, index, count, nxt, kept, freed, n_freed, left, llse)
    step()
    torch.cuda.synchronize()
    eager = [x.clone() for x in results] + [c.pool.gpu_rows().clone(), table.clone()]
    # against the plain forms
    path_rows = c.pool.gpu_rows().clone()
    for b in range(B):
        masks = tree[b].tolist()
        path, token = M.verify(tokens[b].tolist(), p[b].tolist(), None, masks, u[b].tolist())
        assert index[b].tolist() == path + [-1] * (T - len(path)) and int(nxt[b]) == token
        n = len(path)
        want = rows[b, path].cpu()
        at = torch.tensor([c.row(b, ctx[b] - T + k) for k in range(n)])
        if dtype == "bf16":
            assert torch.equal(path_rows[at].cpu(), want.view(torch.uint8))
        else:
            assert torch.equal(path_rows[at].cpu(), P.quantise(want)[0].view(torch.uint8))
        stay, gone = M.evict(c.table[b], [-1] * c.P, weights[b].tolist(), ctx[b], int(budget[b]), 1, 2, False)
        assert [x for x in kept[b].tolist() if x >= 0] == stay and int(n_freed[b]) == len(gone)
        assert freed[b, :len(gone)].tolist() == [int(c.table[b, x]) for x in gone]
        for t in range(T):
            pos = torch.cat([torch.arange(x * 64, min(ctx[b], x * 64 + 64)) for x in stay])
            pos = pos[P.seen_mask(ctx[b], T, masks, t)[pos]]
            ref = P.attention(q[b, t].double(), c.kv(b, pos), torch.ones(len(pos), dtype=torch.bool, device="cuda"), SCALE)
            P.check_attention(left[b, t], llse[b, t], *ref, what=f"request {b} token {t}")

    def reset():
        c.pool.gpu_rows().copy_(start)
        if scales is not None:
            c.pool.gpu_scales().copy_(scales)
        table.copy_(full_table)
        for x in results:
            x.fill_(-7)

    side = torch.cuda.Stream()
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        reset()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(list(results) + [c.pool.gpu_rows(), table], eager):
            assert torch.equal(x, y)
    # the windowed attention and the weights saw the rows as they were first put in
    c.pool.gpu_rows().copy_(start)
    if scales is not None:
        c.pool.gpu_scales().copy_(scales)
    c.pool.append_rows(rows, req)
    torch.cuda.synchronize()
    check_window(c, q, eager[0], eager[1], window, n_sink, tree)
    check_weights(c, eager[4], q, eager[3], tree, prior=before, decay=0.5)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_calls_on_two_streams_at_once(dtype):
    B, T, H = 4, 4, 96  # weights: two groups, through the workspace
    c = Cache(dtype, [9000, 5000, 8000, 3000])
    q = [normal(81 + i, B, T, H, P.DIM) for i in range(2)]
    lse = [lse_of(c, x) for x in q]
    want = [run_weights(c, x, y) for x, y in zip(q, lse)]
    wout = [attend_window(c, x, 3000, 4) for x in q]
    req = torch.arange(B, **I32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.full_like(want[0], -7.0) for _ in range(2)]
    outs = [(torch.zeros_like(wout[0][0]), torch.zeros_like(wout[0][1])) for _ in range(2)]
    ws = [[workspace(c.hs.hs_weights_workspace_bytes(c.pool.handle, B, T, H)),
           workspace(c.hs.hs_window_workspace_bytes(c.pool.handle, B, T, H, 3000, 4))] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            c.pool.page_weights(q[i], lse[i], req, None, SCALE, got[i], None, 1.0, ws[i][0], stream=s)
            c.pool.page_mla_decode_window(q[i], req, None, 3000, 4, SCALE, *outs[i], ws[i][1], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i])
        assert torch.equal(outs[i][0], wout[i][0]) and torch.equal(outs[i][1], wout[i][1])
    c.close()


def test_refusals():
    """Arguments that the calls refuse: a status, and nothing is launched."""
    c = Cache("bf16", [200, 100])
    hs, pool = c.hs, c.pool
    q = normal(91, 2, 3, 16, P.DIM)
    req = torch.arange(2, **I32)
    out, lse = torch.full((2, 3, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 3, 16), 7.0, device="cuda")
    tree = torch.ones(2, 3, dtype=torch.int64, device="cuda")
    w = torch.full((2, c.P), 7.0, device="cuda")
    big = workspace(1 << 22)

    def status(call):
        with pytest.raises(hs.HsError) as e:
            call()
        return e.value.status

    inval, unsup = hs.HS_ERR_INVALID_ARG, hs.HS_ERR_UNSUPPORTED
    for window, sink in ((0, 0), (-5, 0), (10, -1)):
        assert status(lambda: pool.page_mla_decode_window(q, req, None, window, sink, SCALE, out, lse, big)) == inval
        assert hs.hs_window_workspace_bytes(pool.handle, 2, 3, 16, window, sink) == 0
    assert status(lambda: pool.page_mla_decode_window(q, req, tree, 2, 0, SCALE, out, lse, big)) == unsup
    long = Cache("bf16", [40000])
    q1 = normal(92, 1, 3, 16, P.DIM)
    need = hs.hs_window_workspace_bytes(long.pool.handle, 1, 3, 16, 30000, 4)
    assert need > 0
    for ws in (None, workspace(need - 1), workspace(need + 8)[8:]):
        assert status(lambda: long.pool.page_mla_decode_window(q1, req[:1], None, 30000, 4, SCALE, out[:1], lse[:1], ws)) == inval
    q33 = normal(93, 2, 33, 16, P.DIM)
    l33 = torch.zeros(2, 33, 16, device="cuda")
    need = hs.hs_weights_workspace_bytes(pool.handle, 2, 33, 16)
    assert need > 0 and hs.hs_weights_workspace_bytes(pool.handle, 2, 16, 16) == 0
    for ws in (None, workspace(need - 1), workspace(need + 8)[8:]):
        assert status(lambda: pool.page_weights(q33, l33, req, None, SCALE, w, None, 1.0, ws)) == inval
    t65 = torch.ones(1, 65, dtype=torch.int64, device="cuda")
    q65 = normal(94, 1, 65, 2, P.DIM)
    assert status(lambda: pool.page_weights(q65, torch.zeros(1, 65, 2, device="cuda"), req[:1], t65, SCALE, w)) == inval
    assert status(lambda: pool.page_mla_decode_window(q65, req[:1], t65, 100, 0, SCALE, torch.zeros(1, 65, 2, 512, dtype=torch.bfloat16, device="cuda"),
                                                      torch.zeros(1, 65, 2, device="cuda"), big)) == inval
    kept, freed, n = torch.full((2, 4), 7, **I32), torch.full((2, c.P), 7, **I32), torch.full((2,), 7, **I32)
    for first, last in ((-1, 0), (0, -1)):
        assert status(lambda: pool.evict_pages(req, req, w, kept, freed, n, first, last)) == inval
    lib, p = hs.load(), C.c_void_p
    assert lib.hs_evict_pages(pool.handle, 2, 4, 0, 0, 4, *(p(x.data_ptr()) for x in (req, req, w, kept, freed, n)), None) == inval
    assert lib.hs_evict_pages(pool.handle, 2, 0, 0, 0, 0, *(p(x.data_ptr()) for x in (req, req, w, kept, freed, n)), None) == inval
    assert lib.hs_evict_pages(pool.handle, -1, 4, 0, 0, 0, *(p(x.data_ptr()) for x in (req, req, w, kept, freed, n)), None) == inval
    assert lib.hs_evict_pages(pool.handle, 2, 4, 0, 0, 0, None, *(p(x.data_ptr()) for x in (req, w, kept, freed, n)), None) == inval
    tok, u = torch.zeros(2, 3, **I32), torch.zeros(2, 3, device="cuda")
    pr, dr = torch.zeros(2, 3, 8, device="cuda"), torch.zeros(2, 2, 8, device="cuda")
    idx, cnt, nxt = torch.full((2, 3), 7, **I32), torch.full((2,), 7, **I32), torch.full((2,), 7, **I32)
    assert status(lambda: pool.verify_drafts(tok, pr, dr, tree, u, idx, cnt, nxt)) == unsup
    a = [p(x.data_ptr()) for x in (pr, dr, tok, u, idx, cnt, nxt)]

    def verify(B=2, T=3, V=8, dtype=0, probs=a[0], ld=8, draft=a[1], dld=8, tokens=a[2], uniform=a[3], nxt=a[6]):
        return lib.hs_verify_drafts(pool.handle, B, T, V, dtype, probs, ld, draft, dld, tokens, None, uniform, a[4], a[5], nxt, None)

    for bad in ({"B": -1}, {"B": 65536}, {"T": 0}, {"T": 65}, {"V": 0}, {"dtype": 2}, {"ld": 7}, {"dld": 7}, {"ld": 1 << 50},
                {"probs": None}, {"tokens": None}, {"uniform": None}, {"nxt": None}, {"probs": p(pr.data_ptr() + 2)}):
        assert verify(**bad) == inval, bad
    with pytest.raises(ValueError):
        pool.verify_drafts(tok, pr, dr.to(torch.bfloat16), None, u, idx, cnt, nxt)
    with pytest.raises(ValueError):
        pool.verify_drafts(tok, pr, pr, None, u, idx, cnt, nxt)
    with pytest.raises(ValueError):
        pool.page_weights(q, lse, req, None, SCALE, w[:1])
    with pytest.raises(ValueError):
        pool.page_weights(q, lse.double(), req, None, SCALE, w)
    with pytest.raises(ValueError):
        pool.evict_pages(req, req, w, kept, freed[:, :1], n)
    # nothing to do is no error
    pool.page_mla_decode_window(q[:0], req[:0], None, 10, 0, SCALE, out[:0], lse[:0])
    pool.page_weights(q[:0], lse[:0], req[:0], None, SCALE, w)
    pool.evict_pages(req[:0], req[:0], w, kept[:0], freed[:0], n[:0])
    pool.verify_drafts(tok[:0], pr[:0], dr[:0], None, u[:0], idx[:0], cnt[:0], nxt[:0])
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((lse == 7).all()) and bool((w == 7).all())
    assert all(bool((x == 7).all()) for x in (kept, freed, n, idx, cnt, nxt))
    long.close()
    c.close()


@pytest.mark.parametrize("ctx,T,H,window,n_sink", [
    ([900, 2], 700, 32, 100, 4), ([3000, 700, 900], 700, 24, 333, 0), ([5000], 1500, 16, 1, 0), ([1301, 1300, 1], 1300, 16, 64, 70),
    ([2700, 650, 30, 0, 900], 600, 17, 500, 1), ([40, 600, 20000, 64], 600, 16, 5000, 64), ([300] * 160, 3, 40, 128, 2),
    ([1] * 100 + [0] * 60 + [3000] * 10, 2, 64, 200, 2)])
def test_window_units_one_after_the_other(ctx, T, H, window, n_sink):
    """More units than two for each pair of CTAs: long ones, ones of a single step, and empty ones in
    any order."""
    B = len(ctx)
    c = Cache("bf16", ctx)
    q = normal(26, B, T, H, P.DIM)
    out, lse = attend_window(c, q, window, n_sink)
    tokens = sorted({0, 1, T // 3, T // 2, T - 2, T - 1}) if T > 3 else None
    check_window(c, q, out, lse, window, n_sink, tokens=tokens)
    for _ in range(3):
        again = attend_window(c, q, window, n_sink)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.close()


def test_window_units_one_after_the_other_with_unknown_requests():
    B = 200
    c = Cache("bf16", [500, 90, 0])
    q = normal(27, B, 1, 128, P.DIM)
    g = torch.Generator().manual_seed(28)
    req = torch.randint(-1, 4, (B,), generator=g).to(torch.int32)
    out, lse = attend_window(c, q, 100, 3, req=req.cuda())
    known = [b for b in range(B) if 0 <= int(req[b]) < 3]
    check_window(c, q[known], out[known], lse[known], 100, 3, req=[int(req[b]) for b in known])
    rest = [b for b in range(B) if b not in known]
    assert not out[rest].any() and bool((lse[rest] == -math.inf).all())
    c.close(c.hs.HS_DEVERR_BAD_REQUEST)
