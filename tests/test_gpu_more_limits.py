"""Windowed attention, page weights, eviction and verification at the edge of what they accept:
offsets past 32 bits, lengths past max_ctx, rows that are not finite beside ones that are seen,
long vocabularies, many requests."""
import math

import numpy as np
import pytest
import torch

import _more as M
import _pages as P
from test_gpu_more import (I32, SCALE, Cache, Tables, a_draft, a_tree, attend_window, check_verify, check_weights,
                           check_window, i32, lse_of, normal, pool, run_evict, run_verify, run_weights, workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("T,H,window,n_sink", [(4, 128, 100, 3), (16, 40, 70, 0)])
def test_window_trees_one_after_the_other(T, H, window, n_sink):
    B = 40
    g = torch.Generator().manual_seed(1)
    ctx = [T + int(x) for x in torch.randint(0, 500, (B,), generator=g)]
    c = Cache("bf16", ctx)
    q, tree = normal(2, B, T, H, P.DIM), a_tree(3, B, T)
    tree[::7, T // 2] = 0
    out, lse = attend_window(c, q, window, n_sink, tree)
    check_window(c, q, out, lse, window, n_sink, tree, tokens=sorted({0, 1, T // 2, T - 1}))
    c.close()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("column", [0, 300, 511, 512, 575])
def test_hidden_rows_that_are_not_finite(bad, column):
    """One value that is not finite in a row that some query tokens do not see: theirs are as if
    it were not there, with zeros and tiny values among the queries, over all pages and in a
    window."""
    T, L = 5, 3 * 64 + 40
    c = Cache("bf16", [L], garbage=False)
    at = L - 2  # seen by the last two query tokens of a chain alone
    c.pool.gpu_rows()[c.row(0, at)].view(torch.bfloat16)[column] = bad
    q = normal(4, 1, T, 16, P.DIM)
    q[0, :, 0] = 0
    q[0, :, 1] *= 2.0 ** -120
    q[0, :, 2, column] = 0
    clean = c.kv(0, range(L))
    clean[at] = 0
    for window in (None, 100):
        if window:
            out, lse = attend_window(c, q, window, 2)
        else:
            out, lse = torch.zeros(1, T, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, T, 16, device="cuda")
            c.pool.page_mla_decode(q, None, i32(0), None, SCALE, out, lse, workspace(c.hs.hs_page_decode_workspace_bytes(1, T, 16, c.P)))
            torch.cuda.synchronize()
        for t in range(T - 2):
            keep = M.window_mask(L, T, None, t, window or 10 ** 9, 2).cuda()
            P.check_attention(out[0, t], lse[0, t], *P.attention(q[0, t].double(), clean, keep, SCALE), what=f"token {t}")
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_rows_past_32_bits(dtype):
    """Pages in blocks whose rows begin past 2^32 bytes."""
    ctx = [300, 500]
    c = Cache(dtype, ctx, garbage=False)
    small, n = c.pool, 120000 if dtype == "fp8" else 60000
    c.pool = c.hs.Pool(dtype=small.cfg.dtype, n_gpu_blocks=n, n_host_blocks=0, max_requests=2, max_ctx=c.max_ctx, max_topk=32)
    c.set_ctx(ctx)
    k = small.cfg.n_gpu_blocks
    assert (n - k) * 64 * small.row_bytes > 2 ** 32
    c.pool.gpu_rows()[-64 * k:] = small.gpu_rows()
    if dtype == "fp8":
        c.pool.gpu_scales()[-64 * k:] = small.gpu_scales()
    c.table[c.table >= 0] += n - k
    for r in range(2):
        c.pool.page_map_range(r, 0, c.table[r], c.table[r] * 0 - 1)
    torch.cuda.synchronize()
    small.close()
    q = normal(5, 2, 3, 16, P.DIM)
    out, lse = attend_window(c, q, 130, 4)
    check_window(c, q, out, lse, 130, 4)
    lse = lse_of(c, q)
    check_weights(c, run_weights(c, q, lse), q, lse)
    big = normal(6, 2, 200, 128, P.DIM)  # units one after the other, FP8 ones by themselves
    out, lse = attend_window(c, big, 130, 4)
    check_window(c, big, out, lse, 130, 4, tokens=[0, 99, 199])
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_lengths_past_max_ctx_are_taken_as_max_ctx(dtype):
    c = Cache(dtype, [256, 200], max_ctx=256)
    c.ctx = [256, 200]
    c.pool.set_ctx_lens(i32(100000, 200))
    hs = c.hs
    q = normal(7, 2, 2, 16, P.DIM)
    out, lse = attend_window(c, q, 70, 3)
    check_window(c, q, out, lse, 70, 3)
    assert c.pool.get_error() == hs.HS_DEVERR_INDEX_RANGE
    big = normal(8, 2, 200, 128, P.DIM)
    out, lse = attend_window(c, big, 70, 3)
    check_window(c, big, out, lse, 70, 3, tokens=[0, 100, 199])
    assert c.pool.get_error() == hs.HS_DEVERR_INDEX_RANGE
    lse = torch.full((2, 2, 16), 5.0, device="cuda")
    check_weights(c, run_weights(c, q, lse), q, lse)
    assert c.pool.get_error() == hs.HS_DEVERR_INDEX_RANGE
    c.pool.set_ctx_lens(i32(-5, 200))
    c.ctx = [0, 200]
    check_weights(c, run_weights(c, q, lse), q, lse)
    out, lse = attend_window(c, q, 70, 3)
    check_window(c, q, out, lse, 70, 3)
    c.close()


def test_weights_of_many_requests():
    B = 3000
    g = torch.Generator().manual_seed(9)
    ctx = torch.randint(0, 200, (B,), generator=g).tolist()
    c = Cache("fp8", ctx, max_ctx=256)
    q = normal(10, B, 1, 8, P.DIM)
    lse = lse_of(c, q)
    w = run_weights(c, q, lse)
    check_weights(c, w, q, lse, which=list(range(0, B, 211)) + [B - 1])
    some = torch.tensor([x > 0 for x in ctx]).cuda()
    total = torch.where(w == -7.0, 0.0, w).sum(1)
    assert bool(((total - 8.0 * some).abs() <= 0.01).all())
    c.close()


@pytest.mark.parametrize("T,H", [(1, 1), (1, 70000), (2000, 16), (5, 333)])
def test_weights_of_few_and_of_very_many_rows(T, H):
    c = Cache("bf16", [max(T, 70), T + 130])
    q = normal(11, 2, T, H, P.DIM)
    lse = torch.full((2, T, H), 6.0, device="cuda")
    check_weights(c, run_weights(c, q, lse), q, lse)
    c.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["draft", "tree"])
@pytest.mark.parametrize("V", [245760, 245761, 700001])
def test_verify_long_vocabularies(pool, dtype, kind, V):
    """Several batches for each kept sum."""
    x = a_draft(12, 2, 3, V, dtype, kind, sharp=0.5)
    check_verify(run_verify(pool, *x), *x)
    tokens, p, q, tree, u = x
    for b in range(2):  # the last values, where only they are left
        p[b, :, :V - 5] = 0
        if q is not None:
            q[b] = 0
    check_verify(run_verify(pool, *x), *x)


def test_verify_rows_past_32_bits(pool):
    """Rows 2^31 elements apart, beside each other and past 2^32 bytes."""
    V, far = 1000, 2 ** 31 + 8
    tokens, p, q, _, u = a_draft(13, 1, 3, V, torch.bfloat16, "draft")
    buf = torch.empty(2 * far + V, dtype=torch.bfloat16, device="cuda")
    wide = buf.as_strided((1, 3, V), (3 * far, far, 1))
    wide.copy_(p)
    check_verify(run_verify(pool, tokens, wide, q, None, u), tokens, p, q, None, u)
    u[0, 1:] = 0  # all accepted: the last row
    got = run_verify(pool, tokens, wide, q, None, u)
    check_verify(got, tokens, p, q, None, u)
    assert got[1] == [3]


@pytest.mark.parametrize("B", [1000, 20000])
def test_verify_many_requests(pool, B):
    tokens, p, q, _, u = a_draft(14, 200, 3, 50, torch.float32, "draft", sharp=2.0)
    want = run_verify(pool, tokens, p, q, None, u)
    n = B // 200
    got = run_verify(pool, tokens.repeat(n, 1), p.repeat(n, 1, 1), q.repeat(n, 1, 1), None, u.repeat(n, 1))
    assert got[0] == want[0] * n and got[1] == want[1] * n and got[2] == want[2] * n


def test_evict_many_requests():
    """More requests than CTAs or clusters at once."""
    for ctx, n in ((900, 400), (70 * 64 * 40, 60)):
        c = Tables([ctx - 64 * (i % 7) for i in range(n)], seed=n)
        w = torch.rand(c.R, c.P, generator=torch.Generator().manual_seed(n))
        kept, freed, count = run_evict(c, list(range(n)), [i % 40 for i in range(n)], w.cuda(), 64, 1, 1, False, True)
        for r in range(0, n, 7):
            stay, gone = M.evict(c.table[r], c.saved[r], w[r].tolist(), c.ctx[r], r % 40, 1, 1, False)
            assert kept[r] == stay + [-1] * (64 - len(stay)) and count[r] == len(gone)
            assert freed[r][:len(gone)] == c.table[r, gone].tolist()
        c.close()


def test_plans_captured_with_one_workspace_and_replayed_in_turn():
    """Two graphs that share their workspaces, replayed one after the other: each writes all that
    it reads."""
    c = Cache("bf16", [9000, 5000])
    B, T, H = 2, 4, 96
    q = [normal(15 + i, B, T, H, P.DIM) for i in range(2)]
    lse = [lse_of(c, x) for x in q]
    want = [(run_weights(c, x, y), *attend_window(c, x, 6000, 4)) for x, y in zip(q, lse)]
    hs, req = c.hs, torch.arange(B, **I32)
    ws = workspace(max(hs.hs_weights_workspace_bytes(c.pool.handle, B, T, H), hs.hs_window_workspace_bytes(c.pool.handle, B, T, H, 6000, 4)))
    outs = [(torch.full_like(want[0][0], -7.0), torch.zeros_like(want[0][1]), torch.zeros_like(want[0][2])) for _ in range(2)]
    graphs, side = [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=side):
            c.pool.page_weights(q[i], lse[i], req, None, SCALE, outs[i][0], None, 1.0, ws)
            c.pool.page_mla_decode_window(q[i], req, None, 6000, 4, SCALE, outs[i][1], outs[i][2], ws)
    for i in (0, 1, 1, 0, 1, 0):
        for x in outs[i]:
            x.fill_(-7)
        ws.fill_(0xFF)
        graphs[i].replay()
        graphs[1 - i].replay()
        torch.cuda.synchronize()
        for j in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[j], want[j]))
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H", [(1, 33), (2, 40), (1, 129), (1, 257), (33, 8), (3, 107), (5, 104), (33, 20), (2, 449)])
def test_weights_of_rows_dealt_to_uneven_groups(dtype, T, H):
    """Groups of 64, 96, 160, 192, 224 columns, the last one not full, over ranges that come to
    several requests; with a tree too."""
    B = 40
    g = torch.Generator().manual_seed(31)
    ctx = [T + int(x) for x in torch.randint(0, 900, (B,), generator=g)]
    ctx[7] = 0
    c = Cache(dtype, ctx)
    q = normal(32, B, T, H, P.DIM)
    for tree in (None, a_tree(33, B, T)):
        lse = lse_of(c, q, tree)
        w = run_weights(c, q, lse, tree)
        check_weights(c, w, q, lse, tree, which=[0, 7, 8, 21, B - 1])
        total, seen = torch.where(w == -7.0, 0.0, w).sum(1), torch.isfinite(lse).sum((1, 2)).float()
        assert bool(((total - seen).abs() <= 2.0 ** -10 * seen).all())
        assert torch.equal(w, run_weights(c, q, lse, tree))
    c.close()


@pytest.mark.parametrize("pages", [31, 33, 64, 255, 511, 512, 513, 537, 2049, 4097])
@pytest.mark.parametrize("kind", ["one value", "two values", "narrow", "a few apart"])
def test_evict_where_many_pages_are_near_the_border(pages, kind):
    """Equal weights in one warp and in several, and bins of the border that hold hundreds of pages."""
    g = torch.Generator().manual_seed(34)
    c = Tables([64 * pages - 5] * 4, seed=35, holes=0.05)
    x = torch.rand(c.R, c.P, generator=g)
    if kind == "one value":
        x.fill_(0.25)
    elif kind == "two values":
        x = (x > 0.5).float()
    elif kind == "narrow":  # 512 values next to each other
        x = (0x3F800000 + (x * 512).int()).view(torch.float32)
    else:  # most pages alike, few of other magnitudes
        x = torch.where(x < 0.02, x * 1e30, torch.where(x < 0.04, x * 1e-30, 1.0 + 2.0 ** -23 * (x * 4).floor()))
    budget = [2, pages // 3, pages - 1, pages // 2 + 1]
    kept, freed, count = run_evict(c, range(4), budget, x.cuda(), c.P, plan=True)
    for r in range(4):
        stay, gone = M.evict(c.table[r], c.saved[r], x[r].tolist(), c.ctx[r], budget[r], 1, 1, False)
        assert kept[r] == stay + [-1] * (c.P - len(stay)) and count[r] == len(gone)
        assert freed[r][:len(gone)] == [int(c.table[r, p]) for p in gone]
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_weights_see_what_was_written_just_before(dtype):
    """Rows appended, lengths set, queries and pages changed directly before each call in the same
    stream, one workspace for all: eager, and as one graph."""
    B, T, H, new = 3, 2, 40, 2000
    lens = [i32(9000, 7000, 8000), i32(8500, 9000, 6001)]
    c = Cache(dtype, [9000, 7000, 8000], max_ctx=9000)
    c.pool.page_map_range(1, 0, np.resize(c.table[1][c.table[1] >= 0], c.P).astype(np.int32), np.full(c.P, -1, np.int32))
    hs, req = c.hs, torch.arange(B, **I32)
    rows = [normal(41 + i, B, new, P.DIM) for i in range(2)]
    q = [normal(43 + i, B, T, H, P.DIM) for i in range(2)]
    c.set_ctx([9000, 7000, 8000])
    lse = torch.full((B, T, H), 3.0, device="cuda")
    ws = workspace(hs.hs_weights_workspace_bytes(c.pool.handle, B, T, H))
    now = torch.empty_like(q[0])

    def step(i, w, sync):
        for call in (lambda: c.pool.set_ctx_lens(lens[i]), lambda: c.pool.append_rows(rows[i], req), lambda: now.copy_(q[i]),
                     lambda: c.pool.page_weights(now, lse, req, None, SCALE, w, None, 1.0, ws)):
            call()
            if sync:
                torch.cuda.synchronize()

    blank = torch.full((c.R, c.P), -7.0, device="cuda")
    want = [blank.clone() for _ in range(2)]
    for i in (0, 1, 0, 1):
        want[i].fill_(-7.0)
        step(i, want[i], True)
    assert not torch.equal(want[0], want[1])
    outs = [blank.clone() for _ in range(12)]
    for i in range(12):
        step(i % 2, outs[i], False)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], want[i % 2]) for i in range(2, 12))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        for i in range(12):
            step(i % 2, outs[i], False)
    for w in outs:
        w.fill_(-7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], want[i % 2]) for i in range(2, 12))
    c.close()
