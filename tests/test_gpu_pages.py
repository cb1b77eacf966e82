"""Append, page means, page selection and attention over pages on the GPU, against
plain forms in 64 bits (tests/_pages.py, which derives the tolerances)."""
import math

import numpy as np
import pytest
import torch

import _pages as P

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(P.DIM)
I32 = {"dtype": torch.int32, "device": "cuda"}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available()


def i32(*v):
    return torch.tensor(v, **I32)


class Cache:
    """A pool with each request's pages at scattered blocks, and its plain mirror."""

    def __init__(self, dtype, ctx, max_ctx=None, host=0, seed=0, garbage=True, extra=0, hot_rows=64, max_topk=32):
        import tiered_sparse_mla_gb300 as hs
        self.hs, self.dtype, self.ctx, self.R = hs, dtype, list(ctx), len(ctx)
        self.max_ctx = max_ctx or max(64, max(ctx))
        self.P = -(-self.max_ctx // 64)
        g = torch.Generator().manual_seed(seed)
        n = max(1, sum(-(-c // 64) for c in ctx)) + extra
        fp8 = dtype == "fp8"
        self.pool = hs.Pool(dtype=hs.HS_FP8_E4M3_ROWSCALE if fp8 else hs.HS_BF16, n_gpu_blocks=n,
                            n_host_blocks=host, max_requests=self.R, max_ctx=self.max_ctx, max_topk=max_topk,
                            hot_rows=hot_rows)
        self.table = np.full((self.R, self.P), -1, np.int32)
        blocks = torch.randperm(n, generator=g).numpy().astype(np.int32)
        at = 0
        for r, c in enumerate(ctx):
            k = -(-c // 64)
            self.table[r, :k] = blocks[at:at + k]
            at += k
            self.pool.page_map_range(r, 0, self.table[r], self.table[r] * 0 - 1)
        self.spare = blocks[at:]
        self.set_ctx(ctx)
        x = torch.randn(n * 64, P.DIM, generator=g)
        rows, scales = self.pool.gpu_rows(), self.pool.gpu_scales()
        if fp8:
            c, s = P.quantise(x.to(torch.bfloat16))
            rows.copy_(c.view(torch.uint8))
            scales.copy_(s)
        else:
            rows.copy_(x.to(torch.bfloat16).view(torch.uint8))
        if garbage:  # rows past a context: NaN bytes, NaN and infinite scales
            for r, c in enumerate(ctx):
                if c % 64:
                    b = int(self.table[r, c // 64]) * 64
                    rows[b + c % 64:b + 64] = 0xFF
                    if fp8:
                        scales[b + c % 64:b + 64] = math.nan
                        scales[b + 63] = math.inf
        torch.cuda.synchronize()

    def set_ctx(self, ctx):
        self.ctx = list(ctx)
        self.pool.set_ctx_lens(torch.tensor(self.ctx, **I32))

    def row(self, r, pos):
        return int(self.table[r, pos // 64]) * 64 + pos % 64

    def values(self):
        return P.values(self.pool.gpu_rows(), self.pool.gpu_scales())

    def kv(self, r, positions):
        t = torch.from_numpy(self.table[r].astype(np.int64)).cuda()
        pos = torch.as_tensor(positions, device="cuda").long()
        at = t[pos // 64] * 64 + pos % 64
        s = self.pool.gpu_scales()
        return P.values(self.pool.gpu_rows()[at], None if s is None else s[at])

    def close(self, err=0):
        torch.cuda.synchronize()
        got = self.pool.get_error()
        self.pool.close()
        assert got == err, f"device error bits {got}, expected {err}"


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def attend(c, q, pages, tree=None, req=None, per_token=False, scale=SCALE, n_pages=0):
    hs = c.hs
    B, T, H = q.shape[:3]
    out = torch.full((B, T, H, 512), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, H), math.nan, device="cuda")
    N = (n_pages or c.P) if pages is None else pages.shape[-1]
    n = hs.hs_page_decode_workspace_bytes(*((B * T, 1) if per_token else (B, T)), H, N)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    req = torch.arange(B, **I32) if req is None else req
    if per_token:
        c.pool.page_mla_decode_per_token(q, pages, req, tree, scale, out, lse, ws)
    else:
        c.pool.page_mla_decode(q, pages, req, tree, scale, out, lse, ws, n_pages=n_pages)
    torch.cuda.synchronize()
    return out, lse


def check(c, q, out, lse, pages_of, tree=None, req=None, scale=SCALE):
    """pages_of(b, t): the list of pages (repeats count), or None for all."""
    B, T = q.shape[:2]
    for b in range(B):
        r = b if req is None else req[b]
        L = c.ctx[r]
        for t in range(T):
            pg = pages_of(b, t)
            pos = torch.arange(L) if pg is None else torch.cat(
                [torch.arange(p * 64, min(L, p * 64 + 64)) for p in pg] + [torch.zeros(0, dtype=torch.long)])
            keep = P.seen_mask(L, T, None if tree is None else tree[b].tolist(), t)[pos] if L else torch.zeros(0, dtype=torch.bool)
            pos = pos[keep]
            kv = c.kv(r, pos)
            ref = P.attention(q[b, t].double(), kv, torch.ones(len(pos), dtype=torch.bool, device="cuda"), scale)
            P.check_attention(out[b, t], lse[b, t], *ref, what=f"request {b} token {t}")


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,pick", [(1, 1, False), (3, 5, True), (2, 64, True), (2, 129, False), (5, 33, False)])
def test_append(dtype, B, T, pick):
    ctx = [T + 100 + 37 * b for b in range(B)]
    c = Cache(dtype, ctx, garbage=False)
    x = normal(1, B, T, P.DIM)
    x[0, 0] = 0  # a row of zeros
    x[-1, -1] *= 2.0 ** -120  # near the smallest values
    index = None
    if pick:
        g = torch.Generator().manual_seed(2)
        index = torch.where(torch.rand(B, T, generator=g) < 0.5, torch.randint(0, T, (B, T), generator=g), -1)
        index = index.to(torch.int32).cuda()
    before, s0 = c.pool.gpu_rows().clone(), None if dtype == "bf16" else c.pool.gpu_scales().clone()
    req = torch.arange(B, **I32).flip(0)  # not in order
    c.pool.append_rows(x, req, None, index)  # positions ctx - T ..
    torch.cuda.synchronize()
    want, ws = before.clone(), None if s0 is None else s0.clone()
    for b in range(B):
        r = B - 1 - b
        for k in range(T):
            i = k if index is None else int(index[b, k])
            if i < 0:
                continue
            at = c.row(r, ctx[r] - T + k)
            if dtype == "bf16":
                want[at] = x[b, i].view(torch.uint8)
            else:
                code, s = P.quantise(x[b, i].cpu())
                want[at] = code.view(torch.uint8).cuda()
                ws[at] = float(s)
    assert torch.equal(c.pool.gpu_rows(), want)  # other rows as they were
    if ws is not None:
        assert torch.equal(c.pool.gpu_scales(), ws)
    # the same rows at the same places, named by their first position
    c.pool.append_rows(x, req, torch.tensor([ctx[int(r)] - T for r in req], **I32), index)
    torch.cuda.synchronize()
    assert torch.equal(c.pool.gpu_rows(), want)
    c.close()


def test_append_fp8_codes_of_every_kind():
    """Wide ranges of magnitudes and exact ties: codes and scales equal the definition's."""
    n = 512
    c = Cache("fp8", [n], garbage=False)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(n, P.DIM, generator=g) * torch.exp2(torch.randint(-130, 120, (n, 1), generator=g).float())
    x[:64] = torch.randint(-480, 481, (64, P.DIM), generator=g).float()  # integers: many ties
    x[64:96] = x[64:96] * torch.exp2(torch.randint(-40, 1, (32, P.DIM), generator=g).float())
    x = x.to(torch.bfloat16)
    c.pool.append_rows(x[None].cuda(), i32(0), i32(0))
    torch.cuda.synchronize()
    code, s = P.quantise(x)
    at = torch.tensor([c.row(0, p) for p in range(n)])
    assert torch.equal(c.pool.gpu_scales().cpu()[at], s)
    got = c.pool.gpu_rows().cpu()[at]
    same = got == code.view(torch.uint8)
    zero = (got & 0x7f == 0) & (code.view(torch.uint8) & 0x7f == 0)  # the sign of a zero
    assert bool((same | zero).all())
    c.close()


def test_append_nonfinite_rows_read_as_nan():
    c = Cache("fp8", [64], garbage=False)
    x = normal(4, 1, 3, P.DIM)
    x[0, 0, 5] = math.inf
    x[0, 1, 575] = math.nan
    c.pool.append_rows(x, i32(0), i32(7))
    torch.cuda.synchronize()
    v = c.kv(0, range(7, 10))
    assert bool(torch.isnan(v[:2]).all()) and bool(torch.isfinite(v[2]).all())
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_append_reaches_host_copy_and_hot_slot(dtype):
    """Pages with a host copy, and positions held in the hot buffer, stay coherent."""
    c = Cache(dtype, [256], host=4, garbage=False, extra=1)
    c.pool.hot_lease(0, [int(c.spare[0])])
    host = np.array([2, 0, 3, 1], np.int32)
    gpu = c.table[0, :4].copy()
    gpu[1] = -1  # page 1: only on the host
    c.pool.page_map_range(0, 0, gpu, host)
    c.pool.host_rows()[:] = 0
    if dtype == "fp8":
        c.pool.host_scales()[:] = 1.0
    # positions 70 and 71 become hot
    top = torch.tensor([[70, 71]], **I32)
    res, cnt = torch.empty(1, 2, **I32), torch.empty(1, 3, **I32)
    c.pool.resolve_topk(i32(0), top, res, None, None, cnt)
    x = normal(5, 1, 20, P.DIM)
    c.pool.append_rows(x, i32(0), i32(55))  # positions 55 .. 74: pages 0 and 1
    torch.cuda.synchronize()
    code = x[0].view(torch.uint8).cpu() if dtype == "bf16" else P.quantise(x[0].cpu())[0].view(torch.uint8)
    rows, hrows = c.pool.gpu_rows().cpu(), c.pool.host_rows()
    for k in range(20):
        pos = 55 + k
        assert np.array_equal(hrows[host[pos // 64] * 64 + pos % 64], code[k].numpy()), pos
        if pos < 64:
            assert torch.equal(rows[c.row(0, pos)], code[k])
    assert int(cnt[0, 2]) == 2
    for i, pos in enumerate((70, 71)):
        assert torch.equal(rows[int(res[0, i])], code[pos - 55])
    c.pool.resolve_topk(i32(0), top, res, None, None, cnt)
    torch.cuda.synchronize()
    assert cnt.tolist() == [[0, 2, 0]]
    c.close()


def test_append_skips_what_it_cannot_place():
    c = Cache("bf16", [100, 60], max_ctx=256, garbage=False)
    hs = c.hs
    before = c.pool.gpu_rows().clone()

    def put(req, start, index=None, T=2):
        x = normal(6, 1, T, P.DIM)
        c.pool.append_rows(x, i32(req), i32(start), None if index is None else torch.tensor([index], **I32))
        return x, c.pool.get_error()

    assert put(7, 0)[1] == hs.HS_DEVERR_BAD_REQUEST
    assert put(-1, 0)[1] == hs.HS_DEVERR_BAD_REQUEST
    assert put(0, 256)[1] == hs.HS_DEVERR_INDEX_RANGE
    assert put(0, -5)[1] == hs.HS_DEVERR_INDEX_RANGE
    assert put(0, 10, [2, -2])[1] == hs.HS_DEVERR_INDEX_RANGE
    assert put(1, 64)[1] == hs.HS_DEVERR_BAD_PAGE  # page 1 of request 1 is not mapped
    assert torch.equal(c.pool.gpu_rows(), before)
    x, err = put(1, 63)  # the first row has a page, the second none
    assert err == hs.HS_DEVERR_BAD_PAGE
    before[c.row(1, 63)] = x[0, 0].view(torch.uint8)
    assert torch.equal(c.pool.gpu_rows(), before)
    c.close()


# ------------------------------------------------------------------ means
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_page_means(dtype):
    ctx = [1, 63, 64, 65, 300, 0]
    c = Cache(dtype, ctx, max_ctx=320, host=2)
    means = torch.full((c.R, c.P, P.DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    pairs = [(r, p) for r, n in enumerate(ctx) for p in range(-(-n // 64))] + [(4, 2)]  # one of them twice
    # a page that is only on the host
    host = np.full(5, -1, np.int32)
    host[1] = 1
    gpu = c.table[4].copy()
    src = c.row(4, 64)
    c.pool.host_rows()[64:128] = c.pool.gpu_rows()[src:src + 64].cpu().numpy()
    if dtype == "fp8":
        c.pool.host_scales()[64:128] = c.pool.gpu_scales()[src:src + 64].cpu().numpy()
    gpu[1] = -1
    c.pool.page_map_range(4, 0, gpu, host)
    c.pool.page_means(i32(*(a for a, _ in pairs)), i32(*(b for _, b in pairs)), means)
    torch.cuda.synchronize()
    done = torch.zeros(c.R, c.P, dtype=torch.bool)
    for r, p in pairs:
        done[r, p] = True
        v = c.kv(r, range(64 * p, min(ctx[r], 64 * p + 64)))
        ref, n = v.mean(0), v.shape[0]
        # one rounding to BF16, and 32-bit sums of n terms
        tol = 2.0 ** -8 * ref.abs() + n * 2.0 ** -23 * v.abs().mean(0)
        assert bool(((means[r, p].double() - ref).abs() <= tol).all()), (r, p)
    assert bool((means[~done.cuda()] == 7.0).all())  # the others as they were
    c.close()


def test_page_means_skips_and_empties():
    c = Cache("bf16", [64, 10], max_ctx=192, garbage=False)
    means = torch.full((2, 3, P.DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    c.set_ctx([0, 10])  # page 0 of request 0 holds no token now
    c.pool.page_means(i32(0, 2, 0, 1, -1), i32(0, 0, 3, 1, 0), means)
    torch.cuda.synchronize()
    assert not means[0, 0].any()
    assert bool((means[0, 1:] == 7.0).all()) and bool((means[1] == 7.0).all())
    c.close(c.hs.HS_DEVERR_BAD_PAGE)


# ------------------------------------------------------------------ selection
def run_select(c, q, means, N, n_first=1, n_last=2, tree=None, req=None, topk=False):
    B, T = q.shape[:2]
    pages = torch.full((B, T, N), -7, **I32)
    tk = torch.full((B, T, N * 64), -7, **I32) if topk else None
    ws = torch.full((c.hs.hs_select_workspace_bytes(c.pool.handle, B, T),), 0xFF, dtype=torch.uint8, device="cuda")
    req = torch.arange(B, **I32) if req is None else req
    c.pool.select_pages(q, means, req, pages, n_first, n_last, tree, tk, ws)
    torch.cuda.synchronize()
    return (pages, tk) if topk else pages


def check_select(c, q, means, pages, n_first, n_last, tree=None, req=None):
    B, T = q.shape[:2]
    N = pages.shape[2]
    for b in range(B):
        r = b if req is None else req[b]
        for t in range(T):
            end = c.ctx[r] if tree is not None else max(0, c.ctx[r] - T + t + 1)
            want = P.select(q[b, t].double(), means[r].double(), -(-end // 64), N, n_first, n_last)
            got = pages[b, t].tolist()
            assert got[:len(want)] == want and got[len(want):] == [-1] * (N - len(want)), (b, t)


def sparse_cache(ctx, max_ctx=None):
    """Selection reads lengths and means alone: no page needs to be mapped."""
    import tiered_sparse_mla_gb300 as hs
    c = Cache.__new__(Cache)
    c.hs, c.R, c.max_ctx = hs, len(ctx), max_ctx or max(ctx)
    c.P = -(-c.max_ctx // 64)
    c.pool = hs.Pool(dtype=hs.HS_BF16, n_gpu_blocks=1, n_host_blocks=0, max_requests=c.R, max_ctx=c.max_ctx,
                     max_topk=32)
    c.set_ctx(ctx)
    return c


@pytest.mark.parametrize("B,T,H,ctx,N", [(1, 1, 16, 4096, 4), (3, 2, 8, 20000, 7), (2, 3, 24, 9000, 20),
                                         (2, 1, 128, 70001, 32), (2, 4, 128, 33000, 16), (1, 5, 100, 8300, 9),
                                         (4, 1, 1, 1000, 3), (2, 2, 16, 300000, 64)])
def test_select(B, T, H, ctx, N):
    lens = [max(1, ctx - 777 * b) for b in range(B)]
    c = sparse_cache(lens)
    means = torch.randn(c.R, c.P, P.DIM, generator=torch.Generator().manual_seed(7)).mul(0.2).to(torch.bfloat16).cuda()
    for r, n in enumerate(lens):  # what lies past a context says nothing
        means[r, -(-n // 64):] = math.nan
    q = normal(8, B, T, H, P.DIM)
    for nf, nl in ((1, 2), (0, 0), (N, 0)):
        if nf + nl <= N:
            check_select(c, q, means, run_select(c, q, means, N, nf, nl), nf, nl)
    c.close()


@pytest.mark.parametrize("B,T,H,long", [(350, 1, 300, 40000), (60, 3, 128, 60000), (33, 2, 16, 20000)])
def test_select_many_requests(B, T, H, long):
    """Lists of many lengths laid end to end: empty requests, one page, several tiles of
    pages, the same request more than once, unknown ones in between."""
    g = torch.Generator().manual_seed(B)
    lens = [0, 1, 64, long, long - 12345] + torch.randint(1, 3000, (15,), generator=g).tolist()
    c = sparse_cache(lens)
    means = normal(15, c.R, c.P, P.DIM)
    for r, n in enumerate(lens):
        means[r, -(-n // 64):] = math.nan
    q = normal(16, B, T, H, P.DIM)
    req = torch.randint(-2, c.R + 3, (B,), generator=g).tolist()
    pages = run_select(c, q, means, 5, req=i32(*req))
    for b, r in enumerate(req):
        if 0 <= r < c.R:
            check_select(c, q[b:b + 1], means, pages[b:b + 1], 1, 2, req=[r])
        else:
            assert bool((pages[b] == -1).all())
    c.close(c.hs.HS_DEVERR_BAD_REQUEST)


def test_select_ties_and_near_ties():
    """Equal scores go to the lower page, and scores that differ by less than 32-bit
    sums can tell are told apart."""
    c = sparse_cache([64 * 4000] * 4)
    g = torch.Generator().manual_seed(9)
    means = torch.zeros(4, c.P, P.DIM)
    means[0] = 1.0                                             # all pages alike
    means[1] = torch.randint(-2, 3, (c.P, 1), generator=g)     # five values
    base = torch.randn(P.DIM, generator=g) * 64                # large terms that cancel, a small rest
    means[2] = base
    means[2, :, 0] = torch.randint(-3, 4, (c.P,), generator=g) * 2.0 ** -9
    means[3] = torch.randn(c.P // 8, P.DIM, generator=g).repeat(8, 1)  # every page eight times
    means = means.to(torch.bfloat16).cuda()
    q = normal(10, 4, 2, 16, P.DIM)
    q[2, :, :, 0] = 1.0
    q[2, :, 1:] = q[2, :, :1]  # heads alike: no head is the best by itself
    q[0, 1] = 0.0
    for N in (5, 40, 700):
        check_select(c, q, means, run_select(c, q, means, N), 1, 2)
    c.close()


def test_select_where_short_sums_lose_the_most():
    """One product so large that sums held beside it lose every other one: the scores of
    two pages are then off by 2^-15.84 |q||c| in opposite directions, and their order in
    exact sums is the other one."""
    c = sparse_cache([64 * 600] * 2)
    small = 2.0 ** -5 * (1 - 2.0 ** -8)
    means = torch.zeros(2, c.P, P.DIM)
    means[:, :, 0] = 512.0
    up, down = means[:, 0].clone(), means[:, 0].clone()
    up[:, 0] = down[:, 0] = 1024.0
    up[:, 2:], down[:, 2:] = small, -small
    down[:, 1] = 35.0 / 32                     # 574 * 2 * small = 35.74 > 35
    for r, (i, j) in enumerate(((100, 300), (300, 100))):
        means[r, i], means[r, j] = up[r], down[r]
    q = torch.ones(2, 1, 8, P.DIM)
    q[..., 0], q[..., 1] = 1024.0, 32.0
    q, means = q.to(torch.bfloat16).cuda(), means.to(torch.bfloat16).cuda()
    pages = run_select(c, q, means, 3, 1, 1)
    check_select(c, q, means, pages, 1, 1)
    assert pages[:, 0, 1].tolist() == [100, 300]
    c.close()


def test_select_with_infinities_and_nan():
    c = sparse_cache([64 * 900] * 3)
    means = torch.randn(3, c.P, P.DIM, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16).cuda()
    means[0, 5, 3] = math.nan
    means[0, 17, 9] = math.inf
    means[0, 400] = -math.inf
    means[1, 20:30] = 3e38  # sums beyond 32 bits
    means[2, :, 7] = math.nan
    q = normal(12, 3, 1, 8, P.DIM)
    check_select(c, q, means, run_select(c, q, means, 12), 1, 2)
    q[0, 0, 3, 0] = math.inf
    q[1, 0, 2, 100] = math.nan
    check_select(c, q, means, run_select(c, q, means, 12), 1, 2)
    c.close()


def test_select_short_contexts_trees_and_positions():
    lens = [0, 1, 64, 65, 500, 3]
    T, N = 4, 5
    c = sparse_cache(lens, max_ctx=1024)
    means = normal(13, 6, c.P, P.DIM)
    q = normal(14, 6, T, 8, P.DIM)
    tree = torch.tensor([[1, 3, 5, 0]] * 6, dtype=torch.int64, device="cuda")
    for tr in (None, tree):
        pages, topk = run_select(c, q, means, N, 1, 1, tr, topk=True)
        check_select(c, q, means, pages, 1, 1, tr)
        for b in range(6):
            for t in range(T):
                mask = P.seen_mask(lens[b], T, None if tr is None else tr[b].tolist(), t)
                want = []
                for p in pages[b, t].tolist():
                    want += [x if 0 <= x < lens[b] and p >= 0 and bool(mask[x]) else -1
                             for x in range(p * 64, p * 64 + 64)]
                assert topk[b, t].tolist() == want, (b, t)
    # requests in another order, one of them unknown
    req = i32(4, 9, 2)
    pages = run_select(c, q[:3], means, N, 1, 1, req=req)
    check_select(c, q[:1], means, pages[:1], 1, 1, req=[4])
    check_select(c, q[2:3], means, pages[2:], 1, 1, req=[2])
    assert bool((pages[1] == -1).all())
    c.close(c.hs.HS_DEVERR_BAD_REQUEST)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,T,H", [([1, 63, 64, 65, 129], 1, 16), ([40, 200, 1], 1, 128), ([500, 77], 3, 24),
                                     ([130, 700, 64, 5], 4, 128), ([9000], 2, 8), ([66, 67], 65, 8),
                                     ([0, 3, 2], 5, 1)])
def test_attention_over_all_pages(dtype, ctx, T, H):
    c = Cache(dtype, ctx, max_ctx=max(ctx) + 70)
    q = normal(15, len(ctx), T, H, P.DIM)
    out, lse = attend(c, q, None)
    check(c, q, out, lse, lambda b, t: None)
    # a plan for fewer or more pages gives the same up to how the splits meet
    out, lse = attend(c, q, None, n_pages=1)
    check(c, q, out, lse, lambda b, t: None)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,ctx", [(1, 8, [100, 1]), (7, 16, [1001, 64, 70]), (33, 24, [200, 33]),
                                     (64, 16, [64, 1000, 127]), (16, 128, [300])])
def test_attention_of_a_tree(dtype, T, H, ctx):
    c = Cache(dtype, ctx)
    B = len(ctx)
    g = torch.Generator().manual_seed(16)
    tree = torch.randint(-2 ** 63, 2 ** 63 - 1, (B, T), generator=g)
    tree[0, 0] = 0          # nothing of the draft
    tree[-1, T - 1] = -1    # all of it, and bits past it
    tree = tree.cuda()
    q = normal(17, B, T, H, P.DIM)
    out, lse = attend(c, q, None, tree)
    check(c, q, out, lse, lambda b, t: None, tree)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_of_a_tree_ignores_hidden_nodes(dtype):
    """A drafted row of NaN reaches the tokens that see it and no other."""
    T, L = 6, 203
    c = Cache(dtype, [L])
    bad = 2  # this node
    at = c.row(0, L - T + bad)
    if dtype == "bf16":
        c.pool.gpu_rows()[at] = 0xFF
    else:
        c.pool.gpu_scales()[at] = math.nan
    tree = [1, 3, 4, 9, 0, 0x24]
    q = normal(18, 1, T, 16, P.DIM)
    tr = torch.tensor([tree], dtype=torch.int64, device="cuda")
    out, lse = attend(c, q, None, tr)
    for t in range(T):
        if tree[t] >> bad & 1:
            assert bool(torch.isnan(out[0, t]).all()) and bool(torch.isnan(lse[0, t]).all())
        else:
            keep = P.seen_mask(L, T, tree, t)
            ref = P.attention(q[0, t].double(), c.kv(0, torch.arange(L)[keep]),
                              torch.ones(int(keep.sum()), dtype=torch.bool, device="cuda"), SCALE)
            P.check_attention(out[0, t], lse[0, t], *ref, what=f"token {t}")
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H,N,ctx", [(1, 1, 16, 4, 4096), (2, 3, 128, 9, 2000), (3, 4, 8, 33, 2100),
                                         (5, 1, 24, 1, 700), (2, 2, 64, 130, 8300)])
def test_attention_over_lists(dtype, B, T, H, N, ctx):
    lens = [ctx - 61 * b for b in range(B)]
    c = Cache(dtype, lens)
    rng = np.random.default_rng(19)
    shared = np.full((B, N), -1, np.int32)
    own = np.full((B, T, N), -1, np.int32)
    for b in range(B):
        n = -(-lens[b] // 64)
        shared[b] = rng.integers(-1, n, N)  # any order, gaps, repeats
        own[b] = rng.integers(-1, n, (T, N))
    own[0, 0] = -1  # nothing at all
    if T > 1:
        own[0, 1, :] = -1
        own[0, 1, N - 1] = (lens[0] - 1) // 64  # the last entry alone, partly seen
    q = normal(20, B, T, H, P.DIM)
    out, lse = attend(c, q, torch.from_numpy(shared).cuda())
    check(c, q, out, lse, lambda b, t: [p for p in shared[b] if p >= 0])
    out, lse = attend(c, q, torch.from_numpy(own).cuda(), per_token=True)
    check(c, q, out, lse, lambda b, t: [p for p in own[b, t] if p >= 0])
    if T > 1:
        tree = torch.tensor([[1 << t | 1 for t in range(T)]] * B, dtype=torch.int64, device="cuda")
        out, lse = attend(c, q, torch.from_numpy(own).cuda(), tree, per_token=True)
        check(c, q, out, lse, lambda b, t: [p for p in own[b, t] if p >= 0], tree)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H", [(30, 1, 16), (12, 2, 128), (21, 3, 40)])
def test_attention_of_medium_batches(dtype, B, T, H):
    """As many lists as leave two splits each: joined inside the clusters. Requests of
    one page leave a split without any; some rows lie past the last 128-row tile."""
    lens = [1500 - 47 * b if b % 5 else (1, 64, 70, 0, T)[b % 4] for b in range(B)]
    c = Cache(dtype, lens, max_ctx=1536)
    q = normal(80, B, T, H, P.DIM)
    out, lse = attend(c, q, None)
    check(c, q, out, lse, lambda b, t: None)
    rng = np.random.default_rng(81)
    own = np.full((B, T, 20), -1, np.int32)
    for b in range(B):
        n = -(-lens[b] // 64)
        for t in range(T):
            k = rng.integers(0, min(n, 20) + 1)
            own[b, t, :k] = np.sort(rng.permutation(n)[:k])
    out, lse = attend(c, q, torch.from_numpy(own).cuda(), per_token=True)
    check(c, q, out, lse, lambda b, t: [p for p in own[b, t] if p >= 0])
    again = attend(c, q, torch.from_numpy(own).cuda(), per_token=True)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H", [(80, 1, 128), (27, 3, 128), (40, 2, 80), (79, 1, 3)])
def test_attention_of_more_lists_than_fit_at_once(dtype, B, T, H):
    """Most lists whole, those of the last round in splits: a list may have tiles of both."""
    lens = [1500 - 17 * b if b % 5 else (1, 64, 70, 0, T)[b % 4] for b in range(B)]
    c = Cache(dtype, lens, max_ctx=1536)
    q = normal(85, B, T, H, P.DIM)
    out, lse = attend(c, q, None)
    check(c, q, out, lse, lambda b, t: None)
    tree = torch.randint(-2 ** 63, 2 ** 63 - 1, (B, T), generator=torch.Generator().manual_seed(86)).cuda()
    out, lse = attend(c, q, None, tree)
    check(c, q, out, lse, lambda b, t: None, tree)
    again = attend(c, q, None, tree)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    c.close()


@pytest.mark.parametrize("factor,scale", [(8.0, SCALE), (32.0, SCALE), (2.0 ** -20, SCALE * 2.0 ** 20), (0.0, SCALE)])
def test_attention_peaked_and_flat(factor, scale):
    for dtype in ("bf16", "fp8"):
        c = Cache(dtype, [1500, 300])
        q = normal(21, 2, 2, 16, P.DIM) * factor
        out, lse = attend(c, q, None, scale=scale)
        check(c, q, out, lse, lambda b, t: None, scale=scale)
        c.close()


def test_attention_fp8_scales_of_many_magnitudes():
    """Weights are even (a tiny factor), so every row's values count by its scale:
    scales that grow and fall over the pages, negative ones, zeros, the smallest one."""
    L = 1300
    c = Cache("fp8", [L, L, L])
    g = torch.Generator().manual_seed(82)
    ramp = torch.linspace(-30, 12, L)
    for r, e in enumerate((ramp, -ramp - 20, torch.randint(-18, 19, (L,), generator=g).float())):
        s = torch.exp2(e) * torch.where(torch.rand(L, generator=g) < 0.3, -1.0, 1.0)
        if r == 2:
            s[::5], s[1::5] = 0.0, 2.0 ** -126
        at = torch.tensor([c.row(r, i) for i in range(L)], device="cuda")
        c.pool.gpu_scales()[at] = s.cuda()
    q = normal(83, 3, 2, 24, P.DIM)
    out, lse = attend(c, q, None, scale=2.0 ** -30)
    check(c, q, out, lse, lambda b, t: None, scale=2.0 ** -30)
    c.pool.gpu_scales().zero_()
    out, lse = attend(c, q, None)
    check(c, q, out, lse, lambda b, t: None)
    c.close()


def test_attention_fp8_keeps_small_weights():
    """The row that takes almost all of the weight has zeros for values: what is left
    are values at a weight of e^-18 = 2^-26. F16's smallest step, 2^-24 of a weight kept
    at 2^10 times itself, puts such a weight off by at most 2^-35 / 2^-26 = 2^-9 of it
    (times 2^-7 / 0.0074, the scales' reference over the row's): less than a weight's
    rounding to BF16, which the check allows."""
    c = Cache("fp8", [2], garbage=False)
    x = torch.zeros(2, P.DIM)
    x[0, 512:] = 6.75  # scores 64 * 6.75 / 24 = 18 above those of the other row
    x[1, :512] = torch.randn(512, generator=torch.Generator().manual_seed(87)).clamp(-3.3, 3.3)
    x[1, 0] = 3.3
    codes, scale = P.quantise(x.to(torch.bfloat16))
    at = torch.tensor([c.row(0, 0), c.row(0, 1)], device="cuda")
    c.pool.gpu_rows()[at] = codes.view(torch.uint8).cuda()
    c.pool.gpu_scales()[at] = scale.cuda()
    q = torch.zeros(1, 1, 16, P.DIM)
    q[..., 512:] = 1.0
    q = q.to(torch.bfloat16).cuda()
    out, lse = attend(c, q, None)
    check(c, q, out, lse, lambda b, t: None)
    c.close()


def test_attention_fp8_queries_with_outliers():
    """A query's values are the sums of two e4m3 codes each, at a power of two that
    brings the row's largest to (224, 448]: values of at least 2^-10 of the largest are
    exact, and smaller ones off by at most half the codes' smallest step, 2^-10 / 224 of
    the largest. Rows of very different magnitudes do not touch each other."""
    L = 700
    c = Cache("fp8", [L])
    q = normal(84, 1, 2, 32, P.DIM)
    big = 2.0 ** torch.arange(0, 8).float()
    for h in range(32):
        q[0, :, h, 37 * h % 576] = float(big[h % 8]) * 3
    q[0, 0, 8:16] *= 2.0 ** -40
    q[0, 0, 16] = 0.0
    q[0, 0, 17, 5], q[0, 0, 18, 7], q[0, 0, 19, 9] = math.inf, -math.inf, math.nan
    out, lse = attend(c, q, None)
    broken = [17, 18, 19]
    assert bool(torch.isnan(out[0, 0, broken]).all()) and bool(torch.isnan(lse[0, 0, broken]).all())
    for t in range(2):
        heads = [h for h in range(32) if t or h not in broken]
        kv = c.kv(0, torch.arange(L - 1 + t))
        for h in heads:
            x = q[0, t, h:h + 1].double()
            ref = P.attention(x, kv, torch.ones(len(kv), dtype=torch.bool, device="cuda"), SCALE)
            small = (x[0].abs() < 2.0 ** -10 * x.abs().max()).double()
            lost = SCALE * float(x.abs().max()) * 2.0 ** -10 / 224 * float((kv.abs() @ small).max())
            P.check_attention(out[0, t, h:h + 1], lse[0, t, h:h + 1], *ref[:3], ref[3] + lost * 2.0 ** 16, what=f"{t} {h}")
    c.close()


def test_attention_skips_entries_it_cannot_read():
    c = Cache("bf16", [300, 300])
    hs = c.hs
    gpu = c.table[0].copy()
    gpu[1] = -1  # not resident
    c.pool.page_map_range(0, 0, gpu, gpu * 0 - 1)
    q = normal(22, 1, 1, 16, P.DIM)
    for pages, good, err in (([0, 1, 3], [0, 3], hs.HS_DEVERR_BAD_PAGE), ([0, 5, -3, 2], [0, 2], hs.HS_DEVERR_INDEX_RANGE),
                             ([1], [], hs.HS_DEVERR_BAD_PAGE)):
        out, lse = attend(c, q, i32(*pages)[None])
        check(c, q, out, lse, lambda b, t: good)
        assert c.pool.get_error() == err
    out, lse = attend(c, q, None)
    check(c, q, out, lse, lambda b, t: [0, 2, 3, 4])
    assert c.pool.get_error() == hs.HS_DEVERR_BAD_PAGE
    # an unknown request, next to a known one
    q2 = normal(23, 2, 1, 16, P.DIM)
    out, lse = attend(c, q2, i32(0, 2, 2, 3).view(2, 2), req=i32(5, 1))
    assert c.pool.get_error() & hs.HS_DEVERR_BAD_REQUEST
    assert not out[0].any() and bool((lse[0] == -math.inf).all())
    check(c, q2[1:], out[1:], lse[1:], lambda b, t: [2, 3], req=[1])
    c.close()


def test_results_repeat_bit_for_bit():
    c = Cache("fp8", [5000, 900])
    q = normal(24, 2, 4, 16, P.DIM)
    a = attend(c, q, None)
    for _ in range(3):
        b = attend(c, q, None)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
    c.close()


# ------------------------------------------------------------------ together
def build_step(c, B, T, H, N, seed):
    """The calls of one serving step on caller-held buffers: returns (run, buffers)."""
    hs = c.hs
    bufs = {
        "x": normal(seed, B, T, P.DIM), "q": normal(seed + 1, B, T, H, P.DIM), "req": torch.arange(B, **I32),
        "means": torch.zeros(c.R, c.P, P.DIM, dtype=torch.bfloat16, device="cuda"),
        "pages": torch.empty(B, T, N, **I32), "topk": torch.empty(B, T, N * 64, **I32),
        "out": torch.empty(B, T, H, 512, dtype=torch.bfloat16, device="cuda"), "lse": torch.empty(B, T, H, device="cuda"),
        "ws1": torch.empty(hs.hs_select_workspace_bytes(c.pool.handle, B, T), dtype=torch.uint8, device="cuda"),
        "ws2": torch.empty(max(1, hs.hs_page_decode_workspace_bytes(B * T, 1, H, N)), dtype=torch.uint8, device="cuda"),
    }
    pairs = [(b, p) for b in range(B) for p in range(-(-c.ctx[b] // 64))]
    bufs["pr"], bufs["pp"] = i32(*(a for a, _ in pairs)), i32(*(p for _, p in pairs))

    def run():
        c.pool.append_rows(bufs["x"], bufs["req"])
        c.pool.page_means(bufs["pr"], bufs["pp"], bufs["means"])
        c.pool.select_pages(bufs["q"], bufs["means"], bufs["req"], bufs["pages"], 1, 1, None, bufs["topk"], bufs["ws1"])
        c.pool.page_mla_decode_per_token(bufs["q"], bufs["pages"], bufs["req"], None, SCALE, bufs["out"], bufs["lse"],
                                         bufs["ws2"])

    return run, bufs


def check_step(c, bufs, N):
    T = bufs["q"].shape[1]
    check_select(c, bufs["q"], bufs["means"], bufs["pages"], 1, 1)
    pages = bufs["pages"].cpu().numpy()
    check(c, bufs["q"], bufs["out"], bufs["lse"], lambda b, t: [p for p in pages[b, t] if p >= 0])
    for b in range(bufs["q"].shape[0]):  # the appended rows are in
        at = c.ctx[b] - T
        v, x = c.kv(b, range(at, at + T)), bufs["x"][b]
        if c.dtype == "bf16":
            assert torch.equal(v, x.double())
        else:
            assert float((v - x.double()).abs().max()) <= 2.0 ** -4 * float(x.double().abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_step_eager_captured_and_on_another_stream(dtype):
    B, T, H, N = 3, 2, 16, 8
    c = Cache(dtype, [3000, 1111, 130], max_topk=2 * 8 * 64, hot_rows=1024)
    run, bufs = build_step(c, B, T, H, N, 30)
    run()
    torch.cuda.synchronize()
    check_step(c, bufs, N)
    want = bufs["out"].clone(), bufs["lse"].clone(), bufs["pages"].clone()
    # two graphs with workspaces of their own, replayed at once on two streams
    run2, bufs2 = build_step(c, B, T, H, N, 30)
    graphs = []
    for f, bb in ((run, bufs), (run2, bufs2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        bb["out"].fill_(0)
        bb["lse"].fill_(0)
        graphs.append(g)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for bb in (bufs, bufs2):
        assert torch.equal(bb["out"].view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(bb["lse"], want[1]) and torch.equal(bb["pages"], want[2])
    # new inputs and a longer context in the same buffers
    c.set_ctx([2999, 1100, 128])
    bufs["q"].copy_(normal(40, B, T, H, P.DIM))
    bufs["x"].copy_(normal(41, B, T, P.DIM))
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    check_step(c, bufs, N)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H,ctx", [(1, 3, 16, 9000), (30, 1, 16, 1500), (3, 40, 128, 700), (2, 64, 24, 333)])
def test_plans_of_every_kind_captured_and_at_once(dtype, B, T, H, ctx):
    """Splits joined by a second kernel, inside a cluster, and no splits: captured and
    replayed with new queries, masks and lengths; two calls at once on two streams."""
    c = Cache(dtype, [ctx - 7 * b for b in range(B)])
    g = torch.Generator().manual_seed(90)

    def trees(n):
        return torch.randint(-2 ** 63, 2 ** 63 - 1, (n, T), generator=g).cuda()

    def buffers(seed):
        return {"q": normal(seed, B, T, H, P.DIM), "tree": trees(B), "req": torch.arange(B, **I32),
                "out": torch.empty(B, T, H, 512, dtype=torch.bfloat16, device="cuda"),
                "lse": torch.empty(B, T, H, device="cuda"),
                "ws": torch.empty(max(1, c.hs.hs_page_decode_workspace_bytes(B, T, H, c.P)), dtype=torch.uint8,
                                  device="cuda")}

    def call(x):
        c.pool.page_mla_decode(x["q"], None, x["req"], x["tree"], SCALE, x["out"], x["lse"], x["ws"])

    a, b = buffers(91), buffers(92)
    call(a)
    torch.cuda.synchronize()
    check(c, a["q"], a["out"], a["lse"], lambda i, t: None, a["tree"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
        call(a)
    for step in range(2):
        a["q"].copy_(normal(93 + step, B, T, H, P.DIM))
        a["tree"].copy_(trees(B))
        c.set_ctx([n - 1 for n in c.ctx])
        a["out"].fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(c, a["q"], a["out"], a["lse"], lambda i, t: None, a["tree"])
    alone = a["out"].clone(), a["lse"].clone()
    call(b)
    torch.cuda.synchronize()
    other = b["out"].clone(), b["lse"].clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(s1):
            graph.replay()
        with torch.cuda.stream(s2):
            call(b)
    torch.cuda.synchronize()
    for got, want in ((a, alone), (b, other)):
        assert torch.equal(got["out"].view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(got["lse"], want[1])
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_selected_positions_through_the_tiered_path(dtype):
    """The selection's positions, resolved as a union and attended to row by row, give
    what attention over the pages gives (same rows, other kernels)."""
    B, T, H, N = 2, 2, 16, 6
    c = Cache(dtype, [2000, 700], max_topk=T * N * 64, hot_rows=1024)
    run, bufs = build_step(c, B, T, H, N, 50)
    run()
    K = N * 64
    topk = bufs["topk"].view(B, T * K)
    res, cnt = torch.empty(B, T * K, **I32), torch.empty(B, 3, **I32)
    c.pool.resolve_topk_union(bufs["req"], topk, res, None, None, cnt)
    out, lse = torch.empty_like(bufs["out"]), torch.empty_like(bufs["lse"])
    ws = torch.empty(max(1, c.hs.hs_decode_workspace_bytes(B * T, 1, H, K)), dtype=torch.uint8, device="cuda")
    c.pool.sparse_mla_decode_per_token(bufs["q"], None, None, res.view(B, T, K), bufs["topk"], bufs["req"], SCALE, out,
                                       lse, ws)
    torch.cuda.synchronize()
    assert int(cnt.sum()) == int((topk >= 0).sum())
    # both within their own roundings (weights, partial results and outputs to BF16) of the exact result
    rel = (out.double() - bufs["out"].double()).norm(dim=-1) / bufs["out"].double().norm(dim=-1)
    assert float(rel.max()) <= 2e-2
    assert float((lse - bufs["lse"]).abs().max()) <= 1e-3
    check_step(c, bufs, N)
    c.close()


def test_a_verified_draft():
    """Drafted rows are appended, attended to as a tree, and the accepted path is
    appended over them: the next chain step sees exactly the path."""
    L, T, H = 500, 8, 16
    c = Cache("bf16", [L], max_ctx=576, garbage=False)
    x = normal(60, 1, T, P.DIM)
    parent = [-1, 0, 0, 1, 2, 4, 5, 1]
    tree = []
    for t, p in enumerate(parent):
        tree.append((tree[p] if p >= 0 else 0) | 1 << t)
    c.set_ctx([L])
    c.pool.append_rows(x, i32(0))  # nodes at L - T ..
    q = normal(61, 1, T, H, P.DIM)
    tr = torch.tensor([tree], dtype=torch.int64, device="cuda")
    out, lse = attend(c, q, None, tr)
    check(c, q, out, lse, lambda b, t: None, tr)
    path = [0, 2, 4, 5]  # ancestors of node 5, and itself
    index = torch.tensor([path + [-1] * (T - len(path))], **I32)
    c.pool.append_rows(x, i32(0), i32(L - T), index)
    c.set_ctx([L - T + len(path)])
    q1 = q[:, 5:6].contiguous()
    o1, l1 = attend(c, q1, None)
    check(c, q1, o1, l1, lambda b, t: None)
    # the same rows in the same order as node 5 saw them in the tree; sums split the same way or not
    assert float((o1[0, 0].double() - out[0, 5].double()).abs().max()) <= 2.0 ** -6 * float(out.double().abs().max())
    assert float((l1[0, 0] - lse[0, 5]).abs().max()) <= 1e-4
    c.close()


# ------------------------------------------------------------------ refusals
def test_refusals():
    c = Cache("bf16", [200], max_ctx=64 * 200, garbage=False)
    hs = c.hs
    lib = hs.load()
    q, pages, req = normal(70, 1, 2, 8, P.DIM), torch.zeros(1, 2, 4, **I32), i32(0)
    out, lse = torch.empty(1, 2, 8, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 2, 8, device="cuda")
    means = torch.zeros(1, c.P, P.DIM, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def status(f, *a, **k):
        with pytest.raises(hs.HsError) as e:
            f(*a, **k)
        return e.value.status

    inval = hs.HS_ERR_INVALID_ARG
    # types and shapes
    for bad in (lambda: c.pool.append_rows(q.float(), req), lambda: c.pool.append_rows(q[:, :, 0], i32(0, 1)),
                lambda: c.pool.append_rows(q[:, :, 0].contiguous(), req, torch.zeros(1, dtype=torch.int64, device="cuda")),
                lambda: c.pool.append_rows(q[:, :, 0].transpose(0, 1), i32(0, 0)),
                lambda: c.pool.page_means(req, req, means[:, 1:].contiguous()),
                lambda: c.pool.select_pages(q, means, req, pages.long(), workspace=ws),
                lambda: c.pool.select_pages(q, means, req, pages, tree=pages, workspace=ws),
                lambda: c.pool.page_mla_decode(q, pages, req, None, SCALE, out, lse, ws),
                lambda: c.pool.page_mla_decode(q, None, req, None, SCALE, out.float(), lse, ws),
                lambda: c.pool.page_mla_decode(q.cpu(), None, req, None, SCALE, out, lse, ws)):
        with pytest.raises(ValueError):
            bad()
    # what the library refuses
    assert status(c.pool.select_pages, q, means, req, pages, 3, 2, workspace=ws) == inval
    assert status(c.pool.select_pages, q, means, req, pages, -1, 2, workspace=ws) == inval
    assert status(c.pool.select_pages, q, means, req, pages, 1, 1, workspace=ws[:64]) == inval
    assert status(c.pool.select_pages, q, means, req, pages, 1, 1) == inval
    assert status(c.pool.select_pages, q, means, req, torch.empty(1, 2, 1025, **I32), workspace=ws) == hs.HS_ERR_CAPACITY
    long = normal(71, 1, 65, 1, P.DIM)
    tree = torch.zeros(1, 65, dtype=torch.int64, device="cuda")
    o65, l65 = torch.empty(1, 65, 1, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 65, 1, device="cuda")
    assert status(c.pool.page_mla_decode, long, None, req, tree, SCALE, o65, l65, ws) == inval
    assert status(c.pool.select_pages, long, means, req, torch.empty(1, 65, 4, **I32), 1, 1, tree, workspace=ws) == inval
    need = hs.hs_page_decode_workspace_bytes(1, 2, 8, c.P)
    assert need > 0
    assert status(c.pool.page_mla_decode, q, None, req, None, SCALE, out, lse, ws[:need - 256]) == inval
    assert status(c.pool.page_mla_decode, q, None, req, None, SCALE, out, lse) == inval
    assert status(c.pool.page_mla_decode, q, None, req, None, SCALE, out, lse, ws[8:]) == inval
    h, qp = c.pool.handle, q.data_ptr()
    assert lib.hs_append_rows(h, 1, 0, qp, req.data_ptr(), None, None, None) == inval
    assert lib.hs_append_rows(h, 1, 1, qp + 2, req.data_ptr(), None, None, None) == inval
    assert lib.hs_append_rows(h, -1, 1, qp, req.data_ptr(), None, None, None) == inval
    assert lib.hs_page_mla_decode_per_token(h, 1, 2, 8, 4, qp, None, req.data_ptr(), None, 0.1, out.data_ptr(),
                                            lse.data_ptr(), ws.data_ptr(), 1 << 20, None) == inval
    # nothing to do
    assert lib.hs_append_rows(h, 0, 1, None, None, None, None, None) == hs.HS_OK
    assert lib.hs_page_means(h, 0, None, None, None, None) == hs.HS_OK
    c.close()
