"""Append, page means, page selection and attention over pages where an input is at the
edge of what the operators accept, or past it. Plain 64-bit forms: tests/_pages.py."""
import math

import numpy as np
import pytest
import torch

import _pages as P
from test_gpu_pages import I32, SCALE, Cache, attend, check, check_select, i32, normal, run_select, sparse_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available()


# ------------------------------------------------------------------ lengths past max_ctx
@pytest.mark.parametrize("max_ctx", [4096, 4070])
def test_select_takes_a_length_past_max_ctx_as_max_ctx(max_ctx):
    """Lengths come from device memory unchecked. The scores' rows end at max_ctx: a
    longer length changes no other list's choice and nothing behind the workspace."""
    hs_lens = [max_ctx, 1000, max_ctx]
    B, T, H, N = 4, 2, 16, 6
    c = sparse_cache(hs_lens, max_ctx=max_ctx)
    means = normal(100, 3, c.P, P.DIM)
    q = normal(101, B, T, H, P.DIM)
    req = i32(0, 1, 2, 1)
    tree = torch.tensor([[1, 3]] * B, dtype=torch.int64, device="cuda")
    for tr in (None, tree):
        c.set_ctx(hs_lens)
        want, want_pos = run_select(c, q, means, N, 1, 2, tr, req, topk=True)
        check_select(c, q, means, want, 1, 2, tr, req=[0, 1, 2, 1])
        assert c.pool.get_error() == 0
        for longer in (max_ctx + 1, max_ctx + 64 * 33, 2 ** 31 - 1):
            c.pool.set_ctx_lens(i32(longer, 1000, longer))
            pages = torch.full((B, T, N), -7, **I32)
            pos = torch.full((B, T, N * 64), -7, **I32)
            need = c.hs.hs_select_workspace_bytes(c.pool.handle, B, T)
            ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
            c.pool.select_pages(q, means, req, pages, 1, 2, tr, pos, ws)
            assert c.pool.get_error() == c.hs.HS_DEVERR_INDEX_RANGE
            assert torch.equal(pages, want) and torch.equal(pos, want_pos)
            assert bool((ws[need:] == 0xA5).all())
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_and_means_take_a_length_past_max_ctx_as_max_ctx(dtype):
    max_ctx = 330
    c = Cache(dtype, [max_ctx, 200], max_ctx=max_ctx)
    q = normal(102, 2, 3, 16, P.DIM)
    lists = torch.tensor([[5, 0, 3], [2, 1, 3]], **I32)
    pr, pp = i32(0, 0, 1), i32(5, 2, 3)

    def means():
        m = torch.zeros(2, c.P, P.DIM, dtype=torch.bfloat16, device="cuda")
        c.pool.page_means(pr, pp, m)
        torch.cuda.synchronize()
        return m

    want = attend(c, q, None), attend(c, q, lists), means()
    assert c.pool.get_error() == 0
    for longer in (max_ctx + 1, 64 * 500, 2 ** 31 - 1):
        c.pool.set_ctx_lens(i32(longer, 200))
        for i, pages in enumerate((None, lists)):
            got = attend(c, q, pages)
            assert c.pool.get_error() == c.hs.HS_DEVERR_INDEX_RANGE
            assert torch.equal(got[0].view(torch.int16), want[i][0].view(torch.int16)) and torch.equal(got[1], want[i][1])
        assert torch.equal(means().view(torch.int16), want[2].view(torch.int16))
        assert c.pool.get_error() == c.hs.HS_DEVERR_INDEX_RANGE
    c.pool.set_ctx_lens(i32(-5, 200))  # a negative one holds nothing
    out, lse = attend(c, q, None)
    assert not out[0].any() and bool((lse[0] == -math.inf).all())
    check(c, q[1:], out[1:], lse[1:], lambda b, t: None, req=[1])
    c.close()


# ------------------------------------------------------------------ selection: very small values
@pytest.mark.parametrize("q_exp,c_exp", [(-70, 0), (-90, 0), (0, -70), (0, -90), (-62, -45)])
def test_select_where_squares_leave_the_normal_range(q_exp, c_exp):
    """Queries or means whose squares are below f32's smallest normal number, with products
    above it: a power of two on all of them changes no choice."""
    c = sparse_cache([64 * 600] * 4)
    small = 2.0 ** -5 * (1 - 2.0 ** -8)
    means = torch.zeros(4, c.P, P.DIM)
    means[:2, :, 0] = 512.0
    up, down = means[0, 0].clone(), means[0, 0].clone()
    up[0] = down[0] = 1024.0
    up[2:], down[2:] = small, -small
    down[1] = 35.0 / 32
    for r, (i, j) in enumerate(((100, 300), (300, 100))):  # short sums have these two in the other order
        means[r, i], means[r, j] = up, down
    g = torch.Generator().manual_seed(103)
    base = torch.randn(P.DIM, generator=g) * 64  # large terms that cancel, a small rest
    means[2] = base
    means[2, :, 0] = torch.randint(-3, 4, (c.P,), generator=g) * 2.0 ** -9
    means[3] = torch.randn(c.P, P.DIM, generator=g)
    q = torch.ones(4, 1, 8, P.DIM)
    q[:2, ..., 0], q[:2, ..., 1] = 1024.0, 32.0
    q[2:] = torch.randn(2, 1, 1, P.DIM, generator=g)
    q[2, ..., 0] = 1.0
    q, means = (q * 2.0 ** q_exp).to(torch.bfloat16).cuda(), (means * 2.0 ** c_exp).to(torch.bfloat16).cuda()
    for N in (3, 40):
        pages = run_select(c, q, means, N, 1, 1)
        check_select(c, q, means, pages, 1, 1)
    c.close()


def test_select_of_zeros():
    """Queries or means of exact zeros: equal scores, so the lowest pages."""
    c = sparse_cache([64 * 5000] * 3)
    means = normal(104, 3, c.P, P.DIM)
    means[1] = 0.0
    means[2, 7::2] = -0.0
    q = normal(105, 3, 2, 16, P.DIM)
    q[0] = 0.0
    q[0, 1, 3] = -0.0
    for N in (5, 700):
        check_select(c, q, means, run_select(c, q, means, N), 1, 2)
    c.close()


def test_select_weighs_every_head_of_a_page_whose_norm_overflows():
    """A thousand equal scores of 1, and one page of 1 + 2^-16 by a head whose 32-bit sum
    says 0 (a pair of 2^30 cancels) next to a head whose sum says 1 - 2^-8."""
    c = sparse_cache([64 * 1000] * 2)
    means = torch.zeros(2, c.P, P.DIM)
    means[..., 3] = 1.0
    for r, p in enumerate((700, 3)):
        u = torch.zeros(P.DIM)
        u[0] = u[128] = 2.0 ** 30
        u[1], u[64], u[2] = 1.0, 2.0 ** -16, 1 - 2.0 ** -8
        u[5] = 3e19  # where no query has a value: the square of the norm is infinite
        means[r, p] = u
    q = torch.zeros(2, 1, 8, P.DIM)
    q[..., 3] = 1.0
    q[:, :, 0, 0], q[:, :, 0, 128] = 1.0, -1.0
    q[:, :, 0, 1] = q[:, :, 0, 64] = 1.0
    q[:, :, 1:, 2] = 1.0
    q, means = q.to(torch.bfloat16).cuda(), means.to(torch.bfloat16).cuda()
    for N in (1, 4):
        pages = run_select(c, q, means, N, 0, 0)
        check_select(c, q, means, pages, 0, 0)
    assert 700 in pages[0, 0].tolist() and 3 in pages[1, 0].tolist()
    c.close()


# ------------------------------------------------------------------ selection: sums near the border
def test_select_tells_sums_apart_that_pairs_of_f32_do_not():
    """A product of 1, nine of nearly 2^-24 and eight of 2^-45 in the places that one lane
    sums: the eight are half the last place of what the nine leave in the sum's second
    word. The other page has 2^-43 in their stead, half as much."""
    c = sparse_cache([64 * 600] * 2)
    order = [2 * 0 + 64 * i + e for i in range(9) for e in (0, 1)]  # lane 0's products
    more = torch.zeros(P.DIM)
    more[order[0]] = 1.0
    more[order[1:10]] = 2.0 ** -24 * (1 - 2.0 ** -8)
    less = more.clone()
    more[order[10:]] = 2.0 ** -45
    less[order[10]] = 2.0 ** -43
    means = torch.zeros(2, c.P, P.DIM)
    for r, (i, j) in enumerate(((100, 300), (300, 100))):
        means[r, i], means[r, j] = more, less
    q, means = torch.ones(2, 1, 8, P.DIM).to(torch.bfloat16).cuda(), means.to(torch.bfloat16).cuda()
    pages = run_select(c, q, means, 3, 1, 1)
    check_select(c, q, means, pages, 1, 1)
    assert pages[:, 0, 1].tolist() == [100, 300]
    c.close()


def test_select_keeps_rests_below_the_normal_range():
    """Products near 2^-113, whose last bits, 2^-127, fall behind a sum of 2^-103: seventeen
    of those bits against one product of 2^-124."""
    c = sparse_cache([64 * 600] * 2)
    lane = [[2 * l + 64 * i + e for i in range(9) for e in (0, 1)] for l in (0, 1)]
    q = torch.ones(P.DIM)
    q[lane[0][1:]] = 1 + 2.0 ** -7
    more, less = torch.zeros(P.DIM), torch.zeros(P.DIM)
    more[lane[0][0]] = less[lane[1][0]] = 2.0 ** -103
    more[lane[0][1:]] = (1 + 2.0 ** -7) * 2.0 ** -113    # products (1 + 2^-6 + 2^-14) 2^-113
    less[lane[1][1:]] = (1 + 2.0 ** -6) * 2.0 ** -113
    less[4] = 2.0 ** -124
    means = torch.zeros(2, c.P, P.DIM)
    for r, (i, j) in enumerate(((100, 300), (300, 100))):
        means[r, i], means[r, j] = more, less
    q = q.expand(2, 1, 8, P.DIM).to(torch.bfloat16).cuda()
    means = means.to(torch.bfloat16).cuda()
    pages = run_select(c, q, means, 3, 1, 1)
    check_select(c, q, means, pages, 1, 1)
    assert pages[:, 0, 1].tolist() == [100, 300]
    c.close()


# ------------------------------------------------------------------ append
def test_append_fp8_keeps_the_sign_of_zeros():
    """Codes equal the definition's, e4m3(x / scale), zeros' signs included, whatever the
    row's largest magnitude."""
    n = 96
    c = Cache("fp8", [n], garbage=False)
    g = torch.Generator().manual_seed(106)
    x = torch.randn(n, P.DIM, generator=g)
    x = torch.where(torch.rand(n, P.DIM, generator=g) < 0.5, x, torch.where(x < 0, -0.0, 0.0))
    x[:, 1::7] *= 2.0 ** -30  # quotients that round to zero
    x[:, 3::9] = torch.sign(x[:, 3::9]) * 2.0 ** -130  # subnormal values
    x[::3] *= 2.0 ** 80
    x[1::3] *= 2.0 ** -80
    x[5] = -0.0
    x = x.to(torch.bfloat16)
    c.pool.append_rows(x[None].cuda(), i32(0), i32(0))
    torch.cuda.synchronize()
    code, s = P.quantise(x)
    at = torch.tensor([c.row(0, p) for p in range(n)])
    assert torch.equal(c.pool.gpu_scales().cpu()[at], s)
    assert torch.equal(c.pool.gpu_rows().cpu()[at], code.view(torch.uint8))
    c.close()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_of_an_unknown_request_reports_nothing_else(dtype):
    c = Cache(dtype, [300])
    q = normal(107, 2, 2, 16, P.DIM)
    lists = torch.tensor([[1, 3, -1], [2, 0, 4]], **I32)
    for bad in (5, -1):
        for pages, per_token in ((None, False), (lists, False), (lists[:, None].expand(2, 2, 3).contiguous(), True)):
            out, lse = attend(c, q, pages, req=i32(bad, 0), per_token=per_token)
            assert c.pool.get_error() == c.hs.HS_DEVERR_BAD_REQUEST
            assert not out[0].any() and bool((lse[0] == -math.inf).all())
            check(c, q[1:], out[1:], lse[1:], lambda b, t: None if pages is None else [2, 0, 4], req=[0])
    c.close()


# ------------------------------------------------------------------ means
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_page_means_are_quotients(dtype):
    """Sums that are exact in f32 over counts that are no powers of two: the mean is half
    way between two BF16 values and goes to the even one."""
    lens = [14, 28, 60, 64 + 26]
    c = Cache(dtype, lens, garbage=False)
    mid = {14: 345, 28: 345, 60: 293, 26: 413}
    means = torch.zeros(4, c.P, P.DIM, dtype=torch.bfloat16, device="cuda")
    want = torch.zeros(4, P.DIM)
    for r, L in enumerate(lens):
        n = L % 64
        m = torch.full((P.DIM,), mid[n])  # odd: m - 1 and m + 1 are BF16 values, m lies between two
        at = torch.tensor([c.row(r, L - n + i) for i in range(n)], device="cuda")
        sign = torch.tensor([1, -1]).repeat(n // 2)
        if dtype == "fp8":  # codes of 1 at those scales
            c.pool.gpu_rows()[at] = torch.ones(n, P.DIM).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            c.pool.gpu_scales()[at] = (mid[n] + sign).float().cuda()
        else:
            m += 4 * (torch.arange(P.DIM) % 4)
            c.pool.gpu_rows()[at] = (m + sign[:, None]).to(torch.bfloat16).view(torch.uint8).cuda()
        want[r] = m
    c.pool.page_means(i32(0, 1, 2, 3), i32(0, 0, 0, 1), means)
    torch.cuda.synchronize()
    for r, L in enumerate(lens):
        assert torch.equal(means[r, L // 64].cpu(), want[r].to(torch.bfloat16)), r
    c.close()


@pytest.mark.parametrize("q_exp,row_exp,peak", [(100, -105, 1), (122, -118, 16), (-100, 100, 1)])
def test_attention_fp8_queries_and_scales_of_opposite_magnitude(q_exp, row_exp, peak):
    """Scores are ordinary numbers although the query times the codes is not one."""
    L = 400
    c = Cache("fp8", [L])
    at = torch.tensor([c.row(0, i) for i in range(L)], device="cuda")
    c.pool.gpu_scales()[at] *= 2.0 ** row_exp
    q = (normal(108, 1, 2, 16, P.DIM).double() * 2.0 ** q_exp).to(torch.bfloat16)
    scale = peak * SCALE * 2.0 ** -(q_exp + row_exp)
    out, lse = attend(c, q, None, scale=scale)
    kv = c.kv(0, torch.arange(L))
    for t in range(2):
        k = kv[:L - 1 + t]
        ref = P.attention(q[0, t].double(), k, torch.ones(len(k), dtype=torch.bool, device="cuda"), scale)
        # The output is as small or large as the rows: compare it at the rows' magnitude.
        # What is below 2^-126 may count as zero: each of at most four splits' partials,
        # their products with the weights, the sum, its quotient and the BF16 value, 11
        # times 2^-126 at most. The check allows 2^-8 of the mass, so 2^8 times that joins it.
        lost = 11 * 2.0 ** -126 * 2.0 ** 8
        P.check_attention((out[0, t].double() * 2.0 ** -row_exp).float(), lse[0, t], ref[0] * 2.0 ** -row_exp, ref[1],
                          (ref[2] + lost) * 2.0 ** -row_exp, ref[3], what=f"token {t}")
    c.close()


@pytest.mark.parametrize("largest", [225.0, 250.0, 256.0, 448.0])
def test_attention_fp8_small_values_beside_a_large_one(largest):
    """A query value of at least 2^-9.8 of its row's largest is taken exactly, a smaller one
    is off by at most 2^-17.8 of the largest. One row of context, 448 where a head has its
    small value and 0 where it has the large one, so that lse is the score itself."""
    H = 128
    c = Cache("fp8", [1], garbage=False)
    x = torch.zeros(P.DIM)
    x[:H] = 448.0
    at = c.row(0, 0)
    c.pool.gpu_rows()[at] = x.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    c.pool.gpu_scales()[at] = 1.0
    v = torch.arange(128, 256).float()[None] * 2.0 ** torch.tensor([-16.0, -17.0, -18.0])[:, None]  # from 2^-11 to 2^-8
    v = (v * largest).to(torch.bfloat16).flatten()[torch.randperm(384, generator=torch.Generator().manual_seed(110))]
    for part in v.view(3, H):
        q = torch.zeros(1, 1, H, P.DIM, dtype=torch.bfloat16)
        q[0, 0, torch.arange(H), torch.arange(H)] = part
        q[..., 575] = largest
        out, lse = attend(c, q.cuda(), None, scale=1.0)
        got, want = lse[0, 0].double().cpu() / 448, part.double()
        off = (got - want).abs()
        exact = want >= largest * 2.0 ** -9.8
        assert bool(exact.any()) and not bool(exact.all())
        # a sum of two products in f32, and lse's two roundings and products with log2(e) and ln(2)
        assert bool((off <= torch.where(exact, 2.0 ** -20 * want, 2.0 ** -20 * want + 2.0 ** -17.8 * largest)).all())
    c.close()


def test_attention_fp8_rows_of_huge_scale_that_do_not_count():
    """Rows at 2^40 times the others' scale whose weights are nothing leave the others'
    weights their bits, whether they come before them, between them or behind."""
    L = 700
    c = Cache("fp8", [L] * 4, garbage=False)
    g = torch.Generator().manual_seed(109)
    q = torch.zeros(4, 1, 16, P.DIM)
    q[..., :64] = torch.randn(4, 1, 16, 64, generator=g)
    q[..., 575] = 8.0
    q = q.to(torch.bfloat16).cuda()
    rows, scales = c.pool.gpu_rows(), c.pool.gpu_scales()

    def check_all(scale):
        out, lse = attend(c, q, None, scale=scale)
        for r in range(4):
            kv = c.kv(r, range(L))
            here = torch.tensor([float(scales[c.row(r, i)]) < 1 for i in range(L)], device="cuda")
            seen = torch.ones(L, dtype=torch.bool, device="cuda")
            ref = P.attention(q[r, 0].double(), kv, seen, scale)
            # the huge rows' scores are far below all others, or exactly zero: the error of
            # a score that counts is that of the others
            reach = P.attention(q[r, 0].double(), kv[here], seen[here], scale)[3]
            P.check_attention(out[r, 0], lse[r, 0], *ref[:3], reach, what=f"request {r}")

    for r, where in enumerate((range(0, 40), range(300, 303), range(L - 5, L), (0, 130, 131, 400, 699))):
        for i in where:
            x = torch.randn(P.DIM, generator=g)
            x[575] = -448.0  # far below every other score
            x[:64] = 0.0
            at = c.row(r, i)
            rows[at] = x.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            scales[at] = 2.0 ** 33
    check_all(SCALE)
    # the first row counts for a moment: the next ones' scores leave it behind
    for r in range(4):
        x = torch.randn(P.DIM, generator=g)
        x[:64] = 0.0
        x[575] = 0.0
        at = c.row(r, 1)
        rows[at] = x.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        scales[at] = 2.0 ** 33
        for i in range(128, L - 5):
            if float(scales[c.row(r, i)]) < 2.0 ** 30:
                at = c.row(r, i)
                v = rows[at].clone()
                v[575] = 0x7e  # code 448, scores that are larger by 8 * 448 * scale / 24, about 1
                rows[at] = v
    check_all(SCALE * 40)
    c.close()


# ------------------------------------------------------------------ sizes
def small_pool(dtype, n_blocks, max_requests, max_ctx):
    import tiered_sparse_mla_gb300 as hs
    return hs, hs.Pool(dtype=hs.HS_FP8_E4M3_ROWSCALE if dtype == "fp8" else hs.HS_BF16, n_gpu_blocks=n_blocks,
                       n_host_blocks=0, max_requests=max_requests, max_ctx=max_ctx, max_topk=32, hot_rows=64)


def one_query(hs, pool, q, pages, req, tree=None):
    B, T, H = q.shape[:3]
    out = torch.full((B, T, H, 512), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, H), math.nan, device="cuda")
    n = hs.hs_page_decode_workspace_bytes(B, T, H, pool.max_pages if pages is None else pages.shape[-1])
    pool.page_mla_decode(q, pages, req, tree, SCALE, out, lse, torch.empty(max(1, n), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("dtype,n", [("bf16", 70000), ("fp8", 140000)])
def test_rows_past_32_bits_of_offset(dtype, n):
    """Pages at both ends of a pool of more than 2^32 bytes."""
    L = 150
    hs, pool = small_pool(dtype, n, 1, 192)
    blocks = [n - 1, 0, n - 2]
    pool.page_map_range(0, 0, blocks, [-1] * 3)
    pool.set_ctx_lens(i32(L))
    x = normal(120, 1, L, P.DIM)
    pool.append_rows(x, i32(0))
    means = torch.zeros(1, 3, P.DIM, dtype=torch.bfloat16, device="cuda")
    pool.page_means(i32(0, 0, 0), i32(0, 1, 2), means)
    torch.cuda.synchronize()
    at = torch.tensor([blocks[i // 64] * 64 + i % 64 for i in range(L)], device="cuda")
    s = pool.gpu_scales()
    kv = P.values(pool.gpu_rows()[at], None if s is None else s[at])
    if dtype == "bf16":
        assert torch.equal(kv, x[0].double())
    else:
        code, scale = P.quantise(x[0].cpu())
        assert torch.equal(pool.gpu_rows()[at].cpu(), code.view(torch.uint8)) and torch.equal(s[at].cpu(), scale)
    for p in range(3):
        v = kv[64 * p:64 * p + 64]
        tol = 2.0 ** -8 * v.mean(0).abs() + len(v) * 2.0 ** -23 * v.abs().mean(0)
        assert bool(((means[0, p].double() - v.mean(0)).abs() <= tol).all())
    q = normal(121, 1, 2, 16, P.DIM)
    out, lse = one_query(hs, pool, q, None, i32(0))
    for t in range(2):
        ref = P.attention(q[0, t].double(), kv[:L - 1 + t], torch.ones(L - 1 + t, dtype=torch.bool, device="cuda"), SCALE)
        P.check_attention(out[0, t], lse[0, t], *ref)
    assert pool.get_error() == 0
    pool.close()


def test_select_among_means_past_32_bits_of_offset():
    """Two requests of two million pages each: 4.8 GB of means."""
    L = 2 ** 27
    c = sparse_cache([L - 5, L], max_ctx=L)
    means = torch.empty(2, c.P, P.DIM, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(122)
    for r in range(2):
        means[r].normal_(generator=g)
    q = normal(123, 2, 2, 8, P.DIM)
    pages = run_select(c, q, means, 20, 1, 2)
    check_select(c, q, means, pages, 1, 2)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_of_the_most_lists(dtype):
    """65,535 lists of one page each, of three requests in turn."""
    B, lens = 65535, [100, 128, 65]
    c = Cache(dtype, lens)
    q = normal(124, B, 1, 1, P.DIM)
    req = torch.arange(B, device="cuda") % 3
    pages = torch.randint(0, 2, (B, 1), generator=torch.Generator().manual_seed(125)).to(torch.int32).cuda()
    out, lse = attend(c, q, pages, req=req.to(torch.int32))
    for r in range(3):
        for p in range(2):
            mine = (req == r) & (pages[:, 0] == p)
            kv = c.kv(r, range(64 * p, min(lens[r], 64 * p + 64)))
            ref = P.attention(q[mine, 0, 0].double(), kv, torch.ones(len(kv), dtype=torch.bool, device="cuda"), SCALE)
            P.check_attention(out[mine, 0, 0], lse[mine, 0, 0], *ref, what=f"request {r} page {p}")
    c.close()


@pytest.mark.parametrize("dtype,T,H", [("bf16", 32767, 1), ("fp8", 32767, 3), ("bf16", 1, 70000), ("fp8", 2, 40000)])
def test_attention_of_the_most_rows(dtype, T, H):
    """As many query tokens as a request may have, each with its own border, and as many
    heads as need hundreds of tiles; every 997th token, or all."""
    L = T + 333
    c = Cache(dtype, [L])
    q = normal(126, 1, T, H, P.DIM)
    out, lse = attend(c, q, None)
    kv = c.kv(0, range(L))
    for t in sorted({*range(0, T, 997), T - 1}):
        k = kv[:L - T + t + 1]
        ref = P.attention(q[0, t].double(), k, torch.ones(len(k), dtype=torch.bool, device="cuda"), SCALE)
        P.check_attention(out[0, t], lse[0, t], *ref, what=f"token {t}")
    c.close()


@pytest.mark.parametrize("T,H", [(32767, 1), (4, 65535)])
def test_select_of_the_most_rows(T, H):
    L = T + 700
    c = sparse_cache([L])
    means = normal(127, 1, c.P, P.DIM)
    q = normal(128, 1, T, H, P.DIM)
    N = 5
    pages = run_select(c, q, means, N, 1, 1)
    m = means[0].double()
    for t in sorted({*range(0, T, 331), T - 1}):
        want = P.select(q[0, t].double(), m, -(-(L - T + t + 1) // 64), N, 1, 1)
        assert pages[0, t].tolist() == want + [-1] * (N - len(want)), t
    c.close()


def test_select_of_the_most_requests():
    """65,535 lists, of five requests in turn, one of them empty and one unknown."""
    B, lens = 65535, [700, 64, 0, 1500]
    c = sparse_cache(lens)
    means = normal(129, 4, c.P, P.DIM)
    q = normal(130, B, 1, 2, P.DIM)
    req = torch.arange(B, device="cuda") % 5
    pages = run_select(c, q, means, 3, 1, 1, req=req.to(torch.int32))[:, 0]
    assert bool((pages[req == 4] == -1).all()) and bool((pages[req == 2] == -1).all())
    assert bool((pages[req == 1] == i32(0, -1, -1)).all())
    for r in (0, 3):
        n = -(-lens[r] // 64)
        s = (q[req == r, 0].double() @ means[r, :n].double().T).amax(1)
        best = s[:, 1:n - 1].argmax(1) + 1
        want = torch.stack([torch.zeros_like(best), best, torch.full_like(best, n - 1)], 1)
        assert torch.equal(pages[req == r].long(), want)
    c.close(c.hs.HS_DEVERR_BAD_REQUEST)


def test_select_with_heads_of_nan():
    """Heads that hold a NaN count for nothing; where all of them do, all scores are equal."""
    c = sparse_cache([64 * 5000, 64 * 700])
    means = normal(131, 2, c.P, P.DIM)
    means[1, 700:] = math.nan
    means[0, 11, 3], means[0, 12, 4], means[1, 5, 6] = math.nan, math.inf, -math.inf
    q = normal(132, 2, 4, 16, P.DIM)
    q[:, 1, 3, 100] = math.nan
    q[:, 2, 1:, 7] = math.nan
    q[:, 3, :, 0] = math.nan
    q[0, 2, 2, 9] = math.inf
    for N in (5, 600):
        check_select(c, q, means, run_select(c, q, means, N, 1, 2), 1, 2)
    q[:, :, 0] = 0.0
    q[:, 0, 1:] = math.nan
    check_select(c, q, means, run_select(c, q, means, 600, 1, 2), 1, 2)
    c.close()
