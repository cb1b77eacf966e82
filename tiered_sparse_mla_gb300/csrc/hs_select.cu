// hs_select.cu -- the pages that each query token attends to: scores of all of a
// request's pages on tcgen05 tensor cores, then an exact top-N.
//
// The score of page p for query token t is s = max_h q[t][h] . c_p, c_p the mean
// row of the page (hs_page_means). The selection is that of the exact sums: the
// tensor cores' sums are within
//     E = 2^-15 * max_h |q_h| * max_p |c_p|
// of them: products of BF16 values are exact, and each of a score's 36 MMAs of depth
// 16 cuts its 16 products and the sum so far at 2^-25 of the largest's power of two
// and then rounds the sum to f32, together less than (16 * 2^-25 + 2^-23) |q||c|, so
// 36 times that, 2^-15.5, in all (2^-15.84 measured with one product of |q||c| and all
// others just below the cut; 2^-22 to 2^-23 with random ones). A page whose score is
// more than 2 E from the border is therefore in or out, and the few nearer ones are
// summed again, as exactly as in 64 bits. Equal scores go to the lower page. Products below
// f32's normal numbers may count as zero. Norms and sums may lose what lies below
// those numbers too: each square at most 2^-126, so 576 of them are added to a norm's
// square, and E gets 2^-116 more (576 products and 36 sums of at most 2^-126). Only
// where all queries, or all means, are exactly zero are the sums exact as they are.
#include <cfloat>
#include <climits>
#include <cstdint>

#include "hs_internal.cuh"
#include "hs_tc.cuh"
#include "hs_tmap.cuh"

namespace {

using namespace hs::tc;
using hs::kDim;
using hs::kPage;

__host__ __device__ __forceinline__ int pages_of(int tokens) {
    return tokens <= 0 ? 0 : (tokens - 1) / kPage + 1;
}

// ---------------------------------------------------------------- scores
// Work unit: a group of whole query tokens of at most 256 rows, the same tokens of
// every request, and a range of the page tiles of all requests laid end to end, run
// by two CTAs whose tensor cores work as one (cta_group::2, M = 256, N up to 256):
// pages are the MMA's M rows, 128 per CTA, so that the maximum over heads runs along
// the registers of the one thread that owns a page, and query rows its N columns,
// half of them supplied by either CTA. The queries stay in shared memory (144 KB a
// CTA) and the pages stream past once through a ring of 16 KB chunks; the scores of
// one tile are reduced while the next is multiplied (two accumulators). Where a range
// goes on to the next request, its queries take their places chunk by chunk behind the
// last tile, so the MMAs hardly pause.
// Bound: one MMA of 256 x 256 x 16 takes 128 clocks, so 256 rows per pass need 4.6k
// clocks per tile of 256 pages; fewer rows are bound by the pages' bytes. 16 requests
// of 16,384 pages with 512 query rows each (155 GFLOP, 302 MB): 92 us by itself, 99 in calls
// back to back, under which the clock falls: 1.68 and 1.56 PFLOP/s.
// Measured there: ranges cut at requests, which fill 64 of 76 pairs, 107 us; four ring
// stages instead of five 105 us; one CTA per 128 pages with the queries streamed past
// each tile, which moves 6x the pages' bytes from L2, about 300 us.
//   warp 0      producer;  warp 1 (CTA 0) MMA issuer;
//   warps 2-5   the pages' |c|^2, from the chunks as they land; their arrival is
//               what the MMA issuer waits for;
//   warps 6-9   maxima over heads, one thread per page, and the group of eight heads
//               that each is in.
constexpr int SP = 256;          // pages per tile (two CTAs)
constexpr int NCH = kDim / 64;   // depth chunks
constexpr int ST = 320;
constexpr int MAXN = 256;        // query rows per pass
constexpr int HG = 8;            // heads per group
constexpr int NST = 5;           // ring stages
constexpr int A_BYTES = 128 * 128;
constexpr int OFF_RING = NCH * 128 * 128;
constexpr int OFF_SBAR = OFF_RING + NST * A_BYTES;
constexpr int SCORE_SMEM = OFF_SBAR + 384 + 1024;
static_assert(SCORE_SMEM <= 232448, "shared memory");

struct ScoreParams {
    const int32_t *req, *ctx;
    const uint4 *means;  // [max_req][max_pages] rows of 72
    float *s1;       // [B*T][Pp] best head's score
    uint32_t *s2;    // [B*T][Pp] best score of another group of heads (BF16, rounded up) << 16 | group
    // [B][Pp] |c_p|^2, zero for rows of zeros alone; [B][Pp / 32] the largest of 32 pages
    // (infinite if one is not finite)
    float *cn, *cm;
    uint32_t *err;
    int B, T, H, tpg, groups, parts;  // tokens per group; groups of tokens; parts of the tiles
    int hpc, N;                     // heads per pass (H, or 256 at most); N: query rows of a pass, rounded up
    int Pp, max_req, max_pages, max_ctx;
};

__global__ void __launch_bounds__(ST, 1)
score_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_q,
             const ScoreParams p) {
    extern __shared__ uint8_t smem_raw[];
    // launched early, and launching early, but only what comes before is complete:
    // a later grid may read what this one's predecessors wrote before it waits
    grid_dep_wait();
    grid_dep_launch();
    const int rank = static_cast<int>(hs::cluster_ctarank());
    const int unit = blockIdx.x >> 1, g = unit % p.groups, part = unit / p.groups;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t raw = hs::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    volatile int32_t *misc = reinterpret_cast<volatile int32_t *>(smem + OFF_SBAR);
    volatile int32_t *sums = reinterpret_cast<volatile int32_t *>(smem + OFF_SBAR + 320);
    constexpr int B_QFULL = 0, B_FULL = B_QFULL + NCH, B_READY = B_FULL + NST, B_FREE = B_READY + NST,
                  B_DFULL = B_FREE + NST, B_DFREE = B_DFULL + 2, B_DRAIN = B_DFREE + 2, NB = B_DRAIN + 1;
    static_assert(32 + 8 * NB <= 320 && ST / 32 * 4 <= 64, "barriers and sums");
    auto bar = [&](int i) { return base + OFF_SBAR + 32u + 8u * (uint32_t)i; };
    const uint32_t lead0 = hs::dsmem_map(smem + OFF_SBAR + 32, 0);
    auto lead = [&](int i) { return lead0 + 8u * (uint32_t)i; };
    // the pages of request b of the list, none if its index is out of range
    auto pages_at = [&](int b, int &r) {
        r = b < p.B ? p.req[b] : -1;
        return r >= 0 && r < p.max_req ? pages_of(hs::context_within(p.ctx[r], p.max_ctx)) : 0;
    };
    auto tiles_of = [](int pages) { return (pages + SP - 1) / SP; };

    const int passes = (p.H + p.hpc - 1) / p.hpc;  // one, unless a token has more than 256 heads
    auto fail = [&]() {
        misc[1] = 1;
        atomicOr(p.err, HS_DEVERR_TIMEOUT);
    };
    uint32_t cols = 32;
    while ((int)cols < 2 * p.N) cols <<= 1;
    if (threadIdx.x == ST - 32) {  // a warp that finds no requests of its own below unless there are hundreds
        for (int i = 0; i < NCH; ++i) mbar_init(bar(B_QFULL + i), 1);
        for (int i = 0; i < NST; ++i) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_READY + i), 8);
            mbar_init(bar(B_FREE + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_DFULL + i), 1);
            mbar_init(bar(B_DFREE + i), 8);
        }
        mbar_init(bar(B_DRAIN), 1);
        misc[1] = 0;
        fence_mbar_init();
        fence_proxy_async();
        prefetch_tmap(&tm_c);
        prefetch_tmap(&tm_q);
    }
    if (warp == 1) tmem_alloc2(base + OFF_SBAR, cols);

    // This pair's range of the requests' tiles, laid end to end, and where it begins.
    const int per = (p.B + ST - 1) / ST;
    int mine = 0, own_r = 0, own_pages = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        own_pages = pages_at((int)threadIdx.x * per + i, own_r);
        mine += tiles_of(own_pages);
    }
    int before = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) sums[warp] = before;
    before -= mine;
    tc_fence_before();
    __syncthreads();
    int all = 0;
#pragma unroll 1
    for (int w = 0; w < ST / 32; ++w) {
        const int x = sums[w];
        before += w < warp ? x : 0;
        all += x;
    }
    const int even = all / p.parts, odd = all - even * p.parts;
    const int f0 = even * part + min(part, odd), f1 = f0 + even + (part < odd ? 1 : 0);
    if (f0 == f1) {
        if (threadIdx.x == 0) misc[2] = misc[3] = misc[4] = misc[5] = 0;
    } else if (f0 >= before && f0 < before + mine) {
        int i = 0, at = before;
        if (per > 1) {
            while (i < per - 1) {
                const int n = tiles_of(pages_at((int)threadIdx.x * per + i, own_r));
                if (f0 < at + n) break;
                at += n;
                ++i;
            }
            own_pages = pages_at((int)threadIdx.x * per + i, own_r);
        }
        misc[2] = (int)threadIdx.x * per + i;
        misc[3] = f0 - at;
        misc[4] = own_r;
        misc[5] = own_pages;
    }
    __syncthreads();
    cluster_sync_relaxed();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);
    const uint32_t tiles = (uint32_t)(f1 - f0) * (uint32_t)passes;  // that this pair multiplies

    // The range's requests, one after the other: every warp walks them for itself.
    struct Walk {
        int b, r, pages, lo, n;  // request, its cache index and pages, first tile, tiles (0: no more)
        int left;                // tiles of the range behind these
    };
    auto take = [&](Walk &w) {
        const int have = tiles_of(w.pages) - w.lo;
        w.n = min(w.left, have);
        w.left -= w.n;
    };
    auto start = [&]() {
        Walk w;
        w.b = misc[2];
        w.lo = misc[3];
        w.r = misc[4];
        w.pages = misc[5];
        w.left = f1 - f0;
        take(w);
        return w;
    };
    auto next = [&](Walk &w) {
        w.n = w.lo = 0;
        if (w.left <= 0) return;
        for (int b0 = w.b + 1; b0 < p.B; b0 += 32) {
            int r;
            const int pages = pages_at(b0 + lane, r);
            const uint32_t some = __ballot_sync(0xffffffffu, pages > 0);
            if (some) {
                const int l = __ffs(some) - 1;
                w.b = b0 + l;
                w.r = __shfl_sync(0xffffffffu, r, l);
                w.pages = __shfl_sync(0xffffffffu, pages, l);
                take(w);
                return;
            }
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // Queries are loaded once for a request (and pass): chunk by chunk, each as
        // soon as the last tile of the request before has used its place, which the
        // ring's wait for a stage NST chunks later has shown.
        Walk w = start();
        uint32_t issued = 0, loads = 0;
        bool ok = true;
        while (w.n > 0 && ok) {
            Walk nx = w;
            next(nx);
            for (int k = 0; k < passes && ok; ++k, ++loads) {
                if (lane == 0) {
                    const bool last = k == passes - 1;
                    auto load_q = [&](int c, int pass, int b) {
                        if (rank == 0) mbar_expect_tx(bar(B_QFULL + c), p.N * 128);
                        tma_load_pair(base + c * (p.N / 2) * 128, &tm_q, 64 * c,
                                      g * p.tpg * p.H + pass * p.hpc + rank * (p.N / 2), b, lead(B_QFULL + c));
                    };
                    for (int i = 0; i < w.n && ok; ++i)
                        for (int c = 0; c < NCH && ok; ++c, ++issued) {
                            const uint32_t s = issued % NST;
                            ok = mbar_wait_inline(bar(B_FREE + s), ((issued / NST) & 1u) ^ 1u);
                            if (!ok) break;
                            if (i == 0 && loads == 0)
                                load_q(c, k, w.b);
                            else if (i == 0 && c < NST)
                                load_q(c + NCH - NST, k, w.b);
                            if (i == w.n - 1 && c >= NST && !(last && nx.n == 0))
                                load_q(c - NST, last ? 0 : k + 1, last ? nx.b : w.b);
                            mbar_expect_tx(bar(B_FULL + s), A_BYTES);
                            tma_load_3d(base + OFF_RING + s * A_BYTES, &tm_c, 64 * c, (w.lo + i) * SP + 128 * rank,
                                        w.r, bar(B_FULL + s));
                        }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            w = nx;
        }
        if (!ok && lane == 0) {
            // the queries' copies are older than the wait that gave up
            fail();
            for (uint32_t u = issued, n = 0; n < NST && u > 0; ++n) {
                --u;
                mbar_wait_inline(bar(B_FULL + u % NST), (u / NST) & 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (CTA 0)
        if (rank == 0) {
            const uint32_t idesc = idesc_f16(1u, 0, SP, p.N);
            const uint64_t d0 = desc_sw128(base, 16, 1024);
            const uint32_t hi = (uint32_t)(d0 >> 32), lo = (uint32_t)d0;
            const uint32_t leader = elect_one();
            const uint32_t qch = (uint32_t)(p.N / 2) * 128u;
            bool ok = true;
            uint32_t u = 0, i = 0, loads = 0;
            const uint32_t last_u = tiles * NCH;
            for (Walk w = start(); w.n > 0 && ok; next(w))
                for (int k = 0; k < passes && ok; ++k, ++loads)
                    for (int j = 0; j < w.n && ok; ++j, ++i) {
                        if (i >= 2)
                            ok = __all_sync(0xffffffffu,
                                            mbar_wait_inline(bar(B_DFREE + (i & 1)), ((i >> 1) & 1u) ^ 1u));
                        if (!ok) break;
                        const uint32_t d = tmem + (i & 1) * (uint32_t)p.N;
                        for (int c = 0; c < NCH && ok; ++c, ++u) {
                            const uint32_t s = u % NST;
                            if (j == 0)
                                ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(B_QFULL + c), loads & 1u));
                            if (ok)
                                ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(B_READY + s), (u / NST) & 1u));
                            if (!ok) break;
                            tc_fence_after();
                            if (leader) {
                                const uint32_t a = lo + ((OFF_RING + s * A_BYTES) >> 4), q = lo + ((c * qch) >> 4);
#pragma unroll
                                for (int e = 0; e < 4; ++e) mma2_ss(d, a + 2 * e, q + 2 * e, hi, idesc, (c | e) != 0);
                                if (u + NST < last_u) commit_both(bar(B_FREE + s));
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        if (leader) commit_both(bar(B_DFULL + (i & 1)));
                        __syncwarp();
                    }
            if (!ok && lane == 0) fail();
            if (leader) {
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 bar(B_DRAIN))
                             : "memory");
                mbar_wait_inline(bar(B_DRAIN), 0);
            }
            __syncwarp();
        }
    } else if (warp < 6) {
        // ------------------------------------------------------------ norms
        const int row = (warp - 2) * 32 + lane;
        bool ok = true;
        uint32_t u = 0;
        for (Walk w = start(); w.n > 0; next(w))
        for (int i = 0; i < passes * w.n; ++i) {
            float n4[4] = {0.f, 0.f, 0.f, 0.f};
            const bool need = i < w.n && (w.lo + i) % p.groups == g;  // the groups share this work
            for (int c = 0; c < NCH; ++c, ++u) {
                const uint32_t s = u % NST;
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(B_FULL + s), (u / NST) & 1u));
                if (ok && need) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 v = ld_shared_v4(base + OFF_RING + s * A_BYTES + row * 128 + ((k ^ (row & 7)) << 4));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = __uint_as_float(w[e] << 16), y = __uint_as_float(w[e] & 0xffff0000u);
                            n4[e] = fmaf(y, y, fmaf(x, x, n4[e]));
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_peer(lead(B_READY + s));
            }
            if (ok && need) {
                const int page = (w.lo + i) * SP + 128 * rank + row;
                const bool in = page < w.pages;
                float cn = (n4[0] + n4[1]) + (n4[2] + n4[3]);
                if (in && cn == 0.f) {  // rare: squares below f32's normal numbers, or zeros
                    const uint4 *c = p.means + ((size_t)w.r * p.max_pages + page) * (2 * kDim / 16);
                    uint32_t any = 0;
#pragma unroll 1
                    for (int k = 0; k < 2 * kDim / 16; ++k) any |= c[k].x | c[k].y | c[k].z | c[k].w;
                    if (any & 0x7fff7fffu) cn = FLT_MIN;
                }
                float m = in ? (cn <= FLT_MAX ? cn : INFINITY) : 0.f;
                m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                if (in) p.cn[(size_t)w.b * p.Pp + page] = cn;
                if (in && lane == 0) p.cm[((size_t)w.b * p.Pp + page) / 32] = m;
            }
        }
        if (!ok && lane == 0) fail();
    } else {
        // ------------------------------------------------------------ maxima over heads
        const int wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        bool ok = true;
        uint32_t i = 0;
        for (Walk w = start(); w.n > 0; next(w))
        for (int k = 0; k < passes; ++k)
        for (int j = 0; j < w.n; ++j, ++i) {
            const int page = (w.lo + j) * SP + 128 * rank + row;
            const int h0 = k * p.hpc, hn = min(p.hpc, p.H - h0);  // heads of this pass
            const int t0 = g * p.tpg, tn = min(p.tpg, p.T - t0);
            const int rows = tn * hn;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(B_DFULL + (i & 1)), (i >> 1) & 1u));
            if (ok) {
                tc_fence_after();
                int t = t0, h = 0, arg = 0;
                float m = -INFINITY, m2 = -INFINITY;  // best group's score and the best of the others
                const uint32_t d0 = tmem + lane_off + (i & 1) * (uint32_t)p.N;
                auto group = [&](float x, int g8) {
                    m2 = fmaxf(m2, fminf(m, x));
                    arg = x > m ? g8 : arg;
                    m = fmaxf(m, x);
                };
                auto flush = [&]() {
                    if (page < w.pages) {
                        const size_t at = ((size_t)w.b * p.T + t) * p.Pp + page;
                        arg += h0 / HG;
                        if (k > 0) {  // with the earlier heads', which this thread stored itself
                            const float o = p.s1[at];
                            const uint32_t x2 = p.s2[at];
                            m2 = fmaxf(fmaxf(m2, __uint_as_float(x2 & 0xffff0000u)), fminf(m, o));
                            arg = m > o ? arg : (int)(x2 & 0xffffu);
                            m = fmaxf(m, o);
                        }
                        p.s1[at] = m;
                        // rounded up: its distance to the best is never overstated
                        p.s2[at] = ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_ru(m2)) << 16) | (uint32_t)arg;
                    }
                    m = m2 = -INFINITY;
                    h = arg = 0;
                    ++t;
                };
                float part = -INFINITY;  // heads that do not come in whole groups
                for (int c0 = 0; c0 < rows; c0 += 32) {
                    uint32_t d[32];
                    HS_TMEM_LD32(d0 + c0, d);
                    HS_TMEM_WAIT_LD32(d);
                    auto f = [&](int e) { return __uint_as_float(d[e]); };
                    if (hn % HG == 0) {
#pragma unroll
                        for (int e = 0; e < 32; e += HG) {
                            if (c0 + e < rows) {
                                group(fmaxf(max3(f(e), f(e + 1), f(e + 2)),
                                            max3(f(e + 3), max3(f(e + 4), f(e + 5), f(e + 6)), f(e + 7))),
                                      h / HG);
                                if ((h += HG) == hn) flush();
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (c0 + e < rows) {
                                part = fmaxf(part, f(e));
                                if (++h % HG == 0 || h == hn) {
                                    group(part, (h - 1) / HG);
                                    part = -INFINITY;
                                }
                                if (h == hn) flush();
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && i + 2 < tiles) mbar_arrive_peer(lead(B_DFREE + (i & 1)));
        }
        if (!ok && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();
    // No CTA leaves while the other's MMAs or arrives may reach it: every arrive on the
    // other's barriers is one that it waits for, so none is on its way any more.
    cluster_arrive_last(misc[1] != 0);
    cluster_wait();
    tc_fence_after();
    if (warp == 1) tmem_dealloc2(tmem, cols);
}

// ---------------------------------------------------------------- selection
// One CTA per (request, query token): 1024 threads, or 256 where they can keep
// all of a request's scores (fewer barrier partners: a call for one list of 64 pages
// takes 10.9 us instead of 13.6). The scores are read once, as integers in the
// scores' order. A histogram of them finds the border's bin (one pass where the
// scores are of one magnitude, three at most), the bin's members give the k-th
// largest score, and a last pass collects the pages above the border's interval
// and those inside it; the latter are summed again (dot64).
constexpr int BINS = 2048;
constexpr int CAP = 512;       // pages near the border that fit in shared memory
constexpr int MAXSEL = 1024;   // pages per list
constexpr int KEEP = 16;       // scores that a thread keeps in registers

struct SelectParams {
    const int32_t *req, *ctx;
    const uint64_t *tree;            // [B][T] or null
    const __nv_bfloat16 *q, *means;  // [B][T][H][576], [max_req][max_pages][576]
    float *s1;
    uint32_t *s2;
    const float *cn, *cm;
    uint64_t *key64;                 // [B*T][Pp] only written when more than CAP pages are near the border
    int32_t *pages, *topk;           // [B][T][N], [B][T][N*64] or null
    uint32_t *err;
    int T, H, N, n_first, n_last, Pp, max_req, max_pages, max_ctx;
};

__device__ __forceinline__ uint32_t order32(float x) {
    const uint32_t u = __float_as_uint(x) == 0x80000000u ? 0u : __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_order32(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr float NORM_LOST = kDim * FLT_MIN;  // of a norm's square
constexpr float SUMS_LOST = 2048.f * FLT_MIN;  // of 2 E
constexpr uint32_t KEY_MOST = 0xff7fffffu, KEY_LEAST = 0x00800000u;  // of the finite scores
// NaN ranks with minus infinity
__device__ __forceinline__ uint64_t order64(double x) {
    if (x != x) x = -(double)INFINITY;
    const uint64_t u = x == 0.0 ? 0ull : (uint64_t)__double_as_longlong(x);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

// f32 arithmetic that keeps numbers below the normal ones (the build flushes them).
__device__ __forceinline__ float add_full(float a, float b) {
    float d;
    asm("add.rn.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float sub_full(float a, float b) {
    float d;
    asm("sub.rn.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float mul_full(float a, float b) {
    float d;
    asm("mul.rn.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ double to_double(float a) {
    double d;
    asm("cvt.f64.f32 %0, %1;" : "=d"(d) : "f"(a));
    return d;
}
// a becomes a + b; returns what its rounding left out, exactly (Knuth's two-sum).
__device__ __forceinline__ float two_sum(float &a, float b) {
    const float t = add_full(a, b), y = sub_full(t, a);
    const float rest = add_full(sub_full(a, sub_full(t, y)), sub_full(b, y));
    a = t;
    return rest;
}

// q . c as exactly as in 64 bits, by a warp (every lane gets the sum). Products of BF16
// values above f32's smallest numbers are exact in f32, and sums are kept in three words:
// what a sum's rounding leaves out goes into the second by another two-sum, and what that
// leaves out into the third. With S the sum of the products' magnitudes, and the adds of
// the first word 23 deep (18 products of a lane, five joins), of the second 28: the second
// word stays below 23 x 2^-24 S, the third below 28 x 2^-24 of that, 2^-38 S, and its
// roundings are below 2^-56 S. With the two of the join in 64 bits, whose arithmetic is
// 1/64 as fast, less than 2^-50 S is lost. (Two words lose up to 2^-39 S.)
__device__ __forceinline__ double dot64(const __nv_bfloat16 *q, const __nv_bfloat16 *c) {
    const int lane = threadIdx.x & 31;
    uint32_t a[kDim / 64], b[kDim / 64];
#pragma unroll
    for (int i = 0; i < kDim / 64; ++i) {
        a[i] = reinterpret_cast<const uint32_t *>(q)[lane + 32 * i];
        b[i] = reinterpret_cast<const uint32_t *>(c)[lane + 32 * i];
    }
    float s = 0.f, r = 0.f, t = 0.f;
    auto add = [&](float x) { t = add_full(t, two_sum(r, two_sum(s, x))); };
#pragma unroll
    for (int i = 0; i < kDim / 64; ++i) {
        add(mul_full(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16)));
        add(mul_full(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u)));
    }
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) {
        const float so = __shfl_xor_sync(0xffffffffu, s, o), ro = __shfl_xor_sync(0xffffffffu, r, o);
        const float to = __shfl_xor_sync(0xffffffffu, t, o);
        add(so);
        t = add_full(t, add_full(two_sum(r, ro), to));
    }
    double acc = to_double(s) + (to_double(r) + to_double(t));
    if (!(fabs(acc) <= (double)FLT_MAX)) {
        // infinities, NaN, or products beyond 32 bits: the same in every lane
        acc = 0.0;
#pragma unroll 1
        for (int i = lane; i < kDim; i += 32)
            acc = fma((double)__bfloat162float(q[i]), (double)__bfloat162float(c[i]), acc);
#pragma unroll 1
        for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    }
    return acc;
}
// The same in 32 bits: off by less than 2^-19 |q||c|, well inside E.
__device__ __forceinline__ float dot32(const __nv_bfloat16 *q, const __nv_bfloat16 *c) {
    const int lane = threadIdx.x & 31;
    float x = 0.f;
#pragma unroll 3
    for (int i = 0; i < kDim / 64; ++i) {
        const uint32_t a = reinterpret_cast<const uint32_t *>(q)[lane + 32 * i];
        const uint32_t b = reinterpret_cast<const uint32_t *>(c)[lane + 32 * i];
        x = fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), x);
        x = fmaf(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u), x);
    }
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int LT>
__global__ void __launch_bounds__(LT) select_kernel(const SelectParams p) {
    constexpr int NW = LT / 32, PB = BINS / LT;
    __shared__ int hist[BINS];
    __shared__ uint32_t lkey[CAP];
    __shared__ int lpage[CAP];
    __shared__ unsigned long long lk64[CAP];
    __shared__ int sel[MAXSEL], sorted[MAXSEL];
    __shared__ int warp_i[32];
    __shared__ uint32_t s_lo, s_hi, s_theta;
    __shared__ int s_need, s_bin, s_m, s_nsel, s_near, s_qn, s_cn;
    const int list = blockIdx.x, b = list / p.T, t = list % p.T;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = p.req[b];
    const bool req_ok = r >= 0 && r < p.max_req;
    const int len = req_ok ? p.ctx[r] : 0, L = hs::context_within(len, p.max_ctx);
    const __nv_bfloat16 *q = p.q + (size_t)list * p.H * kDim;
    const long long end = p.tree ? (long long)L : (long long)L - p.T + t + 1;
    const int n = end <= 0 ? 0 : pages_of((int)end);  // pages that hold a token this one may see
    const bool all = n <= p.N;
    const int k = p.N - p.n_first - p.n_last;
    const int c0 = p.n_first, cnt = n - p.n_last - c0;  // candidates (when not all)
    if (!req_ok && tid == 0) atomicOr(p.err, HS_DEVERR_BAD_REQUEST);
    if (len > p.max_ctx && tid == 0) atomicOr(p.err, HS_DEVERR_INDEX_RANGE);
    if (tid == 0) {
        s_nsel = s_m = s_near = 0;
        s_lo = 0xffffffffu;
        s_hi = 0u;
        s_qn = __float_as_int(-1.f);
        s_cn = 0;
    }
    if (all) {
        for (int i = tid; i < p.N; i += LT) sorted[i] = i < n ? i : -1;
    } else {
        for (int i = tid; i < p.n_first; i += LT) sel[k + i] = i;
        for (int i = tid; i < p.n_last; i += LT) sel[k + p.n_first + i] = n - p.n_last + i;
    }
    __syncthreads();
    if (!all && k > 0) {
        // max |q_h|^2; the queries were there before the scores' kernel began. A head that
        // holds a NaN has no sum that counts, so its norm does not either.
        float mx = -1.f;
        for (int h = warp; h < p.H; h += NW) {
            const uint32_t *qr = reinterpret_cast<const uint32_t *>(q + (size_t)h * kDim);
            float x = 0.f, y = 0.f;
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < kDim / 64; ++i) {
                const uint32_t w = qr[lane + 32 * i];
                any |= w & 0x7fff7fffu;
                const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
                x = fmaf(lo, lo, x);
                y = fmaf(hi, hi, y);
            }
            x += y;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (x == 0.f && __any_sync(0xffffffffu, any)) x = FLT_MIN;  // not a row of zeros
            mx = fmaxf(mx, x);  // NaN drops out
            if (mx == INFINITY) break;
        }
        // as an integer: the order of those that are not negative, and -1.f below them
        if (lane == 0) atomicMax(&s_qn, __float_as_int(mx));
    }
    grid_dep_wait();  // the scores
    grid_dep_launch();
    if (!all && k > 0) {
        float *s1 = p.s1 + (size_t)list * p.Pp + c0;
        uint32_t *s2 = p.s2 + (size_t)list * p.Pp + c0;
        const float *cn = p.cn + (size_t)b * p.Pp + c0, *cm = p.cm + (size_t)b * p.Pp / 32;
        const __nv_bfloat16 *means = p.means + ((size_t)r * p.max_pages + c0) * kDim;
        // one reading of the scores, all loads at once; candidates are numbered from 0
        uint32_t v[KEEP];
        auto load = [&]() {
            float x[KEEP];
#pragma unroll
            for (int u = 0; u < KEEP; ++u) x[u] = tid + u * LT < cnt ? s1[tid + u * LT] : 0.f;
#pragma unroll
            for (int u = 0; u < KEEP; ++u) v[u] = order32(x[u]);
        };
        auto each = [&](auto f) {
#pragma unroll
            for (int u = 0; u < KEEP; ++u)
                if (tid + u * LT < cnt) f(tid + u * LT, v[u]);
            for (int i = tid + KEEP * LT; i < cnt; i += LT) f(i, order32(s1[i]));
        };
        // the same for the few that satisfy `is`: little code in the unrolled part
        // (instructions that run once come from memory)
        auto pick = [&](auto is, auto f) {
            uint32_t mask = 0;
#pragma unroll
            for (int u = 0; u < KEEP; ++u) mask |= (tid + u * LT < cnt && is(v[u]) ? 1u : 0u) << u;
            while (mask) {
                const int i = tid + (__ffs(mask) - 1) * LT;
                mask &= mask - 1;
                f(i, order32(s1[i]));
            }
            for (int i = tid + KEEP * LT; i < cnt; i += LT) {
                const uint32_t key = order32(s1[i]);
                if (is(key)) f(i, key);
            }
        };
        load();
        uint32_t lo = 0xffffffffu, hi = 0u;
        float cmx = 0.f;
        for (int i = tid; i < (n + 31) / 32; i += LT) cmx = fmaxf(cmx, cm[i]);
        each([&](int, uint32_t key) {
            lo = min(lo, key);
            hi = max(hi, key);
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        cmx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(cmx)));
        if (lane == 0) {
            atomicMin(&s_lo, lo);
            atomicMax(&s_hi, hi);
            atomicMax(&s_cn, __float_as_int(cmx));
        }
        __syncthreads();
        lo = s_lo;
        hi = s_hi;
        // a page whose score or norm is not finite says nothing in 32 bits
        // (where every head holds a NaN, all scores are minus infinity)
        const float qn = __int_as_float(s_qn);
        const bool some_unknown = qn >= 0.f && (lo < KEY_LEAST || hi > KEY_MOST || __int_as_float(s_cn) > FLT_MAX);
        if (some_unknown) {
            // those pages' scores in 64 bits; what stands for them in 32 is the
            // rounded sum
            __syncthreads();
            if (tid == 0) {
                s_lo = 0xffffffffu;
                s_hi = 0u;
                s_cn = 0;
            }
            __syncthreads();
            for (int i0 = warp * 32; i0 < cnt; i0 += LT) {
                const int i = i0 + lane;
                float s = i < cnt ? s1[i] : 0.f;
                const float c = i < cnt ? cn[i] : 0.f;
                const bool mine = i < cnt && (!(fabsf(s) <= FLT_MAX) || !(c <= FLT_MAX));
                unsigned todo = __ballot_sync(0xffffffffu, mine);
                while (todo) {
                    const int who = __ffs(todo) - 1, pg = i0 + who;
                    todo &= todo - 1;
                    double best = -(double)INFINITY;
                    for (int h = 0; h < p.H; ++h) {
                        const double d = dot64(q + (size_t)h * kDim, means + (size_t)pg * kDim);
                        best = d > best ? d : best;
                    }
                    if (lane == who) {
                        s = __double2float_rn(best);
                        s1[pg] = s;
                        s2[pg] = 0x7f800000u;  // another group's may be as good
                    }
                }
                if (i < cnt) {
                    const uint32_t key = order32(s);
                    atomicMin(&s_lo, key);
                    atomicMax(&s_hi, key);
                    if (!mine) atomicMax(&s_cn, __float_as_int(c));
                }
            }
            __syncthreads();
            load();
            lo = s_lo;
            hi = s_hi;
        }
        // ------------------------------------------------ the border's bin
        int need = k, m = cnt;
        while (m > CAP && lo != hi) {
            const int bits = 32 - __clz((int)(hi - lo));
            const int sh = bits > 11 ? bits - 11 : 0;
            for (int i = tid; i < BINS; i += LT) hist[i] = 0;
            __syncthreads();
            const uint32_t span = hi - lo;
            each([&](int, uint32_t key) {
                if (key - lo <= span) atomicAdd(&hist[(key - lo) >> sh], 1);
            });
            __syncthreads();
            // from the top: a thread's PB bins, the highest first
            const int b0 = BINS - 1 - PB * tid;
            int hb[PB], own = 0;
#pragma unroll
            for (int e = 0; e < PB; ++e) own += hb[e] = hist[b0 - e];
            int sum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += x;
            }
            if (lane == 31) warp_i[warp] = sum;
            __syncthreads();
            int above = sum - own;  // members above this thread's bins
            for (int w = 0; w < warp; ++w) above += warp_i[w];
#pragma unroll
            for (int e = 0; e < PB; ++e) {
                if (above < need && above + hb[e] >= need) {
                    s_bin = b0 - e;
                    s_need = need - above;
                    s_m = hb[e];
                }
                above += hb[e];
            }
            __syncthreads();
            need = s_need;
            m = s_m;
            lo = lo + ((uint32_t)s_bin << sh);
            hi = min(hi, lo + ((sh ? (1u << sh) : 1u) - 1u));
            __syncthreads();
        }
        // the k-th largest score: the need-th of the bin
        if (tid == 0) {
            s_m = 0;
            s_theta = lo;
        }
        __syncthreads();
        if (lo != hi) {
            const uint32_t span = hi - lo;
            pick([&](uint32_t key) { return key - lo <= span; },
                 [&](int, uint32_t key) { lkey[atomicAdd(&s_m, 1)] = key; });
            __syncthreads();
            for (int i = tid; i < m; i += LT) {
                int above = 0, equal = 0;
                const uint32_t mine = lkey[i];
                for (int j = 0; j < m; ++j) {
                    above += lkey[j] > mine;
                    equal += lkey[j] == mine;
                }
                if (above < need && above + equal >= need) s_theta = mine;
            }
            __syncthreads();
        }
        // ------------------------------------------------ above it, and near it
        // The interval's bounds are rounded outwards; a bound that is NaN (norms
        // beyond 32 bits) makes every page near.
        const float theta = from_order32(s_theta), cmost = __int_as_float(s_cn);
        const bool same = qn < 0.f || ((qn == 0.f || cmost == 0.f) && !some_unknown);  // the sums are exact as they are
        const float qc = __fmul_ru(__fsqrt_ru(__fadd_ru(qn, NORM_LOST)), __fsqrt_ru(__fadd_ru(cmost, NORM_LOST)));
        const float e2 = same ? 0.f : __fadd_ru(__fmul_ru(2.f / 32768.f * 1.001f, qc), SUMS_LOST);
        const float slack = __fadd_ru(e2, __fmul_ru(fabsf(theta), 1.f / 4194304.f));
        const float fup = __fadd_ru(theta, slack), fdn = __fadd_rd(theta, -slack);
        const uint32_t up = fup == fup ? order32(fup) : 0xffffffffu, dn = fdn == fdn ? order32(fdn) : 0u;
        pick([&](uint32_t key) { return key >= dn; },
             [&](int i, uint32_t key) {
                 if (key > up) {
                     sel[atomicAdd(&s_nsel, 1)] = c0 + i;
                 } else {
                     const int j = atomicAdd(&s_near, 1);
                     if (j < CAP) lpage[j] = i;
                 }
             });
        __syncthreads();
        const int first = s_nsel;
        need = k - first;
        m = s_near;
        if (m == need && m <= CAP) {
            for (int i = tid; i < m; i += LT) sel[first + i] = c0 + lpage[i];
        } else if (m <= CAP) {
            for (int i = tid; i < m; i += LT) lk64[i] = same ? order64((double)s1[lpage[i]]) : 0ull;
            __syncthreads();
            if (!same) {
                // The heads in question: those of the best group, or all where
                // another group comes near it. A warp takes one at a time.
                for (int e = 0; e < m; ++e) {
                    const int pg = lpage[e];
                    const uint32_t w = s2[pg];
                    const bool one = s1[pg] - __uint_as_float(w & 0xffff0000u) > e2;
                    const int h0 = one ? (int)(w & 0xffffu) * HG : 0, hn = one ? min(HG, p.H - h0) : p.H;
                    // entries begin at different warps, so that they run at once
                    for (int h = (warp + NW - e * HG % NW) % NW; h < hn; h += NW) {
                        const double y = dot64(q + (size_t)(h0 + h) * kDim, means + (size_t)pg * kDim);
                        if (lane == 0) atomicMax(&lk64[e], (unsigned long long)order64(y));
                    }
                }
                __syncthreads();
            }
            for (int i = tid; i < m; i += LT) {
                int better = 0;
                for (int j = 0; j < m; ++j)
                    better += lk64[j] > lk64[i] || (lk64[j] == lk64[i] && lpage[j] < lpage[i]);
                if (better < need) sel[first + better] = c0 + lpage[i];
            }
        } else {
            // very many equal or nearly equal scores: keys of all candidates in
            // memory, the need-th largest by bisection, ties by position
            uint64_t *k64 = p.key64 + (size_t)list * p.Pp;
            for (int i = warp; i < cnt; i += NW) {
                const uint32_t key32 = order32(s1[i]);
                uint64_t key = 0;
                if (key32 >= dn && key32 <= up) {
                    if (same) {
                        key = order64((double)s1[i]);
                    } else {
                        const __nv_bfloat16 *c = means + (size_t)i * kDim;
                        // the heads whose 32-bit sums come near the best; all of them
                        // where e2 does not bound this page's sums
                        const bool bounded = cn[i] <= FLT_MAX;
                        float best = -INFINITY;
                        for (int h = 0; h < p.H && bounded; ++h) best = fmaxf(best, dot32(q + (size_t)h * kDim, c));
                        for (int h = 0; h < p.H; ++h) {
                            const __nv_bfloat16 *qh = q + (size_t)h * kDim;
                            if (bounded && dot32(qh, c) < best - e2) continue;
                            const uint64_t y = order64(dot64(qh, c));
                            key = y > key ? y : key;
                        }
                    }
                }
                if (lane == 0) k64[i] = key;
            }
            __syncthreads();
            auto count = [&](uint64_t at_least) {  // by the whole CTA
                int c = 0;
                for (int i = tid; i < cnt; i += LT) c += k64[i] >= at_least;
                c = __reduce_add_sync(0xffffffffu, c);
                if (lane == 0) warp_i[warp] = c;
                __syncthreads();
                c = 0;
                for (int w = 0; w < NW; ++w) c += warp_i[w];
                __syncthreads();
                return c;
            };
            uint64_t tau = 0;  // the largest key that at least `need` pages reach
            for (int bit = 63; bit >= 0; --bit) {
                const uint64_t mid = tau | (1ull << bit);
                if (count(mid) >= need) tau = mid;
            }
            int room = need - count(tau + 1);  // of those equal to it, the lowest pages
            if (tid == 0) s_m = 0;
            __syncthreads();
            for (int i0 = 0; i0 < cnt; i0 += LT) {
                const int i = i0 + tid;
                const uint64_t key = i < cnt ? k64[i] : 0;
                int total;
                const int rank = hs::block_scan_flag<LT>(i < cnt && key == tau, warp_i, total);
                if (i < cnt && (key > tau || (key == tau && rank < room)))
                    sel[first + atomicAdd(&s_m, 1)] = c0 + i;
                room -= total;
            }
        }
    }
    __syncthreads();
    if (!all) {
        // ascending order
        for (int i = tid; i < p.N; i += LT) {
            const int mine = sel[i];
            int at = 0;
            for (int j = 0; j < p.N; ++j) at += sel[j] < mine;
            sorted[at] = mine;
        }
        __syncthreads();
    }
    for (int i = tid; i < p.N; i += LT) p.pages[(size_t)list * p.N + i] = sorted[i];
    if (p.topk) {
        const uint64_t tree = p.tree ? p.tree[list] : 0;
        int32_t *o = p.topk + (size_t)list * p.N * kPage;
        for (int i = tid; i < p.N * kPage; i += LT) {
            const int pg = sorted[i / kPage];
            int pos = -1;
            if (pg >= 0) {
                const long long x = (long long)pg * kPage + i % kPage, node = x - ((long long)L - p.T);
                const bool seen = p.tree ? (node < 0 || (node < p.T && ((tree >> node) & 1))) : x < end;
                if (seen) pos = (int)x;
            }
            o[i] = pos;
        }
    }
}

struct Ws {
    int Pp;
    size_t s1, s2, cn, cm, k64, total;
};
Ws workspace(const hs_pool *pool, int64_t B, int64_t T) {
    Ws w{};
    w.Pp = (pool->max_pages + 31) & ~31;
    const size_t lists = (size_t)B * T, row = (size_t)w.Pp;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    w.s1 = 0;
    w.s2 = up(lists * row * 4);
    w.cn = w.s2 + up(lists * row * 4);
    w.cm = w.cn + up((size_t)B * row * 4);
    w.k64 = w.cm + up((size_t)B * row / 32 * 4);
    w.total = w.k64 + up(lists * row * 8);
    return w;
}

// Parts that the page tiles of all requests are cut into, each worked through by one
// pair of CTAs per group: the count that a model of the launch makes shortest. A tile
// takes a pair about 2.8 us (the pages' bytes at the card's rate, or 256 query rows'
// products), its start and the queries 4 us. Groups of one part run side by side and
// share its pages in L2.
int score_parts(int64_t groups, int64_t tiles) {
    const int64_t pairs = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
    double best = 1e300;
    int64_t parts = 1;
    for (int64_t w = 1; w <= 8; ++w) {
        int64_t n = w * pairs / groups;
        n = n < 1 ? 1 : (n > tiles ? tiles : n);
        const double waves = (double)((groups * n + pairs - 1) / pairs);
        const double t = waves * ((double)((tiles + n - 1) / n) * 2.8 + 4.0);
        if (t < best * 0.98) {
            best = t;
            parts = n;
        }
    }
    return (int)parts;
}

hs_status score_attr(int dev) {
    static std::atomic<int> state[64];
    if (dev < 0 || dev >= 64) return HS_ERR_UNSUPPORTED;
    if (state[dev].load(std::memory_order_acquire) == 1) return HS_OK;
    HS_CUDA_TRY(cudaFuncSetAttribute(score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SCORE_SMEM));
    state[dev].store(1, std::memory_order_release);
    return HS_OK;
}

}  // namespace

extern "C" size_t hs_select_workspace_bytes(hs_pool_t pool, int32_t B, int32_t T) {
    if (!pool || B < 1 || B > 65535 || T < 1 || T > 32767) return 0;
    return workspace(pool, B, T).total;
}

extern "C" hs_status hs_select_pages(hs_pool_t pool, int32_t B, int32_t T, int32_t H, int32_t N,
                                     int32_t n_first, int32_t n_last, const void *d_q,
                                     const void *d_means, const int32_t *d_req_ids,
                                     const uint64_t *d_tree, int32_t *d_pages, int32_t *d_topk_idx,
                                     void *d_workspace, size_t ws_bytes, void *stream) {
    if (!pool || B < 0 || B > 65535 || T < 1 || T > 32767 || H < 1 || H > 65535 ||
        (int64_t)T * H > (1 << 22) || (int64_t)B * T > INT32_MAX || N < 1 || n_first < 0 ||
        n_last < 0 || (int64_t)n_first + n_last > N || (d_tree && T > 64))
        return HS_ERR_INVALID_ARG;
    if (N > MAXSEL) return HS_ERR_CAPACITY;
    if (B == 0) return HS_OK;
    if (!d_q || !d_means || !d_req_ids || !d_pages || !d_workspace) return HS_ERR_INVALID_ARG;
    if (((uintptr_t)d_q | (uintptr_t)d_means) & 15u) return HS_ERR_INVALID_ARG;
    const Ws w = workspace(pool, B, T);
    if (ws_bytes < w.total || ((uintptr_t)d_workspace & 255u)) return HS_ERR_INVALID_ARG;
    int dev = -1;
    HS_CUDA_TRY(cudaGetDevice(&dev));
    if (dev != pool->device) return HS_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(d_workspace);

    if (pool->max_pages > N && N > n_first + n_last) {
        const hs_status st = score_attr(dev);
        if (st != HS_OK) return st;
        ScoreParams p{};
        p.req = d_req_ids;
        p.ctx = pool->d_ctx;
        p.means = static_cast<const uint4 *>(d_means);
        p.s1 = reinterpret_cast<float *>(ws + w.s1);
        p.s2 = reinterpret_cast<uint32_t *>(ws + w.s2);
        p.cn = reinterpret_cast<float *>(ws + w.cn);
        p.err = pool->d_err;
        p.cm = reinterpret_cast<float *>(ws + w.cm);
        p.B = B;
        p.T = T;
        p.H = H;
        p.hpc = H < MAXN ? H : MAXN;
        p.tpg = MAXN / p.hpc < T ? MAXN / p.hpc : T;
        p.groups = (T + p.tpg - 1) / p.tpg;
        p.N = (p.tpg * p.hpc + 31) & ~31;
        const int64_t tiles = (int64_t)B * ((pool->max_pages + SP - 1) / SP);
        p.parts = score_parts(p.groups, tiles);
        const int64_t units = (int64_t)p.groups * p.parts;
        if (2 * units > INT32_MAX || tiles > INT32_MAX) return HS_ERR_INVALID_ARG;
        p.Pp = w.Pp;
        p.max_req = pool->cfg.max_requests;
        p.max_pages = pool->max_pages;
        p.max_ctx = pool->cfg.max_ctx;
        CUtensorMap tc, tq;
        if (!make_map(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_means, kDim, pool->max_pages,
                      pool->cfg.max_requests, 2 * kDim, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_q, kDim, (uint64_t)T * H, B, 2 * kDim, 64, p.N / 2,
                      CU_TENSOR_MAP_SWIZZLE_128B))
            return HS_ERR_CUDA;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(2 * units), 1, 1);
        cfg.blockDim = dim3(ST, 1, 1);
        cfg.dynamicSmemBytes = SCORE_SMEM;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        if (cudaLaunchKernelEx(&cfg, score_kernel, tc, tq, p) != cudaSuccess) return HS_ERR_CUDA;
    }
    SelectParams p{};
    p.req = d_req_ids;
    p.ctx = pool->d_ctx;
    p.tree = d_tree;
    p.q = static_cast<const __nv_bfloat16 *>(d_q);
    p.means = static_cast<const __nv_bfloat16 *>(d_means);
    p.s1 = reinterpret_cast<float *>(ws + w.s1);
    p.s2 = reinterpret_cast<uint32_t *>(ws + w.s2);
    p.cn = reinterpret_cast<const float *>(ws + w.cn);
    p.cm = reinterpret_cast<const float *>(ws + w.cm);
    p.key64 = reinterpret_cast<uint64_t *>(ws + w.k64);
    p.pages = d_pages;
    p.topk = d_topk_idx;
    p.err = pool->d_err;
    p.T = T;
    p.H = H;
    p.N = N;
    p.n_first = n_first;
    p.n_last = n_last;
    p.Pp = w.Pp;
    p.max_req = pool->cfg.max_requests;
    p.max_pages = pool->max_pages;
    p.max_ctx = pool->cfg.max_ctx;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)B * T), 1, 1);
    const bool few = pool->max_pages <= KEEP * 256;
    cfg.blockDim = dim3(few ? 256 : 1024, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    // its first part needs nothing of the scores' kernel
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pool->max_pages > N && N > n_first + n_last ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, few ? select_kernel<256> : select_kernel<1024>, p) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}
