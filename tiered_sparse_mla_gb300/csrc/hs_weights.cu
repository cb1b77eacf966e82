// hs_weights.cu -- the attention weight that each page gets, on tcgen05 tensor cores:
//   W'[r][p] = decay W[r][p] + sum over query rows m and the page's keys j that m sees of
//              exp(scale q_m.k_j - lse_m).
// With the attention's lse no running maximum is needed and no product with values: one
// pass over the keys, whose scores are exponentiated and added up where they arise.
//
// Work unit: a group of at most 256 query rows and a range of the key tiles (four pages)
// of all requests laid end to end, run by two CTAs whose tensor cores work as one
// (cta_group::2, M = 256): keys are the MMA's M rows, 128 (two pages) per CTA, so that a
// key's sum runs along the registers of the threads that own it, and query rows its N
// columns, half of them supplied by either CTA. The queries stay in shared memory (up to
// 144 KB a CTA), the keys stream past once, and one tile's exponentials run while the next
// is multiplied (two accumulators). Several groups' sums meet in a second grid; the rows are
// dealt to them evenly (12 x 27,929 FP8 keys, 264 rows: 64 us with 160 columns each, 79 with 192;
// 16 rows of 16 x 3,000: 11.4 with 32 columns, 12.7 with 64). Where a
// range goes on to another request, each chunk of its queries comes as soon as the last tile's
// MMAs have read that chunk of the one before (8 x 8,000 BF16 keys, 512 rows: 34.2 -> 30.7 us
// against all chunks after the last tile; a second place for them, up to 128 rows, changes nothing).
//   warp 0      producer: key chunks;
//   warp 1      (CTA 0) MMA issuer: one lane, waits and all. With the warp's 32 lanes agreeing on each wait
//               it cannot keep up with chunks of 192 or fewer columns (4 x 20,000 BF16 keys, 528 rows: 48 us
//               instead of 39);
//   warps 2-9   per request: the columns' terms; per tile: the sums, thread = key and half of
//               the columns;
//   warp 10     producer: queries.
// FP8: scores from the e4m3 codes themselves (kind::f8f6f4). A query value times its row's
// power of two, which brings the row's largest to (224, 448], is the sum of two codes: exact
// from 2^-9.8 of that largest on, off by at most 2^-17.8 of it below. A grid of its own makes the
// codes of each row once, in the workspace; pairs that did so for themselves at each request took
// 4 to 5 us each time (30 x 6,000 keys, 256 rows: 46 -> 37 us; 40 x 1,000, 32 rows: 15.0 -> 12.8).
// Only 64 x 500 keys, 256 rows, where every pair has one request, were faster so (22 against 24).
// Bound: the keys' bytes, or for 256 rows of codes 36 MMAs of 128 clocks per tile. 4 x 74,160 BF16
// keys, 256 rows: 62 us, tiles at the copy rate from 7 us on; 8 x 131,072 FP8 keys, 512 rows: 310 to
// 400 us with the clock, 1.96 to 1.52 PFLOP/s. Pages asked into L2 two tiles ahead: 85 instead of 67 us.
// Ranges cut at half tiles or at pages, whose last tiles are not full: 8 x 8,000 BF16 keys, 512 rows
// 28.1 instead of 26.1 us, 4 x 74,160 the same.
// Every wait is bounded; on expiry the kernel sets HS_DEVERR_TIMEOUT, drains its own
// copies and MMAs and returns.
#include <cuda_bf16.h>

#include <atomic>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "hs_internal.cuh"
#include "hs_pages.cuh"
#include "hs_tc.cuh"
#include "hs_tmap.cuh"

namespace {

using namespace hs::tc;
using hs::kDim;
using hs::kPage;

constexpr int TP = 4;            // pages per tile (two CTAs)
constexpr int NCH = kDim / 64;   // depth chunks
constexpr int MAXN = 256;        // query rows per group
constexpr int NEW = 8;           // warps for the sums
constexpr int WT = 96 + 32 * NEW;
constexpr int MAXST = 16;        // ring stages, one chunk of 128 keys each
constexpr int SMEM_MOST = 232448;

template <bool FP8>
struct WCfg {
    static constexpr int STAGE = FP8 ? 128 * 64 : 128 * 128;
    static constexpr int OFF_A = 0;                               // FP8 f32 [256]: scale over the rows' powers
    static constexpr int OFF_B = OFF_A + (FP8 ? MAXN * 4 : 0);    // f32 [256]: -lse, in log2 units
    static constexpr int OFF_PS = OFF_B + MAXN * 4;               // f32 [2][8]: sums of a tile, by warp
    static constexpr int OFF_DEAD = OFF_PS + 2 * NEW * 4;         // u32 [8]: columns that add nothing
    static constexpr int OFF_MISC = OFF_DEAD + 32;                // TMEM base, abort flag
    static constexpr int OFF_BAR = OFF_MISC + 16;
    static constexpr int B_QFULL = 0, B_QFREE = NCH, B_DRAIN = 2 * NCH, B_DFULL = B_DRAIN + 1, B_DFREE = B_DFULL + 2,
                         B_FULL = B_DFREE + 2, B_FREE = B_FULL + MAXST, NBAR = B_FREE + MAXST;
    static constexpr int HEAD = OFF_BAR + 8 * NBAR;
    __host__ __device__ static int stages(int N) {
        const int room = SMEM_MOST - 1024 - HEAD - NCH * (N / 2) * 128, n = room / STAGE;
        return n < MAXST ? n : MAXST;
    }
    static_assert(OFF_BAR % 8 == 0 && OFF_B % 16 == 0, "alignment");
};
static_assert((SMEM_MOST - 1024 - WCfg<false>::HEAD - NCH * 128 * 128) / WCfg<false>::STAGE >= 5, "ring");
static_assert((SMEM_MOST - 1024 - WCfg<true>::HEAD - NCH * 128 * 128) / WCfg<true>::STAGE >= 9, "ring");

struct WeightParams {
    const int32_t *req, *ctx;
    const int2 *table;
    const float *powers;          // FP8 [B][T*H]: the query rows' powers of two, inverted
    const uint64_t *tree;         // [B][T] or null
    const float *lse;             // [B][T*H]
    const float *scales;          // FP8: the pool's row scales
    const float *prior;           // [max_req][max_pages] or null
    float *weights;               // [max_req][max_pages]
    float *part;                  // [groups][B][max_pages] where there are several groups
    uint32_t *err;
    int B, T, H, M, groups, parts, N, nst;
    int max_req, max_pages, max_ctx, zero_block;
    float scale_log2, decay;
};

// a = a c + e, b = b d + f
__device__ __forceinline__ void fma2(float &a, float &b, float c, float d, float e, float f) {
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mov.b64 z, {%4, %5};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d), "f"(e), "f"(f));
}
// FP8: the query rows' codes, laid out as the rows were: per chunk of 64 values the first codes,
// then the second ones; and the inverses of their powers of two. One warp per row.
__global__ void __launch_bounds__(256)
weight_codes_kernel(const uint4 *q, uint2 *codes, float *powers, int64_t rows) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t m = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (m >= rows) return;
    constexpr int UNITS = kDim / 8;
    uint4 y[3];
    uint32_t top = 0;  // the largest magnitude; NaN if there is one
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int u = lane + 32 * k;
        y[k] = u < UNITS ? q[m * UNITS + u] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const uint32_t z[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(z[e] & 0x7fff7fffu));
    }
    // bits of magnitudes are in their order, infinities and NaN above all
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    const uint32_t pow2 = query_power(top);
    if (lane == 0) powers[m] = query_back(top);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int u = lane + 32 * k;
        if (u >= UNITS) break;
        uint2 z, r;
        bf16x4_to_e4m3(y[k].x, y[k].y, pow2, z.x, r.x);
        bf16x4_to_e4m3(y[k].z, y[k].w, pow2, z.y, r.y);
        uint2 *to = codes + m * (2 * UNITS) + (u >> 3) * 16 + (u & 7);
        to[0] = z;
        to[8] = r;
    }
}

template <bool FP8>
__global__ void __launch_bounds__(WT, 1)
weight_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, const WeightParams p) {
    using C = WCfg<FP8>;
    extern __shared__ uint8_t smem_raw[];
    const int rank = static_cast<int>(hs::cluster_ctarank());
    const int unit = blockIdx.x >> 1, g = unit % p.groups, part = unit / p.groups;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t raw = hs::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // queries, ring, then the small things
    const uint32_t qall = NCH * (uint32_t)(p.N / 2) * 128u;
    const uint32_t ring = base + qall, head = ring + (uint32_t)(p.nst * C::STAGE);
    uint8_t *small = smem_raw + (head - raw);
    volatile int32_t *misc = reinterpret_cast<volatile int32_t *>(small + C::OFF_MISC);
    auto bar = [&](int i) { return head + C::OFF_BAR + 8u * (uint32_t)i; };
    const uint32_t lead0 = cluster_address(head + C::OFF_BAR, 0);
    auto lead = [&](int i) { return lead0 + 8u * (uint32_t)i; };
    const uint32_t nst = (uint32_t)p.nst;
    auto fail = [&]() {
        misc[1] = 1;
        atomicOr(p.err, HS_DEVERR_TIMEOUT);
    };
    uint32_t cols = 32;
    while ((int)cols < 2 * p.N) cols <<= 1;
    if (warp == 0) {
        for (int i = lane; i < C::NBAR; i += 32) {
            uint32_t n = 1;
            if (i == C::B_DFREE || i == C::B_DFREE + 1) n = 2 * NEW;  // both CTAs'
            mbar_init(bar(i), n);
        }
        fence_mbar_init();
        fence_proxy_async();
        if (lane == 0) {
            misc[1] = 0;
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_q);
        }
        __syncwarp();
    }
    if (warp == 1) tmem_alloc2(head + C::OFF_MISC, cols);
    // FP8: the launch before is the one that makes the codes, begun when all before it had ended;
    // those who read codes or powers wait for it.
    if (!FP8) grid_dep_wait();
    grid_dep_launch();

    // The requests' tiles laid end to end: how many, and where this pair's range begins.
    // Every warp finds that, and walks the range, for itself.
    uint32_t bad = 0;
    auto request = [&](int b, int &r) {  // context length of request b of the list
        r = b < p.B ? p.req[b] : -1;
        if (r < 0 || r >= p.max_req) {
            if (b < p.B) bad |= HS_DEVERR_BAD_REQUEST;
            return 0;
        }
        const int len = p.ctx[r];
        if (len > p.max_ctx) bad |= HS_DEVERR_INDEX_RANGE;
        return hs::context_within(len, p.max_ctx);
    };
    auto tiles_of = [](int pages) { return (pages + TP - 1) / TP; };
    struct Walk {
        int b, r, L, lo, n;  // request, its cache index and context, first tile, tiles (0: no more)
        int left;            // tiles of the range behind these
    };
    Walk begin{};
    int total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        int r;
        const int n = tiles_of(pages_of(request(b0 + lane, r)));
        total += __reduce_add_sync(0xffffffffu, n);
    }
    const int even = total / p.parts, odd = total - even * p.parts;
    const int f0 = even * part + min(part, odd), f1 = f0 + even + (part < odd ? 1 : 0);
    auto take = [&](Walk &w) {
        w.n = min(w.left, tiles_of(pages_of(w.L)) - w.lo);
        w.left -= w.n;
    };
    if (f1 > f0) {
        int at = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            int r;
            const int L = request(b0 + lane, r), n = tiles_of(pages_of(L));
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, at + incl > f0);
            if (past) {
                const int l = __ffs(past) - 1;
                begin.b = b0 + l;
                begin.r = __shfl_sync(0xffffffffu, r, l);
                begin.L = __shfl_sync(0xffffffffu, L, l);
                begin.lo = f0 - at - __shfl_sync(0xffffffffu, incl - n, l);
                begin.left = f1 - f0;
                take(begin);
                break;
            }
            at += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    auto next = [&](Walk &w) {
        w.n = w.lo = 0;
        if (w.left <= 0) return;
        for (int b0 = w.b + 1; b0 < p.B; b0 += 32) {
            int r;
            const int L = request(b0 + lane, r);
            const uint32_t some = __ballot_sync(0xffffffffu, L > 0);
            if (some) {
                const int l = __ffs(some) - 1;
                w.b = b0 + l;
                w.r = __shfl_sync(0xffffffffu, r, l);
                w.L = __shfl_sync(0xffffffffu, L, l);
                take(w);
                return;
            }
        }
    };
    const uint32_t tiles = (uint32_t)(f1 - f0);  // that this pair multiplies
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, bad);
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);
    const uint32_t qch = (uint32_t)(p.N / 2) * 128u;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        Walk w = begin;
        uint32_t u = 0, s = 0, turn = 1;  // chunks asked for; ring stage and the phase before its own
        bool ok = true;
        while (w.n > 0 && ok) {
            const int2 *table = p.table + (size_t)w.r * p.max_pages;
            const int pages = pages_of(w.L);
            int blk = 0;
            for (int i = 0; i < w.n; ++i) {
                // blocks of this CTA's pages, 16 tiles ahead
                if (i % 16 == 0) {
                    const int page = TP * (w.lo + i + (lane >> 1)) + 2 * rank + (lane & 1);
                    const int x = page < pages ? table[page].x : -1;
                    blk = x >= 0 ? x : p.zero_block;
                }
                const int row0 = __shfl_sync(0xffffffffu, blk, 2 * (i % 16)) * kPage;
                const int row1 = __shfl_sync(0xffffffffu, blk, 2 * (i % 16) + 1) * kPage;
                if (lane == 0) {
                    for (int c = 0; c < NCH && ok; ++c, ++u) {
                        ok = mbar_wait_inline(bar(C::B_FREE + (int)s), turn);
                        if (!ok) break;
                        // both CTAs' bytes complete on CTA 0's barrier
                        if (rank == 0) mbar_expect_tx(bar(C::B_FULL + (int)s), 2 * C::STAGE);
                        tma_load_pair(ring + s * C::STAGE, &tm_k, 0, row0, c, lead(C::B_FULL + (int)s));
                        tma_load_pair(ring + s * C::STAGE + C::STAGE / 2, &tm_k, 0, row1, c, lead(C::B_FULL + (int)s));
                        if (++s == nst) {
                            s = 0;
                            turn ^= 1u;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
            }
            next(w);
        }
        if (lane == 0 && !ok) {
            fail();
            for (uint32_t k = 0, v = u; rank == 0 && k < nst && v > 0; ++k) {
                --v;
                mbar_wait_inline(bar(C::B_FULL + (int)(v % nst)), (v / nst) & 1u);
            }
        }
    } else if (warp == 2 + NEW) {
        // ------------------------------------------------------------ queries' producer
        uint32_t n = 0;  // chunks asked for
        bool ok = true;
        uint32_t x = 0;
        if (FP8) grid_dep_wait();
        for (Walk w = begin; w.n > 0 && ok; next(w), ++x) {
            if (lane == 0) {
                for (int c = 0; c < NCH && ok; ++c) {
                    // the MMAs of the request before are done with the chunk's place
                    if (x > 0) ok = mbar_wait_inline(bar(C::B_QFREE + c), (x - 1) & 1u);
                    if (!ok) break;
                    if (rank == 0) mbar_expect_tx(bar(C::B_QFULL + c), 2 * qch);  // both CTAs' bytes
                    tma_load_pair(base + c * qch, &tm_q, 64 * c, g * p.N + rank * (p.N / 2), w.b, lead(C::B_QFULL + c));
                    ++n;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
        }
        if (lane == 0) {
            if (!ok) fail();
            // the copies begun have landed before the CTA may end
            for (uint32_t k = n > NCH ? n - NCH : 0; k < n && rank == 0; ++k)
                mbar_wait_inline(bar(C::B_QFULL + (int)(k % NCH)), (k / NCH) & 1u);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (CTA 0)
        if (rank == 0 && tiles > 0) {
            const uint32_t idesc = idesc_f16(FP8 ? 0u : 1u, 0, 256, p.N);
            const uint64_t d0 = desc_sw128(base, 16, 1024);
            const uint32_t hi = (uint32_t)(d0 >> 32), lo = (uint32_t)d0;
            const uint32_t khi = FP8 ? (uint32_t)(desc_sw64(base, 16, 512) >> 32) : hi;
            const uint32_t leader = elect_one();
            bool ok = true;
            uint32_t i = 0, seg = 0, s = 0, turn = 0;  // ring stage and its phase
            uint32_t keep = tiles * NCH > nst ? tiles * NCH - nst : 0;  // chunks whose stages are filled again
            for (Walk w = begin; w.n > 0 && ok; ++seg) {
                Walk nx = w;
                next(nx);
                if (leader) {
                    for (int j = 0; j < w.n && ok; ++j) {
                        const uint32_t k = i + (uint32_t)j, d = tmem + (k & 1u) * (uint32_t)p.N;
                        if (k >= 2) ok = mbar_wait_inline(bar(C::B_DFREE + (int)(k & 1u)), ((k >> 1) & 1u) ^ 1u);
#pragma unroll 1
                        for (int c = 0; c < NCH && ok; ++c) {
                            if (j == 0) ok = mbar_wait_inline(bar(C::B_QFULL + c), seg & 1u);
                            if (ok) ok = mbar_wait_inline(bar(C::B_FULL + (int)s), turn);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t a = lo + ((ring - base + s * C::STAGE) >> 4), q = lo + ((c * qch) >> 4);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (FP8)  // both codes of the queries with the same 32 codes of the keys
                                    mma2_ss_e4m3(d, a + 2 * (e & 1), khi, q + 2 * e, hi, idesc, (c | e) != 0);
                                else
                                    mma2_ss(d, a + 2 * e, q + 2 * e, hi, idesc, (c | e) != 0);
                            }
                            if (keep > 0) {
                                commit_both(bar(C::B_FREE + (int)s));
                                --keep;
                            }
                            // the next request's queries take the place of these
                            if (j == w.n - 1 && nx.n > 0) commit_both(bar(C::B_QFREE + c));
                            if (++s == nst) {
                                s = 0;
                                turn ^= 1u;
                            }
                        }
                        if (ok) commit_both(bar(C::B_DFULL + (int)(k & 1u)));
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                i += (uint32_t)w.n;
                w = nx;
            }
            if (!ok && lane == 0) fail();
            if (leader) {
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 bar(C::B_DRAIN))
                             : "memory");
                mbar_wait_inline(bar(C::B_DRAIN), 0);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ the sums
        const int wq = warp & 3, hf = (warp - 2) >> 2, tid = (warp - 2) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const int mid = (p.N / 2 + 31) & ~31, c_lo = hf * mid, c_hi = min(hf ? p.N : mid, p.M - g * p.N);
        volatile float *psum = reinterpret_cast<volatile float *>(small + C::OFF_PS);
        volatile uint32_t *dead = reinterpret_cast<volatile uint32_t *>(small + C::OFF_DEAD);
        const bool writer = hf == 0 && (wq & 1) == 0 && lane == 0;  // of one page of the tile
        bool ok = true;
        uint32_t i = 0;
        const int m_own = g * p.N + tid;  // this thread's column
        float lse = 0.f, pw = 0.f;
        auto fetch = [&](const Walk &v) {  // its terms
            if (tid >= p.N || m_own >= p.M || v.n <= 0) return;
            lse = p.lse[(size_t)v.b * p.M + m_own];
            if (FP8) pw = p.powers[(size_t)v.b * p.M + m_own];
        };
        if (FP8) grid_dep_wait();
        fetch(begin);
        for (Walk w = begin, nx; w.n > 0; w = nx) {
            nx = w;
            next(nx);
            // The columns' terms. All warps are done with the last segment's.
            const bool fin = fabsf(lse) < INFINITY;
            const uint32_t out = __ballot_sync(0xffffffffu, !fin);
            if (tid < p.N)
                st_shared_f1(head + C::OFF_B + 4 * tid, fin && m_own < p.M ? -lse * 1.4426950408889634f : -INFINITY);
            if (FP8 && tid < p.N) st_shared_f1(head + C::OFF_A + 4 * tid, p.scale_log2 * pw);
            if (lane == 0) dead[warp - 2] = out;
            fetch(nx);
            named_bar_sync(1, 32 * NEW);
            const uint32_t terms = head + C::OFF_B, tab = head + C::OFF_A;

            const int pages = pages_of(w.L), draft = w.L - p.T;
            const int2 *table = p.table + (size_t)w.r * p.max_pages;
            auto block_at = [&](int tile) {
                const int page = TP * tile + 2 * rank + (wq >> 1);
                return page < pages ? table[page].x : -1;
            };
            int blk = block_at(w.lo);
            for (int j = 0; j < w.n; ++j, ++i) {
                const int page = TP * (w.lo + j) + 2 * rank + (wq >> 1);
                const int pos = page * kPage + 32 * (wq & 1) + lane;
                const bool live = blk >= 0;  // the same in a warp
                float ks = p.scale_log2;
                if (FP8 && live) ks = p.scales[(size_t)blk * kPage + 32 * (wq & 1) + lane];
                const int blk_next = j + 1 < w.n ? block_at(w.lo + j + 1) : -1;
                float before = 0.f;
                if (writer && page < pages && p.groups == 1 && p.prior && p.decay != 0.f)
                    before = p.decay * p.prior[(size_t)w.r * p.max_pages + page];
                const bool all = (pos | 31) < draft;  // every query token sees these keys
                const int node = pos - draft;
                // Which of the query rows m .. m + 31 see this key. A word of them ahead of the sums: asked at
                // each row, the tiles at a context's end took 5 us more (13 x 304 keys, 512 rows: 14.3 -> 9.9 us).
                auto sees = [&](int m) {
                    if (!p.tree) {  // the tokens from the key's own on
                        const int first = max(node, 0) * p.H - m;
                        return first <= 0 ? ~0u : first < 32 ? ~0u << first : 0u;
                    }
                    if (node < 0) return ~0u;
                    uint32_t x = 0;
                    if (node < p.T)
                        for (int t = m / p.H; t < p.T && t * p.H < m + 32; ++t) {
                            const int lo = max(t * p.H - m, 0), n = min((t + 1) * p.H - m, 32) - lo;
                            if ((p.tree[(size_t)w.b * p.T + t] >> node) & 1) x |= (n < 32 ? (1u << n) - 1u : ~0u) << lo;
                        }
                    return x;
                };
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_DFULL + (int)(i & 1)), (i >> 1) & 1u));
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
                if (ok && live) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
                        uint32_t d[32];
                        HS_TMEM_LD32(tmem + lane_off + (i & 1) * (uint32_t)p.N + c0, d);
                        HS_TMEM_WAIT_LD32(d);
                        const uint32_t gone = dead[c0 >> 5];
                        // the columns that count: with a key that is not finite the others hold NaN
                        uint32_t live = ~gone & (c_hi - c0 < 32 ? (1u << (c_hi - c0)) - 1u : ~0u);
                        if (!all) live &= sees(g * p.N + c0);
                        auto sums = [&](auto whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 b = ld_shared_f4(terms + 4 * (c0 + e));
                                float a0 = ks, a1 = ks, a2 = ks, a3 = ks;
                                if (FP8) {  // the two scales first: their product with a sum may be the only one in range
                                    const float4 a = ld_shared_f4(tab + 4 * (c0 + e));
                                    mul2(a0, a1, a.x, a.y);
                                    mul2(a2, a3, a.z, a.w);
                                }
                                float x0 = __uint_as_float(d[e]), x1 = __uint_as_float(d[e + 1]);
                                float x2 = __uint_as_float(d[e + 2]), x3 = __uint_as_float(d[e + 3]);
                                fma2(x0, x1, a0, a1, b.x, b.y);
                                fma2(x2, x3, a2, a3, b.z, b.w);
                                float y0 = ex2(x0), y1 = ex2(x1), y2 = ex2(x2), y3 = ex2(x3);
                                if (!decltype(whole)::value) {
                                    y0 = (live >> e) & 1u ? y0 : 0.f;
                                    y1 = (live >> (e + 1)) & 1u ? y1 : 0.f;
                                    y2 = (live >> (e + 2)) & 1u ? y2 : 0.f;
                                    y3 = (live >> (e + 3)) & 1u ? y3 : 0.f;
                                }
                                add2(s0, s1, y0, y1);
                                add2(s2, s3, y2, y3);
                            }
                        };
                        if (__all_sync(0xffffffffu, live == ~0u))
                            sums(std::true_type{});
                        else
                            sums(std::false_type{});
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && i + 2 < tiles) mbar_arrive_peer(lead(C::B_DFREE + (int)(i & 1)));
                float sum = (s0 + s1) + (s2 + s3);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const int at = (int)(i & 1) * NEW;
                if (lane == 0) psum[at + 4 * hf + wq] = sum;
                named_bar_sync(1, 32 * NEW);
                if (writer && page < pages && ok) {
                    const float got = (psum[at + wq] + psum[at + wq + 1]) + (psum[at + 4 + wq] + psum[at + 5 + wq]);
                    if (p.groups == 1)
                        p.weights[(size_t)w.r * p.max_pages + page] = before + got;
                    else
                        p.part[((size_t)g * p.B + w.b) * p.max_pages + page] = got;
                }
                blk = blk_next;
            }
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

// The groups' sums of each page, in order. One thread per page.
__global__ void __launch_bounds__(256)
weight_join_kernel(const float *part, const int32_t *req, const int32_t *ctx, const float *prior, float *weights, int B,
                   int groups, int max_req, int max_pages, int max_ctx, float decay) {
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.y, r = req[b];
    if (r < 0 || r >= max_req) return;
    const int pages = pages_of(hs::context_within(ctx[r], max_ctx));
    for (int page = blockIdx.x * 256 + threadIdx.x; page < pages; page += gridDim.x * 256) {
        const size_t at = (size_t)r * max_pages + page;
        float sum = 0.f;
        for (int g = 0; g < groups; ++g) sum += part[((size_t)g * B + b) * max_pages + page];
        weights[at] = (prior && decay != 0.f ? decay * prior[at] : 0.f) + sum;
    }
}

bool takes(int64_t B, int64_t T, int64_t H) {
    return B >= 0 && B <= 65535 && T >= 1 && T <= 32767 && H >= 1 && T * H <= (1 << 22);
}
// The query rows are dealt evenly to as few groups as hold them: rows of a group, a multiple of 32.
int rows_of(int64_t M) {
    const int64_t groups = (M + MAXN - 1) / MAXN;
    return (int)((M + groups - 1) / groups + 31) & ~31;
}
int groups_of(int64_t M) { return (int)((M + rows_of(M) - 1) / rows_of(M)); }

// Parts that the key tiles of all requests are cut into, each worked through by one pair of
// CTAs per group: the count that a model of the launch makes shortest. A tile takes a
// pair us_tile, its start and the queries 5 us.
int parts_of(int64_t groups, int64_t tiles, double us_tile) {
    const int64_t pairs = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
    double best = 1e300;
    int64_t parts = 1;
    for (int64_t w = 1; w <= 8; ++w) {
        int64_t n = w * pairs / groups;
        n = n < 1 ? 1 : (n > tiles ? tiles : n);
        const double waves = (double)((groups * n + pairs - 1) / pairs);
        const double t = waves * ((double)((tiles + n - 1) / n) * us_tile + 5.0);
        if (t < best * 0.98) {
            best = t;
            parts = n;
        }
    }
    return (int)parts;
}

template <bool FP8>
hs_status launch_weights(int dev, cudaStream_t s, const CUtensorMap &tk, const CUtensorMap &tq, const WeightParams &p) {
    static std::atomic<int> state[64];
    if (dev < 0 || dev >= 64) return HS_ERR_UNSUPPORTED;
    if (state[dev].load(std::memory_order_acquire) != 1) {
        HS_CUDA_TRY(cudaFuncSetAttribute(weight_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MOST));
        state[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * p.groups * p.parts), 1, 1);
    cfg.blockDim = dim3(WT, 1, 1);
    cfg.dynamicSmemBytes =
        (size_t)(1024 + NCH * (p.N / 2) * 128 + p.nst * WCfg<FP8>::STAGE + WCfg<FP8>::HEAD);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, weight_kernel<FP8>, tk, tq, p) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
// FP8: the queries' codes and powers, before the groups' sums in the workspace
size_t code_bytes(int64_t B, int64_t T, int64_t H) {
    const size_t rows = (size_t)B * T * H;
    return up256(rows * 2 * kDim) + up256(rows * 4);
}

}  // namespace

extern "C" size_t hs_weights_workspace_bytes(hs_pool_t pool, int32_t B, int32_t T, int32_t H) {
    if (!pool || B < 1 || !takes(B, T, H)) return 0;
    const int groups = groups_of((int64_t)T * H);
    const size_t parts = groups == 1 ? 0 : (size_t)groups * B * pool->max_pages * 4;
    return up256(parts) + (pool->cfg.dtype == HS_FP8_E4M3_ROWSCALE ? code_bytes(B, T, H) : 0);
}

extern "C" hs_status hs_page_weights(hs_pool_t pool, int32_t B, int32_t T, int32_t H, const void *d_q,
                                     const float *d_lse, const int32_t *d_req_ids, const uint64_t *d_tree,
                                     float sm_scale, float decay, const float *d_prior, float *d_weights,
                                     void *d_workspace, size_t ws_bytes, void *stream) {
    if (!pool || !takes(B, T, H) || (d_tree && T > 64)) return HS_ERR_INVALID_ARG;
    if (B == 0) return HS_OK;
    if (!d_q || !d_lse || !d_req_ids || !d_weights || ((uintptr_t)d_q & 15u)) return HS_ERR_INVALID_ARG;
    const size_t need = hs_weights_workspace_bytes(pool, B, T, H);
    if (need && (!d_workspace || ws_bytes < need || ((uintptr_t)d_workspace & 255u))) return HS_ERR_INVALID_ARG;
    int dev = -1;
    HS_CUDA_TRY(cudaGetDevice(&dev));
    if (dev != pool->device) return HS_ERR_INVALID_ARG;
    const bool fp8 = pool->cfg.dtype == HS_FP8_E4M3_ROWSCALE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    WeightParams p{};
    p.req = d_req_ids;
    p.ctx = pool->d_ctx;
    p.table = reinterpret_cast<const int2 *>(pool->d_page);
    p.tree = d_tree;
    p.lse = d_lse;
    p.scales = pool->d_scales;
    p.prior = d_prior;
    p.weights = d_weights;
    const int64_t rows = (int64_t)B * T * H;
    uint8_t *ws = static_cast<uint8_t *>(d_workspace);
    float *powers = fp8 ? reinterpret_cast<float *>(ws + up256((size_t)rows * 2 * kDim)) : nullptr;
    p.powers = powers;
    p.part = reinterpret_cast<float *>(ws + (fp8 ? code_bytes(B, T, H) : 0));  // read with several groups only
    p.err = pool->d_err;
    p.B = B;
    p.T = T;
    p.H = H;
    p.M = T * H;
    p.groups = groups_of(p.M);
    p.N = rows_of(p.M);
    p.nst = fp8 ? WCfg<true>::stages(p.N) : WCfg<false>::stages(p.N);
    const int64_t tiles = (int64_t)B * ((pool->max_pages + TP - 1) / TP);
    // the keys' bytes at the card's rate, or the products
    const double us_mma = 2.5 * p.N / 256, us_bytes = (fp8 ? 148e3 : 295e3) / 85e3;
    p.parts = parts_of(p.groups, tiles, us_mma > us_bytes ? us_mma : us_bytes);
    if (2ll * p.groups * p.parts > INT32_MAX || rows > 8ll * INT32_MAX || tiles > INT32_MAX / 32) return HS_ERR_INVALID_ARG;
    p.max_req = pool->cfg.max_requests;
    p.max_pages = pool->max_pages;
    p.max_ctx = pool->cfg.max_ctx;
    p.zero_block = (int)pool->cfg.n_gpu_blocks;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.decay = decay;
    CUtensorMap tk, tq;
    if (!make_page_map(&tk, fp8, pool->d_rows, (uint64_t)(pool->cfg.n_gpu_blocks + 1) * kPage, 1,
                       fp8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT16, fp8 ? ws : d_q, kDim, (uint64_t)p.M, B, 2 * kDim, 64, p.N / 2,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return HS_ERR_CUDA;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    if (fp8) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((rows + 7) / 8), 1, 1);
        cfg.blockDim = dim3(256, 1, 1);
        cfg.stream = s;
        cfg.attrs = pdl;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, weight_codes_kernel, static_cast<const uint4 *>(d_q), reinterpret_cast<uint2 *>(ws), powers,
                               rows) != cudaSuccess)
            return HS_ERR_CUDA;
    }
    const hs_status st = fp8 ? launch_weights<true>(dev, s, tk, tq, p) : launch_weights<false>(dev, s, tk, tq, p);
    if (st != HS_OK || p.groups == 1) return st;
    cudaLaunchConfig_t cfg = {};
    const int64_t blocks = ((int64_t)pool->max_pages + 255) / 256;
    cfg.gridDim = dim3((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)B, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weight_join_kernel, (const float *)p.part, d_req_ids, (const int32_t *)pool->d_ctx,
                              d_prior, d_weights, (int)B, p.groups, p.max_req, p.max_pages, p.max_ctx, decay) == cudaSuccess
               ? HS_OK
               : HS_ERR_CUDA;
}
