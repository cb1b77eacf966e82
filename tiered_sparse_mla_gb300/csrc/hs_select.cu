// hs_select.cu -- the pages that each query token attends to: scores of all of a
// request's pages on tcgen05 tensor cores, then an exact top-N.
//
// The score of page p for query token t is s = max_h q[t][h] . c_p, c_p the mean
// row of the page (hs_page_means). The selection is that of the exact sums: the
// tensor cores' sums are within
//     E = 2^-16 * max_h |q_h| * max_p |c_p|
// of them (36 MMAs of depth 16 per score; products of BF16 values are exact in
// f32, and each MMA adds at most 2^-22 of the sums' largest possible magnitude
// |q||c|, so 36 * 2^-22 < 2^-16 of it in all), so a page whose score is more
// than 2 E from the border is in or out, and the few nearer ones are summed
// again in 64 bits (of which 576 exact products lose nothing that BF16 inputs
// can tell apart but ties). Equal scores go to the lower page.
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
// One CTA per (128 pages, request). The pages are the MMA's M rows, the query
// rows (token x head) its N columns, so that the maximum over heads runs along
// the registers of the one thread that owns a page. Chunks of 64 depth columns
// stream through a ring (pages 16 KB, query rows up to 32 KB a stage); two CTAs
// share an SM, so one's loads cover the other's epilogue.
constexpr int SP = 128;          // pages per tile
constexpr int NCH = kDim / 64;   // depth chunks
constexpr int ST = 192;          // threads: producer, MMA, four epilogue warps
constexpr int MAXN = 256;        // query rows per group
constexpr int MAXST = 5;         // ring stages
constexpr int A_BYTES = SP * 128;
constexpr int RING_BYTES = 98304;
constexpr int SCORE_SMEM = RING_BYTES + 1024 + 256;

struct ScoreParams {
    const int32_t *req, *ctx;
    float *s1;       // [B*T][Pp] best head's score
    uint32_t *s2;    // [B*T][Pp] second best (BF16, rounded up) << 16 | best head
    float *cn;       // [B][Pp]   |c_p|^2
    uint32_t *err;
    int T, H, M, N, groups, nst, Pp, max_req;
};

__global__ void __launch_bounds__(ST, 2)
score_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_q,
             const ScoreParams p) {
    extern __shared__ uint8_t smem_raw[];
    grid_dep_launch();
    const int b = blockIdx.y, tile = blockIdx.x;
    const int r = p.req[b];
    if (r < 0 || r >= p.max_req) return;
    const int pages = pages_of(p.ctx[r]);
    if (tile * SP >= pages) return;
    const uint32_t raw = hs::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    volatile int32_t *misc = reinterpret_cast<volatile int32_t *>(smem + RING_BYTES);
    auto bar = [&](int i) { return base + RING_BYTES + 16u + 8u * (uint32_t)i; };
    constexpr int B_FULL = 0, B_EMPTY = MAXST, B_NREAD = 2 * MAXST, B_DFULL = 3 * MAXST,
                  B_DEMPTY = B_DFULL + 1, B_DRAIN = B_DEMPTY + 1, NB = B_DRAIN + 1;
    static_assert(16 + 8 * NB <= 256, "barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage = A_BYTES + p.N * 128;
    const int uses = p.groups * NCH;
    auto fail = [&]() {
        misc[1] = 1;
        atomicOr(p.err, HS_DEVERR_TIMEOUT);
    };
    uint32_t cols = 32;
    while ((int)cols < p.N) cols <<= 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.nst; ++i) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_EMPTY + i), 1);
            mbar_init(bar(B_NREAD + i), 4);
        }
        mbar_init(bar(B_DFULL), 1);
        mbar_init(bar(B_DEMPTY), 4);
        mbar_init(bar(B_DRAIN), 1);
        misc[1] = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_c);
        prefetch_tmap(&tm_q);
    }
    if (warp == 1) tmem_alloc(base + RING_BYTES, cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int issued = 0;
            bool ok = true;
            for (int u = 0; u < uses && ok; ++u) {
                const int s = u % p.nst;
                const uint32_t ph = (uint32_t)(u / p.nst) & 1u;
                ok = mbar_wait(bar(B_EMPTY + s), ph ^ 1u) && !misc[1];
                // a stage of the first group is also read by the norms
                if (ok && u >= p.nst && u - p.nst < NCH) ok = mbar_wait(bar(B_NREAD + s), ph ^ 1u);
                if (!ok) break;
                const int g = u / NCH, c = u % NCH;
                mbar_expect_tx(bar(B_FULL + s), stage);
                tma_load_3d(base + s * stage, &tm_c, 64 * c, tile * SP, r, bar(B_FULL + s));
                tma_load_3d(base + s * stage + A_BYTES, &tm_q, 64 * c, g * p.N, b, bar(B_FULL + s));
                ++issued;
            }
            if (!ok) {
                fail();
                for (int u = issued - 1; u >= 0 && u >= issued - p.nst; --u)
                    mbar_wait(bar(B_FULL + u % p.nst), (uint32_t)(u / p.nst) & 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = idesc_f16(1u, 0, SP, p.N);
            bool ok = true;
            for (int u = 0; u < uses && ok; ++u) {
                const int s = u % p.nst, g = u / NCH, c = u % NCH;
                if (c == 0 && g > 0) ok = mbar_wait(bar(B_DEMPTY), (uint32_t)(g - 1) & 1u);
                ok = ok && mbar_wait(bar(B_FULL + s), (uint32_t)(u / p.nst) & 1u) && !misc[1];
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = desc_sw128(base + s * stage, 16, 1024);
                const uint64_t q = desc_sw128(base + s * stage + A_BYTES, 16, 1024);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_f16(tmem, a + 2 * k, q + 2 * k, idesc, (c | k) != 0);
                mma_commit(bar(B_EMPTY + s));
                if (c == NCH - 1) mma_commit(bar(B_DFULL));
            }
            if (!ok) fail();
            mma_commit(bar(B_DRAIN));
            mbar_wait(bar(B_DRAIN), 0);
        }
    } else {
        // ------------------------------------------------------------ norms, epilogue
        const int wq = warp & 3, row = wq * 32 + lane;
        const int page = tile * SP + row;
        bool ok = true;
        // |c_p|^2 of this thread's page, from the chunks as they pass
        float cn = 0.f;
        for (int u = 0; u < NCH; ++u) {
            const int s = u % p.nst;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_FULL + s), (uint32_t)(u / p.nst) & 1u) &&
                                                     !misc[1]);
            if (ok) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 v = ld_shared_v4(base + s * stage + row * 128 + ((c ^ (row & 7)) << 4));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xffff0000u);
                        cn = fmaf(lo, lo, cn);
                        cn = fmaf(hi, hi, cn);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_NREAD + s));
        }
        if (ok && page < pages) p.cn[(size_t)b * p.Pp + page] = cn;
        int t = 0, h = 0, arg = 0;
        float m1 = -INFINITY, m2 = -INFINITY;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        for (int g = 0; g < p.groups; ++g) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_DFULL), (uint32_t)g & 1u) && !misc[1]);
            if (ok) {
                tc_fence_after();
                const int left = min(p.N, p.M - g * p.N);
                for (int c0 = 0; c0 < left; c0 += 16) {
                    uint32_t d[16];
                    HS_TMEM_LD16(tmem + lane_off + c0, d);
                    HS_TMEM_WAIT_LD16(d);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (c0 + e >= left) break;
                        const float v = __uint_as_float(d[e]);
                        m2 = fmaxf(m2, fminf(m1, v));
                        arg = v > m1 ? h : arg;
                        m1 = fmaxf(m1, v);
                        if (++h == p.H) {
                            if (page < pages) {
                                const size_t at = ((size_t)b * p.T + t) * p.Pp + page;
                                p.s1[at] = m1;
                                // rounded up: its distance to the best is never overstated
                                p.s2[at] = ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_ru(m2)) << 16) | (uint32_t)arg;
                            }
                            m1 = m2 = -INFINITY;
                            h = arg = 0;
                            ++t;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DEMPTY));
        }
        if (!ok) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, cols);
}

// ---------------------------------------------------------------- selection
// One CTA per (request, query token). A histogram of the scores' bits, as
// integers in the scores' order, finds the border's bin (one pass where the
// scores are of one magnitude, three at most); the bin's members give the k-th
// largest score; a last pass collects the pages above the border's interval and
// those inside it, and the latter are summed again in 64 bits.
constexpr int LT = 1024;       // threads
constexpr int NW = LT / 32;
constexpr int BINS = 2048;
constexpr int CAP = 512;       // pages near the border that fit in shared memory
constexpr int MAXSEL = 1024;   // pages per list

struct SelectParams {
    const int32_t *req, *ctx;
    const uint64_t *tree;            // [B][T] or null
    const __nv_bfloat16 *q, *means;  // [B][T][H][576], [max_req][max_pages][576]
    float *s1;
    uint32_t *s2;
    const float *cn;
    uint64_t *key64;                 // [B*T][Pp] only written when more than CAP pages are near the border
    int32_t *pages, *topk;           // [B][T][N], [B][T][N*64] or null
    uint32_t *err;
    int T, H, N, n_first, n_last, Pp, max_req, max_pages;
};

__device__ __forceinline__ uint32_t order32(float x) {
    const uint32_t u = __float_as_uint(x) == 0x80000000u ? 0u : __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_order32(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// NaN ranks with minus infinity
__device__ __forceinline__ uint64_t order64(double x) {
    if (x != x) x = -(double)INFINITY;
    const uint64_t u = x == 0.0 ? 0ull : (uint64_t)__double_as_longlong(x);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

// q . c in 64 bits, by a warp (every lane gets the sum)
__device__ __forceinline__ double dot64(const __nv_bfloat16 *q, const __nv_bfloat16 *c) {
    const int lane = threadIdx.x & 31;
    double acc = 0.0;
#pragma unroll
    for (int i = 0; i < kDim / 64; ++i) {
        const uint32_t a = reinterpret_cast<const uint32_t *>(q)[lane + 32 * i];
        const uint32_t b = reinterpret_cast<const uint32_t *>(c)[lane + 32 * i];
        acc = fma((double)__uint_as_float(a << 16), (double)__uint_as_float(b << 16), acc);
        acc = fma((double)__uint_as_float(a & 0xffff0000u), (double)__uint_as_float(b & 0xffff0000u), acc);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    return acc;
}

__global__ void __launch_bounds__(LT) select_kernel(const SelectParams p) {
    __shared__ int hist[BINS];
    __shared__ uint32_t lkey[CAP];
    __shared__ int lpage[CAP];
    __shared__ unsigned long long lk64[CAP];
    __shared__ int sel[MAXSEL], sorted[MAXSEL];
    __shared__ int warp_i[NW];
    __shared__ float warp_f[NW];
    __shared__ uint32_t s_lo, s_hi, s_theta;
    __shared__ int s_need, s_bin, s_m, s_nsel, s_unknown;
    __shared__ float s_qn, s_cn;
    const int list = blockIdx.x, b = list / p.T, t = list % p.T;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = p.req[b];
    const bool req_ok = r >= 0 && r < p.max_req;
    const int L = req_ok ? p.ctx[r] : 0;
    const __nv_bfloat16 *q = p.q + (size_t)list * p.H * kDim;
    const long long end = p.tree ? (long long)L : (long long)L - p.T + t + 1;
    const int n = end <= 0 ? 0 : pages_of((int)end);  // pages that hold a token this one may see
    const bool all = n <= p.N;
    const int k = p.N - p.n_first - p.n_last;
    const int c0 = p.n_first, c1 = n - p.n_last;  // candidates (when not all)
    if (!req_ok && tid == 0) atomicOr(p.err, HS_DEVERR_BAD_REQUEST);
    if (tid == 0) {
        s_nsel = 0;
        s_m = 0;
        s_unknown = 0;
        s_lo = 0xffffffffu;
        s_hi = 0u;
        s_cn = 0.f;
    }
    if (!all && k > 0) {
        // max |q_h|^2; the queries were there before the scores' kernel began
        float mx = 0.f;
        for (int h = warp; h < p.H; h += NW) {
            const uint32_t *qr = reinterpret_cast<const uint32_t *>(q + (size_t)h * kDim);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kDim / 64; ++i) {
                const uint32_t w = qr[lane + 32 * i];
                const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
                s = fmaf(lo, lo, s);
                s = fmaf(hi, hi, s);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            mx = s == s ? fmaxf(mx, s) : INFINITY;
            if (mx == INFINITY) break;
        }
        if (lane == 0) warp_f[warp] = mx;
        __syncthreads();
        if (tid == 0) {
            float m = 0.f;
            for (int w = 0; w < NW; ++w) m = fmaxf(m, warp_f[w]);
            s_qn = m;
        }
    }
    grid_dep_wait();  // the scores
    __syncthreads();

    if (all) {
        for (int i = tid; i < p.N; i += LT) sorted[i] = i < n ? i : -1;
    } else {
        for (int i = tid; i < p.n_first; i += LT) sel[k + i] = i;
        for (int i = tid; i < p.n_last; i += LT) sel[k + p.n_first + i] = n - p.n_last + i;
    }
    if (!all && k > 0) {
        float *s1 = p.s1 + (size_t)list * p.Pp;
        uint32_t *s2 = p.s2 + (size_t)list * p.Pp;
        const float *cn = p.cn + (size_t)b * p.Pp;
        const __nv_bfloat16 *means = p.means + (size_t)r * p.max_pages * kDim;
        // a page whose score or norm is not finite says nothing in 32 bits
        auto unknown = [&](float s, float c) { return !(fabsf(s) <= FLT_MAX) || !(c <= FLT_MAX); };
        uint32_t lo = 0xffffffffu, hi = 0u;
        float cm = 0.f;
        int unk = 0;
        for (int i = c0 + tid; i < c1; i += LT) {
            const float s = s1[i], c = cn[i];
            if (unknown(s, c)) {
                unk = 1;
            } else {
                const uint32_t key = order32(s);
                lo = min(lo, key);
                hi = max(hi, key);
                cm = fmaxf(cm, c);
            }
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        cm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(cm)));  // not negative
        unk = __any_sync(0xffffffffu, unk);
        if (lane == 0) {
            atomicMin(&s_lo, lo);
            atomicMax(&s_hi, hi);
            atomicMax(reinterpret_cast<int *>(&s_cn), __float_as_int(cm));
            if (unk) s_unknown = 1;
        }
        __syncthreads();
        if (s_unknown) {
            // those pages' scores in 64 bits; what stands for them in 32 is the
            // rounded sum, with a second best that names no head
            for (int i0 = c0 + warp * 32; i0 < c1; i0 += LT) {
                const int i = i0 + lane;
                unsigned todo = __ballot_sync(0xffffffffu, i < c1 && unknown(s1[i < c1 ? i : c0], cn[i < c1 ? i : c0]));
                while (todo) {
                    const int pg = i0 + __ffs(todo) - 1;
                    todo &= todo - 1;
                    double best = -(double)INFINITY;
                    for (int h = 0; h < p.H; ++h) {
                        const double d = dot64(q + (size_t)h * kDim, means + (size_t)pg * kDim);
                        best = d > best ? d : best;
                    }
                    const float s = __double2float_rn(best);
                    if (lane == 0) {
                        s1[pg] = s;
                        s2[pg] = 0x7f800000u;
                        const uint32_t key = order32(s);
                        atomicMin(&s_lo, key);
                        atomicMax(&s_hi, key);
                    }
                }
            }
            __syncthreads();
        }
        // ------------------------------------------------ the border's bin
        int need = k;
        lo = s_lo;
        hi = s_hi;
        int m = 0;
        for (;;) {
            const int bits = 32 - __clz((int)(hi - lo));
            const int sh = bits > 11 ? bits - 11 : 0;
            for (int i = tid; i < BINS; i += LT) hist[i] = 0;
            __syncthreads();
            for (int i = c0 + tid; i < c1; i += LT) {
                const uint32_t key = order32(s1[i]);
                if (key >= lo && key <= hi) atomicAdd(&hist[(key - lo) >> sh], 1);
            }
            __syncthreads();
            // from the top: thread i holds bins BINS-1-2i and the one below
            const int b0 = BINS - 1 - 2 * tid;
            const int h0 = hist[b0], h1 = hist[b0 - 1];
            int sum = h0 + h1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += x;
            }
            if (lane == 31) warp_i[warp] = sum;
            __syncthreads();
            int before = 0;
            for (int w = 0; w < warp; ++w) before += warp_i[w];
            const int a = before + sum - h0 - h1;  // members above bin b0
            if (a < need && a + h0 >= need) {
                s_bin = b0;
                s_need = need - a;
                s_m = h0;
            } else if (a + h0 < need && a + h0 + h1 >= need) {
                s_bin = b0 - 1;
                s_need = need - a - h0;
                s_m = h1;
            }
            __syncthreads();
            need = s_need;
            m = s_m;
            lo = lo + ((uint32_t)s_bin << sh);
            hi = min(hi, lo + ((sh ? (1u << sh) : 1u) - 1u));
            __syncthreads();
            if (sh == 0 || m <= CAP) break;
        }
        // the k-th largest score: the need-th of the bin
        if (lo == hi) {
            if (tid == 0) s_theta = lo;
        } else {
            if (tid == 0) s_m = 0;
            __syncthreads();
            for (int i = c0 + tid; i < c1; i += LT) {
                const uint32_t key = order32(s1[i]);
                if (key >= lo && key <= hi) lkey[atomicAdd(&s_m, 1)] = key;
            }
            __syncthreads();
            if (tid < m) {
                int above = 0, equal = 0;
                for (int j = 0; j < m; ++j) {
                    above += lkey[j] > lkey[tid];
                    equal += lkey[j] == lkey[tid];
                }
                if (above < need && above + equal >= need) s_theta = lkey[tid];
            }
        }
        if (tid == 0) s_m = 0;
        __syncthreads();
        // ------------------------------------------------ above it, and near it
        const float theta = from_order32(s_theta);
        const double e2 = 2.0 * (1.0 / 65536.0) * sqrt((double)s_qn) * sqrt((double)s_cn) * 1.0001;
        const double slack = e2 + fabs((double)theta) * (1.0 / 4194304.0);
        const double up = (double)theta + slack, dn = (double)theta - slack;
        for (int i = c0 + tid; i < c1; i += LT) {
            const double s = (double)s1[i];
            if (s > up) {
                sel[atomicAdd(&s_nsel, 1)] = i;
            } else if (!(s < dn)) {
                const int j = atomicAdd(&s_m, 1);
                if (j < CAP) lpage[j] = i;
            }
        }
        __syncthreads();
        need = k - s_nsel;
        m = s_m;
        // exact score of a near page: the best head alone where the second best is further off
        const bool same = e2 == 0.0 && !s_unknown;  // the sums are exact as they are
        auto ambiguous = [&](int pg) {
            const float second = __uint_as_float(s2[pg] & 0xffff0000u);
            return !((double)s1[pg] - (double)second > e2);
        };
        if (m <= CAP) {
            if (m == need) {
                if (tid < m) sel[s_nsel + tid] = lpage[tid];
            } else {
                if (tid < m) lk64[tid] = same ? order64((double)s1[lpage[tid]]) : 0ull;
                __syncthreads();
                if (!same) {
                    for (int j = 0; j < m; ++j) {
                        const int pg = lpage[j];
                        const bool amb = ambiguous(pg);
                        const int step = amb ? NW : p.H;
                        for (int h = amb ? warp : (warp == j % NW ? (int)(s2[pg] & 0xffffu) : p.H); h < p.H; h += step) {
                            const double d = dot64(q + (size_t)h * kDim, means + (size_t)pg * kDim);
                            if (lane == 0) atomicMax(&lk64[j], (unsigned long long)order64(d));
                        }
                    }
                    __syncthreads();
                }
                if (tid < m) {
                    int better = 0;
                    for (int j = 0; j < m; ++j)
                        better += lk64[j] > lk64[tid] || (lk64[j] == lk64[tid] && lpage[j] < lpage[tid]);
                    if (better < need) sel[s_nsel + better] = lpage[tid];
                }
            }
        } else {
            // very many equal or nearly equal scores: keys of all candidates in
            // memory, the need-th largest by bisection, ties by position
            uint64_t *k64 = p.key64 + (size_t)list * p.Pp;
            for (int i = c0 + warp; i < c1; i += NW) {
                const double s = (double)s1[i];
                uint64_t key = 0;
                if (!(s > up) && !(s < dn)) {
                    if (same) {
                        key = order64(s);
                    } else {
                        const bool amb = ambiguous(i);
                        const int h0 = amb ? 0 : (int)(s2[i] & 0xffffu), h1 = amb ? p.H : h0 + 1;
                        for (int h = h0; h < h1; ++h) {
                            const uint64_t d = order64(dot64(q + (size_t)h * kDim, means + (size_t)i * kDim));
                            key = d > key ? d : key;
                        }
                    }
                }
                if (lane == 0) k64[i] = key;
            }
            __syncthreads();
            auto count = [&](uint64_t at_least) {  // by the whole CTA
                int c = 0;
                for (int i = c0 + tid; i < c1; i += LT) c += k64[i] >= at_least;
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
            const int first = s_nsel;
            if (tid == 0) s_m = 0;
            __syncthreads();
            for (int i0 = c0; i0 < c1; i0 += LT) {
                const int i = i0 + tid;
                const uint64_t key = i < c1 ? k64[i] : 0;
                int total;
                const int rank = hs::block_scan_flag<LT>(i < c1 && key == tau, warp_i, total);
                if (i < c1 && (key > tau || (key == tau && rank < room)))
                    sel[first + atomicAdd(&s_m, 1)] = i;
                room -= total;
            }
        }
        __syncthreads();
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
    }
    __syncthreads();
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
    size_t s1, s2, cn, k64, total;
};
Ws workspace(const hs_pool *pool, int64_t B, int64_t T) {
    Ws w{};
    w.Pp = (pool->max_pages + 31) & ~31;
    const size_t lists = (size_t)B * T, row = (size_t)w.Pp;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    w.s1 = 0;
    w.s2 = up(lists * row * 4);
    w.cn = w.s2 + up(lists * row * 4);
    w.k64 = w.cn + up((size_t)B * row * 4);
    w.total = w.k64 + up(lists * row * 8);
    return w;
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
    if (!pool || B < 1 || T < 1) return 0;
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
        p.s1 = reinterpret_cast<float *>(ws + w.s1);
        p.s2 = reinterpret_cast<uint32_t *>(ws + w.s2);
        p.cn = reinterpret_cast<float *>(ws + w.cn);
        p.err = pool->d_err;
        p.T = T;
        p.H = H;
        p.M = T * H;
        p.groups = (p.M + MAXN - 1) / MAXN;
        p.N = ((p.M + p.groups - 1) / p.groups + 15) & ~15;
        p.nst = RING_BYTES / (A_BYTES + p.N * 128);
        if (p.nst > MAXST) p.nst = MAXST;
        p.Pp = w.Pp;
        p.max_req = pool->cfg.max_requests;
        CUtensorMap tc, tq;
        if (!make_map(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_means, kDim, pool->max_pages,
                      pool->cfg.max_requests, 2 * kDim, 64, SP, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_q, kDim, p.M, B, 2 * kDim, 64, p.N,
                      CU_TENSOR_MAP_SWIZZLE_128B))
            return HS_ERR_CUDA;
        const dim3 grid((pool->max_pages + SP - 1) / SP, B);
        score_kernel<<<grid, ST, SCORE_SMEM, s>>>(tc, tq, p);
        if (cudaGetLastError() != cudaSuccess) return HS_ERR_CUDA;
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)B * T), 1, 1);
    cfg.blockDim = dim3(LT, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    // its first part needs nothing of the scores' kernel
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pool->max_pages > N && N > n_first + n_last ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, select_kernel, p) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}
