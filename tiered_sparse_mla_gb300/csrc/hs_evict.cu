// hs_evict.cu -- which pages a request keeps on the GPU, by the attention weight that
// they have got (hs_page_weights), and the release of the others.
//
// Kept are the first n_first and the last n_last pages of the context, with SAVED_ONLY
// those without a host copy too, and then the others by descending weight, equal weights by
// ascending page, until there are `budget`. The weights become keys whose unsigned order is
// theirs. Bound: the latencies of the call; 16,384 pages are 12 bytes each.
//   512 pages at most: one CTA, a thread per page, which counts the keys before its own;
//   more: a cluster of CTAs, a slice of the pages each. A histogram of the range that the
//   keys are in, added over the cluster, gives the bin that the border is in; as soon as
//   a bin has no more than CANDS keys all CTAs take them and count (mostly after one
//   histogram). With g pages above the border and e on it before a page, min(e, room) + g
//   kept ones are before that page; the histograms say g and e of the slices before.
// The pool's pages say which, a request's own are known on the device alone: 64 pages take 3.0 us in a
// pool of up to 512 pages a request, 5.4 to 5.7 in one of 513 to 16,384. 500 pages 7.6 (13.7 with equal keys'
// places looked at one by one); 16 requests of 16,384 pages: 12.2 us (one CTA of 1,024 threads for everything
// 27; histograms of 2,048 bins, whose exchange takes 3 each, 23; the slices' counts in an
// exchange of their own and loads behind the length 14.2).
#include <atomic>
#include <cstdint>

#include "hs_internal.cuh"
#include "hs_tc.cuh"

namespace {

using hs::kPage;

constexpr int ET = 512;        // threads per CTA
constexpr int NW = ET / 32;
constexpr int BINS = 512;      // one per thread
constexpr int CANDS = 256;     // 512: 13.2 instead of 6.7 us where 537 pages leave as many; 64: 12.8 instead of 12.2 for 16,384
constexpr int CAP = 20480;     // keys of a slice that are kept in shared memory, with their blocks
constexpr int MAXG = 8;
constexpr uint32_t ABSENT = 0u, MUST = 0xffffffffu;

struct EvictParams {
    int2 *table;
    const int32_t *ctx, *req, *budget;
    const float *weights;
    int32_t *kept, *freed, *n_freed;
    uint32_t *err;
    int N, n_first, n_last, max_req, max_pages, max_ctx, cap;
    bool saved_only, plan;
};

// Keys in the weights' order: -inf and NaN lowest, above ABSENT; zeros of either sign equal.
__device__ __forceinline__ uint32_t key_of(float w) {
    uint32_t b = __float_as_uint(w);
    if ((b & 0x7fffffffu) > 0x7f800000u) b = 0xff800000u;  // NaN
    if (b == 0x80000000u) b = 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t key_at(const EvictParams &p, int page, int P, float w, int2 where) {
    if (where.x < 0) return ABSENT;
    const bool must = page < p.n_first || page >= P - p.n_last || (p.saved_only && where.y < 0);
    return must ? MUST : key_of(w);
}
// Request i's cache index, or -1 with its outputs written; its pages.
__device__ __forceinline__ int request_of(const EvictParams &p, int i, bool first, int &P, int &budget) {
    const int r = p.req[i];
    budget = p.budget[i];
    if (r < 0 || r >= p.max_req) {
        if (first) {
            for (int k = threadIdx.x; k < p.N; k += ET) p.kept[(size_t)i * p.N + k] = -1;
            if (threadIdx.x == 0) {
                p.n_freed[i] = 0;
                atomicOr(p.err, HS_DEVERR_BAD_REQUEST);
            }
        }
        return -1;
    }
    const int len = p.ctx[r], L = hs::context_within(len, p.max_ctx);
    P = L <= 0 ? 0 : (L - 1) / kPage + 1;
    if (first && threadIdx.x == 0) {
        uint32_t bad = len > p.max_ctx ? HS_DEVERR_INDEX_RANGE : 0u;
        if (budget < 0) bad |= HS_DEVERR_BAD_PAGE;
        if (bad) atomicOr(p.err, bad);
    }
    return r;
}

// At most ET pages: one CTA per request.
__global__ void __launch_bounds__(ET)
evict_few_kernel(const EvictParams p) {
    hs::tc::grid_dep_wait();
    hs::tc::grid_dep_launch();
    __shared__ __align__(16) uint32_t keys[ET];
    __shared__ int32_t warp_kept[NW], warp_all[NW], warp_must[NW];
    const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int P, budget;
    const int r = request_of(p, i, true, P, budget);
    if (r < 0) return;
    int2 *table = p.table + (size_t)r * p.max_pages;
    int2 where = make_int2(-1, -1);
    uint32_t key = ABSENT;
    if (tid < P) {
        where = table[tid];
        key = key_at(p, tid, P, p.weights[(size_t)r * p.max_pages + tid], where);
    }
    keys[tid] = key;
    const int must_n = __popc(__ballot_sync(0xffffffffu, key == MUST));
    const uint32_t here = __ballot_sync(0xffffffffu, key != ABSENT);
    if (lane == 0) {
        warp_must[warp] = must_n;
        warp_all[warp] = __popc(here);
    }
    __syncthreads();
    int must = 0, cand = 0, all_before = __popc(here & ((1u << lane) - 1u));
    for (int w = 0; w < NW; ++w) {
        must += warp_must[w];
        all_before += w < warp ? warp_all[w] : 0;
        cand += warp_all[w];
    }
    // how many of the pages that need not stay come before this one
    int rank = -must;
    if (key != ABSENT && key != MUST) {
        const uint4 *k4 = reinterpret_cast<const uint4 *>(keys);
        const int here0 = 32 * warp;
#pragma unroll 4
        for (int k = 0; k < here0; k += 4) {
            const uint4 v = k4[k >> 2];
            rank += (v.x >= key) + (v.y >= key) + (v.z >= key) + (v.w >= key);
        }
#pragma unroll 4
        for (int k = here0; k < P; k += 4) {
            const uint4 v = k4[k >> 2];
            rank += (v.x > key) + (v.y > key) + (v.z > key) + (v.w > key);
        }
    }
    rank += __popc(__match_any_sync(0xffffffffu, key) & ((1u << lane) - 1u));  // equal ones of this warp, before it
    // a negative budget frees nothing
    const bool stay = key == MUST || (key != ABSENT && (budget < 0 || rank < budget - must));
    const uint32_t kept = __ballot_sync(0xffffffffu, stay);
    if (lane == 0) warp_kept[warp] = __popc(kept);
    __syncthreads();
    int before = __popc(kept & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < NW; ++w) {
        before += w < warp ? warp_kept[w] : 0;
        total += warp_kept[w];
    }
    if (stay) {
        if (before < p.N) p.kept[(size_t)i * p.N + before] = tid;
    } else if (key != ABSENT) {
        p.freed[(size_t)i * p.max_pages + all_before - before] = where.x;
        if (!p.plan) table[tid].x = -1;
    }
    for (int k = total + tid; k < p.N; k += ET) p.kept[(size_t)i * p.N + k] = -1;
    if (tid == 0) {
        p.n_freed[i] = cand - total;
        if (total > p.N) atomicOr(p.err, HS_DEVERR_CAPACITY);
    }
}

// A cluster of G CTAs per request, a slice of the pages each: the same for any length, so that
// its first pages are on their way before the length is known.
constexpr int EARLY = 4;

__global__ void __launch_bounds__(ET)
evict_kernel(const EvictParams p, const int G) {
    // Once all CTAs of the cluster have come here, each may write to the others' shared memory: a
    // CTA that has not begun has none. The wait is directly before the first such write, behind the
    // loads that lead to it.
    hs::tc::cluster_arrive_relaxed();
    hs::tc::grid_dep_wait();
    hs::tc::grid_dep_launch();
    extern __shared__ uint32_t keys[];  // [cap] of the slice, and their blocks
    __shared__ uint32_t hist[2][BINS];  // one is read by the others while the next is filled
    __shared__ uint32_t own[CANDS];     // the slice's candidates
    __shared__ __align__(16) uint32_t cands[CANDS];
    __shared__ int32_t wsum[NW][3], s_bin, s_over, s_n, s_same;
    __shared__ uint32_t s_border, s_room, wkey[NW][2];
    __shared__ int32_t counts[MAXG][4], lists[MAXG];  // of all CTAs
    const int i = blockIdx.x / G, rank = (int)hs::cluster_ctarank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t *blocks = reinterpret_cast<int32_t *>(keys) + p.cap;
    const int per = ((p.max_pages + 32 * G - 1) / (32 * G)) * 32, p0 = min(rank * per, p.max_pages), slots = min(per, p.max_pages - p0);
    const int maybe = p.req[i], at_r = maybe >= 0 && maybe < p.max_req ? maybe : 0;
    int2 *table = p.table + (size_t)at_r * p.max_pages;
    const float *weights = p.weights + (size_t)at_r * p.max_pages;
    float w_early[EARLY];
    int2 t_early[EARLY];
#pragma unroll
    for (int u = 0; u < EARLY; ++u) {
        const int k = tid + u * ET;
        if (k < slots) {
            w_early[u] = weights[p0 + k];
            t_early[u] = table[p0 + k];
        }
    }
    int P, budget;
    const int r = request_of(p, i, rank == 0, P, budget);
    if (r < 0) {  // the whole cluster
        hs::cluster_wait();
        return;
    }
    int32_t *kept = p.kept + (size_t)i * p.N, *freed = p.freed + (size_t)i * p.max_pages;
    const int n = max(min(P - p0, slots), 0);
    auto key = [&](int k) {
        return k < p.cap ? keys[k] : key_at(p, p0 + k, P, weights[p0 + k], table[p0 + k]);
    };
    hist[0][tid] = hist[1][tid] = 0;
    if (tid == 0) s_n = 0;
    int cand = 0, must = 0;
    uint32_t lo = MUST, hi = ABSENT;  // of the keys that need not stay
    auto take = [&](int k, float w, int2 where) {
        const uint32_t x = key_at(p, p0 + k, P, w, where);
        if (k < p.cap) {
            keys[k] = x;
            blocks[k] = where.x;
        }
        cand += x != ABSENT;
        must += x == MUST;
        if (x != ABSENT && x != MUST) {
            lo = min(lo, x);
            hi = max(hi, x);
        }
    };
#pragma unroll
    for (int u = 0; u < EARLY; ++u)
        if (tid + u * ET < n) take(tid + u * ET, w_early[u], t_early[u]);
#pragma unroll 4
    for (int k = tid + EARLY * ET; k < n; k += ET) take(k, weights[p0 + k], table[p0 + k]);
    cand = __reduce_add_sync(0xffffffffu, cand);
    must = __reduce_add_sync(0xffffffffu, must);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        wsum[warp][0] = cand;
        wsum[warp][1] = must;
        wkey[warp][0] = lo;
        wkey[warp][1] = hi;
    }
    __syncthreads();
    hs::cluster_wait();
    if (warp == 0) {
        cand = __reduce_add_sync(0xffffffffu, lane < NW ? wsum[lane][0] : 0);
        must = __reduce_add_sync(0xffffffffu, lane < NW ? wsum[lane][1] : 0);
        lo = __reduce_min_sync(0xffffffffu, lane < NW ? wkey[lane][0] : MUST);
        hi = __reduce_max_sync(0xffffffffu, lane < NW ? wkey[lane][1] : ABSENT);
        if (lane < G) {
            hs::dsmem_st(hs::dsmem_map(&counts[rank][0], lane), cand);
            hs::dsmem_st(hs::dsmem_map(&counts[rank][1], lane), must);
            hs::dsmem_st(hs::dsmem_map(&counts[rank][2], lane), (int32_t)lo);
            hs::dsmem_st(hs::dsmem_map(&counts[rank][3], lane), (int32_t)hi);
        }
    }
    hs::cluster_arrive();
    hs::cluster_wait();
    // of all slices, and (..0) of those before this one
    cand = must = 0;
    int cand0 = 0, must0 = 0;
    lo = MUST;
    hi = ABSENT;
    for (int g = 0; g < G; ++g) {
        if (g == rank) {
            cand0 = cand;
            must0 = must;
        }
        cand += counts[g][0];
        must += counts[g][1];
        lo = min(lo, (uint32_t)counts[g][2]);
        hi = max(hi, (uint32_t)counts[g][3]);
    }
    // of the pages that need not stay, the `need` of the largest keys do; a negative budget
    // frees nothing
    const int others = cand - must, need = budget < 0 ? others : min(max(budget - must, 0), others);
    uint32_t border = ABSENT;  // keys above it stay, and of those equal to it the first `room`
    int room = 0;
    int g0 = cand0, e0 = 0;  // keys above the border, and on it, before this slice
    if (need == 0) {
        border = MUST - 1;
        g0 = must0;
    } else if (need < others) {
        int left = need, inside = others;  // of the keys in lo .. hi
        int above = 0;                     // this thread's share of those above it before this slice
        int same = cand0 - must0;          // before this slice, in lo .. hi
#pragma unroll 1
        for (int d = 0; lo < hi && inside > CANDS; ++d) {
            const int wide = 32 - __clz((int)(hi - lo)), shift = wide > 9 ? wide - 9 : 0;
            uint32_t *h = hist[d & 1];
            for (int k = tid; k < n; k += ET) {
                const uint32_t x = key(k);
                if (x >= lo && x <= hi) atomicAdd(&h[(x - lo) >> shift], 1u);
            }
            hs::cluster_arrive();
            hs::cluster_wait();
            // bins from the top, one a thread, over all slices
            const int bin = BINS - 1 - tid;
            int mine = 0, before = 0;
#pragma unroll
            for (int g = 0; g < MAXG; ++g)
                if (g < G) {
                    const int x = hs::dsmem_ld(hs::dsmem_map(&h[bin], (uint32_t)g));
                    mine += x;
                    before += g < rank ? x : 0;
                }
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) wsum[warp][0] = incl;
            hist[(d & 1) ^ 1][tid] = 0;  // read by the others before the last barrier
            __syncthreads();
            const int over = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane][0] : 0) + incl - mine;  // in higher bins
            if (over < left && over + mine >= left) {
                s_bin = bin;
                s_over = over;
                s_n = mine;
                s_same = before;
            }
            __syncthreads();
            above += bin > s_bin ? before : 0;
            lo += (uint32_t)s_bin << shift;
            hi = min(hi, lo + ((1u << shift) - 1u));
            left -= s_over;
            inside = s_n;
            same = s_same;
            __syncthreads();
        }
        border = lo;  // where one key is left
        room = left;
        int on = 0;
        if (lo < hi) {
            if (tid == 0) s_n = 0;
            __syncthreads();
            for (int k = tid; k < n; k += ET) {
                const uint32_t x = key(k);
                if (x >= lo && x <= hi) own[atomicAdd(&s_n, 1)] = x;
            }
            __syncthreads();
            if (tid < G) hs::dsmem_st(hs::dsmem_map(&lists[rank], (uint32_t)tid), s_n);
            hs::cluster_arrive();
            hs::cluster_wait();
            // all slices' candidates, slice by slice; within one in any order
            if (tid < CANDS) cands[tid] = ABSENT;
            __syncthreads();
            int at = 0;
            for (int g = 0; g < G; ++g) {
                const int m = lists[g];
                if (tid < m) cands[at + tid] = (uint32_t)hs::dsmem_ld(hs::dsmem_map(&own[tid], (uint32_t)g));
                at += m;
            }
            __syncthreads();
            uint32_t x = ABSENT;
            if (tid < inside) {
                x = cands[tid];
                const uint4 *c4 = reinterpret_cast<const uint4 *>(cands);
                int more = 0, equal = 0;
                for (int k = 0; k < inside; k += 4) {
                    const uint4 v = c4[k >> 2];
                    more += (v.x > x) + (v.y > x) + (v.z > x) + (v.w > x);
                    equal += (v.x == x) + (v.y == x) + (v.z == x) + (v.w == x);
                }
                if (more < left && more + equal >= left) {  // equal ones write the same
                    s_border = x;
                    s_room = (uint32_t)(left - more);
                }
            }
            __syncthreads();
            border = s_border;
            room = (int)s_room;
            if (tid < same) {  // those of the slices before this one come first
                above += x > border;
                on = x == border;
            }
        }
        above = __reduce_add_sync(0xffffffffu, above);
        on = __reduce_add_sync(0xffffffffu, on);
        if (lane == 0) {
            wsum[warp][0] = above;
            wsum[warp][1] = on;
        }
        __syncthreads();
        above = __reduce_add_sync(0xffffffffu, lane < NW ? wsum[lane][0] : 0);
        on = __reduce_add_sync(0xffffffffu, lane < NW ? wsum[lane][1] : 0);
        g0 = must0 + above;
        e0 = lo < hi ? on : same;
    }
    hs::cluster_arrive();  // the last that this CTA reads of another

    // each warp a run of rows of 32 pages: how many are above the border, on it, there at all
    const int rows = (n + 31) / 32, row0 = rows * warp / NW, row1 = rows * (warp + 1) / NW;
    int g_n = 0, e_n = 0, a_n = 0;
    for (int row = row0; row < row1; ++row) {
        const int k = 32 * row + lane;
        const uint32_t x = k < n ? key(k) : ABSENT;
        g_n += __popc(__ballot_sync(0xffffffffu, x > border));
        e_n += __popc(__ballot_sync(0xffffffffu, x == border && x != ABSENT));
        a_n += __popc(__ballot_sync(0xffffffffu, x != ABSENT));
    }
    __syncthreads();  // wsum has been read
    if (lane < 3) wsum[warp][lane] = lane == 0 ? g_n : (lane == 1 ? e_n : a_n);
    __syncthreads();
    int g = g0, e = e0, a = cand0;
    for (int w = 0; w < warp; ++w) g += wsum[w][0], e += wsum[w][1], a += wsum[w][2];
    for (int row = row0; row < row1; ++row) {
        const int k = 32 * row + lane, page = p0 + k;
        const uint32_t x = k < n ? key(k) : ABSENT, lower = (1u << lane) - 1u;
        const bool isg = x > border, ise = x == border && x != ABSENT, isa = x != ABSENT;
        const uint32_t bg = __ballot_sync(0xffffffffu, isg), be = __ballot_sync(0xffffffffu, ise), ba = __ballot_sync(0xffffffffu, isa);
        const int on = e + __popc(be & lower), before = g + __popc(bg & lower) + min(on, room);  // kept pages before this one
        if (isg || (ise && on < room)) {
            if (before < p.N) kept[before] = page;
        } else if (isa) {
            freed[a + __popc(ba & lower) - before] = k < p.cap ? blocks[k] : table[page].x;
            if (!p.plan) table[page].x = -1;
        }
        g += __popc(bg);
        e += __popc(be);
        a += __popc(ba);
    }
    const int stay = must + need;
    for (int k = stay + rank * ET + tid; k < p.N; k += G * ET) kept[k] = -1;
    if (rank == 0 && tid == 0) {
        p.n_freed[i] = cand - stay;
        if (stay > p.N) atomicOr(p.err, HS_DEVERR_CAPACITY);
    }
    hs::cluster_wait();  // nobody reads this CTA's memory any more
}

}  // namespace

extern "C" hs_status hs_evict_pages(hs_pool_t pool, int32_t n, int32_t N, int32_t n_first, int32_t n_last,
                                    uint32_t flags, const int32_t *d_req, const int32_t *d_budget,
                                    const float *d_weights, int32_t *d_kept, int32_t *d_freed,
                                    int32_t *d_n_freed, void *stream) {
    if (!pool || n < 0 || N < 1 || n_first < 0 || n_last < 0 || (flags & ~(HS_EVICT_SAVED_ONLY | HS_EVICT_PLAN)))
        return HS_ERR_INVALID_ARG;
    if (n == 0) return HS_OK;
    if (!d_req || !d_budget || !d_weights || !d_kept || !d_freed || !d_n_freed) return HS_ERR_INVALID_ARG;
    int dev = -1;
    HS_CUDA_TRY(cudaGetDevice(&dev));
    if (dev != pool->device) return HS_ERR_INVALID_ARG;
    static std::atomic<int> state[64];
    if (dev < 0 || dev >= 64) return HS_ERR_UNSUPPORTED;
    if (state[dev].load(std::memory_order_acquire) != 1) {
        HS_CUDA_TRY(cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CAP * 8));
        state[dev].store(1, std::memory_order_release);
    }
    EvictParams p{};
    p.table = reinterpret_cast<int2 *>(pool->d_page);
    p.ctx = pool->d_ctx;
    p.req = d_req;
    p.budget = d_budget;
    p.weights = d_weights;
    p.kept = d_kept;
    p.freed = d_freed;
    p.n_freed = d_n_freed;
    p.err = pool->d_err;
    p.N = N;
    p.n_first = n_first;
    p.n_last = n_last;
    p.max_req = pool->cfg.max_requests;
    p.max_pages = pool->max_pages;
    p.max_ctx = pool->cfg.max_ctx;
    // CTAs of a cluster: one for 2,048 pages, up to eight
    const int G = pool->max_pages <= 2048 ? 1 : (pool->max_pages <= 4096 ? 2 : (pool->max_pages <= 8192 ? 4 : MAXG));
    const bool few = pool->max_pages <= ET;
    if ((int64_t)n * G > INT32_MAX) return HS_ERR_INVALID_ARG;
    const int64_t slice = ((int64_t)pool->max_pages + 32 * G - 1) / (32 * G) * 32;
    p.cap = slice < CAP ? (int)slice : CAP;
    p.saved_only = flags & HS_EVICT_SAVED_ONLY;
    p.plan = flags & HS_EVICT_PLAN;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(few ? n : n * G), 1, 1);
    cfg.blockDim = dim3(ET, 1, 1);
    cfg.dynamicSmemBytes = few ? 0 : (size_t)p.cap * 8;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)G;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = few ? 1 : 2;
    return (few ? cudaLaunchKernelEx(&cfg, evict_few_kernel, p) : cudaLaunchKernelEx(&cfg, evict_kernel, p, G)) == cudaSuccess
               ? HS_OK
               : HS_ERR_CUDA;
}
