// hs_evict.cu -- which pages a request keeps on the GPU, by the attention weight that
// they have got (hs_page_weights), and the release of the others.
//
// Kept are the first n_first and the last n_last pages of the context, with SAVED_ONLY
// those without a host copy too, and then the others by descending weight, equal weights by
// ascending page, until there are `budget`. One CTA per request: the weights become keys
// whose unsigned order is theirs, three histograms of 11, 11 and 10 bits find the key at the
// border, and one scan over rows of 32 pages gives every page its place in the two lists:
// with g pages above the border before it and e on it, a page has min(e, room) + g kept
// ones before it. Bound: the latencies of the call; 16,384 pages are 12 bytes each, 196 KB,
// which one CTA reads in two microseconds.
#include <atomic>
#include <cstdint>

#include "hs_internal.cuh"
#include "hs_tc.cuh"

namespace {

using hs::kPage;

constexpr int ET = 1024;       // threads per CTA
constexpr int NW = ET / 32;
constexpr int BINS = 2048;
constexpr int ROWS = 1024;     // rows of 32 pages per scan
constexpr int CAP = 40960;     // keys that are kept in shared memory: 2.6 million tokens
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

__global__ void __launch_bounds__(ET)
evict_kernel(const EvictParams p) {
    hs::tc::grid_dep_wait();
    hs::tc::grid_dep_launch();
    extern __shared__ uint32_t keys[];  // [cap]
    __shared__ uint32_t hist[BINS];
    __shared__ int32_t above[ROWS], equal[ROWS], all[ROWS];
    __shared__ int32_t wsum[NW], s_bin, s_over, s_cand, s_must;
    const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = p.req[i];
    int32_t *kept = p.kept + (size_t)i * p.N, *freed = p.freed + (size_t)i * p.max_pages;
    if (r < 0 || r >= p.max_req) {
        for (int k = tid; k < p.N; k += ET) kept[k] = -1;
        if (tid == 0) {
            p.n_freed[i] = 0;
            atomicOr(p.err, HS_DEVERR_BAD_REQUEST);
        }
        return;
    }
    const int len = p.ctx[r], L = hs::context_within(len, p.max_ctx);
    const int budget = p.budget[i];
    const int P = L <= 0 ? 0 : (L - 1) / kPage + 1;
    int2 *table = p.table + (size_t)r * p.max_pages;
    const float *weights = p.weights + (size_t)r * p.max_pages;
    auto make = [&](int page, float w, int2 where) {
        if (where.x < 0) return ABSENT;
        const bool must = page < p.n_first || page >= P - p.n_last || (p.saved_only && where.y < 0);
        return must ? MUST : key_of(w);
    };
    auto key_at = [&](int page) { return page < p.cap ? keys[page] : make(page, weights[page], table[page]); };
    if (tid == 0) {
        s_cand = s_must = 0;
        uint32_t bad = len > p.max_ctx ? HS_DEVERR_INDEX_RANGE : 0u;
        if (budget < 0) bad |= HS_DEVERR_BAD_PAGE;
        if (bad) atomicOr(p.err, bad);
    }
    for (int k = tid; k < BINS; k += ET) hist[k] = 0;
    __syncthreads();

    int cand = 0, must = 0;
#pragma unroll 4
    for (int page = tid; page < P; page += ET) {
        const uint32_t k = make(page, weights[page], table[page]);
        if (page < p.cap) keys[page] = k;
        cand += k != ABSENT;
        must += k == MUST;
    }
    cand = __reduce_add_sync(0xffffffffu, cand);
    must = __reduce_add_sync(0xffffffffu, must);
    if (lane == 0 && cand) {
        atomicAdd(&s_cand, cand);
        atomicAdd(&s_must, must);
    }
    __syncthreads();
    // of the pages that need not stay, the `need` of the largest keys do; a negative budget
    // frees nothing
    const int others = s_cand - s_must;
    const int need = budget < 0 ? others : max(budget - s_must, 0);
    uint32_t border = ABSENT;  // keys above it stay, and of those equal to it the first `room`
    int room = 0;
    if (need == 0) {
        border = MUST - 1;
    } else if (need < others) {
        int left = need;
        uint32_t prefix = 0;
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0), bits = d == 2 ? 10 : 11;
            for (int page = tid; page < P; page += ET) {
                const uint32_t k = key_at(page);
                if (k != ABSENT && k != MUST && (d == 0 || (k >> (shift + bits)) == prefix))
                    atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            // bins from the top: thread t has bins 2047 - 2t and 2046 - 2t
            const int h0 = (int)hist[BINS - 1 - 2 * tid], h1 = (int)hist[BINS - 2 - 2 * tid];
            int incl = h0 + h1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) wsum[warp] = incl;
            __syncthreads();
            const int w = lane < warp ? wsum[lane] : 0;
            const int over = __reduce_add_sync(0xffffffffu, w) + incl - h0 - h1;  // keys in higher bins
            if (over < left && over + h0 >= left) {
                s_bin = BINS - 1 - 2 * tid;
                s_over = over;
            } else if (over + h0 < left && over + h0 + h1 >= left) {
                s_bin = BINS - 2 - 2 * tid;
                s_over = over + h0;
            }
            hist[BINS - 1 - 2 * tid] = hist[BINS - 2 - 2 * tid] = 0;
            __syncthreads();
            prefix = (prefix << bits) | (uint32_t)s_bin;
            left -= s_over;
        }
        border = prefix;
        room = left;
    }
    // border is ABSENT where all stay

    int base_g = 0, base_e = 0, base_a = 0;
    for (int p0 = 0; p0 < P; p0 += 32 * ROWS) {
        const int rows = min(ROWS, (P - p0 + 31) / 32);
        for (int row = warp; row < rows; row += NW) {
            const int page = p0 + 32 * row + lane;
            const uint32_t k = page < P ? key_at(page) : ABSENT;
            const uint32_t g = __ballot_sync(0xffffffffu, k > border);
            const uint32_t e = __ballot_sync(0xffffffffu, k == border && k != ABSENT);
            const uint32_t a = __ballot_sync(0xffffffffu, k != ABSENT);
            if (lane == 0) {
                above[row] = __popc(g);
                equal[row] = __popc(e);
                all[row] = __popc(a);
            }
        }
        __syncthreads();
        if (warp < 3) {  // exclusive sums of the rows, 32 per lane
            int32_t *v = warp == 0 ? above : (warp == 1 ? equal : all);
            int mine = 0;
            for (int k = 0; k < ROWS / 32; ++k) {
                const int at = k * 32 + lane;
                // 32 rows at a time: their sums so far
                int x = at < rows ? v[at] : 0, incl = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (at < rows) v[at] = mine + incl - x;
                mine += __shfl_sync(0xffffffffu, incl, 31);
                if ((k + 1) * 32 >= rows) break;
            }
            if (lane == 0) wsum[warp] = mine;
        }
        __syncthreads();
        for (int row = warp; row < rows; row += NW) {
            const int page = p0 + 32 * row + lane;
            const uint32_t k = page < P ? key_at(page) : ABSENT;
            const bool isg = k > border, ise = k == border && k != ABSENT, isa = k != ABSENT;
            const uint32_t lower = (1u << lane) - 1u;
            const int g = base_g + above[row] + __popc(__ballot_sync(0xffffffffu, isg) & lower);
            const int e = base_e + equal[row] + __popc(__ballot_sync(0xffffffffu, ise) & lower);
            const int a = base_a + all[row] + __popc(__ballot_sync(0xffffffffu, isa) & lower);
            const int before = g + min(e, room);  // kept pages before this one
            if (isg || (ise && e < room)) {
                if (before < p.N) kept[before] = page;
            } else if (isa) {
                freed[a - before] = table[page].x;
                if (!p.plan) table[page].x = -1;
            }
        }
        base_g += wsum[0];
        base_e += wsum[1];
        base_a += wsum[2];
        __syncthreads();
    }
    const int stay = base_g + min(base_e, room);
    for (int k = stay + tid; k < p.N; k += ET) kept[k] = -1;
    if (tid == 0) {
        p.n_freed[i] = base_a - stay;
        if (stay > p.N) atomicOr(p.err, HS_DEVERR_CAPACITY);
    }
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
        HS_CUDA_TRY(cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CAP * 4));
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
    p.cap = pool->max_pages < CAP ? pool->max_pages : CAP;
    p.saved_only = flags & HS_EVICT_SAVED_ONLY;
    p.plan = flags & HS_EVICT_PLAN;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n, 1, 1);
    cfg.blockDim = dim3(ET, 1, 1);
    cfg.dynamicSmemBytes = (size_t)p.cap * 4;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel, p) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}
