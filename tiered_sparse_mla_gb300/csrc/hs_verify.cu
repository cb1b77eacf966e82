// hs_verify.cu -- drafted tokens against the target's probabilities, from given
// random numbers, and the token that follows them.
//
// A drafted token x with draft probability q(x) and target probability p(x) stays where
// u q(x) < p(x). At the first one that does not, the next token is drawn from
// r(v) = max(p(v) - q(v), 0); where all stay, from the last row of p. A draft without
// probabilities is a sure guess: q is 1 at x, or, for the later children of a tree's
// node, what the children before them left of p; the draw then goes by p without the
// refused children. The drawn token is the first v whose r(0) + .. + r(v) passes u_0 times
// the sum of all.
//
// Only one row of V values (two with a draft's) is read in full for a request: 64 requests
// of 128,000 values, 65.5 MB, whose bytes are the bound, after two dependent loads that
// say which row it is.
//
// Sums are integers: a probability is a multiple of 2^-62 in 64 bits (floats from 2^-38 on
// are such multiples exactly), so that their order does not matter, and no sum differs
// between a search's two steps. They saturate near 4, which the sums of
// probabilities do not reach.
#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>

#include "hs_internal.cuh"
#include "hs_tc.cuh"

namespace {

constexpr int VT = 512;          // threads per CTA
constexpr int NW = VT / 32;
constexpr int BATCH = 256;       // values that a warp adds up at a time
constexpr int MAXB = 512;        // sums per CTA: longer slices take several batches for each
constexpr int MAXT = 64;
constexpr int MAXG = 8;          // CTAs per request

struct VerifyParams {
    const void *probs, *draft;  // rows of V values, ld and draft_ld apart
    const int32_t *tokens;
    const uint64_t *tree;
    const float *uniform;
    int32_t *index, *count, *next;
    uint32_t *err;
    int64_t ld, draft_ld;
    int T, V, per;  // per: batches for each sum
};

__device__ __forceinline__ uint64_t add_sat(uint64_t a, uint64_t b) {
    const uint64_t s = a + b;
    return s < a ? ~0ull : s;
}
__device__ __forceinline__ uint64_t shuffle64(uint64_t x, int src) {
    return (uint64_t)__shfl_sync(0xffffffffu, (unsigned long long)x, src);
}

// A probability's bits: NaN and negative ones are 0, ones above 1 are 1.
__device__ __forceinline__ uint32_t clean(uint32_t b) {
    return b > 0x7f800000u ? 0u : min(b, 0x3f800000u);
}
// In units of 2^-62, the rest cut off.
__device__ __forceinline__ uint64_t fixed(uint32_t b) {
    const uint32_t top = ((b & 0x7fffffu) | 0x800000u) << 7;  // 2^62 for 1.0, with 32 zeros behind it
    uint64_t r;
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"((uint64_t)top << 32), "r"(127u - (b >> 23)));  // beyond 63: 0
    return r;
}
template <typename P>
__device__ __forceinline__ uint32_t bits_at(const void *row, int64_t i);
template <>
__device__ __forceinline__ uint32_t bits_at<float>(const void *row, int64_t i) {
    return static_cast<const uint32_t *>(row)[i];
}
template <>
__device__ __forceinline__ uint32_t bits_at<__nv_bfloat16>(const void *row, int64_t i) {
    return (uint32_t)static_cast<const uint16_t *>(row)[i] << 16;
}
// floor(u total) for u in [0, 1), exactly
__device__ __forceinline__ uint64_t part_of(float u, uint64_t total) {
    u = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
    const uint32_t b = __float_as_uint(u), e = b >> 23;
    if (e == 0) return 0;
    const uint64_t m = (b & 0x7fffffu) | 0x800000u, lo = m * total, hi = __umul64hi(m, total);
    const uint32_t s = 150u - e;  // at least 24
    return s < 64 ? (hi << (64 - s)) | (lo >> s) : (s < 128 ? hi >> (s - 64) : 0);
}

// Cluster of gridDim.x CTAs per request (blockIdx.y): each finds the accepted path by
// itself, adds up its slice of the row, and the one that holds the border draws.
template <typename P>
__global__ void __launch_bounds__(VT)
verify_kernel(const VerifyParams p) {
    hs::tc::grid_dep_wait();
    hs::tc::grid_dep_launch();
    __shared__ uint64_t sums[MAXB], totals[MAXG];
    __shared__ int32_t gone[MAXT];     // refused children's tokens
    __shared__ int32_t s_row, s_minus, s_gone;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.y, G = gridDim.x, rank = blockIdx.x, T = p.T, V = p.V;

    if (warp == 0) {
        // nodes lane and lane + 32
        int tok[2], par[2];
        float u[2], px[2], qx[2];
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = lane + 32 * k;
            tok[k] = -1;
            par[k] = -1;
            u[k] = px[k] = qx[k] = 0.f;
            if (t >= 1 && t < T) {
                const int x = p.tokens[(int64_t)b * T + t];
                u[k] = p.uniform[(int64_t)b * T + t];
                if (p.tree) {  // the last of the nodes above it
                    const uint64_t above = p.tree[(int64_t)b * T + t] & ((1ull << t) - 1);
                    par[k] = 63 - __clzll((long long)above);
                } else {
                    par[k] = t - 1;
                }
                bad = bad || x < -1 || x >= V;
                if (x >= 0 && x < V && par[k] >= 0) {
                    tok[k] = x;
                    const P *row = static_cast<const P *>(p.probs) + ((int64_t)b * T + par[k]) * p.ld;
                    px[k] = __uint_as_float(clean(bits_at<P>(row, x)));
                    if (p.draft)
                        qx[k] = __uint_as_float(clean(bits_at<P>(
                            static_cast<const P *>(p.draft) + ((int64_t)b * (T - 1) + t - 1) * p.draft_ld, x)));
                }
            }
            u[k] = u[k] > 0.f ? fminf(u[k], 0x1.fffffep-1f) : 0.f;
        }
        auto both = [&](bool lo, bool hi) {
            return (uint64_t)__ballot_sync(0xffffffffu, lo) | (uint64_t)__ballot_sync(0xffffffffu, hi) << 32;
        };
        uint64_t path = 1;
        int end = 0, minus = 0, ngone = 0;
        if (p.draft) {  // a chain: up to the first that has no token or is refused
            // u q has 48 bits: exact in 64
            const bool s0 = tok[0] >= 0 && (double)u[0] * (double)qx[0] < (double)px[0];
            const bool s1 = tok[1] >= 0 && (double)u[1] * (double)qx[1] < (double)px[1];
            const uint64_t stop = both(lane > 0 && !s0, !s1);  // nodes from T on have no token
            const uint64_t there = both(tok[0] >= 0, tok[1] >= 0);
            const int n = stop ? __ffsll((long long)stop) - 1 : MAXT;
            path = n < 64 ? (1ull << n) - 1 : ~0ull;
            end = n - 1;
            minus = n < 64 && ((there >> n) & 1);
        } else {
            for (int node = 0; node >= 0;) {
                uint64_t kids = both(par[0] == node && tok[0] >= 0, par[1] == node && tok[1] >= 0);
                double left = 1.0;
                int go = -1;
                ngone = 0;
                while (kids && go < 0) {
                    const int c = __ffsll((long long)kids) - 1;
                    kids &= kids - 1;
                    const int x = __shfl_sync(0xffffffffu, c < 32 ? tok[0] : tok[1], c & 31);
                    float pc = __shfl_sync(0xffffffffu, c < 32 ? px[0] : px[1], c & 31);
                    const float uc = __shfl_sync(0xffffffffu, c < 32 ? u[0] : u[1], c & 31);
                    // a token that an earlier child had is gone already
                    const uint64_t same = both(par[0] == node && tok[0] == x, par[1] == node && tok[1] == x);
                    if (same & ((1ull << c) - 1)) pc = 0.f;
                    if ((double)uc * left < (double)pc) {
                        go = c;
                    } else {
                        left = fmax(left - (double)pc, 0.0);
                        if (lane == 0) gone[ngone] = x;
                        ++ngone;
                    }
                }
                end = node;
                if (go >= 0) path |= 1ull << go;
                node = go;
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0 && rank == 0) atomicOr(p.err, HS_DEVERR_INDEX_RANGE);
        if (lane == 0) {
            s_row = end;
            s_minus = minus;
            s_gone = ngone;
        }
        if (rank == 0) {
            const int n = __popcll(path);
            if (lane == 0) p.count[b] = n;
            for (int i = lane; i < T; i += 32) {
                int at = -1;
                if (i < n) {  // the i-th node of the path
                    uint64_t rest = path;
                    for (int k = 0; k < i; ++k) rest &= rest - 1;
                    at = __ffsll((long long)rest) - 1;
                }
                p.index[(int64_t)b * T + i] = at;
            }
        }
    }
    __syncthreads();
    const P *row = static_cast<const P *>(p.probs) + ((int64_t)b * T + s_row) * p.ld;
    const P *guess = p.draft && s_minus ? static_cast<const P *>(p.draft) + ((int64_t)b * (T - 1) + s_row) * p.draft_ld : nullptr;
    int ngone = s_gone;
    const float u0 = p.uniform[(int64_t)b * T];
    const int64_t unit = (int64_t)BATCH * p.per, units = (V + unit - 1) / unit;
    const int first = (int)(units * rank / G), n = (int)(units * (rank + 1) / G) - first;

    for (int attempt = 0;; ++attempt) {
        for (int i = warp; i < n; i += NW) {
            uint64_t sum = 0;
#pragma unroll 1
            for (int k = 0; k < p.per; ++k) {
                const int64_t v0 = (first + i) * unit + (int64_t)k * BATCH;
                uint32_t x[8], y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t v = v0 + 32 * e + lane;
                    x[e] = v < V ? bits_at<P>(row, v) : 0u;
                    y[e] = guess && v < V ? bits_at<P>(guess, v) : 0u;
                }
                // the refused children's tokens among these
                for (int g = 0; g < ngone; ++g) {
                    const int64_t at = gone[g] - v0;
                    if (at >= 0 && at < BATCH && (at & 31) == lane) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = (at >> 5) == e ? 0u : x[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t a = clean(x[e]), c = clean(y[e]);
                    const uint64_t r = a > c ? fixed(a) - fixed(c) : 0ull;
                    sum = add_sat(sum, r);
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum = add_sat(sum, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)sum, o));
            if (lane == 0) sums[i] = sum;
        }
        __syncthreads();
        uint64_t mine = 0;  // of lane's sums: 16 in a row
        if (warp == 0) {
            for (int k = 0; k < MAXB / 32; ++k) {
                const int i = lane * (MAXB / 32) + k;
                mine = add_sat(mine, i < n ? sums[i] : 0ull);
            }
            uint64_t all = mine;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) all = add_sat(all, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)all, o));
            if (lane < G) {
                const uint32_t at = hs::dsmem_map(&totals[rank], lane);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(all) : "memory");
            }
        }
        hs::cluster_arrive();
        hs::cluster_wait();
        uint64_t before = 0, total = 0;
        for (int g = 0; g < G; ++g) {
            if (g == rank) before = total;
            total = add_sat(total, totals[g]);
        }
        if (total == 0 && attempt == 0 && (guess || ngone)) {
            // nothing is left beside the draft: by the row itself
            guess = nullptr;
            ngone = 0;
            hs::cluster_arrive();  // the totals are read before they are written again
            hs::cluster_wait();
            continue;
        }
        if (warp != 0) return;
        if (total == 0) {
            if (rank == 0 && lane == 0) {
                p.next[b] = -1;
                atomicOr(p.err, HS_DEVERR_INDEX_RANGE);
            }
            return;
        }
        const uint64_t border = part_of(u0, total);
        if (border < before || border - before >= totals[rank]) return;
        // which lane's sums, which of them, which batch, which lane's values, which value:
        // each time the first whose inclusive sum passes the border
        uint64_t rest = border - before;
        auto locate = [&](uint64_t x) {  // lane; rest becomes what is left in it
            uint64_t incl = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = (uint64_t)__shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
                if (lane >= o) incl = add_sat(incl, y);
            }
            const uint32_t past = __ballot_sync(0xffffffffu, incl > rest);
            const int l = past ? __ffs(past) - 1 : -1;
            if (l > 0) rest -= shuffle64(incl, l - 1);
            return l;
        };
        int l = locate(mine);
        if (l < 0) return;  // cannot be: the sums are the same ones
        int i = l * (MAXB / 32);
        while (i < n - 1 && sums[i] <= rest) rest -= sums[i++];
        for (int k = 0; k < p.per; ++k) {
            const int64_t v0 = (first + i) * unit + (int64_t)k * BATCH + 8 * lane;
            uint64_t r[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t v = v0 + e;
                uint32_t a = v < V ? clean(bits_at<P>(row, v)) : 0u;
                const uint32_t c = guess && v < V ? clean(bits_at<P>(guess, v)) : 0u;
                for (int g = 0; g < ngone; ++g) a = gone[g] == v ? 0u : a;
                r[e] = a > c ? fixed(a) - fixed(c) : 0ull;
                sum = add_sat(sum, r[e]);
            }
            l = locate(sum);
            if (l < 0) {  // a later batch: all of this one lies before the border
                uint64_t all = sum;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) all = add_sat(all, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)all, o));
                rest -= all;
                continue;
            }
            if (lane == l) {
                int e = 0;
#pragma unroll
                for (int j = 0; j < 7; ++j)
                    if (e == j && r[j] <= rest) {
                        rest -= r[j];
                        ++e;
                    }
                p.next[b] = (int32_t)(v0 + e);
            }
            return;
        }
        return;
    }
}

}  // namespace

extern "C" hs_status hs_verify_drafts(hs_pool_t pool, int32_t B, int32_t T, int32_t V, int32_t dtype,
                                      const void *d_probs, int64_t probs_ld, const void *d_draft_probs,
                                      int64_t draft_ld, const int32_t *d_tokens, const uint64_t *d_tree,
                                      const float *d_uniform, int32_t *d_index, int32_t *d_count,
                                      int32_t *d_next, void *stream) {
    if (!pool || B < 0 || B > 65535 || T < 1 || T > MAXT || V < 1 || (dtype != HS_PROB_F32 && dtype != HS_PROB_BF16) ||
        probs_ld < V || (d_draft_probs && draft_ld < V))
        return HS_ERR_INVALID_ARG;
    // offsets in bytes fit 63 bits
    if (probs_ld > (1ll << 38) || (d_draft_probs && draft_ld > (1ll << 38))) return HS_ERR_INVALID_ARG;
    if (d_draft_probs && d_tree) return HS_ERR_UNSUPPORTED;
    if (B == 0) return HS_OK;
    if (!d_probs || !d_tokens || !d_uniform || !d_index || !d_count || !d_next) return HS_ERR_INVALID_ARG;
    const uintptr_t mis = (uintptr_t)d_probs | (uintptr_t)d_draft_probs;
    if (mis & (dtype == HS_PROB_F32 ? 3u : 1u)) return HS_ERR_INVALID_ARG;
    int dev = -1;
    HS_CUDA_TRY(cudaGetDevice(&dev));
    if (dev != pool->device) return HS_ERR_INVALID_ARG;
    VerifyParams p{};
    p.probs = d_probs;
    p.draft = T > 1 ? d_draft_probs : nullptr;
    p.tokens = d_tokens;
    p.tree = d_tree;
    p.uniform = d_uniform;
    p.index = d_index;
    p.count = d_count;
    p.next = d_next;
    p.err = pool->d_err;
    p.ld = probs_ld;
    p.draft_ld = draft_ld;
    p.T = T;
    p.V = V;
    const int64_t batches = ((int64_t)V + BATCH - 1) / BATCH;
    // CTAs per request: one for as many batches as it has warps, eight at most
    const int G = (int)(batches <= NW ? 1 : (batches <= 2 * NW ? 2 : (batches <= 4 * NW ? 4 : MAXG)));
    p.per = (int)((batches + (int64_t)G * MAXB - G - 1) / ((int64_t)G * MAXB - G));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)G, (unsigned)B, 1);
    cfg.blockDim = dim3(VT, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)G;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto kernel = dtype == HS_PROB_F32 ? verify_kernel<float> : verify_kernel<__nv_bfloat16>;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}
