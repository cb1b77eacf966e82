// hs_rows.cu -- new latent rows into the tiered cache, and the mean row of a page.
//
// hs_append_rows puts the rows of new tokens at their positions in every tier
// that holds them; hs_page_means reduces a page's 64 rows to one, the cheap key
// that hs_select_pages scores.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cfloat>
#include <cstdint>

#include "hs_internal.cuh"
#include "hs_tc.cuh"

namespace {

using hs::kDim;
using hs::kPage;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// ---------------------------------------------------------------- append
// Eight lanes per row, nine 16-byte pieces (72 BF16 values) per lane: a warp
// reads four rows in nine loads of 4 x 128 contiguous bytes, all in flight
// before the first is used, and the row's largest magnitude is three shuffles.
constexpr int AT = 128;              // threads per CTA
constexpr int ARW = 4;               // rows per warp
constexpr int ARB = AT / 32 * ARW;   // rows per CTA

struct AppendParams {
    const uint8_t *src;                        // [B][T][576] BF16
    const int32_t *req, *start, *index, *ctx;  // start, index: may be null
    const int2 *page;
    const int32_t *hot_blocks, *p2s;
    uint8_t *rows, *host_rows;
    float *scales, *host_scales;
    uint32_t *err;
    int64_t n;  // B * T
    int T, max_req, max_pages, max_ctx, C, HB;
};

// Eight BF16 values (one 16-byte piece) to eight e4m3 codes of value / scale.
// The definition is the quotient rounded to 32 bits, then to e4m3. `inv` is
// 1 / scale rounded to nearest: one product and one residual correction
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990, theorem on division with a correctly rounded reciprocal)
// give the correctly rounded quotient as long as no step leaves the normal
// range, which the caller ensures; otherwise the divide instruction is used (checked in
// exact arithmetic for every pair of a value's and a scale's significands). The
// residual is taken with the other sign: that of a zero is +0, and -0 less +0 stays -0.
template <bool SAFE>
__device__ __forceinline__ uint2 quantise8(uint4 v, float scale, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = bf16_lo(w[e]), b = bf16_hi(w[e]);
        float qa, qb;
        if (SAFE) {
            qa = __fmul_rn(a, inv);
            qb = __fmul_rn(b, inv);
            qa = __fmaf_rn(-__fmaf_rn(qa, scale, -a), inv, qa);
            qb = __fmaf_rn(-__fmaf_rn(qb, scale, -b), inv, qb);
        } else {  // subnormal operands kept (the build flushes them elsewhere)
            asm("div.rn.f32 %0, %1, %2;" : "=f"(qa) : "f"(a), "f"(scale));
            asm("div.rn.f32 %0, %1, %2;" : "=f"(qb) : "f"(b), "f"(scale));
        }
        c[e] = __nv_cvt_float2_to_fp8x2(make_float2(qa, qb), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <bool FP8>
__global__ void __launch_bounds__(AT) append_kernel(const AppendParams p) {
    constexpr int RB = FP8 ? kDim : 2 * kDim;
    hs::tc::grid_dep_wait();  // may be launched while the stream's last kernel runs
    hs::tc::grid_dep_launch();
    const int lane = threadIdx.x & 31, part = lane & 7;
    const int64_t i = (int64_t)blockIdx.x * ARB + (threadIdx.x >> 5) * ARW + (lane >> 3);
    // whole warps run to the shuffles; rows that write nothing have go = false
    bool go = i < p.n;
    const int64_t b = go ? i / p.T : 0;
    const int k = go ? (int)(i - b * p.T) : 0;
    int from = k;
    if (go && p.index) from = p.index[i];
    uint32_t bad = 0;
    if (go && (from < -1 || from >= p.T)) bad = HS_DEVERR_INDEX_RANGE;
    go = go && from >= 0 && from < p.T;
    uint4 v[9];
    if (go) {
        const uint8_t *s = p.src + ((size_t)b * p.T + from) * (2 * kDim) + part * 16;
#pragma unroll
        for (int u = 0; u < 9; ++u) v[u] = hs::ld_once_v4(s + 128 * u);
    } else {
#pragma unroll
        for (int u = 0; u < 9; ++u) v[u] = make_uint4(0u, 0u, 0u, 0u);
    }
    // where the row goes: its page's GPU block, its host copy, its hot slot
    int64_t gpu = -1, host = -1, hot = -1;
    if (go) {
        const int r = p.req[b];
        if (r < 0 || r >= p.max_req) {
            bad = HS_DEVERR_BAD_REQUEST;
        } else {
            const int64_t pos = (p.start ? (int64_t)p.start[b] : (int64_t)p.ctx[r] - p.T) + k;
            if (pos < 0 || pos >= p.max_ctx) {
                bad = HS_DEVERR_INDEX_RANGE;
            } else {
                const int2 e = p.page[(size_t)r * p.max_pages + pos / kPage];
                const int slot = p.p2s[(size_t)r * p.max_ctx + pos];
                const int off = (int)(pos % kPage);
                if (e.x >= 0) gpu = (int64_t)e.x * kPage + off;
                if (e.y >= 0) host = (int64_t)e.y * kPage + off;
                if (slot >= 0 && slot < p.C) {
                    const int hb = p.hot_blocks[(size_t)r * p.HB + slot / kPage];
                    if (hb >= 0) hot = (int64_t)hb * kPage + slot % kPage;
                }
                if (gpu < 0 && host < 0) bad = HS_DEVERR_BAD_PAGE;
            }
        }
    }
    if (bad && part == 0) atomicOr(p.err, bad);
    const bool wr = go && !bad;
    if (!FP8) {
        if (!wr) return;
#pragma unroll
        for (int u = 0; u < 9; ++u) {
            const int o = 16 * part + 128 * u;
            if (gpu >= 0) hs::st_v4(p.rows + gpu * RB + o, v[u]);
            if (host >= 0) hs::st_v4(p.host_rows + host * RB + o, v[u]);
            if (hot >= 0) hs::st_v4(p.rows + hot * RB + o, v[u]);
        }
        return;
    }
    // FP8: the largest magnitude as BF16 bits (their order is that of the values)
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 9; ++u) {
        m = __vmaxu2(m, v[u].x & 0x7fff7fffu);
        m = __vmaxu2(m, v[u].y & 0x7fff7fffu);
        m = __vmaxu2(m, v[u].z & 0x7fff7fffu);
        m = __vmaxu2(m, v[u].w & 0x7fff7fffu);
    }
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!wr) return;
    const uint32_t top = max(m & 0xffffu, m >> 16);
    const float amax = __uint_as_float(top << 16);
    float scale;
    asm("div.rn.f32 %0, %1, %2;" : "=f"(scale) : "f"(amax), "f"(448.f));
    // a row of zeros, or of values below 448 * 2^-126, keeps the smallest normal
    // scale: value = code * scale stays exact where the codes are
    scale = scale >= FLT_MIN ? scale : FLT_MIN;
    if (top >= 0x7f80u) scale = __uint_as_float(0x7fc00000u);  // an infinity or NaN: the row is NaN
    float inv = 0.f;
    // 2^-60 <= amax <= 2^60: with |value| >= amax * 2^-20 (smaller ones become
    // code 0 whatever the quotient's last bit) every step below is normal
    const bool safe = top >= 0x2180u && top <= 0x5d80u;
    if (safe) inv = __frcp_rn(scale);
#pragma unroll
    for (int u = 0; u < 9; ++u) {
        const uint2 c = safe ? quantise8<true>(v[u], scale, inv) : quantise8<false>(v[u], scale, inv);
        const int o = 8 * part + 64 * u;
        if (gpu >= 0) *reinterpret_cast<uint2 *>(p.rows + gpu * RB + o) = c;
        if (host >= 0) *reinterpret_cast<uint2 *>(p.host_rows + host * RB + o) = c;
        if (hot >= 0) *reinterpret_cast<uint2 *>(p.rows + hot * RB + o) = c;
    }
    if (part == 0) {
        if (gpu >= 0) p.scales[gpu] = scale;
        if (host >= 0) p.host_scales[host] = scale;
        if (hot >= 0) p.scales[hot] = scale;
    }
}

// ---------------------------------------------------------------- page means
// One CTA per page. A thread owns one 16-byte column piece of the row and every
// G-th row of the page, all of them loaded before the first is used, so a page
// (72 KB BF16, 36 KB FP8) is in flight at once; the G partial sums meet in
// shared memory. Sums in f32 in a fixed order, a quotient rounded to f32 (a product with
// a rounded 1/n puts means half way between two BF16 values on the wrong one), and one
// rounding to BF16 at the end.
constexpr int MT = 288;

template <bool FP8>
__global__ void __launch_bounds__(MT)
means_kernel(const uint8_t *rows, const float *scales, const uint8_t *host_rows, const float *host_scales,
             const int2 *page, const int32_t *ctx, int max_req, int max_pages, int max_ctx, const int32_t *req,
             const int32_t *pg, __nv_bfloat16 *means, uint32_t *err) {
    constexpr int RB = FP8 ? kDim : 2 * kDim;
    constexpr int V = RB / 16;       // pieces of a row: 72, or 36
    constexpr int G = MT / V;        // row groups: 4, or 8
    constexpr int NR = kPage / G;    // rows per thread: 16, or 8
    constexpr int E = FP8 ? 16 : 8;  // values per piece
    __shared__ float part[G][kDim + 4];
    hs::tc::grid_dep_wait();
    hs::tc::grid_dep_launch();
    const int r = req[blockIdx.x], p = pg[blockIdx.x];
    const bool in_range = r >= 0 && r < max_req && p >= 0 && p < max_pages;
    const size_t at = (size_t)(in_range ? r : 0) * max_pages + (in_range ? p : 0);
    const int2 e = in_range ? page[at] : make_int2(-1, -1);
    if (e.x < 0 && e.y < 0) {
        if (threadIdx.x == 0) atomicOr(err, HS_DEVERR_BAD_PAGE);
        return;
    }
    const int len = ctx[r], left = hs::context_within(len, max_ctx) - p * kPage;
    const int n = left <= 0 ? 0 : (left < kPage ? left : kPage);  // rows that hold a token
    if (len > max_ctx && threadIdx.x == 0) atomicOr(err, HS_DEVERR_INDEX_RANGE);
    const bool dev = e.x >= 0;
    const size_t row0 = (size_t)(dev ? e.x : e.y) * kPage;
    const uint8_t *src = (dev ? rows : host_rows) + row0 * RB;
    const int piece = threadIdx.x % V, g = threadIdx.x / V;
    uint4 v[NR];
    float sc[NR];
#pragma unroll
    for (int u = 0; u < NR; ++u) {
        const int k = u * G + g;
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        sc[u] = 0.f;
        if (k < n) {  // rows past the context hold no token and are not read
            v[u] = hs::ld_once_v4(src + (size_t)k * RB + piece * 16);
            if (FP8) sc[u] = (dev ? scales : host_scales)[row0 + k];
        }
    }
    float sum[E];
#pragma unroll
    for (int j = 0; j < E; ++j) sum[j] = 0.f;
#pragma unroll
    for (int u = 0; u < NR; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (FP8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(
                        (__nv_fp8x2_storage_t)(w[q] >> (16 * h)), __NV_E4M3);
                    const float2 f = __half22float2(__half2(x));
                    sum[4 * q + 2 * h] = fmaf(f.x, sc[u], sum[4 * q + 2 * h]);
                    sum[4 * q + 2 * h + 1] = fmaf(f.y, sc[u], sum[4 * q + 2 * h + 1]);
                }
            } else {
                sum[2 * q] += bf16_lo(w[q]);
                sum[2 * q + 1] += bf16_hi(w[q]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < E; ++j) part[g][piece * E + j] = sum[j];
    __syncthreads();
    const float count = n > 0 ? (float)n : 1.f;
    for (int c = threadIdx.x; c < kDim / 2; c += MT) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int q = 0; q < G; ++q) {
            a += part[q][2 * c];
            b += part[q][2 * c + 1];
        }
        *reinterpret_cast<__nv_bfloat162 *>(means + at * kDim + 2 * c) =
            __floats2bfloat162_rn(__fdiv_rn(a, count), __fdiv_rn(b, count));
    }
}

// A launch that may begin while the stream's previous kernel still runs (the kernels
// wait for it before they read or write anything, and read nothing through the
// read-only path, which may hold or fetch what was there before).
template <typename... P, typename... A>
hs_status launch(void (*kernel)(P...), unsigned grid, int threads, void *stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

bool on_pool_device(const hs_pool *pool) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == pool->device;
}

}  // namespace

extern "C" hs_status hs_append_rows(hs_pool_t pool, int32_t B, int32_t T, const void *d_rows,
                                    const int32_t *d_req_ids, const int32_t *d_start,
                                    const int32_t *d_index, void *stream) {
    if (!pool || B < 0 || T < 1) return HS_ERR_INVALID_ARG;
    if (B == 0) return HS_OK;
    if (!d_rows || !d_req_ids || ((uintptr_t)d_rows & 15u)) return HS_ERR_INVALID_ARG;
    const int64_t n = (int64_t)B * T;
    if (n > (int64_t)INT32_MAX * ARB || !on_pool_device(pool)) return HS_ERR_INVALID_ARG;
    AppendParams p{};
    p.src = static_cast<const uint8_t *>(d_rows);
    p.req = d_req_ids;
    p.start = d_start;
    p.index = d_index;
    p.ctx = pool->d_ctx;
    p.page = reinterpret_cast<const int2 *>(pool->d_page);
    p.hot_blocks = pool->d_hot_blocks;
    p.p2s = pool->d_p2s;
    p.rows = pool->d_rows;
    p.host_rows = pool->hd_rows;
    p.scales = pool->d_scales;
    p.host_scales = pool->hd_scales;
    p.err = pool->d_err;
    p.n = n;
    p.T = T;
    p.max_req = pool->cfg.max_requests;
    p.max_pages = pool->max_pages;
    p.max_ctx = pool->cfg.max_ctx;
    p.C = pool->cfg.hot_rows;
    p.HB = pool->hb;
    const unsigned grid = (unsigned)((n + ARB - 1) / ARB);
    return launch(pool->cfg.dtype == HS_BF16 ? append_kernel<false> : append_kernel<true>, grid, AT, stream, p);
}

extern "C" hs_status hs_page_means(hs_pool_t pool, int32_t n, const int32_t *d_req,
                                   const int32_t *d_page, void *d_means, void *stream) {
    if (!pool || n < 0) return HS_ERR_INVALID_ARG;
    if (n == 0) return HS_OK;
    if (!d_req || !d_page || !d_means || ((uintptr_t)d_means & 15u) || !on_pool_device(pool))
        return HS_ERR_INVALID_ARG;
    return launch(pool->cfg.dtype == HS_BF16 ? means_kernel<false> : means_kernel<true>, (unsigned)n, MT, stream,
                  pool->d_rows, pool->d_scales, pool->hd_rows, pool->hd_scales,
                  reinterpret_cast<const int2 *>(pool->d_page), pool->d_ctx, pool->cfg.max_requests, pool->max_pages,
                  pool->cfg.max_ctx, d_req, d_page, static_cast<__nv_bfloat16 *>(d_means), pool->d_err);
}
