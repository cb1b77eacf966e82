// hs_page_decode.cu -- MLA decode over whole pages of the pool, on tcgen05 tensor
// cores: a list of pages per query token or per request, or all of a request's
// pages, with the drafted tokens a chain or a tree.
//
// One 64-row page is one key tile: its rows lie together in the pool, so TMA
// brings them as boxes of 64 rows x 64 columns with no per-row ids.
//   S[128 x 64] = Q[128 x 576] K^T,  O[128 x 512] += P V,  V = K[:, 0:512].
//
// Work unit: (list, 128 query rows, split of the list), run by two CTAs. CTA h
// holds O for the value columns [256 h, 256 h + 256) and both compute the whole
// of S: 832 instead of 544 columns of depth per key, but no exchange of scores
// between the two. O takes 256 of the 512 TMEM columns, S 64, P 32 and five of
// the nine 64-column chunks of Q the other 160; Q's other four stay in shared
// memory (the MMA reads A from either).
//   warp 0      producer: Q, then per page five boxes of the columns that only
//               S needs (the other CTA's value columns and the 64 rope columns)
//               and one of this CTA's four value chunks, which stay until PV;
//   warp 1      MMA issuer: S_j = Q K_j^T, then O += P_{j-1} V_{j-1}: the pipe
//               works on the latter while the softmax warps read S_j;
//   warps 4-7   softmax, one thread per query row: mask, online softmax with a
//               conditional rescale, P to TMEM; then the epilogue;
//   warps 8-15  (FP8) converters: e4m3 codes of each landed chunk to BF16, the
//               chunks alternating between two groups of four warps.
// FP8: the codes become BF16 exactly; a row's fp32 scale multiplies its scores
// in f32 and its probability before that is rounded to BF16 (the MMA's operand
// type; the probabilities' sum is that of the unrounded ones).
// Every wait is bounded; on expiry the kernel sets HS_DEVERR_TIMEOUT, drains its
// own copies and MMAs and returns.
#include <cuda_bf16.h>

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

constexpr int BM = 128, BN = kPage;
constexpr int QCH = BM * 128;   // a 64-column chunk of Q
constexpr int KCH = BN * 128;   // a 64-column chunk of a page, BF16
constexpr int CCH = BN * 64;    // the same as e4m3 codes
constexpr int NX = 5, NVC = 4;  // chunks that only S needs; chunks of this CTA's value columns
constexpr int NSM = 128;        // softmax threads
constexpr int NT_RING = 4;      // tiles whose page number and scales are held
constexpr float TAU2 = 8.f;     // rescale threshold, log2 units: P <= 2^8
constexpr uint32_t TM_O = 0, TM_S = 256, TM_P = 320, TM_Q = 352;

template <bool FP8>
struct PCfg {
    static constexpr int THREADS = FP8 ? 512 : 256;
    static constexpr int NV = FP8 ? 2 : 3;   // stages of value chunks
    static constexpr int NXS = FP8 ? 6 : 8;  // slots of the other chunks
    static constexpr int NC = FP8 ? 11 : 1;  // slots of codes
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_V = OFF_Q + NVC * QCH;
    static constexpr int OFF_X = OFF_V + NV * NVC * KCH;
    static constexpr int OFF_C = OFF_X + NXS * KCH;
    static constexpr int OFF_SC = OFF_C + (FP8 ? NC * CCH : 0);        // f32 [NT_RING][64]
    static constexpr int OFF_PG = OFF_SC + (FP8 ? NT_RING * BN * 4 : 0);  // int32 [NT_RING]
    static constexpr int OFF_BAR = OFF_PG + NT_RING * 4;
    static constexpr int B_QFULL = 0, B_QREADY = 1, B_SFULL = 2, B_SFREE = 3, B_PFULL = 4,
                         B_PVDONE = 5, B_DRAIN = 6, B_TFULL = 7, B_TFREE = B_TFULL + NT_RING,
                         B_VFULL = B_TFREE + NT_RING, B_VFREE = B_VFULL + NV,
                         B_XFULL = B_VFREE + NV, B_XFREE = B_XFULL + NXS,
                         B_CFULL = B_XFREE + NXS, B_CFREE = B_CFULL + NC, NBAR = B_CFREE + NC;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;  // TMEM base, abort flag, tiles, first tile
    static constexpr int SMEM = OFF_MISC + 16;
    static constexpr int SMEM_ALLOC = SMEM + 1024;
    static_assert(OFF_BAR % 8 == 0 && OFF_MISC % 4 == 0, "alignment");
    static_assert(NX * QCH <= OFF_C - OFF_V, "staging of Q");
    static_assert(SMEM_ALLOC <= 232448, "shared memory");
};

struct PageParams {
    const int32_t *pages;  // [lists][N] or null: pages 0, 1, ...
    const int32_t *req, *ctx;
    const int2 *table;
    const uint64_t *tree;  // [B][T] or null
    const float *scales;   // FP8: the pool's row scales
    __nv_bfloat16 *out;
    float *lse, *ws_o, *ws_lse;
    uint32_t *err;
    int T, H, N, M, lists, nsplit, max_req, max_pages, zero_block;
    int tpl;               // lists per request: list i is token i % tpl of request i / tpl
    float scale_log2;
};

// f32 bulk copy of one page's scales into shared memory
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

template <bool FP8>
__global__ void __launch_bounds__(PCfg<FP8>::THREADS, 1)
page_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k1,
                   const __grid_constant__ CUtensorMap tm_k4, const PageParams p) {
    using C = PCfg<FP8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = hs::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = blockIdx.x & 1, split = blockIdx.x >> 1, mt = blockIdx.y, list = blockIdx.z;
    volatile int32_t *misc = reinterpret_cast<volatile int32_t *>(smem + C::OFF_MISC);
    volatile int32_t *ring_pg = reinterpret_cast<volatile int32_t *>(smem + C::OFF_PG);
    auto bar = [&](int i) { return base + C::OFF_BAR + 8u * (uint32_t)i; };
    auto fail = [&]() {
        misc[1] = 1;
        atomicOr(p.err, HS_DEVERR_TIMEOUT);
    };

    const int req = p.req[list / p.tpl];
    const bool req_ok = req >= 0 && req < p.max_req;
    const int L = req_ok ? p.ctx[req] : 0;
    const int npages = L <= 0 ? 0 : (L - 1) / kPage + 1;
    const int32_t *entries = p.pages ? p.pages + (size_t)list * p.N : nullptr;

    if (threadIdx.x == 32) {
        mbar_init(bar(C::B_QFULL), 1);
        mbar_init(bar(C::B_QREADY), NSM);
        mbar_init(bar(C::B_SFULL), 1);
        mbar_init(bar(C::B_SFREE), NSM);
        mbar_init(bar(C::B_PFULL), NSM);
        mbar_init(bar(C::B_PVDONE), 1);
        mbar_init(bar(C::B_DRAIN), 1);
        for (int i = 0; i < NT_RING; ++i) {
            mbar_init(bar(C::B_TFULL + i), 1);
            mbar_init(bar(C::B_TFREE + i), NSM);
        }
        for (int i = 0; i < C::NV; ++i) {
            mbar_init(bar(C::B_VFULL + i), FP8 ? 128 * NVC : 1);
            mbar_init(bar(C::B_VFREE + i), 1);
        }
        for (int i = 0; i < C::NXS; ++i) {
            mbar_init(bar(C::B_XFULL + i), FP8 ? 128 : 1);
            mbar_init(bar(C::B_XFREE + i), 1);
        }
        for (int i = 0; i < C::NC; ++i) {
            mbar_init(bar(C::B_CFULL + i), 1);
            mbar_init(bar(C::B_CFREE + i), 128);
        }
        misc[1] = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k1);
        if (!FP8) prefetch_tmap(&tm_k4);
    }
    if (warp == 0) {
        // the list's end: past its last entry that names a page
        int end = npages;
        if (entries) {
            end = 0;
            for (int i = lane; i < p.N; i += 32)
                if (entries[i] != -1) end = i + 1;
            end = __reduce_max_sync(0xffffffffu, end);
        }
        if (lane == 0) {
            const int a = (int)((long long)end * split / p.nsplit);
            misc[2] = (int)((long long)end * (split + 1) / p.nsplit) - a;
            misc[3] = a;
        }
    }
    if (warp == 1) tmem_alloc(base + C::OFF_MISC, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);
    const int ntiles = misc[2], first = misc[3];
    // chunk i of the order in which a page's chunks are used
    auto chunk_of = [&](int i) { return i < 4 ? 4 * (1 - half) + i : (i == 4 ? 8 : 4 * half + i - 5); };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (ntiles > 0) {
            if (lane == 0) {
                mbar_expect_tx(bar(C::B_QFULL), 9 * QCH);
                for (int i = 0; i < 9; ++i)
                    tma_load_3d(i < NX ? base + C::OFF_V + i * QCH : base + C::OFF_Q + (i - NX) * QCH, &tm_q,
                                64 * chunk_of(i), mt * BM, list, bar(C::B_QFULL));
            }
            // page number and block of the next 32 entries, one per lane
            uint32_t bad = 0;
            auto fetch = [&](int i0, int &pg, int &blk) {
                const int i = i0 + lane;
                pg = -1;
                blk = p.zero_block;
                if (i < ntiles) {
                    const int x = entries ? entries[first + i] : first + i;
                    if (x < -1 || x >= npages) {
                        bad |= HS_DEVERR_INDEX_RANGE;
                    } else if (x >= 0) {
                        const int g = p.table[(size_t)req * p.max_pages + x].x;
                        if (g >= 0) {
                            pg = x;
                            blk = g;
                        } else {
                            bad |= HS_DEVERR_BAD_PAGE;  // not resident: the entry is skipped
                        }
                    }
                }
            };
            int pg, blk, npg, nblk;
            fetch(0, npg, nblk);
            int ux = 0, uc = 0, tiles_done = 0;  // chunk loads and tiles begun
            bool ok = true;
            for (int j = 0; j < ntiles && ok; ++j) {
                if (j % 32 == 0) {
                    pg = npg;
                    blk = nblk;
                    fetch(j + 32, npg, nblk);
                }
                const int tpg = __shfl_sync(0xffffffffu, pg, j & 31), tblk = __shfl_sync(0xffffffffu, blk, j & 31);
                if (lane == 0) {
                    const int row0 = tblk * kPage;
                    const int ti = j % NT_RING;
                    ok = mbar_wait(bar(C::B_TFREE + ti), ((uint32_t)(j / NT_RING) & 1u) ^ 1u) && !misc[1];
                    if (ok) {
                        ring_pg[ti] = tpg;
                        if (FP8) {
                            mbar_expect_tx(bar(C::B_TFULL + ti), BN * 4);
                            bulk_load(base + C::OFF_SC + ti * BN * 4, p.scales + (size_t)row0, BN * 4, bar(C::B_TFULL + ti));
                        } else {
                            mbar_arrive(bar(C::B_TFULL + ti));
                        }
                        tiles_done = j + 1;
                    }
                    if (FP8) {
                        for (int i = 0; i < 9 && ok; ++i, ++uc) {
                            const int s = uc % C::NC;
                            ok = mbar_wait(bar(C::B_CFREE + s), ((uint32_t)(uc / C::NC) & 1u) ^ 1u) && !misc[1];
                            if (!ok) break;
                            mbar_expect_tx(bar(C::B_CFULL + s), CCH);
                            tma_load_3d(base + C::OFF_C + s * CCH, &tm_k1, 0, row0, chunk_of(i), bar(C::B_CFULL + s));
                        }
                    } else {
                        for (int i = 0; i < NX && ok; ++i, ++ux) {
                            const int s = ux % C::NXS;
                            ok = mbar_wait(bar(C::B_XFREE + s), ((uint32_t)(ux / C::NXS) & 1u) ^ 1u) && !misc[1];
                            if (!ok) break;
                            mbar_expect_tx(bar(C::B_XFULL + s), KCH);
                            tma_load_3d(base + C::OFF_X + s * KCH, &tm_k1, 0, row0, chunk_of(i), bar(C::B_XFULL + s));
                        }
                        const int s = j % C::NV;
                        if (ok && j == 0) ok = mbar_wait(bar(C::B_QREADY), 0);  // Q was staged there
                        if (ok) ok = mbar_wait(bar(C::B_VFREE + s), ((uint32_t)(j / C::NV) & 1u) ^ 1u) && !misc[1];
                        if (ok) {
                            mbar_expect_tx(bar(C::B_VFULL + s), NVC * KCH);
                            tma_load_3d(base + C::OFF_V + s * NVC * KCH, &tm_k4, 0, row0, 4 * half, bar(C::B_VFULL + s));
                            uc = j + 1;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            if (!ok && lane == 0) {
                fail();
                // the copies begun have landed before the CTA may end
                mbar_wait(bar(C::B_QFULL), 0);
                if (FP8) {
                    for (int i = tiles_done - 1; i >= 0 && i >= tiles_done - NT_RING; --i)
                        mbar_wait(bar(C::B_TFULL + i % NT_RING), (uint32_t)(i / NT_RING) & 1u);
                    for (int i = uc - 1; i >= 0 && i >= uc - C::NC; --i)
                        mbar_wait(bar(C::B_CFULL + i % C::NC), (uint32_t)(i / C::NC) & 1u);
                } else {
                    for (int i = ux - 1; i >= 0 && i >= ux - C::NXS; --i)
                        mbar_wait(bar(C::B_XFULL + i % C::NXS), (uint32_t)(i / C::NXS) & 1u);
                    for (int i = uc - 1; i >= 0 && i >= uc - C::NV; --i)
                        mbar_wait(bar(C::B_VFULL + i % C::NV), (uint32_t)(i / C::NV) & 1u);
                }
            }
            bad = __reduce_or_sync(0xffffffffu, bad);
            if (bad && lane == 0) atomicOr(p.err, bad);
        }
        if (lane == 0 && !req_ok) atomicOr(p.err, HS_DEVERR_BAD_REQUEST);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && ntiles > 0) {
            constexpr uint32_t ID_QK = idesc_f16(1u, 0, BM, BN), ID_PV = idesc_f16(1u, 1, BM, 256);
            bool ok = mbar_wait(bar(C::B_QREADY), 0);
            tc_fence_after();
            const uint64_t dq = desc_sw128(base + C::OFF_Q, 16, 1024);
            auto pv = [&](int j) {
                ok = mbar_wait(bar(C::B_PFULL), (uint32_t)j & 1u) && !misc[1];
                if (!ok) return;
                tc_fence_after();
                const int s = j % C::NV;
                const uint64_t v = desc_sw128(base + C::OFF_V + s * NVC * KCH, KCH, 1024);
#pragma unroll
                for (int k = 0; k < 4; ++k)  // 16 keys: 8 columns of P, 2 KB of V
                    mma_f16_ts(tmem + TM_O, tmem + TM_P + 8u * k, v + (uint64_t)(128 * k), ID_PV, (j | k) != 0);
                mma_commit(bar(C::B_VFREE + s));
                mma_commit(bar(C::B_PVDONE));
            };
            int ux = 0;
            for (int j = 0; j < ntiles && ok; ++j) {
                if (j > 0) ok = mbar_wait(bar(C::B_SFREE), (uint32_t)(j - 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                for (int i = 0; i < NX && ok; ++i, ++ux) {
                    const int s = ux % C::NXS;
                    ok = mbar_wait(bar(C::B_XFULL + s), (uint32_t)(ux / C::NXS) & 1u) && !misc[1];
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t kd = desc_sw128(base + C::OFF_X + s * KCH, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16_ts(tmem + TM_S, tmem + TM_Q + 32u * i + 8u * k, kd + 2 * k, ID_QK, (i | k) != 0);
                    mma_commit(bar(C::B_XFREE + s));
                }
                const int s = j % C::NV;
                if (ok) ok = mbar_wait(bar(C::B_VFULL + s), (uint32_t)(j / C::NV) & 1u) && !misc[1];
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = desc_sw128(base + C::OFF_V + s * NVC * KCH, 16, 1024);
#pragma unroll
                for (int i = 0; i < NVC; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16(tmem + TM_S, dq + (uint64_t)((i * QCH + 32 * k) >> 4),
                                vd + (uint64_t)((i * KCH + 32 * k) >> 4), ID_QK, 1u);
                mma_commit(bar(C::B_SFULL));
                if (j > 0) pv(j - 1);
            }
            if (ok) pv(ntiles - 1);
            if (!ok) fail();
            mma_commit(bar(C::B_DRAIN));
            mbar_wait(bar(C::B_DRAIN), 0);
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ softmax, epilogue
        const int wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const int mg = mt * BM + row;
        const bool vrow = mg < p.M;
        const int b = list / p.tpl;
        const int nt = p.T * p.tpl;  // query tokens of the request
        const int t = (vrow ? mg / p.H : 0) + list % p.tpl;
        const long long draft = (long long)L - nt;  // position of the first query token
        uint64_t tree = 0;
        if (p.tree) {
            tree = p.tree[(size_t)b * nt + t];
            if (nt < 64) tree &= (1ull << nt) - 1;
        }
        bool ok = true;
        float m2 = -INFINITY, l = 0.f;
        if (ntiles > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_QFULL), 0));
            if (ok) {
#pragma unroll 1
                for (int i = 0; i < NX; ++i) {
                    uint32_t w[32];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const uint4 v = ld_shared_v4(base + C::OFF_V + i * QCH + row * 128 + ((u ^ (row & 7)) << 4));
                        w[4 * u] = v.x;
                        w[4 * u + 1] = v.y;
                        w[4 * u + 2] = v.z;
                        w[4 * u + 3] = v.w;
                    }
                    HS_TMEM_ST32(tmem + lane_off + TM_Q + 32u * i, w);
                }
                tmem_wait_st();
            }
            fence_proxy_async();  // the staging space is refilled by TMA next
            tc_fence_before();
            mbar_arrive(bar(C::B_QREADY));
        }
        for (int j = 0; j < ntiles; ++j) {
            const int ti = j % NT_RING;
            float s[BN];
            if (ok)
                ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_TFULL + ti), (uint32_t)(j / NT_RING) & 1u) &&
                                                 mbar_wait(bar(C::B_SFULL), (uint32_t)j & 1u) && !misc[1]);
            if (ok) {
                tc_fence_after();
                uint32_t ra[32], rb[32];
                HS_TMEM_LD32(tmem + lane_off + TM_S, ra);
                HS_TMEM_LD32(tmem + lane_off + TM_S + 32, rb);
                HS_TMEM_WAIT_LD32(ra);
                HS_TMEM_WAIT_LD32(rb);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    s[e] = __uint_as_float(ra[e]) * p.scale_log2;
                    s[32 + e] = __uint_as_float(rb[e]) * p.scale_log2;
                }
            }
            tc_fence_before();
            mbar_arrive(bar(C::B_SFREE));  // S_{j+1} may be written
            uint32_t pk[BN / 2];
            bool need = false;
            float alpha = 1.f;
            if (ok) {
                const int pg = ring_pg[ti];
                const uint32_t sc_at = base + C::OFF_SC + ti * BN * 4;
                if (FP8) {
#pragma unroll
                    for (int e = 0; e < BN / 4; ++e) {
                        const float4 f = ld_shared_f4(sc_at + 16 * e);
                        s[4 * e] *= f.x;
                        s[4 * e + 1] *= f.y;
                        s[4 * e + 2] *= f.z;
                        s[4 * e + 3] *= f.w;
                    }
                }
                // the keys that this row sees, as bits
                const long long base_pos = (long long)pg * kPage;
                const bool tail = pg >= 0 && base_pos + kPage > draft;  // some row may not see some key
                uint64_t seen = ~0ull;
                if (pg < 0) {
                    seen = 0;
                } else if (tail) {
                    const long long d = draft - base_pos;  // < 64
                    if (p.tree) {
                        if (d >= 0)
                            seen = ((1ull << d) - 1) | (tree << d);
                        else
                            seen = d > -64 ? tree >> -d : 0ull;
                    } else {
                        const long long n = d + t + 1;
                        seen = n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1);
                    }
                }
                if (!__all_sync(0xffffffffu, seen == ~0ull)) {
                    const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        s[e] = (lo >> e) & 1u ? s[e] : -INFINITY;
                        s[32 + e] = (hi >> e) & 1u ? s[32 + e] : -INFINITY;
                    }
                }
                float mx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mx[e] = fmaxf(fmaxf(s[e], s[e + 8]), fmaxf(s[e + 16], s[e + 24]));
                    mx[e] = fmaxf(mx[e], fmaxf(fmaxf(s[e + 32], s[e + 40]), fmaxf(s[e + 48], s[e + 56])));
                }
#pragma unroll
                for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
                    for (int e = 0; e < w; ++e) mx[e] = fmaxf(mx[e], mx[e + w]);
                const float tmax = mx[0];
                if (j == 0) {
                    m2 = tmax;
                } else if (tmax > m2 + TAU2) {
                    need = true;
                    alpha = exp2f(m2 - tmax);
                    l *= alpha;
                    m2 = tmax;
                }
                const float mref = m2 == -INFINITY ? 0.f : m2;
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < BN / 4; ++e) {
                    float a0 = exp2f(s[4 * e] - mref), a1 = exp2f(s[4 * e + 1] - mref);
                    float a2 = exp2f(s[4 * e + 2] - mref), a3 = exp2f(s[4 * e + 3] - mref);
                    ls[e & 3] += (a0 + a1) + (a2 + a3);
                    if (FP8) {
                        float4 f = ld_shared_f4(sc_at + 16 * e);
                        if (tail) {  // a row that is not seen may have any scale
                            f.x = fabsf(f.x) <= FLT_MAX ? f.x : 0.f;
                            f.y = fabsf(f.y) <= FLT_MAX ? f.y : 0.f;
                            f.z = fabsf(f.z) <= FLT_MAX ? f.z : 0.f;
                            f.w = fabsf(f.w) <= FLT_MAX ? f.w : 0.f;
                        }
                        a0 *= f.x;
                        a1 *= f.y;
                        a2 *= f.z;
                        a3 *= f.w;
                    }
                    pk[2 * e] = pack_bf16(a0, a1);
                    pk[2 * e + 1] = pack_bf16(a2, a3);
                }
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                if (tail && !FP8) {
                    // A row that some query does not see may hold infinities or
                    // NaN, and 0 x NaN would reach that query's sum: they become
                    // zeros here (S_j is done with them; a query that does see
                    // them has them in its scores).
                    const uint32_t v0 = base + C::OFF_V + (j % C::NV) * NVC * KCH + row * 16;
#pragma unroll 4
                    for (int u = 0; u < 16; ++u) {
                        uint4 v = ld_shared_v4(v0 + 2048 * u);
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        bool hit = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool a = (w[e] & 0x7f80u) == 0x7f80u, c = (w[e] & 0x7f800000u) == 0x7f800000u;
                            hit = hit || a || c;
                            w[e] = (a ? 0u : w[e] & 0xffffu) | (c ? 0u : w[e] & 0xffff0000u);
                        }
                        if (hit) st_shared_v4(v0 + 2048 * u, w[0], w[1], w[2], w[3]);
                    }
                    fence_proxy_async();
                }
                // P and O are free once the previous PV is done
                if (j > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_PVDONE), (uint32_t)(j - 1) & 1u));
            }
            mbar_arrive(bar(C::B_TFREE + ti));
            if (ok) {
                tc_fence_after();
                HS_TMEM_ST32(tmem + lane_off + TM_P, pk);
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll 1
                    for (int cc = 0; cc < 8; ++cc) {
                        uint32_t o[32];
                        const uint32_t at = tmem + lane_off + TM_O + 32 * cc;
                        HS_TMEM_LD32(at, o);
                        HS_TMEM_WAIT_LD32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        HS_TMEM_ST32(at, o);
                    }
                }
                tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(bar(C::B_PFULL));
        }
        if (ok && ntiles > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_PVDONE), (uint32_t)(ntiles - 1) & 1u));
            tc_fence_after();
        }
        if (!ok) fail();
        // rows that see nothing: out 0, lse -inf
        const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
        const bool one = p.nsplit == 1;
        if (ok && (one || ntiles > 0)) {
            const size_t orow = one ? (size_t)list * p.M + mg : ((size_t)split * p.lists + list) * p.M + mg;
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {
                uint32_t o[32];
                if (ntiles > 0) {
                    HS_TMEM_LD32(tmem + lane_off + TM_O + 32 * cc, o);
                    HS_TMEM_WAIT_LD32(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (!vrow) continue;
                const size_t at = orow * 512 + 256 * half + 32 * cc;
                if (one) {
                    uint4 *d = reinterpret_cast<uint4 *>(p.out + at);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16(__uint_as_float(o[8 * u + 2 * e]) * inv,
                                             __uint_as_float(o[8 * u + 2 * e + 1]) * inv);
                        d[u] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    // partials stay f32: a third rounding to BF16 would show next to
                    // those of P and of the output
                    float4 *d = reinterpret_cast<float4 *>(p.ws_o + at);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        d[u] = make_float4(__uint_as_float(o[4 * u]) * inv, __uint_as_float(o[4 * u + 1]) * inv,
                                           __uint_as_float(o[4 * u + 2]) * inv, __uint_as_float(o[4 * u + 3]) * inv);
                }
            }
        }
        if (vrow && half == 0) {
            const float lse = (!ok || l == 0.f) ? -INFINITY : (m2 + __log2f(l)) * 0.69314718055994531f;
            if (one)
                p.lse[(size_t)list * p.M + mg] = lse;
            else
                p.ws_lse[((size_t)split * p.lists + list) * p.M + mg] = lse;
        }
    } else if (FP8 && warp >= 8) {
        // ------------------------------------------------------------ converters
        const int grp = (warp - 8) >> 2, tid = threadIdx.x & 127;
        bool ok = ntiles > 0 && __all_sync(0xffffffffu, mbar_wait(bar(C::B_QREADY), 0));  // Q was staged there
        const int total = 9 * ntiles;
        for (int u = grp; u < total; u += 2) {
            const int j = u / 9, i = u % 9, cs = u % C::NC;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_CFULL + cs), (uint32_t)(u / C::NC) & 1u) && !misc[1]);
            uint4 w[2];
            if (ok) {
                w[0] = ld_shared_v4(base + C::OFF_C + cs * CCH + 16 * tid);
                w[1] = ld_shared_v4(base + C::OFF_C + cs * CCH + 16 * (tid + 128));
            }
            mbar_arrive(bar(C::B_CFREE + cs));
            uint32_t dst, full;
            if (i < NX) {
                const int ux = NX * j + i, s = ux % C::NXS;
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_XFREE + s), ((uint32_t)(ux / C::NXS) & 1u) ^ 1u));
                dst = base + C::OFF_X + s * KCH;
                full = bar(C::B_XFULL + s);
            } else {
                const int s = j % C::NV;
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_VFREE + s), ((uint32_t)(j / C::NV) & 1u) ^ 1u));
                dst = base + C::OFF_V + (s * NVC + i - NX) * KCH;
                full = bar(C::B_VFULL + s);
            }
            if (ok) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int un = tid + 128 * k, key = un >> 2, part = un & 3;
                    uint32_t o[8];
                    e4m3x4_to_bf16(w[k].x, o[0], o[1]);
                    e4m3x4_to_bf16(w[k].y, o[2], o[3]);
                    e4m3x4_to_bf16(w[k].z, o[4], o[5]);
                    e4m3x4_to_bf16(w[k].w, o[6], o[7]);
                    st_shared_v4(dst + key * 128 + (((2 * part) ^ (key & 7)) << 4), o[0], o[1], o[2], o[3]);
                    st_shared_v4(dst + key * 128 + (((2 * part + 1) ^ (key & 7)) << 4), o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async();
            }
            mbar_arrive(full);
        }
        if (!ok && ntiles > 0) fail();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the splits: out = sum_s w_s O_s / sum_s w_s, w_s = exp(lse_s - max), in
// the splits' order. Four columns of a row per thread.
__global__ void __launch_bounds__(256)
page_combine_kernel(const float *__restrict__ ws_o, const float *__restrict__ ws_lse, int nsplit, int rows,
                    __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i >> 7;
    const int c = (int)(i & 127) * 4;
    if (row >= rows) return;
    float mx = -INFINITY;
    bool nan = false;
    for (int s = 0; s < nsplit; ++s) {
        const float v = ws_lse[(size_t)s * rows + row];
        nan = nan || v != v;
        mx = fmaxf(mx, v);
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
    if (mx != -INFINITY) {
#pragma unroll 4
        for (int s = 0; s < nsplit; ++s) {
            const float v = ws_lse[(size_t)s * rows + row];
            if (v == -INFINITY) continue;  // that split's partial was not written
            const float4 o = *reinterpret_cast<const float4 *>(ws_o + ((size_t)s * rows + row) * 512 + c);
            const float w = exp2f((v - mx) * 1.4426950408889634f);
            sum += w;
            acc[0] = fmaf(w, o.x, acc[0]);
            acc[1] = fmaf(w, o.y, acc[1]);
            acc[2] = fmaf(w, o.z, acc[2]);
            acc[3] = fmaf(w, o.w, acc[3]);
        }
    }
    const float inv = nan ? __uint_as_float(0x7fc00000u) : (sum > 0.f ? __fdividef(1.f, sum) : 0.f);
    *reinterpret_cast<uint2 *>(out + row * 512 + c) =
        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    if (c == 0) lse[row] = nan ? inv : (sum > 0.f ? mx + __logf(sum) : -INFINITY);
}

// ---------------------------------------------------------------- host side
struct PagePlan {
    int M, mtiles, nsplit;
    size_t ws_o_bytes, ws_bytes;
};

// Splits of a list of N pages: the count that a model of the launch makes
// shortest. A page takes a CTA about 1 us, a CTA's start and epilogue 5 us, a
// second launch 3 us and the partials' write and read about 5 MB per us.
PagePlan page_plan(int64_t lists, int64_t T, int64_t H, int64_t N) {
    PagePlan pl{};
    pl.M = (int)(T * H);
    pl.mtiles = (pl.M + BM - 1) / BM;
    const int64_t sms = sm_count(), units = lists * pl.mtiles * 2;
    const int64_t most = N < 128 ? N : 128;
    double best = 1e300;
    pl.nsplit = 1;
    for (int64_t ns = 1; ns <= most; ++ns) {
        const double waves = (double)((units * ns + sms - 1) / sms);
        double t = waves * ((double)((N + ns - 1) / ns) * 1.0 + 5.0);
        if (ns > 1) t += 3.0 + (double)ns * lists * pl.M * 512 * 8 / 5e6;
        if (t < best * 0.98) {
            best = t;
            pl.nsplit = (int)ns;
        }
        if (units * ns > 8 * sms) break;
    }
    if (pl.nsplit > 1) {
        const size_t rows = (size_t)pl.nsplit * lists * pl.M;
        pl.ws_o_bytes = (rows * 512 * sizeof(float) + 255) & ~size_t(255);
        pl.ws_bytes = pl.ws_o_bytes + ((rows * sizeof(float) + 255) & ~size_t(255));
    }
    return pl;
}

// [rows][9 chunks][64] seen as (element, row, chunk), boxes of 64 x 64 x n
bool make_page_map(CUtensorMap *m, bool fp8, const void *rows, uint64_t n_rows, uint32_t nchunks) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t rb = fp8 ? kDim : 2 * kDim;
    cuuint64_t dims[3] = {64, n_rows, 9};
    cuuint64_t strides[2] = {rb, rb / 9};
    cuuint32_t box[3] = {64, (cuuint32_t)BN, nchunks};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void *>(rows), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8>
hs_status launch_pages(dim3 grid, int dev, cudaStream_t s, const CUtensorMap &tq, const CUtensorMap &k1,
                       const CUtensorMap &k4, const PageParams &p) {
    static std::atomic<int> state[64];
    if (dev < 0 || dev >= 64) return HS_ERR_UNSUPPORTED;
    if (state[dev].load(std::memory_order_acquire) != 1) {
        HS_CUDA_TRY(cudaFuncSetAttribute(page_decode_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PCfg<FP8>::SMEM_ALLOC));
        state[dev].store(1, std::memory_order_release);
    }
    page_decode_kernel<FP8><<<grid, PCfg<FP8>::THREADS, PCfg<FP8>::SMEM_ALLOC, s>>>(tq, k1, k4, p);
    return cudaGetLastError() == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

// `lists` lists of T query tokens each; tpl > 1 (with T = 1): lists / tpl
// requests whose tpl tokens each have their own list.
hs_status page_entry(hs_pool_t pool, int64_t lists, int32_t T, int32_t tpl, int32_t H, int32_t N,
                     const void *d_q, const int32_t *d_pages, const int32_t *d_req_ids,
                     const uint64_t *d_tree, float sm_scale, void *d_out, float *d_lse,
                     void *d_workspace, size_t ws_bytes, void *stream) {
    if (!pool || lists < 0 || lists > 65535 || T < 1 || T > 32767 || H < 1 || N < 0 ||
        (int64_t)T * H > (int64_t)BM * 65535 || (d_tree && (int64_t)T * tpl > 64))
        return HS_ERR_INVALID_ARG;
    if (d_pages ? N < 1 : false) return HS_ERR_INVALID_ARG;
    if (lists == 0) return HS_OK;
    if (!d_q || !d_req_ids || !d_out || !d_lse) return HS_ERR_INVALID_ARG;
    if (((uintptr_t)d_q | (uintptr_t)d_out) & 15u) return HS_ERR_INVALID_ARG;
    int dev = -1;
    HS_CUDA_TRY(cudaGetDevice(&dev));
    if (dev != pool->device) return HS_ERR_INVALID_ARG;
    const bool fp8 = pool->cfg.dtype == HS_FP8_E4M3_ROWSCALE;
    const PagePlan pl = page_plan(lists, T, H, N < 1 ? pool->max_pages : N);
    if (lists * pl.M > INT32_MAX) return HS_ERR_INVALID_ARG;
    if (pl.nsplit > 1 && (!d_workspace || ws_bytes < pl.ws_bytes || ((uintptr_t)d_workspace & 255u)))
        return HS_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap tq, k1, k4;
    const uint64_t rows = (uint64_t)(pool->cfg.n_gpu_blocks + 1) * kPage;
    if (!make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_q, kDim, pl.M, lists, 2 * kDim, 64, BM,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_page_map(&k1, fp8, pool->d_rows, rows, 1) || !make_page_map(&k4, fp8, pool->d_rows, rows, NVC))
        return HS_ERR_CUDA;
    PageParams p{};
    p.pages = d_pages;
    p.req = d_req_ids;
    p.ctx = pool->d_ctx;
    p.table = reinterpret_cast<const int2 *>(pool->d_page);
    p.tree = d_tree;
    p.scales = pool->d_scales;
    p.out = static_cast<__nv_bfloat16 *>(d_out);
    p.lse = d_lse;
    p.ws_o = pl.nsplit > 1 ? static_cast<float *>(d_workspace) : nullptr;
    p.ws_lse = pl.nsplit > 1 ? reinterpret_cast<float *>(static_cast<uint8_t *>(d_workspace) + pl.ws_o_bytes)
                             : nullptr;
    p.err = pool->d_err;
    p.T = T;
    p.H = H;
    p.N = N;
    p.M = pl.M;
    p.lists = (int)lists;
    p.nsplit = pl.nsplit;
    p.max_req = pool->cfg.max_requests;
    p.max_pages = pool->max_pages;
    p.zero_block = (int)pool->cfg.n_gpu_blocks;
    p.tpl = tpl;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    const dim3 grid(2 * pl.nsplit, pl.mtiles, (unsigned)lists);
    const hs_status st = fp8 ? launch_pages<true>(grid, dev, s, tq, k1, k4, p)
                             : launch_pages<false>(grid, dev, s, tq, k1, k4, p);
    if (st != HS_OK || pl.nsplit == 1) return st;
    const int n = (int)(lists * pl.M);
    page_combine_kernel<<<(unsigned)(((int64_t)n * 128 + 255) / 256), 256, 0, s>>>(p.ws_o, p.ws_lse, pl.nsplit, n,
                                                                                   p.out, d_lse);
    return cudaGetLastError() == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

}  // namespace

extern "C" size_t hs_page_decode_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t N) {
    if (B < 1 || T < 1 || H < 1 || N < 1) return 0;
    return page_plan(B, T, H, N).ws_bytes;
}

extern "C" hs_status hs_page_mla_decode(hs_pool_t pool, int32_t B, int32_t T, int32_t H, int32_t N,
                                        const void *d_q, const int32_t *d_pages, const int32_t *d_req_ids,
                                        const uint64_t *d_tree, float sm_scale, void *d_out, float *d_lse,
                                        void *d_workspace, size_t ws_bytes, void *stream) {
    return page_entry(pool, B, T, 1, H, N, d_q, d_pages, d_req_ids, d_tree, sm_scale, d_out, d_lse,
                      d_workspace, ws_bytes, stream);
}

extern "C" hs_status hs_page_mla_decode_per_token(hs_pool_t pool, int32_t B, int32_t T, int32_t H, int32_t N,
                                                  const void *d_q, const int32_t *d_pages,
                                                  const int32_t *d_req_ids, const uint64_t *d_tree,
                                                  float sm_scale, void *d_out, float *d_lse,
                                                  void *d_workspace, size_t ws_bytes, void *stream) {
    // request b's T lists are lists b*T .. b*T+T-1 of one query token each
    if (B < 0 || T < 1 || (int64_t)B * T > 65535 || !d_pages) return HS_ERR_INVALID_ARG;
    return page_entry(pool, (int64_t)B * T, 1, T, H, N, d_q, d_pages, d_req_ids, d_tree, sm_scale, d_out,
                      d_lse, d_workspace, ws_bytes, stream);
}
