// hs_page_decode.cu -- MLA decode over whole pages of the pool, on tcgen05 tensor
// cores: a list of pages per query token or per request, or all of a request's
// pages, with the drafted tokens a chain or a tree; or a sliding window of positions with
// the first ones beside it.
//
// A 64-row page lies together in the pool, so TMA brings it as boxes of 64 rows x
// 64 columns with no per-row ids. Per step, two pages (128 keys):
//   S[128 x 128] = Q[128 x 576] K^T,  O[128 x 512] += P V,  V = K[:, 0:512].
//
// Work unit: (list, 128 query rows, split of the list), run by a pair of CTAs of a
// cluster whose tensor cores work as one (cta_group::2): CTA r holds the query rows
// [64 r, 64 r + 64) with their S (64 TMEM columns), O (256) and six of the nine
// 64-column chunks of Q (192; the other three stay in shared memory), and no
// score leaves its CTA. With M = 128 over two CTAs the accumulator of CTA r has
// row i in lane i for the first half of the MMA's columns and in lane 64 + i for
// the second; A in tensor memory is wanted in both.
//   K: CTA r supplies the keys of page r of the step, all nine chunks, through a
//      ring of chunk slots that S frees at once;
//   V: CTA r supplies the value columns 128 r + {0..127, 256..383} of both pages,
//      loaded apart (the second reading comes from L2) into a buffer that PV frees.
// Bound: an MMA of 128 keys takes 45 clocks (256 value columns: 64), so a step is
// 36 x 45 + 16 x 64 = 2.7k clocks, and its shared-memory traffic (the MMAs' operands,
// the copies, FP8's conversions) about as many at 128 bytes a clock. Measured: BF16
// 2.8k-3.0k clocks a step (8 x 32 tokens x 128 heads over 16,384 rows: 732 us, 1.44
// PFLOP/s), FP8 2.9k-3.2k (4 x 8 tokens x 16 heads over 131,072 rows: 111 us). An earlier
// form, one CTA per half of the value columns and both computing S, was bound by the
// issue of its 80 smaller MMAs per 128 keys and by their operands' shared-memory reads.
// Roles in each CTA:
//   warps 0, 3  producers: the K chunks and the V chunks of each step by TMA;
//   warp 1      (CTA 0) MMA issuer for both CTAs: S_j = Q K_j^T, then
//               O += P_{j-1} V_{j-1}, during which the softmax reads S_j;
//   warps 4-11  softmax: thread = (row, page of the step, half of its keys): mask,
//               online softmax with a conditional rescale, P as BF16 (FP8: F16)
//               to shared memory; epilogue;
//   warp 2      (FP8) the largest of the landed scales, by 32 keys;
//   warps 12-15 (FP8) converters: V's e4m3 codes to F16, half the columns at a time
//               (four more warps leave the softmax 96 registers: 33.9 -> 34.8 us for 16 x 4
//               lists of 2,048 rows).
// FP8: S is taken from the e4m3 codes themselves (kind::f8f6f4), so K needs no
// conversion (with K's chunks converted to F16 like V's, the shared-memory traffic and
// the converters' issue made a step 4.0k clocks: 44 us for 16 x 4 lists of 2,048 rows of
// 128 heads, which now take 34).
//   Q: a value times the row's power of two, which brings the row's largest to
//      (224, 448], is the sum of two e4m3 codes, and an MMA of depth 32 takes either
//      with the same keys: as many MMAs as one of F16. Values that come to 1/4 or more
//      are exact, their last bit is at least the codes' smallest step: 2^-9.8 of the
//      row's largest. Smaller ones are off by at most half that step, 2^-17.8 of that
//      largest. A row that is not finite becomes NaN.
//   V: F16, which every code is exactly and to which the hardware converts two codes
//      per instruction (24 against 72 clocks per 16 codes and warp for placing BF16
//      bits with integer instructions). Two e4m3 codes per weight would spare this
//      too, but lose small weights below 2^-10 of the codes' unit.
//   P: F16, 2^10 exp2(score - reference) * scale / c, c a power of two that a query row
//      keeps for the weights times scales as it does the reference for the scores. The
//      reference follows where a score passes it by 4. c is at most 16 times the row's
//      largest weight times scale so far, so that rows of large scale and little weight
//      leave the others' their bits, and within that not below half the largest scale
//      alone, which is cheap to look up: only where a scale passes 2 c, or the reference
//      moves, are the products themselves looked at. So P <= 2^15; it is off by at most
//      2^-11 of it, or by 2^-35 c. The probabilities' sum has the unrounded ones.
// Window (WIN): a query token at position x sees the positions from x - window + 1 on, and
// those below n_sink. A unit's entries are then the pages that some row of it sees, the first
// ones and those of its window, found by arithmetic; rows are masked from below too on
// the few pages where a row's window may begin.
// Every wait is bounded; on expiry the kernel sets HS_DEVERR_TIMEOUT, drains its
// own copies and MMAs and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
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

constexpr int BM = 128, RM = 64;  // query rows per work unit, per CTA
constexpr int CH = 64 * 128;      // 64 rows (of Q, of a page, of P) x 64 BF16 columns
constexpr int CCH = 64 * 64;      // 64 rows x 64 e4m3 codes
constexpr int NK = 9, NVC = 4;    // K chunks of a page; V chunks of a page in this CTA
constexpr int NQT = 6;            // chunks of Q in tensor memory
constexpr int NTI = 3;            // steps whose page numbers and scales are held
constexpr int NSW = 8;            // softmax warps
constexpr int NCW = 4;            // FP8: converter warps
constexpr uint32_t JOIN_BYTES = RM * 256 * 4 + RM * 4;  // half the columns of a partial, and its lse
// A row's reference follows where its scores' maximum passes the old one by this much
// (log2 units): P <= 2^8, FP8: 2^15.
template <bool FP8>
constexpr float TAU2 = FP8 ? 4.f : 8.f;
constexpr int P_EXP = 10;  // FP8: a weight at both references is 2^10
constexpr float C_MOST = 16.f;  // FP8: of the scales' reference, over the largest weight times scale
constexpr uint32_t TM_O = 0, TM_S = 256, TM_Q = 320;

template <bool FP8>
struct PCfg {
    static constexpr int THREADS = 128 + 32 * NSW + (FP8 ? 32 * NCW : 0);
    static constexpr int NV = 2;              // V's buffers: two steps; FP8: the two halves of one step's columns
    // K chunks per barrier. FP8: three; BF16: the rope chunk by itself, then the
    // value chunks in twos (fewer waits and copies to issue)
    static constexpr int GK = FP8 ? 3 : 2;
    static constexpr int GV = 4;              // FP8: V chunks converted together (half the columns)
    static constexpr int NXG = 4;             // groups of K chunks; BF16: group 0 is the rope's
    static constexpr int NCV = FP8 ? 4 : 0;   // groups of V codes: two per half of the columns
    static constexpr int XB = FP8 ? NXG * GK * CCH : (2 * NXG - 1) * CH;  // bytes of K chunks
    static constexpr int RK = FP8 ? NXG : NXG - 1, RV = FP8 ? NCV : NV;  // the producers' rings
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + (NK - NQT) * CH;  // [2 pages] rows x keys
    static constexpr int OFF_V = OFF_P + 2 * CH;           // [steps][2 pages][NVC]
    static constexpr int OFF_X = OFF_V + (FP8 ? 1 : 2) * 2 * NVC * CH;
    static constexpr int OFF_C = OFF_X + XB;                // FP8: V's codes
    static constexpr int OFF_SC = OFF_C + NCV * GV * CCH;                 // f32 [NTI][2][64] the rows' scales
    static constexpr int OFF_SP = OFF_SC + (FP8 ? NTI * 2 * 64 * 4 : 0);  // f32 [NTI][4] their largest, by 32 keys
    static constexpr int OFF_XM = OFF_SP + (FP8 ? NTI * 16 : 0);          // f32 [softmax threads], FP8: twice
    static constexpr int OFF_WM = OFF_XM + (FP8 ? 2 : 1) * 32 * NSW * 4;  // f32 [RM] FP8: a row's largest weight times scale
    static constexpr int OFF_PG = OFF_WM + (FP8 ? RM * 4 : 0);            // int32 [NTI][2]
    static constexpr int OFF_BAR = (OFF_PG + NTI * 8 + 7) & ~7;
    static constexpr int B_QFULL = 0, B_QDONE = 1, B_QREADY = 2, B_SFULL = 3, B_SFREE = 4, B_PFULL = 5,
                         B_PVDONE = 6, B_DRAIN = 7, B_JOIN = 8, B_EFREE = 9, B_TFULL = 10, B_TFREE = B_TFULL + NTI,
                         B_TREADY = B_TFREE + NTI, B_VFULL = B_TREADY + NTI, B_VFREE = B_VFULL + NV, B_XFULL = B_VFREE + NV,
                         B_XFREE = B_XFULL + NXG, B_CFULL = B_XFREE + NXG, B_CFREE = B_CFULL + NCV,
                         NBAR = B_CFREE + NCV;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;  // TMEM base, abort flag, steps
    static constexpr int SMEM = OFF_MISC + 32;
    static constexpr int SMEM_ALLOC = SMEM + 1024;
    // where box i (32 columns, 64 rows, 8 KB) of the other split's partial lands:
    // behind the own one, and where Q was
    static constexpr int NJB = FP8 ? 6 : 7;
    __device__ static int join_box(int i) {
        return i < NJB ? OFF_V + RM * 512 * 4 + i * 8192 : OFF_Q + (i - NJB) * 8192;
    }
    static constexpr int OFF_QST = OFF_V + (FP8 ? 0 : 1) * 2 * NVC * CH;  // Q is staged in the last V stage
    static_assert(OFF_BAR % 8 == 0 && OFF_SC % 16 == 0, "alignment");
    static_assert(NQT * CH <= 2 * NVC * CH, "staging of Q");
    static_assert(OFF_SC - OFF_V >= RM * 512 * 4, "staging of O");
    static_assert(OFF_SC - OFF_V >= RM * 512 * 4 + NJB * 8192 && (8 - NJB) * 8192 <= OFF_P - OFF_Q, "the other split's partial");
    static_assert(SMEM_ALLOC <= 232448, "shared memory");
};

struct PageParams {
    const int32_t *pages;  // [lists][N] or null: pages 0, 1, ...
    const int32_t *req, *ctx;
    const int2 *table;
    const uint64_t *tree;  // [B][T] or null
    const float *scales;   // FP8: the pool's row scales
    __nv_bfloat16 *out;    // written here when the splits are joined inside the cluster
    float *lse, *ws_lse;
    uint32_t *err;
    int inside;            // 2: the two splits are joined inside the cluster; or 0
    int T, H, N, M, mtiles, nsplit, max_req, max_pages, max_ctx, zero_block;
    int n_full;            // units (128 query rows of a list) not split; the others are, nsplit ways
    int ws_list0, ws_lists;  // the lists that the partials' space holds
    int tpl;               // lists per request: list i is token i % tpl of request i / tpl
    int window, n_sink;    // WIN
    int units;             // LOOP
    const uint8_t *q;
    float scale_log2;
};

// This CTA's shared memory to another CTA's, completing on a barrier there.
__device__ __forceinline__ void bulk_push(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Four e4m3 codes to F16, exactly; the NaN codes (rows that no query sees may hold
// any byte) become a finite value.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const uint32_t most = 0x5f805f80u;  // 480, above every code
    asm("min.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(most));
    asm("min.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(most));
}
// f32 bulk copy of one page's scales into shared memory
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
// a and b plus 0 times c and d: NaN where one is not finite
__device__ __forceinline__ void zeros_of(float &a, float &b, float c, float d) {
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mov.b64 z, {%4, %4};\n"
        " fma.rn.f32x2 x, y, z, x;\n mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d), "f"(0.f));
}
// Whether any of the softmax threads says so (named barrier 1).
__device__ __forceinline__ bool any_softmax(bool x) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(32 * NSW)
        : "memory");
    return r != 0;
}

// O's 128 columns from `at` in this thread's lane times alpha. Out of line: it
// runs where a row's reference grows, and inside the loop it costs the scores'
// registers.
__device__ __noinline__ void rescale_o(uint32_t at, float alpha) {
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        HS_TMEM_LD32(at + c, o);
        HS_TMEM_WAIT_LD32(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
        HS_TMEM_ST32(at + c, o);
    }
    tmem_wait_st();
}

template <bool FP8, bool WIN, bool LOOP>
__global__ void __launch_bounds__(PCfg<FP8>::THREADS, 1)
page_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k1,
                   const __grid_constant__ CUtensorMap tm_k2, const __grid_constant__ CUtensorMap tm_o,
                   const __grid_constant__ CUtensorMap tm_w, const PageParams p) {
    static_assert(!LOOP || (!FP8 && WIN), "units one after the other");
    using C = PCfg<FP8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = hs::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // a cluster is one pair of CTAs, or both splits' pairs
    const uint32_t crank = hs::cluster_ctarank(), pair0 = crank & ~1u;
    const int rank = static_cast<int>(crank & 1u);
    // whole units first, then the others' splits
    const int pair = blockIdx.x >> 1, past = pair - p.n_full;
    const int nsplit = past < 0 ? 1 : p.nsplit, split = past < 0 ? 0 : past % p.nsplit;
    int unit = past < 0 ? pair : p.n_full + past / p.nsplit;
    int list = unit / p.mtiles, mt = unit - list * p.mtiles;
    volatile int32_t *misc = reinterpret_cast<volatile int32_t *>(smem + C::OFF_MISC);
    volatile int32_t *ring_pg = reinterpret_cast<volatile int32_t *>(smem + C::OFF_PG);
    auto bar = [&](int i) { return base + C::OFF_BAR + 8u * (uint32_t)i; };
    // the same barrier in the pair's CTA 0, whose warp 1 issues the MMAs
    const uint32_t lead0 = cluster_address(base + C::OFF_BAR, pair0);
    const uint16_t both = (uint16_t)(3u << pair0);
    auto lead = [&](int i) { return lead0 + 8u * (uint32_t)i; };
    auto fail = [&]() {
        st_shared_b32(base + C::OFF_MISC + 4, 1u);
        atomicOr(p.err, HS_DEVERR_TIMEOUT);
    };

    if (warp == 1) {
        for (int i = lane; i < C::NBAR; i += 32) {
            uint32_t n = 1;
            if (i == C::B_QDONE || i == C::B_EFREE || (i >= C::B_TFREE && i < C::B_TFREE + NTI)) n = NSW;
            // both CTAs' softmax warps
            if (i == C::B_QREADY || i == C::B_SFREE || i == C::B_PFULL) n = 2 * NSW;
            // FP8: four converter warps of each CTA
            if (FP8 && i >= C::B_VFULL && i < C::B_VFREE) n = 8;
            if (FP8 && i >= C::B_CFREE) n = 4;
            mbar_init(bar(i), n);
        }
        if (lane == 0) misc[1] = 0;
        fence_mbar_init();
        fence_proxy_async();
        __syncwarp();
        grid_dep_wait();
        if (lane == 0) {  // Q by TMA at once: its barrier is this CTA's own
            if (p.inside) mbar_expect_tx(bar(C::B_JOIN), JOIN_BYTES);
            mbar_expect_tx(bar(C::B_QFULL), NK * CH);
            for (int i = 0; i < NK; ++i)
                tma_load_3d(i < NQT ? base + C::OFF_QST + i * CH : base + C::OFF_Q + (i - NQT) * CH, &tm_q, 64 * i,
                            mt * BM + RM * rank, list, bar(C::B_QFULL));
        }
        __syncwarp();
    }
    if (warp == 2) tmem_alloc2(base + C::OFF_MISC, 512);
    // What the earlier kernels of the stream wrote is read from here on: this grid
    // may be launched while the last of them still runs. It lets no later grid begin
    // before it ends: the splits' join, placed on SMs that were done early, kept the
    // next call's CTAs from theirs (76 x 27 steps: 129 against 144 us a call).
    grid_dep_wait();
    // The loads that lead to the first copy, as early and as parallel as they go:
    // entries and request, then the table (its bounds do not need the context's
    // length) and the length.
    const int32_t *entries = p.pages ? p.pages + (size_t)list * p.N : nullptr;
    const bool loader = warp == 0 || warp == 3;
    // WIN, a tree: of this lane's tokens, the fewest nodes that one sees, and the last node
    auto tree_nodes = [&](int list_u, int &few, int &last) {
        const uint64_t *masks = p.tree + (size_t)list_u * p.T, nodes = p.T < 64 ? (1ull << p.T) - 1 : ~0ull;
        for (int t = lane; t < p.T; t += 32) {
            const uint64_t m = masks[t] & nodes;
            few = min(few, __popcll(m));
            last = max(last, 63 - __clzll((long long)m));
        }
    };
    int few = 64, last = -1;
    if (WIN && loader && p.tree) tree_nodes(list, few, last);
    int e0 = -1;  // entry `lane`
    if (loader && entries && lane < p.N) e0 = entries[lane];
    const int req = p.req[list / p.tpl];
    bool req_ok = req >= 0 && req < p.max_req;
    const int len = req_ok ? p.ctx[req] : 0;
    int L = hs::context_within(len, p.max_ctx);
    const int2 *table = p.table + (size_t)(req_ok ? req : 0) * p.max_pages;
    int nsteps = 0, first = 0, end = 0, npages = 0;
    int wskip = 0, wsinks = INT_MAX;  // WIN: entries from wsinks on are pages wskip later
    uint32_t bad = len > p.max_ctx ? HS_DEVERR_INDEX_RANGE : 0u;
    // page number and block of the entries from i0 on, one per lane
    auto fetch = [&](int i0, int &pg, int &blk) {
        const int i = first + i0 + lane;
        const bool in = i < end && i < first + 2 * nsteps;
        const int kept = __shfl_sync(0xffffffffu, e0, i & 31);
        int x = -1, g = -1;
        if (in) x = entries ? (i < 32 ? kept : entries[i]) : i;
        if (WIN && in) x = i < wsinks ? i : i + wskip;
        if (x >= 0 && x < p.max_pages) g = table[x].x;
        pg = -1;
        blk = p.zero_block;
        if (x < -1 || x >= npages) {
            bad |= HS_DEVERR_INDEX_RANGE;
        } else if (x >= 0) {
            if (g >= 0) {
                pg = x;
                blk = g;
            } else {
                bad |= HS_DEVERR_BAD_PAGE;  // not resident: the entry is skipped
            }
        }
    };
    // WIN: a unit's entries, of the context's pages `e`; the others are left out
    auto window_pages = [&](int len_u, int mt_u, int few_u, int last_u, int &e, int &sinks_u, int &skip_u) {
        sinks_u = INT_MAX;
        skip_u = 0;
        if (e <= 0) return;
        // The positions that some row sees: up to its last token's, and from its first token's
        // window on. A tree: up to the last node that some token sees (-1: none sees any), and from the
        // window of the token that sees the fewest on. No page in between is without a row
        // that some token sees: where the context's last ones are in no window, all tokens see all nodes.
        int t0 = mt_u * BM / p.H, t1 = (min(p.M, mt_u * BM + BM) - 1) / p.H;
        if (p.tree) {
            t0 = __reduce_min_sync(0xffffffffu, few_u) - 1;
            t1 = __reduce_max_sync(0xffffffffu, last_u);
        }
        const int top = len_u - p.T + t1, low = (int)max((long long)len_u - p.T + t0 - p.window + 1, 0ll);
        e = top < 0 ? 0 : top / kPage + 1;
        const int sinks = min((int)(((long long)p.n_sink + kPage - 1) / kPage), e);
        if (low / kPage > sinks) {
            sinks_u = sinks;
            skip_u = low / kPage - sinks;
            e -= skip_u;
        }
    };
    // LOOP: this pair's units are `apart`. Each role walks them for itself: `it` counts them and
    // g0 the steps before this one's; the barriers' phases run on. The next one is looked up
    // (peek), and worked out (look), while this one runs.
    const int apart = (int)(gridDim.x >> 1);
    int it = 0, g0 = 0, req_next = 0, len_next = 0;
    struct {
        int list, mt, L, end, npages, sinks, skip;
        bool there, ok;
    } nx{};
    auto peek = [&]() {
        nx.there = LOOP && unit + apart < p.units;
        if (!nx.there) return;
        nx.list = (unit + apart) / p.mtiles;
        req_next = p.req[nx.list];
        len_next = req_next >= 0 && req_next < p.max_req ? p.ctx[req_next] : 0;
    };
    auto look = [&]() {
        if (!nx.there) return;
        nx.mt = unit + apart - nx.list * p.mtiles;
        nx.ok = req_next >= 0 && req_next < p.max_req;
        if (!nx.ok) bad |= HS_DEVERR_BAD_REQUEST;
        if (len_next > p.max_ctx) bad |= HS_DEVERR_INDEX_RANGE;
        nx.L = hs::context_within(len_next, p.max_ctx);
        nx.npages = nx.end = nx.L <= 0 ? 0 : (nx.L - 1) / kPage + 1;
        int few_u = 64, last_u = -1;
        if (p.tree) tree_nodes(nx.list, few_u, last_u);
        window_pages(nx.L, nx.mt, few_u, last_u, nx.end, nx.sinks, nx.skip);
    };
    auto enter = [&]() {  // false: there is no next one
        if (!nx.there) return false;
        unit += apart;
        list = nx.list;
        mt = nx.mt;
        L = nx.L;
        table = p.table + (size_t)(nx.ok ? req_next : 0) * p.max_pages;
        g0 += nsteps;
        ++it;
        npages = nx.npages;
        end = nx.end;
        wsinks = nx.sinks;
        wskip = nx.skip;
        nsteps = (end + 1) / 2;
        return true;
    };
    int npg = -1, nblk = p.zero_block;
    if (loader) {
        // the list's end: past its last entry that names a page
        if (entries) {
            end = e0 != -1 ? lane + 1 : 0;
            for (int i = lane + 32; i < p.N; i += 32)
                if (entries[i] != -1) end = i + 1;
            end = __reduce_max_sync(0xffffffffu, end);
        } else {
            end = L <= 0 ? 0 : (L - 1) / kPage + 1;
        }
        if (WIN) window_pages(L, mt, few, last, end, wsinks, wskip);
        // splits begin at even entries: a step is two pages
        const long long steps = (end + 1) / 2;
        const int z = (int)(steps * (split + 1) / nsplit);
        first = (int)(steps * split / nsplit);
        nsteps = z - first;
        first *= 2;
        npages = L <= 0 ? 0 : (L - 1) / kPage + 1;
        fetch(0, npg, nblk);
        if (warp == 0 && lane == 0) misc[2] = nsteps;
    }
    tc_fence_before();
    __syncthreads();
    // Both CTAs' barriers and tensor memory are there. What the peer needs of this
    // CTA are its barriers, released by the fence above: a releasing arrive would
    // wait for everything in flight (measured 3k clocks).
    cluster_sync_relaxed();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);
    nsteps = misc[2];

    if (loader) {
        // ------------------------------------------------------------ producers
        // warp 0: page numbers, scales, K; warp 3: V. Each looks up the pages'
        // blocks itself, 32 entries at a time, ahead of their use.
        const bool kw = warp == 0;
        int pg, blk;
        int ul = 0, ut = 0, ux = 0;  // loads, steps and (BF16) rope loads begun
        bool ok = true;
        if (LOOP && !req_ok) bad |= HS_DEVERR_BAD_REQUEST;
        do {
            peek();
            if (LOOP && nx.there && !kw && lane == 1) {
                // the next unit's Q into L2, so that it comes at once when there is a place for it
                const int row0 = (unit + apart - nx.list * p.mtiles) * BM + RM * rank, n = min(RM, p.M - row0);
                if (n > 0) prefetch_l2(p.q + ((size_t)nx.list * p.M + row0) * (2 * kDim), (uint32_t)n * (2 * kDim));
            }
            if (LOOP && it > 0) {
                fetch(0, npg, nblk);
                if (lane == 0 && !kw) {
                    // Q goes where this unit's first V will: free once the step before the last
                    // is done with it; the chunks that stay, once the last scores are.
                    const int s = g0 % C::NV;
                    ok = mbar_wait_inline(bar(C::B_VFREE + s), ((uint32_t)(g0 / C::NV) & 1u) ^ 1u);
                    if (ok && g0 > 0) ok = mbar_wait_inline(bar(C::B_SFULL), (uint32_t)(g0 - 1) & 1u);
                    if (ok) {
                        mbar_expect_tx(bar(C::B_QFULL), NK * CH);
                        for (int i = 0; i < NK; ++i)
                            tma_load_3d(i < NQT ? base + C::OFF_V + s * 2 * NVC * CH + i * CH : base + C::OFF_Q + (i - NQT) * CH,
                                        &tm_q, 64 * i, mt * BM + RM * rank, list, bar(C::B_QFULL));
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            for (int j = 0; j < nsteps && ok; ++j) {
                const int gj = g0 + j;
                if (j % 16 == 0) {
                    pg = npg;
                    blk = nblk;
                    fetch(2 * j + 32, npg, nblk);
                }
                const int src = 2 * (j % 16);
                const int pg0 = __shfl_sync(0xffffffffu, pg, src), pg1 = __shfl_sync(0xffffffffu, pg, src + 1);
                const int row0 = __shfl_sync(0xffffffffu, blk, src) * kPage;
                const int row1 = __shfl_sync(0xffffffffu, blk, src + 1) * kPage;
                if (lane == 0 && kw) {
                    const int own = rank ? row1 : row0, ti = gj % NTI;
                    ok = mbar_wait_inline(bar(C::B_TFREE + ti), ((uint32_t)(gj / NTI) & 1u) ^ 1u);
                    if (ok) {
                        ring_pg[2 * ti] = pg0;
                        ring_pg[2 * ti + 1] = pg1;
                        if (FP8) {
                            const uint32_t sc = base + C::OFF_SC + ti * 512;
                            mbar_expect_tx(bar(C::B_TFULL + ti), 512);
                            bulk_load(sc, p.scales + (size_t)row0, 256, bar(C::B_TFULL + ti));
                            bulk_load(sc + 256, p.scales + (size_t)row1, 256, bar(C::B_TFULL + ti));
                        } else {
                            mbar_arrive(bar(C::B_TFULL + ti));
                        }
                        ut = gj + 1;
                    }
                    // both CTAs' bytes complete on CTA 0's barrier
                    if (FP8) {
                        for (int i = 0; i < NK && ok; i += C::GK, ++ul) {
                            const int s = ul % C::RK;
                            ok = mbar_wait_inline(bar(C::B_XFREE + s), ((uint32_t)(ul / C::RK) & 1u) ^ 1u);
                            if (!ok) break;
                            if (rank == 0) mbar_expect_tx(bar(C::B_XFULL + s), 2 * C::GK * CCH);
                            tma_load_pair(base + C::OFF_X + s * C::GK * CCH, &tm_k1, 0, own, i, lead(C::B_XFULL + s));
                        }
                    } else {
                        if (ok) ok = mbar_wait_inline(bar(C::B_XFREE), ((uint32_t)gj & 1u) ^ 1u);
                        if (ok) {
                            if (rank == 0) mbar_expect_tx(bar(C::B_XFULL), 2 * CH);
                            tma_load_pair(base + C::OFF_X, &tm_k1, 0, own, 8, lead(C::B_XFULL));
                            ux = gj + 1;
                        }
                        for (int i = 0; i < 8 && ok; i += 2, ++ul) {
                            const int s = 1 + ul % C::RK;
                            ok = mbar_wait_inline(bar(C::B_XFREE + s), ((uint32_t)(ul / C::RK) & 1u) ^ 1u);
                            if (!ok) break;
                            if (rank == 0) mbar_expect_tx(bar(C::B_XFULL + s), 4 * CH);
                            tma_load_pair(base + C::OFF_X + (2 * s - 1) * CH, &tm_k2, 0, own, i, lead(C::B_XFULL + s));
                        }
                    }
                } else if (lane == 0) {
                    if (FP8) {
                        for (int i = 0; i < 2 && ok; ++i, ++ul) {  // half the columns: two chunks of either page
                            const int cs = ul % C::RV;
                            const uint32_t dst = base + C::OFF_C + cs * C::GV * CCH;
                            ok = mbar_wait_inline(bar(C::B_CFREE + cs), ((uint32_t)(ul / C::RV) & 1u) ^ 1u);
                            if (!ok) break;
                            mbar_expect_tx(bar(C::B_CFULL + cs), C::GV * CCH);
                            tma_load_3d(dst, &tm_k2, 0, row0, 4 * i + 2 * rank, bar(C::B_CFULL + cs));
                            tma_load_3d(dst + 2 * CCH, &tm_k2, 0, row1, 4 * i + 2 * rank, bar(C::B_CFULL + cs));
                        }
                    } else {
                        const int s = gj % C::RV;
                        if (j == 1 && it == 0) ok = mbar_wait_inline(bar(C::B_QDONE), 0);  // Q was staged there
                        if (LOOP && j == 0 && it > 0) ok = mbar_wait_inline(bar(C::B_QDONE), (uint32_t)it & 1u);
                        // the last unit's output was
                        if (LOOP && j == 1 && it > 0) ok = mbar_wait_inline(bar(C::B_EFREE), (uint32_t)(it - 1) & 1u);
                        if (ok) ok = mbar_wait_inline(bar(C::B_VFREE + s), ((uint32_t)(gj / C::RV) & 1u) ^ 1u);
                        if (ok) {
                            const uint32_t dst = base + C::OFF_V + s * 2 * NVC * CH;
                            mbar_expect_tx(bar(C::B_VFULL + s), 2 * NVC * CH);
                            tma_load_3d(dst, &tm_k2, 0, row0, 2 * rank, bar(C::B_VFULL + s));
                            tma_load_3d(dst + 2 * CH, &tm_k2, 0, row0, 4 + 2 * rank, bar(C::B_VFULL + s));
                            tma_load_3d(dst + 4 * CH, &tm_k2, 0, row1, 2 * rank, bar(C::B_VFULL + s));
                            tma_load_3d(dst + 6 * CH, &tm_k2, 0, row1, 4 + 2 * rank, bar(C::B_VFULL + s));
                            ul = gj + 1;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            if (LOOP && lane == 0 && !kw && ok && nx.there) {
                // Each phase is waited for once, in order: those that short units have left.
                // (Behind the last unit nothing holds the next phase back.)
                if (it == 0 && nsteps < 2) ok = mbar_wait_inline(bar(C::B_QDONE), 0);
                if (it > 0 && nsteps == 0) ok = mbar_wait_inline(bar(C::B_QDONE), (uint32_t)it & 1u);
                if (ok && it > 0 && nsteps < 2) ok = mbar_wait_inline(bar(C::B_EFREE), (uint32_t)(it - 1) & 1u);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            look();
        } while (ok && enter());
        if (LOOP && lane == 0 && ok) {
            // what the MMA issuer says of the last loads: on its way until it is here
            const int ring = kw ? C::RK : C::RV, b0 = kw ? C::B_XFREE + 1 : C::B_VFREE;
            for (int i = ul - 1; i >= 0 && i >= ul - ring; --i) mbar_wait_inline(bar(b0 + i % ring), (uint32_t)(i / ring) & 1u);
            if (kw && ux > 0) mbar_wait_inline(bar(C::B_XFREE), (uint32_t)(ux - 1) & 1u);
        }
        if (lane == 0) {
            // the copies begun have landed before the CTA may end
            if (LOOP ? !kw : kw) mbar_wait_inline(bar(C::B_QFULL), (uint32_t)it & 1u);
            if (!ok) {
                fail();
                const int ring = kw ? C::RK : C::RV;
                const int b0 = kw ? (FP8 ? C::B_XFULL : C::B_XFULL + 1) : (FP8 ? C::B_CFULL : C::B_VFULL);
                for (int i = ul - 1; (!kw || rank == 0) && i >= 0 && i >= ul - ring; --i)
                    mbar_wait_inline(bar(b0 + i % ring), (uint32_t)(i / ring) & 1u);
                if (!FP8 && kw && rank == 0 && ux > 0) mbar_wait_inline(bar(C::B_XFULL), (uint32_t)(ux - 1) & 1u);
                for (int i = ut - 1; FP8 && kw && i >= 0 && i >= ut - NTI; --i)
                    mbar_wait_inline(bar(C::B_TFULL + i % NTI), (uint32_t)(i / NTI) & 1u);
            }
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (lane == 0 && kw) {
            if (!LOOP && !req_ok) bad = HS_DEVERR_BAD_REQUEST;  // it has no context that an entry could lie outside of
            if (bad) atomicOr(p.err, bad);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (CTA 0)
        if (rank == 0 && (LOOP || nsteps > 0)) {
            constexpr uint32_t ID_QK = idesc_f16(FP8 ? 0u : 1u, 0, BM, 128), ID_PV = idesc_f16(FP8 ? 0u : 1u, 1, BM, 256);
            const uint64_t dk = desc_sw128(base, 16, 1024), dv = desc_sw128(base, CH, 1024);
            const uint32_t hi = (uint32_t)(dk >> 32), klo = (uint32_t)dk, vlo = (uint32_t)dv;
            const uint32_t chi = (uint32_t)(desc_sw64(base, 16, 512) >> 32);  // K's codes
            const uint32_t leader = elect_one();
            bool ok = true;
            auto pv = [&](int j) {
                const int gj = g0 + j;
                ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_PFULL), (uint32_t)gj & 1u));
                if (!ok) return;
                tc_fence_after();
                const uint32_t v = vlo + ((C::OFF_V + (FP8 ? 0 : gj % C::NV) * 2 * NVC * CH) >> 4);
                const uint32_t a = klo + (C::OFF_P >> 4);
#pragma unroll
                for (int nh = 0; nh < 2; ++nh) {  // 256 value columns each
                    if (FP8) {  // each half is there, and free again, by itself
                        ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_VFULL + nh), (uint32_t)j & 1u));
                        if (!ok) return;
                        tc_fence_after();
                    }
                    if (leader) {
#pragma unroll
                        for (int pgi = 0; pgi < 2; ++pgi)
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // 16 keys: 32 bytes of P, 2 KB of V
                                mma2_ss(tmem + TM_O + 128u * nh, a + ((pgi * CH + 32 * k) >> 4),
                                        v + ((pgi * NVC * CH + nh * 2 * CH + 2048 * k) >> 4), hi, ID_PV,
                                        (j | pgi | k) != 0);
                        if (FP8 && j + 1 < nsteps) commit_both(bar(C::B_VFREE + nh), both);
                        if (!FP8 && nh == 1 && (LOOP || j + C::NV < nsteps)) commit_both(bar(C::B_VFREE + gj % C::NV), both);
                        if (nh == 1) commit_both(bar(C::B_PVDONE), both);
                    }
                    __syncwarp();
                }
                __syncwarp();
            };
            constexpr int PER = FP8 ? NK / C::GK : 8 / C::GK;  // groups of K chunks per step
            int s = 0;
            uint32_t ph = 0, ready = 0;  // units with steps so far
            do {
                peek();
                if (!LOOP || nsteps > 0) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_QREADY), ready++ & 1u));
                tc_fence_after();
                for (int j = 0; j < nsteps && ok; ++j) {
                    const int gj = g0 + j;
                    if (gj > 0) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_SFREE), (uint32_t)(gj - 1) & 1u));
                    tc_fence_after();
                    auto qk = [&](int c, uint32_t slot, bool fresh) {  // one chunk: four MMAs
                        const uint32_t kd = klo + ((C::OFF_X + slot * (FP8 ? CCH : CH)) >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // FP8: both pieces of Q with the same 32 codes
                            const uint32_t tq = tmem + TM_Q + 32u * c + 8u * k, sq = klo + ((C::OFF_Q + (c - NQT) * CH + 32 * k) >> 4);
                            const bool acc = !(fresh && k == 0);
                            if (FP8 && c < NQT)
                                mma2_ts_e4m3(tmem + TM_S, tq, kd + 2 * (k & 1), chi, ID_QK, acc);
                            else if (FP8)
                                mma2_ss_e4m3(tmem + TM_S, sq, hi, kd + 2 * (k & 1), chi, ID_QK, acc);
                            else if (c < NQT)
                                mma2_ts(tmem + TM_S, tq, kd + 2 * k, hi, ID_QK, acc);
                            else
                                mma2_ss(tmem + TM_S, sq, kd + 2 * k, hi, ID_QK, acc);
                        }
                    };
                    if (!FP8) {
                        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_XFULL), (uint32_t)gj & 1u));
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            qk(8, 0, true);
                            if (LOOP || j + 1 < nsteps) commit_both(bar(C::B_XFREE), both);
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int c = 0; c < (FP8 ? NK : 8); c += C::GK) {
                        const int b0 = (FP8 ? 0 : 1) + s;
                        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_XFULL + b0), ph));
                        if (ok) {
                            tc_fence_after();
                            if (leader) {
#pragma unroll
                                for (int g = 0; g < C::GK; ++g) qk(c + g, (FP8 ? s * C::GK : 1 + 2 * s) + g, FP8 && c + g == 0);
                                if (LOOP || PER * j + c / C::GK + C::RK < PER * nsteps) commit_both(bar(C::B_XFREE + b0), both);
                            }
                            __syncwarp();
                        }
                        if (++s == (FP8 ? C::NXG : C::NXG - 1)) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (leader) commit_both(bar(C::B_SFULL), both);
                    __syncwarp();
                    if (j > 0) pv(j - 1);
                }
                look();
                if (ok && (!LOOP || nsteps > 0)) pv(nsteps - 1);
            } while (ok && enter());
            // LOOP: the last arrives of both CTAs are here
            if (LOOP && ok && g0 + nsteps > 0)
                ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_SFREE), (uint32_t)(g0 + nsteps - 1) & 1u));
            if (!ok && lane == 0) fail();
            if (leader) {
                // every MMA issued has finished before shared and tensor memory go
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 bar(C::B_DRAIN))
                             : "memory");
                mbar_wait_inline(bar(C::B_DRAIN), 0);
            }
            __syncwarp();
        }
    } else if (FP8 && warp == 2) {
        // ------------------------------------------------------------ the scales' maxima
        bool ok = true;
        for (int j = 0; j < nsteps; ++j) {
            const int ti = j % NTI;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_TFULL + ti), (uint32_t)(j / NTI) & 1u));
            if (!ok) break;
            const float4 f = ld_shared_f4(base + C::OFF_SC + ti * 512 + lane * 16);
            float m = fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w)));
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((lane & 7) == 0) reinterpret_cast<volatile float *>(smem + C::OFF_SP)[4 * ti + (lane >> 3)] = m;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_TREADY + ti));
        }
        if (!ok && lane == 0) fail();
    } else if (warp >= 4 && warp < 4 + NSW) {
        // ------------------------------------------------------------ softmax, epilogue
        // warp w reaches the tensor memory lanes 32 (w % 4) .. + 31
        const int wq = warp & 3, hf = (warp - 4) >> 2, tid = hf * 128 + wq * 32 + lane;
        const int row = tid & 63, kh = wq >> 1;  // query row of this CTA; page of the step
        constexpr int KT = 32;                   // keys per thread: 32 hf .. of the page
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        // 32-bit shared addresses throughout: the loop has no registers to spare
        const uint32_t xm = base + C::OFF_XM;
        auto xm_row = [&](int o) { return xm + 4u * (uint32_t)(o + row); };
        // What the MMAs read was written through this CTA's shared or tensor memory
        // and fenced for the async proxy by its writers: the arrive needs no
        // cluster-scope release, which takes 1-2k clocks a time.
        auto arrive_lead = [&](uint32_t cluster_bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(cluster_bar);
        };
        bool ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_QFULL), 0));
        auto q_at = [&](int i) { return base + (i < NQT ? C::OFF_QST + i * CH : C::OFF_Q + (i - NQT) * CH) + row * 128; };
        float q_back = 1.f;
        if (FP8) {
            // Q's values become codes in place. thread = (row, quarter of each chunk), so that a row
            // is in one warp and is read once: the two pieces of each value, 64 first ones and then
            // 64 second ones, lie where they are read as 128 bytes of a row of A.
            const int crow = tid >> 2, part = 2 * (tid & 3);
            auto at = [&](int i, int u) {
                return base + (i < NQT ? C::OFF_QST + i * CH : C::OFF_Q + (i - NQT) * CH) + crow * 128 + ((u ^ (crow & 7)) << 4);
            };
            uint4 v[NK][2];
            uint32_t m = 0;  // the row's largest magnitude; NaN if there is one
#pragma unroll
            for (int i = 0; i < NK; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    v[i][u] = ok ? ld_shared_v4(at(i, part + u)) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v[i][u].x, v[i][u].y, v[i][u].z, v[i][u].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[e] & 0x7fff7fffu));
                }
            // bits of magnitudes are in their order, infinities and NaN above all
            uint32_t top = max(m & 0xffffu, m >> 16);
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));  // all have read
            const uint32_t q_pow = query_power(top);
            if (part == 0) st_shared_f1(xm + 4 * crow, query_back(top));
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                uint32_t w[4], r[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    bf16x4_to_e4m3(v[i][u].x, v[i][u].y, q_pow, w[2 * u], r[2 * u]);
                    bf16x4_to_e4m3(v[i][u].z, v[i][u].w, q_pow, w[2 * u + 1], r[2 * u + 1]);
                }
                if (ok) {
                    st_shared_v4(at(i, part >> 1), w[0], w[1], w[2], w[3]);
                    st_shared_v4(at(i, 4 + (part >> 1)), r[0], r[1], r[2], r[3]);
                }
            }
            named_bar_sync(1, 32 * NSW);
            q_back = ld_shared_f1(xm_row(0));
        }
        if (ok && nsteps > 0) {
#pragma unroll 1
            for (int i = hf; i < NQT; i += 2) {
                uint32_t w[32];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint4 v = ld_shared_v4(q_at(i) + ((u ^ (row & 7)) << 4));
                    w[4 * u] = v.x;
                    w[4 * u + 1] = v.y;
                    w[4 * u + 2] = v.z;
                    w[4 * u + 3] = v.w;
                }
                HS_TMEM_ST32(tmem + lane_off + TM_Q + 32u * i, w);
            }
            tmem_wait_st();
        }
        // A unit without steps is not announced to the MMA issuer: nothing would hold the softmax back until the
        // issuer has looked, and a phase missed is waited for without end.
        auto q_moved = [&](bool steps) {
            fence_proxy_async();  // the staging space is refilled next
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_QDONE));
            if (steps) arrive_lead(lead(C::B_QREADY));
        };
        q_moved(nsteps > 0);

        const int tpl = LOOP ? 1 : p.tpl;
        auto token_of = [&](int g) { return g < p.M ? g / p.H : 0; };
        int t_row = token_of(mt * BM + RM * rank + row), t_end = WIN ? (min(p.M, mt * BM + BM) - 1) / p.H : 0;
        bool owed = false;  // LOOP: the last unit's output may still be read from shared memory
        auto pay = [&]() {
            if (!LOOP || !owed) return;
            if (lane == 0) {
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                mbar_arrive(bar(C::B_EFREE));
            }
            __syncwarp();
            owed = false;
        };
        do {
            peek();
            // this row's query token and its mask
            const int mg = mt * BM + RM * rank + row;
            const bool vrow = mg < p.M;
            const int nt = p.T * tpl;  // query tokens of the request
            const int t = t_row + list % tpl, draft = L - nt;
            uint64_t tree = 0;
            if (p.tree) {
                tree = p.tree[(size_t)(list / tpl) * nt + t];
                if (nt < 64) tree &= (1ull << nt) - 1;
            }
            // WIN: the row's first position, and the last of its CTA pair's rows' first ones
            auto from = [&](int at) { return (int)max((long long)draft + at - p.window + 1, 0ll); };
            const int low = WIN ? from(p.tree ? __popcll(tree) - 1 : t) : 0;
            const int low_max = WIN ? from(p.tree ? nt - 1 : t_end) : 0;
            float m2 = -INFINITY, l = 0.f;
            float cref = 0.f, fac = 0.f;  // FP8: the scales' reference, a power of two, and 2^10 over it
            const uint32_t wm = base + C::OFF_WM + 4u * (uint32_t)row;
            if (FP8 && tid < RM) st_shared_f1(wm, 0.f);  // read behind a barrier
            const float row_scale = p.scale_log2 * q_back;
            for (int j = 0; j < nsteps; ++j) {
                const int gj = g0 + j, ti = gj % NTI;
                float s[KT];
                const uint32_t sc_at = base + C::OFF_SC + ti * 512 + kh * 256 + hf * 128;
                if (ok)
                    ok = __all_sync(0xffffffffu, mbar_wait_inline(bar((FP8 ? C::B_TREADY : C::B_TFULL) + ti), (uint32_t)(gj / NTI) & 1u) &&
                                                     mbar_wait_inline(bar(C::B_SFULL), (uint32_t)gj & 1u));
                if (ok) {
                    tc_fence_after();
                    uint32_t ra[32];
                    HS_TMEM_LD32(tmem + lane_off + TM_S + 32u * hf, ra);
                    HS_TMEM_WAIT_LD32(ra);
#pragma unroll
                    for (int e = 0; e < KT; e += 4) {
                        float4 f = FP8 ? ld_shared_f4(sc_at + 4 * e) : make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[e + i] = __uint_as_float(ra[e + i]);
                        if (FP8) {
                            // the two scales first: the codes' sum, up to 2^27, times a large
                            // row's alone may be beyond f32 where the score is not
                            mul2(f.x, f.y, row_scale, row_scale);
                            mul2(f.z, f.w, row_scale, row_scale);
                        }
                        mul2(s[e], s[e + 1], f.x, f.y);
                        mul2(s[e + 2], s[e + 3], f.z, f.w);
                    }
                }
                tc_fence_before();
                if (LOOP || j + 1 < nsteps) arrive_lead(lead(C::B_SFREE));  // S_{j+1} may be written
                if (j == 0) pay();
                const int pg = ok ? (int)ld_shared_b32(base + C::OFF_PG + 4 * (2 * ti + kh)) : -1;
                // the keys that this row sees, as bits
                const int d = draft - max(pg, 0) * kPage;  // the first query token's position in the page
                // WIN: some row's window may begin in the page
                const bool head = WIN && pg >= 0 && low_max > pg * kPage && p.n_sink - kPage < pg * kPage;
                const bool tail = (pg >= 0 && d < kPage) || head;  // some row may not see some key
                float tmax = -INFINITY, cmax = 0.f;
                uint32_t mine = ~0u;
                if (pg < 0) {
                    mine = 0;
                } else if (tail) {
                    uint64_t seen;
                    if (p.tree) {
                        if (WIN && d >= 64)
                            seen = ~0ull;
                        else if (d >= 0)
                            seen = ((1ull << d) - 1) | (tree << d);
                        else
                            seen = d > -64 ? tree >> -d : 0ull;
                    } else {
                        const int n = d + t + 1;
                        seen = n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1);
                    }
                    if (WIN && head) {
                        const int a = low - pg * kPage, n = p.n_sink - pg * kPage;
                        const uint64_t on = a >= 64 ? 0ull : (a <= 0 ? ~0ull : ~0ull << a);
                        seen &= on | (n <= 0 ? 0ull : (1ull << n) - 1);  // n is below 64 here
                    }
                    mine = (uint32_t)(seen >> (KT * hf));
                }
                const bool hide = !__all_sync(0xffffffffu, mine == ~0u);
                // BF16: a key that holds an infinity or NaN has no finite score, with any query
                bool odd = false;
                if (!FP8 && ok && tail) {
                    float z0 = 0.f, z1 = 0.f;
#pragma unroll
                    for (int e = 0; e < KT; e += 2) zeros_of(z0, z1, s[e], s[e + 1]);
                    odd = !(z0 + z1 == 0.f);
                }
                if (ok) {
                    if (hide) {
#pragma unroll
                        for (int e = 0; e < KT; ++e) s[e] = (mine >> e) & 1u ? s[e] : -INFINITY;
                    }
                    float mx[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        mx[e] = max3(s[e], s[e + 4], s[e + 8]);
                        mx[e] = max3(mx[e], s[e + 12], s[e + 16]);
                        mx[e] = max3(mx[e], s[e + 20], s[e + 24]);
                        mx[e] = fmaxf(mx[e], s[e + 28]);
                    }
                    tmax = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                    if (FP8) {
                        cmax = ld_shared_f1(base + C::OFF_SP + 4 * (4 * ti + 2 * kh + hf));
                        if (hide) {  // a hidden row's scale may be anything
                            cmax = 0.f;
#pragma unroll
                            for (int e = 0; e < KT; e += 4) {
                                const float4 f = ld_shared_f4(sc_at + 4 * e);
                                cmax = fmaxf(cmax, (mine >> e) & 1u ? fabsf(f.x) : 0.f);
                                cmax = fmaxf(cmax, (mine >> (e + 1)) & 1u ? fabsf(f.y) : 0.f);
                                cmax = fmaxf(cmax, (mine >> (e + 2)) & 1u ? fabsf(f.z) : 0.f);
                                cmax = fmaxf(cmax, (mine >> (e + 3)) & 1u ? fabsf(f.w) : 0.f);
                            }
                        }
                    }
                }
                // A row's four threads share its references: where some row of the CTA may
                // outgrow its own, the rows' four maxima meet in shared memory.
                float alpha = 1.f;
                auto outgrown = [](float x, float ref) { return x > ref + TAU2<FP8> || (ref == -INFINITY && x != -INFINITY); };
                const bool grow = any_softmax(outgrown(tmax, m2) || (FP8 && cmax > 2.f * cref) || odd);
                if (grow) {
                    if (!FP8) odd = any_softmax(odd);  // either half of the keys
                    st_shared_f1(xm + 4 * tid, tmax);
                    if (FP8) st_shared_f1(xm + 4 * (32 * NSW + tid), cmax);
                    named_bar_sync(1, 32 * NSW);
                    auto of_row = [&](int o) {
                        return fmaxf(fmaxf(ld_shared_f1(xm_row(o)), ld_shared_f1(xm_row(o + 64))),
                                     fmaxf(ld_shared_f1(xm_row(o + 128)), ld_shared_f1(xm_row(o + 192))));
                    };
                    const float tall = of_row(0), call = FP8 ? of_row(32 * NSW) : 0.f;
                    named_bar_sync(1, 32 * NSW);  // read before the next writes
                    if (outgrown(tall, m2)) {
                        alpha = exp2f(m2 - tall);  // 0 where the row had seen nothing
                        l *= alpha;
                        m2 = tall;
                    }
                    if (FP8) {
                        float w = 0.f;  // the largest weight times scale (NaN drops out)
                        if (ok) {
                            const float mneg = m2 == -INFINITY ? 0.f : -m2;
#pragma unroll
                            for (int e = 0; e < KT; e += 4) {
                                const float4 f = ld_shared_f4(sc_at + 4 * e);
                                w = max3(w, ex2(s[e] + mneg) * fabsf(f.x), ex2(s[e + 1] + mneg) * fabsf(f.y));
                                w = max3(w, ex2(s[e + 2] + mneg) * fabsf(f.z), ex2(s[e + 3] + mneg) * fabsf(f.w));
                            }
                        }
                        st_shared_f1(xm + 4 * tid, w);
                        named_bar_sync(1, 32 * NSW);
                        const float most = fmaxf(of_row(0), ld_shared_f1(wm) * alpha);
                        named_bar_sync(1, 32 * NSW);
                        if (hf == 0 && kh == 0) st_shared_f1(wm, most);
                        const float want = fminf(fmaxf(call, most), C_MOST * most);
                        if (want > 2.f * cref || cref > C_MOST * most) {
                            // at least 2^-107: its inverse, and the epilogue's factor, are normal
                            const uint32_t e = max(__float_as_uint(want) >> 23, 20u);
                            fac = __uint_as_float((254u + P_EXP - e) << 23);
                            alpha = alpha * cref * fac * (1.f / (1 << P_EXP));
                            cref = __uint_as_float(e << 23);
                        }
                    }
                }
                uint32_t pk[KT / 2];
                if (ok) {
                    const float mneg = m2 == -INFINITY ? 0.f : -m2;
                    float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
                    for (int e = 0; e < KT; e += 4) {
                        float a0 = s[e], a1 = s[e + 1], a2 = s[e + 2], a3 = s[e + 3];
                        add2(a0, a1, mneg, mneg);
                        add2(a2, a3, mneg, mneg);
                        a0 = ex2(a0);
                        a1 = ex2(a1);
                        a2 = ex2(a2);
                        a3 = ex2(a3);
                        add2(l0, l1, a0, a1);
                        add2(l2, l3, a2, a3);
                        if (FP8) {
                            float4 f = ld_shared_f4(sc_at + 4 * e);
                            mul2(f.x, f.y, fac, fac);
                            mul2(f.z, f.w, fac, fac);
                            mul2(a0, a1, f.x, f.y);
                            mul2(a2, a3, f.z, f.w);
                            pk[e / 2] = pack_f16(a0, a1);
                            pk[e / 2 + 1] = pack_f16(a2, a3);
                        } else {
                            pk[e / 2] = pack_bf16(a0, a1);
                            pk[e / 2 + 1] = pack_bf16(a2, a3);
                        }
                    }
                    l += (l0 + l1) + (l2 + l3);
                    if (FP8 && hide) {
                        // a hidden row's scale may be NaN
#pragma unroll
                        for (int e = 0; e < KT / 2; ++e)
                            pk[e] &= ((mine >> (2 * e)) & 1u ? 0xffffu : 0u) | ((mine >> (2 * e + 1)) & 1u ? 0xffff0000u : 0u);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_TFREE + ti));
                // P and O are free once the previous PV is done; BF16: this CTA's V has
                // landed (FP8: its converters tell the MMA issuer themselves)
                if (ok && j > 0) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_PVDONE), (uint32_t)(gj - 1) & 1u));
                if (ok && !FP8)
                    ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_VFULL + gj % C::NV), (uint32_t)(gj / C::NV) & 1u));
                if (ok) {
                    tc_fence_after();
                    const uint32_t pr = base + C::OFF_P + kh * CH + row * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared_v4(pr + (((c + 4 * hf) ^ (row & 7)) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                    if (!FP8 && tail && odd) {
                        // A row that some query does not see may hold infinities or
                        // NaN, and 0 x NaN would reach that query's sum: in V they
                        // become zeros (a query that does see them has them in its
                        // scores). The page's 32 KB, by its 128 threads, where a score says so
                        // (on every page that some query does not see all of, 4 of the 19 of
                        // a window of 1,024, 2 x 1,999 tokens of 16 heads took 206 us instead of 145).
                        const uint32_t v0 = base + C::OFF_V + (gj % C::NV) * 2 * NVC * CH + kh * NVC * CH + (row + 64 * hf) * 16;
#pragma unroll 4
                        for (int u = 0; u < 16; ++u) {
                            const uint4 v = ld_shared_v4(v0 + 2048 * u);
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
                    }
                    fence_proxy_async();
                    if (grow && j > 0 && __any_sync(0xffffffffu, alpha != 1.f))
                        rescale_o(tmem + lane_off + TM_O + 128u * hf, alpha);
                }
                tc_fence_before();
                arrive_lead(lead(C::B_PFULL));
            }
            // LOOP: the next unit's Q into tensor memory while the last PV runs, so that its first
            // scores are multiplied during this unit's epilogue
            const int g1 = g0 + nsteps;
            pay();
            if (LOOP && nx.there) {
                look();
                t_row = token_of(nx.mt * BM + RM * rank + row);
                t_end = (min(p.M, nx.mt * BM + BM) - 1) / p.H;
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_QFULL), (uint32_t)(it + 1) & 1u));
                if (ok) {
#pragma unroll 1
                    for (int i = hf; i < NQT; i += 2) {
                        uint32_t w[32];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const uint4 v = ld_shared_v4(base + C::OFF_V + (g1 % C::NV) * 2 * NVC * CH + i * CH + row * 128 + ((u ^ (row & 7)) << 4));
                            w[4 * u] = v.x;
                            w[4 * u + 1] = v.y;
                            w[4 * u + 2] = v.z;
                            w[4 * u + 3] = v.w;
                        }
                        HS_TMEM_ST32(tmem + lane_off + TM_Q + 32u * i, w);
                    }
                    tmem_wait_st();
                }
                q_moved(nx.end > 0);
            }
            if (ok && nsteps > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_PVDONE), (uint32_t)(g1 - 1) & 1u));
                tc_fence_after();
            }
            if (!ok && lane == 0) fail();
            __syncwarp();
            if (p.inside) cluster_arrive_relaxed();  // what this warp needed of this CTA's memory is used
            // The row's sum over its four threads' keys. LOOP: the last unit's have been read: before a unit's
            // steps its barriers say so, a unit without steps has this one.
            if (LOOP && nsteps == 0) named_bar_sync(1, 32 * NSW);
            st_shared_f1(xm + 4 * tid, l);
            named_bar_sync(1, 32 * NSW);
            l = (ld_shared_f1(xm_row(0)) + ld_shared_f1(xm_row(64))) + (ld_shared_f1(xm_row(128)) + ld_shared_f1(xm_row(192)));
            // rows that see nothing: out 0, lse -inf
            const float inv = l == 0.f ? 0.f : __fdividef(FP8 ? cref * (1.f / (1 << P_EXP)) : 1.f, l);
            const bool one = nsplit == 1;
            // The columns that the other split joins go there as they are staged, once all
            // CTAs are done with the memory they land in (where nothing was computed, what
            // is sent is not used).
            const uint32_t other = crank ^ 2u;
            uint32_t theirs = 0;
            if (p.inside) {
                cluster_wait();
                theirs = cluster_address(bar(C::B_JOIN), other);
            }
            if (p.inside || (ok && (one || nsteps > 0))) {
                // O / l through shared memory, idle by now, in 32-row boxes of 128
                // swizzled bytes per row: this thread's value columns are
                // 256 hf + 128 kh + (0..127). Rows past M are clipped by the map.
                const int wr = wq & 1;  // which 32 rows
                // LOOP: the buffer that the next unit's Q and first V are not in
                const uint32_t stage = base + C::OFF_V + (LOOP ? ((g1 + 1) % C::NV) * 2 * NVC * CH : 0);
                const uint32_t st0 = stage + wr * 4096 + (uint32_t)(row & 31) * 128u;
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t o[32];
                    if (nsteps > 0) {
                        HS_TMEM_LD32(tmem + lane_off + TM_O + 128 * hf + 32 * cc, o);
                        HS_TMEM_WAIT_LD32(o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    const int col = 256 * hf + 128 * kh + 32 * cc;
                    if (one) {
                        const uint32_t at = st0 + (uint32_t)(col >> 6) * 8192u;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack_bf16(__uint_as_float(o[8 * u + 2 * e]) * inv,
                                                 __uint_as_float(o[8 * u + 2 * e + 1]) * inv);
                            const int c = ((col & 32) >> 3) + u;
                            st_shared_v4(at + (uint32_t)((c ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        // partials stay f32: a third rounding to BF16 would show next to
                        // those of P and of the output
                        const uint32_t at = st0 + (uint32_t)(col >> 5) * 8192u;
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            st_shared_v4(at + (uint32_t)((u ^ (row & 7)) << 4), __float_as_uint(__uint_as_float(o[4 * u]) * inv),
                                         __float_as_uint(__uint_as_float(o[4 * u + 1]) * inv),
                                         __float_as_uint(__uint_as_float(o[4 * u + 2]) * inv),
                                         __float_as_uint(__uint_as_float(o[4 * u + 3]) * inv));
                        if (p.inside && hf != split) {
                            fence_proxy_async();
                            __syncwarp();
                            const int box = 4 * kh + cc;
                            if (lane == 0)
                                bulk_push(cluster_address(base + C::join_box(box) + wr * 4096, other),
                                          base + C::OFF_V + (uint32_t)(8 * hf + box) * 8192u + wr * 4096, 4096, theirs);
                        }
                    }
                    if (!p.inside && (!one || (cc & 1))) {  // a box is staged: its store runs behind the next one's
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) {
                            const int box = one ? col >> 6 : col >> 5;
                            tma_store_3d(one ? &tm_o : &tm_w, stage + (uint32_t)box * 8192u + wr * 4096,
                                         one ? 64 * box : 32 * box, mt * BM + RM * rank + 32 * wr,
                                         one ? list : split * p.ws_lists + list - p.ws_list0);
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                    }
                }
                // the stores have read shared memory before the CTA may end
                if (!LOOP && lane == 0 && !p.inside) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
            }
            if (kh == 0 && hf == 0 && (vrow || p.inside)) {
                const float lse = (!ok || l == 0.f) ? -INFINITY : (m2 + __log2f(l)) * 0.69314718055994531f;
                if (one)
                    p.lse[(size_t)list * p.M + mg] = lse;
                else if (!p.inside)
                    p.ws_lse[((size_t)split * p.ws_lists + list - p.ws_list0) * p.M + mg] = lse;
                else
                    st_shared_f1(base + C::OFF_P + 4 * row, lse);  // P is done with
            }
            owed = LOOP;
            if (p.inside && kh == 0 && hf == 0) {
                fence_proxy_async();
                __syncwarp();
                const int wr = wq & 1;
                if (lane == 0)
                    bulk_push(cluster_address(base + C::OFF_P + 1024 + wr * 128, other), base + C::OFF_P + wr * 128, 128, theirs);
                __syncwarp();
            }
        } while (enter());
        pay();
    } else if (FP8 && warp >= 4 + NSW) {
        // ------------------------------------------------------------ converters
        // Half of V's columns at a time; the next half's codes are loaded while its buffer
        // is still read.
        const int tid = threadIdx.x & 127;
        constexpr int BY = NCW / 4;
        // V's space held the staged Q
        bool ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_QDONE), 0));
        constexpr int G = C::GV;
        static_assert(!FP8 || (NVC == G && C::NCV % 2 == 0 && NK % C::GK == 0), "groups of chunks");
        uint4 w[G][2];
        auto load = [&](int u) {
            const int cs = u % C::RV;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_CFULL + cs), (uint32_t)(u / C::RV) & 1u));
            const uint32_t src = base + C::OFF_C + cs * G * CCH + 16 * tid;
            if (ok) {
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    w[g][0] = ld_shared_v4(src + g * CCH);
                    w[g][1] = ld_shared_v4(src + g * CCH + 2048);
                }
            }
        };
        const int u0 = (warp - 4 - NSW) >> 2;
        if (nsteps > 0) load(u0);
#pragma unroll 1
        for (int u = u0; u < 2 * nsteps; u += BY) {
            const int half = u & 1;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_VFREE + half), ((uint32_t)(u >> 1) & 1u) ^ 1u));
            if (ok) {
                const uint32_t dst = base + C::OFF_V + half * 2 * CH + (tid >> 2) * 128;
                const int key = (tid >> 2) & 7, part = 2 * (tid & 3);  // rows key and key + 32: the same swizzle
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // two chunks of the first page, two of the second
                        const uint32_t at = dst + ((g >> 1) * NVC + (g & 1)) * CH + k * 4096;
                        uint32_t o[8];
                        e4m3x4_to_f16(w[g][k].x, o[0], o[1]);
                        e4m3x4_to_f16(w[g][k].y, o[2], o[3]);
                        e4m3x4_to_f16(w[g][k].z, o[4], o[5]);
                        e4m3x4_to_f16(w[g][k].w, o[6], o[7]);
                        st_shared_v4(at + ((part ^ key) << 4), o[0], o[1], o[2], o[3]);
                        st_shared_v4(at + (((part + 1) ^ key) << 4), o[4], o[5], o[6], o[7]);
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_CFREE + u % C::RV));
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(lead(C::B_VFULL + half));
            if (u + BY < 2 * nsteps) load(u + BY);
        }
        if (!ok && lane == 0) fail();
    }

    if (p.inside) {
        // Each CTA joins half the columns of its rows, its own split's with the other's,
        // w_s = exp(lse_s - max) / sum. No workspace is written or read and no second
        // grid waits.
        if (warp < 4 || warp >= 4 + NSW) {
            __syncwarp();
            cluster_arrive_relaxed();
            cluster_wait();
        }
        bool ok = __all_sync(0xffffffffu, mbar_wait_inline(bar(C::B_JOIN), 0));
        __syncthreads();
        if (!ok && lane == 0) fail();
        __syncwarp();
        // What was sent has been read, and nothing more comes: the others may end once
        // this CTA has come here.
        cluster_arrive_last(misc[1] != 0);
        const float *lses = reinterpret_cast<const float *>(smem + C::OFF_P);
        float *wts = reinterpret_cast<float *>(smem + C::OFF_P + 2048);  // [rows]: own, the other's
        if (threadIdx.x < RM) {
            const int row = threadIdx.x, mg = mt * BM + RM * rank + row;
            const float mine = lses[row], theirs = lses[256 + row];
            const bool nan = mine != mine || theirs != theirs;
            const float mx = fmaxf(mine, theirs);
            const float wm = mine == -INFINITY ? 0.f : ex2((mine - mx) * 1.4426950408889634f);
            const float wt = theirs == -INFINITY ? 0.f : ex2((theirs - mx) * 1.4426950408889634f);
            const float sum = wm + wt;
            const float inv = nan ? __uint_as_float(0x7fc00000u) : (sum > 0.f ? __fdividef(1.f, sum) : 0.f);
            wts[2 * row] = wm * inv;
            wts[2 * row + 1] = wt * inv;
            if (split == 0 && mg < p.M)
                p.lse[(size_t)list * p.M + mg] = nan ? inv : (sum > 0.f ? mx + __logf(sum) : -INFINITY);
        }
        __syncthreads();
#pragma unroll 4
        for (int i = threadIdx.x; i < RM * 64; i += C::THREADS) {  // four columns each
            const int row = i >> 6, box = (i >> 3) & 7, mg = mt * BM + RM * rank + row;
            if (mg >= p.M) continue;
            const uint32_t at = (uint32_t)((row >> 5) * 4096 + (row & 31) * 128 + (((i & 7) ^ (row & 7)) << 4));
            const float wm = wts[2 * row], wt = wts[2 * row + 1];
            float4 m = make_float4(0.f, 0.f, 0.f, 0.f), t = m;
            // a weight of 0: that split saw nothing and wrote nothing, or does not count
            if (wm != 0.f) m = ld_shared_f4(base + C::OFF_V + (8 * split + box) * 8192 + at);
            if (wt != 0.f) t = ld_shared_f4(base + C::join_box(box) + at);
            *reinterpret_cast<uint2 *>(p.out + ((size_t)list * p.M + mg) * 512 + 256 * split + 4 * (i & 63)) =
                make_uint2(pack_bf16(m.x * wm + t.x * wt, m.y * wm + t.y * wt),
                           pack_bf16(m.z * wm + t.z * wt, m.w * wm + t.w * wt));
        }
    }
    tc_fence_before();
    __syncthreads();
    // No CTA leaves while the other's MMAs or arrives may reach it. Every arrive on the
    // other CTA's barriers is one that it waits for (none is made for a step or a slot
    // that does not come), so none is on its way any more and the barrier need not
    // release; after a wait that gave up it does.
    if (!p.inside) cluster_arrive_last(misc[1] != 0);
    cluster_wait();
    tc_fence_after();
    if (warp == 2) tmem_dealloc2(tmem, 512);
}

// Joins the splits: out = sum_s w_s O_s / sum_s w_s, w_s = exp(lse_s - max), in a
// fixed order, for the rows from `skip` on of the partials' space. Four columns of a row per
// thread, JU splits at a time, whose loads are all issued before the first is used;
// between them the sums move to the larger maximum. JU: 2, 4 or 8, the smallest that
// takes all splits at once (8 splits of 112 rows: 4 and 16 at a time made a call 0.15 and
// 1.2 us longer, a block per row with four groups of threads 0.6 us; two splits of
// 32,768 rows: 8 at a time, whose registers leave fewer threads, 20 us longer than 2).
template <int JU>
__global__ void __launch_bounds__(256)
join_kernel(const float *ws_o, const float *ws_lse, int nsplit, int rows, int skip, __nv_bfloat16 *out, float *lse) {
    grid_dep_wait();  // the splits' partials
    grid_dep_launch();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = (i >> 7) + skip;
    const int c = (int)(i & 127) * 4;
    if (row >= rows) return;
    float mx = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    bool nan = false;
#pragma unroll 1
    for (int s0 = 0; s0 < nsplit; s0 += JU) {
        float v[JU];
        float4 o[JU];
#pragma unroll
        for (int s = 0; s < JU; ++s) {
            v[s] = -INFINITY;
            o[s] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s0 + s < nsplit) {
                v[s] = ws_lse[(size_t)(s0 + s) * rows + row];
                o[s] = __ldcs(reinterpret_cast<const float4 *>(ws_o + ((size_t)(s0 + s) * rows + row) * 512 + c));
            }
        }
        float top = mx;
#pragma unroll
        for (int s = 0; s < JU; ++s) {
            nan = nan || v[s] != v[s];
            top = fmaxf(top, v[s]);
        }
        if (top == -INFINITY) continue;
        const float back = exp2f((mx - top) * 1.4426950408889634f);  // 0 where nothing was seen before
        mx = top;
        sum *= back;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] *= back;
#pragma unroll
        for (int s = 0; s < JU; ++s)
            if (v[s] != -INFINITY) {  // otherwise that split's partial was not written
                const float w = exp2f((v[s] - mx) * 1.4426950408889634f);
                sum += w;
                acc[0] = fmaf(w, o[s].x, acc[0]);
                acc[1] = fmaf(w, o[s].y, acc[1]);
                acc[2] = fmaf(w, o[s].z, acc[2]);
                acc[3] = fmaf(w, o[s].w, acc[3]);
            }
    }
    const float inv = nan ? __uint_as_float(0x7fc00000u) : (sum > 0.f ? __fdividef(1.f, sum) : 0.f);
    *reinterpret_cast<uint2 *>(out + row * 512 + c) =
        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    if (c == 0) lse[row] = nan ? inv : (sum > 0.f ? mx + __logf(sum) : -INFINITY);
}

// ---------------------------------------------------------------- host side
struct PagePlan {
    int M, mtiles, nsplit, n_full, list0;
    double us;  // the model's time
    size_t ws_o_bytes, ws_bytes;
};

int64_t pairs_at_once() { return sm_count() / 2 > 0 ? sm_count() / 2 : 1; }

// A model of the launch's time, in us: two pages take a pair of CTAs about 1.6,
// their start and epilogue 7.
constexpr double US_STEP = 1.6, US_ENDS = 7.0;

// Splits of a list of N pages joined through the workspace by a second grid: the
// count that the model makes shortest; the join is 3.5 us and about 5 MB of
// partials written and read per us. Where there are more units than pairs of CTAs at
// once, those of the last, partly filled round may be split by themselves
// (8 x 32 tokens of 128 heads, 256 units on 76 pairs, 16,384 rows: 732 us a call
// against 757 with all units in two).
PagePlan page_plan(int64_t lists, int64_t T, int64_t H, int64_t N) {
    PagePlan pl{};
    pl.M = (int)(T * H);
    pl.mtiles = (pl.M + BM - 1) / BM;
    const int64_t pairs = pairs_at_once(), units = lists * pl.mtiles;
    const int64_t steps = (N + 1) / 2, most = steps < 128 ? steps : 128;
    pl.us = 1e300;
    pl.nsplit = 1;
    auto rounds = [&](int64_t u, int64_t ns) {
        return (double)((u * ns + pairs - 1) / pairs) * ((double)((steps + ns - 1) / ns) * US_STEP + US_ENDS);
    };
    auto join = [&](int64_t rows, int64_t ns) { return ns > 1 ? 3.5 + (double)ns * rows * 512 * 8 / 5e6 : 0.0; };
    auto consider = [&](double t, int64_t full, int64_t ns) {
        if (t >= pl.us * 0.98) return;
        pl.us = t;
        pl.nsplit = (int)ns;
        pl.n_full = (int)full;
    };
    for (int64_t ns = 1; ns <= most || ns == 1; ++ns) {
        consider(rounds(units, ns) + join(lists * pl.M, ns), 0, ns);
        if (units * ns > 8 * pairs) break;
    }
    const int64_t rest = units % pairs;
    if (units > pairs && rest)
        for (int64_t ns = 2; ns <= most && rest * ns <= 8 * pairs; ++ns)
            consider(rounds(units - rest, 1) + rounds(rest, ns) + join(rest * BM, ns), units - rest, ns);
    pl.list0 = pl.n_full / pl.mtiles;
    if (pl.nsplit > 1) {
        const size_t rows = (size_t)pl.nsplit * (lists - pl.list0) * pl.M;
        pl.ws_o_bytes = (rows * 512 * sizeof(float) + 255) & ~size_t(255);
        pl.ws_bytes = pl.ws_o_bytes + ((rows * sizeof(float) + 255) & ~size_t(255));
    }
    return pl;
}

// How many clusters of two pairs of CTAs the device holds at once.
template <bool FP8, bool WIN>
int clusters_of_four(int dev) {
    static std::atomic<int> cached[64];
    int n = cached[dev].load(std::memory_order_acquire);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(4, 1, 1024);
        cfg.blockDim = dim3(PCfg<FP8>::THREADS, 1, 1);
        cfg.dynamicSmemBytes = PCfg<FP8>::SMEM_ALLOC;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 4;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, page_decode_kernel<FP8, WIN, false>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        n = n > 0 ? n : -1;
        cached[dev].store(n, std::memory_order_release);
    }
    return n;
}

template <bool FP8, bool WIN, bool LOOP>
hs_status launch_pages(int dev, cudaStream_t s, const CUtensorMap &tq, const CUtensorMap &k1,
                       const CUtensorMap &k2, int64_t units, const void *d_out, void *ws, const PagePlan &pl, PageParams p) {
    static std::atomic<int> state[64];
    if (dev < 0 || dev >= 64) return HS_ERR_UNSUPPORTED;
    if (state[dev].load(std::memory_order_acquire) != 1) {
        HS_CUDA_TRY(cudaFuncSetAttribute(page_decode_kernel<FP8, WIN, LOOP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PCfg<FP8>::SMEM_ALLOC));
        state[dev].store(1, std::memory_order_release);
    }
    // Two splits joined inside a cluster, where all clusters run at once and the model
    // says so: 1.5 us instead of the second grid's 3.5 and the partials' bytes
    // (32 lists of 2,048 rows, 128 heads: 28.2 against 32.0 us). Four splits in a cluster of
    // eight CTAs were slower than eight splits and the second grid.
    if (pl.nsplit > 1) {
        const int64_t steps = ((p.N < 1 ? p.max_pages : p.N) + 1) / 2;
        const double t = (double)((steps + 1) / 2) * US_STEP + US_ENDS + 1.5;
        if (steps >= 2 && t < pl.us && units <= clusters_of_four<FP8, WIN>(dev)) p.inside = p.nsplit = 2;
    }
    if (p.inside) p.n_full = 0;
    const int64_t lists = (int64_t)units / pl.mtiles;
    // the output (units of one split), and the splits' f32 partials
    CUtensorMap to, tw;
    const bool direct = p.nsplit == 1 || p.n_full > 0, split = p.nsplit > 1 && !p.inside;
    if (direct && !make_map(&to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_out, 512, pl.M, lists, 1024, 64, 32,
                            CU_TENSOR_MAP_SWIZZLE_128B))
        return HS_ERR_CUDA;
    if (split && !make_map(&tw, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws, 512, pl.M, (uint64_t)p.ws_lists * p.nsplit, 2048, 32,
                           32, CU_TENSOR_MAP_SWIZZLE_128B))
        return HS_ERR_CUDA;
    if (!direct) to = split ? tw : tq;  // not used
    if (!split) tw = to;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (p.n_full + (units - p.n_full) * p.nsplit)), 1, 1);
    if (LOOP) {
        cfg.gridDim.x = (unsigned)(2 * pairs_at_once());
        p.units = (int)units;
    }
    cfg.blockDim = dim3(PCfg<FP8>::THREADS, 1, 1);
    cfg.dynamicSmemBytes = PCfg<FP8>::SMEM_ALLOC;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.inside ? 2 * p.inside : 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, page_decode_kernel<FP8, WIN, LOOP>, tq, k1, k2, to, tw, p) != cudaSuccess) return HS_ERR_CUDA;
    if (!split) return HS_OK;
    const int n = p.ws_lists * pl.M, skip = (p.n_full % pl.mtiles) * BM;
    cudaLaunchConfig_t cc = {};
    cc.gridDim = dim3((unsigned)(((int64_t)(n - skip) * 128 + 255) / 256), 1, 1);
    cc.blockDim = dim3(256, 1, 1);
    cc.stream = s;
    cudaLaunchAttribute ca[1];
    ca[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ca[0].val.programmaticStreamSerializationAllowed = 1;
    cc.attrs = ca;
    cc.numAttrs = 1;
    auto join = p.nsplit <= 2 ? join_kernel<2> : (p.nsplit <= 4 ? join_kernel<4> : join_kernel<8>);
    const size_t row0 = (size_t)p.ws_list0 * pl.M;
    return cudaLaunchKernelEx(&cc, join, (const float *)ws, (const float *)p.ws_lse, p.nsplit, n, skip,
                              p.out + row0 * 512, p.lse + row0) == cudaSuccess
               ? HS_OK
               : HS_ERR_CUDA;
}

// Sizes that the attention takes: a plan's row counts fit 32 bits.
bool takes(int64_t lists, int64_t T, int64_t H) {
    return lists >= 0 && lists <= 65535 && T >= 1 && T <= 32767 && H >= 1 && T * H <= (int64_t)BM * 65535 &&
           lists * T * H <= INT32_MAX;
}

// The most pages of a window's unit: those of the window of the unit's first token and of the
// tokens behind it, at the worst alignment, and those of the first positions.
int64_t window_pages(const hs_pool *pool, int64_t T, int64_t H, int64_t window, int64_t n_sink) {
    const int64_t tokens = (BM - 1) / H + 2 < T ? (BM - 1) / H + 2 : T;
    const int64_t n = (window + tokens + 61) / kPage + 1 + (n_sink + kPage - 1) / kPage;
    return n < pool->max_pages ? n : pool->max_pages;
}

// Windows over BF16 rows with two units or more for each pair of CTAs may be taken one after the
// other by a pair, none of them split: the next unit's queries and keys come, and its first
// scores are multiplied, during the last one's end, so that a unit's ends take 4 us instead of 7
// (2 x 1,999 tokens of 16 heads, windows of 1,024: 127 us against 148 with a launch's CTAs for each
// unit). But units are dealt out beforehand, and those of requests of other lengths are not
// evened out: requests of one unit lose about a unit's time, less the more units a request
// has, since its own are alike and go to all pairs. Measured one after the other / each by itself, contexts
// spread over 1 to 8,192: 608 requests of one unit, windows of 512 97-105 / 108-111, of 4,096
// 258-295 / 202-217; 38 of 16, windows of 4,096 192-231 / 150-186; 9 of 63, 95-197 / 115-203.
// Equal contexts of 8,192 and windows of 4,096: 160 requests 216 / 181 (the last 8 units split), 608 592 / 614.
constexpr double US_NEXT = 4.0;

PagePlan window_plan(bool fp8, int64_t lists, int64_t T, int64_t H, int64_t N, bool &loop) {
    const PagePlan each = page_plan(lists, T, H, N);
    const int64_t mtiles = each.mtiles, pairs = pairs_at_once(), units = lists * mtiles;
    const double steps = (double)((N + 1) / 2) * US_STEP, uneven = 1.0 - 2.0 * (double)mtiles / (double)pairs;
    loop = !fp8 && units >= 2 * pairs &&
           (double)((units + pairs - 1) / pairs) * (steps + US_NEXT) + (uneven > 0 ? uneven * steps : 0.0) < each.us;
    if (!loop) return each;
    PagePlan pl{};
    pl.M = each.M;
    pl.mtiles = each.mtiles;
    pl.nsplit = 1;
    return pl;
}

// `lists` lists of T query tokens each; tpl > 1 (with T = 1): lists / tpl
// requests whose tpl tokens each have their own list. window > 0: N pages a unit at most.
hs_status page_entry(hs_pool_t pool, int64_t lists, int32_t T, int32_t tpl, int32_t H, int32_t N,
                     const void *d_q, const int32_t *d_pages, const int32_t *d_req_ids,
                     const uint64_t *d_tree, int32_t window, int32_t n_sink, float sm_scale, void *d_out,
                     float *d_lse, void *d_workspace, size_t ws_bytes, void *stream) {
    if (!pool || !takes(lists, T, H) || N < 0 || (d_tree && (int64_t)T * tpl > 64)) return HS_ERR_INVALID_ARG;
    if (d_pages ? N < 1 : false) return HS_ERR_INVALID_ARG;
    if (lists == 0) return HS_OK;
    if (!d_q || !d_req_ids || !d_out || !d_lse) return HS_ERR_INVALID_ARG;
    if (((uintptr_t)d_q | (uintptr_t)d_out) & 15u) return HS_ERR_INVALID_ARG;
    int dev = -1;
    HS_CUDA_TRY(cudaGetDevice(&dev));
    if (dev != pool->device) return HS_ERR_INVALID_ARG;
    const bool fp8 = pool->cfg.dtype == HS_FP8_E4M3_ROWSCALE;
    bool loop = false;
    const PagePlan pl = window > 0 ? window_plan(fp8, lists, T, H, N, loop) : page_plan(lists, T, H, N < 1 ? pool->max_pages : N);
    if (pl.nsplit > 1 && (!d_workspace || ws_bytes < pl.ws_bytes || ((uintptr_t)d_workspace & 255u)))
        return HS_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap tq;
    const uint64_t rows = (uint64_t)(pool->cfg.n_gpu_blocks + 1) * kPage;
    if (!make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_q, kDim, pl.M, lists, 2 * kDim, 64, RM,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return HS_ERR_CUDA;
    // the pool's own maps, once
    static_assert(sizeof(pool->page_maps[0]) == sizeof(CUtensorMap), "size of a tensor map");
    CUtensorMap *maps = reinterpret_cast<CUtensorMap *>(pool->page_maps);
    if (!pool->page_maps_made) {
        if (!make_page_map(&maps[0], fp8, pool->d_rows, rows, fp8 ? PCfg<true>::GK : 1,
                           fp8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_page_map(&maps[1], fp8, pool->d_rows, rows, 2,
                           fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
            return HS_ERR_CUDA;
        pool->page_maps_made = true;
    }
    PageParams p{};
    p.pages = d_pages;
    p.req = d_req_ids;
    p.ctx = pool->d_ctx;
    p.table = reinterpret_cast<const int2 *>(pool->d_page);
    p.tree = d_tree;
    p.scales = pool->d_scales;
    p.out = static_cast<__nv_bfloat16 *>(d_out);
    p.lse = d_lse;
    p.ws_lse = pl.nsplit > 1 ? reinterpret_cast<float *>(static_cast<uint8_t *>(d_workspace) + pl.ws_o_bytes)
                             : nullptr;
    p.err = pool->d_err;
    p.T = T;
    p.H = H;
    p.N = N;
    p.M = pl.M;
    p.mtiles = pl.mtiles;
    p.nsplit = pl.nsplit;
    p.n_full = pl.n_full;
    p.ws_list0 = pl.list0;
    p.ws_lists = (int)lists - pl.list0;
    p.max_req = pool->cfg.max_requests;
    p.max_pages = pool->max_pages;
    p.max_ctx = pool->cfg.max_ctx;
    p.zero_block = (int)pool->cfg.n_gpu_blocks;
    p.tpl = tpl;
    p.window = window;
    p.q = static_cast<const uint8_t *>(d_q);
    p.n_sink = n_sink;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    const int64_t units = lists * pl.mtiles;
    auto launch = window > 0 ? (fp8 ? launch_pages<true, true, false> : (loop ? launch_pages<false, true, true> : launch_pages<false, true, false>))
                             : (fp8 ? launch_pages<true, false, false> : launch_pages<false, false, false>);
    return launch(dev, s, tq, maps[0], maps[1], units, d_out, d_workspace, pl, p);
}

}  // namespace

extern "C" size_t hs_page_decode_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t N) {
    if (B < 1 || N < 1 || !takes(B, T, H)) return 0;
    return page_plan(B, T, H, N).ws_bytes;
}

extern "C" hs_status hs_page_mla_decode(hs_pool_t pool, int32_t B, int32_t T, int32_t H, int32_t N,
                                        const void *d_q, const int32_t *d_pages, const int32_t *d_req_ids,
                                        const uint64_t *d_tree, float sm_scale, void *d_out, float *d_lse,
                                        void *d_workspace, size_t ws_bytes, void *stream) {
    return page_entry(pool, B, T, 1, H, N, d_q, d_pages, d_req_ids, d_tree, 0, 0, sm_scale, d_out, d_lse,
                      d_workspace, ws_bytes, stream);
}

extern "C" hs_status hs_page_mla_decode_per_token(hs_pool_t pool, int32_t B, int32_t T, int32_t H, int32_t N,
                                                  const void *d_q, const int32_t *d_pages,
                                                  const int32_t *d_req_ids, const uint64_t *d_tree,
                                                  float sm_scale, void *d_out, float *d_lse,
                                                  void *d_workspace, size_t ws_bytes, void *stream) {
    // request b's T lists are lists b*T .. b*T+T-1 of one query token each
    if (B < 0 || T < 1 || (int64_t)B * T > 65535 || !d_pages) return HS_ERR_INVALID_ARG;
    return page_entry(pool, (int64_t)B * T, 1, T, H, N, d_q, d_pages, d_req_ids, d_tree, 0, 0, sm_scale,
                      d_out, d_lse, d_workspace, ws_bytes, stream);
}

extern "C" size_t hs_window_workspace_bytes(hs_pool_t pool, int32_t B, int32_t T, int32_t H, int32_t window,
                                            int32_t n_sink) {
    if (!pool || B < 1 || !takes(B, T, H) || window < 1 || n_sink < 0) return 0;
    bool loop;
    return window_plan(pool->cfg.dtype == HS_FP8_E4M3_ROWSCALE, B, T, H, window_pages(pool, T, H, window, n_sink), loop).ws_bytes;
}

extern "C" hs_status hs_page_mla_decode_window(hs_pool_t pool, int32_t B, int32_t T, int32_t H, int32_t window,
                                               int32_t n_sink, const void *d_q, const int32_t *d_req_ids,
                                               const uint64_t *d_tree, float sm_scale, void *d_out,
                                               float *d_lse, void *d_workspace, size_t ws_bytes, void *stream) {
    if (!pool || !takes(B, T, H) || window < 1 || n_sink < 0) return HS_ERR_INVALID_ARG;
    if (d_tree && T <= 64 && window < T) return HS_ERR_UNSUPPORTED;  // drafted nodes would leave the window
    return page_entry(pool, B, T, 1, H, (int32_t)window_pages(pool, T, H, window, n_sink), d_q, nullptr,
                      d_req_ids, d_tree, window, n_sink, sm_scale, d_out, d_lse, d_workspace, ws_bytes, stream);
}
