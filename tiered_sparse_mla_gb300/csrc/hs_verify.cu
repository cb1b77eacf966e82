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
// Only one row of V values (two where a draft's probabilities refuse a token) is read in full for
// a request, a run of it by each warp of a cluster. 64 requests of 128,000 F32 values, 29 of which
// read two rows: 47.7 MB, 7.2 us at the copy rate, take 17. Two dependent loads say which row it is
// (1.5 us); the rows then come until 12, at about 4.5 TB/s: a warp asks for a batch or two by loads of
// one value each, and adds them up before it asks again; the slowest CTA, the barrier and the search take the
// rest. BF16, half the bytes, takes as long (18.6 with 31 such requests): loads are as many. (The
// whole runs asked into L2 at the start: 19.7 us. Copies of 16 bytes through shared memory, 30 us: twice
// the instructions.)
//
// A search by sums has to add the same way each time. Here a value counts in whole steps of
// 2^-58, what is below them is cut off, and sums are integers: eight values of a lane are cut into
// digits of f32, multiples of 2^-20 (to which adding and taking away 12 rounds a value in [0, 1]),
// then of 2^-41, whose sums of eight are exact, and a rest below 2^-42, which an addition rounded
// down leaves as an integer in the low bits. (Integer shifts, at half
// the rate of additions and twice as many, made 64 requests of 128,000 values 22.7 us.)
// Integer sums saturate at 64, which those of probabilities do not reach.
#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>

#include "hs_internal.cuh"
#include "hs_tc.cuh"

namespace {

constexpr int VT = 256;          // threads per CTA
constexpr int NW = VT / 32;
constexpr int BATCH = 256;       // values that a warp takes at a time
constexpr int UNITS = 16;        // of a warp's run of batches: each lane's sum of each is kept
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
    int T, V, per;  // per: batches in a unit
};

__device__ __forceinline__ uint64_t add_sat(uint64_t a, uint64_t b) {
    const uint64_t s = a + b;
    return s < a ? ~0ull : s;
}
__device__ __forceinline__ uint64_t shuffle64(uint64_t x, int src) {
    return (uint64_t)__shfl_sync(0xffffffffu, (unsigned long long)x, src);
}

// The sum over the lanes up to this one.
__device__ __forceinline__ uint64_t sum_up(uint64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = (uint64_t)__shfl_up_sync(0xffffffffu, (unsigned long long)x, o);
        if (lane >= o) x = add_sat(x, y);
    }
    return x;
}

// A probability's bits: NaN and negative ones are 0, ones above 1 are 1.
__device__ __forceinline__ uint32_t clean(uint32_t b) {
    return b > 0x7f800000u ? 0u : min(b, 0x3f800000u);
}
// In [0, 1]; NaN is 0.
__device__ __forceinline__ float within(float x) {
    float y;
    asm("add.sat.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of f32 in one register pair, and operations on both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(lo), "f"(hi));
    return x;
}
__device__ __forceinline__ float both_of(uint64_t x) {  // their sum
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
    return lo + hi;
}
__device__ __forceinline__ uint64_t plus(uint64_t a, uint64_t b) {
    uint64_t c;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(a), "l"(b));
    return c;
}
__device__ __forceinline__ uint64_t less(uint64_t a, uint64_t b) {  // a - b
    uint64_t c;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(c) : "l"(b), "l"(0xbf800000bf800000ull), "l"(a));
    return c;
}
__device__ __forceinline__ uint64_t plus_down(uint64_t a, uint64_t b) {
    uint64_t c;
    asm("add.rm.f32x2 %0, %1, %2;" : "=l"(c) : "l"(a), "l"(b));
    return c;
}
// Two values' digits: the multiples of 2^-20 and 2^-41, and the rest's whole steps of 2^-58 above
// the bits of 1.5 2^-35, whose last bit is one step.
constexpr uint32_t C3 = 0x2e400000u;
struct Digits {
    uint64_t h, m, l;
};
__device__ __forceinline__ uint32_t steps_of(uint64_t l) { return (uint32_t)l + (uint32_t)(l >> 32); }  // of both values, and twice C3
__device__ __forceinline__ Digits digits_of(uint64_t x) {
    constexpr uint64_t C1 = 0x4140000041400000ull, C2 = 0x36c0000036c00000ull, SIGNS = 0x8000000080000000ull;  // 12, 1.5 2^-18
    Digits d;
    d.h = plus(plus(x, C1), C1 ^ SIGNS);
    x = less(x, d.h);
    d.m = plus(plus(x, C2), C2 ^ SIGNS);
    d.l = plus_down(less(x, d.m), (uint64_t)C3 << 32 | C3);
    return d;
}
// In units of 2^-58, the rest cut off.
__device__ __forceinline__ uint64_t fixed(uint32_t b) {
    const uint32_t top = ((b & 0x7fffffu) | 0x800000u) << 3;  // 2^58 for 1.0, with 32 zeros behind it
    uint64_t r;
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"((uint64_t)top << 32), "r"(127u - (b >> 23)));  // beyond 63: 0
    return r;
}
// A value that is not negative as m 2^e.
__device__ __forceinline__ uint32_t parts(float x, int &e) {
    const uint32_t b = __float_as_uint(x), ex = b >> 23;
    e = (int)max(ex, 1u) - 150;
    return (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
}
// u b 2^eb < p, exactly, for b below 2^60: the integers u's times b and p's times 2^k.
__device__ __forceinline__ bool below(float u, uint64_t b, int eb, float p) {
    int eu, ep;
    const uint64_t mu = parts(u, eu), mp = parts(p, ep), lo = mu * b, hi = __umul64hi(mu, b);
    const int k = min(max(ep - eu - eb, -24), 100);  // further on nothing changes: u's times b is below 2^84
    uint64_t plo, phi = 0;
    if (k <= 0) {
        plo = (mp + (1u << -k) - 1) >> -k;  // rounded up: the other side is a whole number
    } else if (k < 64) {
        plo = mp << k;
        phi = mp >> (64 - k);
    } else {
        plo = 0;
        phi = mp << (k - 64);
    }
    return hi < phi || (hi == phi && lo < plo);
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
__global__ void __launch_bounds__(VT, 4)
verify_kernel(const VerifyParams p) {
    // Once all CTAs of the cluster have come here, each may write to the others' shared memory: a
    // CTA that has not begun has none. The wait is directly before the first such write, behind the
    // row's sums.
    hs::tc::cluster_arrive_relaxed();
    hs::tc::grid_dep_wait();
    hs::tc::grid_dep_launch();
    __shared__ uint64_t sums[NW][UNITS][33];   // of a warp's units, by lane
    __shared__ uint64_t totals[MAXG * NW], s_path;  // of the cluster's warps
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
            u[k] = __uint_as_float(min(clean(__float_as_uint(u[k])), 0x3f7fffffu));  // on bits: arithmetic makes subnormal numbers 0
        }
        auto both = [&](bool lo, bool hi) {
            return (uint64_t)__ballot_sync(0xffffffffu, lo) | (uint64_t)__ballot_sync(0xffffffffu, hi) << 32;
        };
        uint64_t path = 1;
        int end = 0, minus = 0, ngone = 0;
        if (p.draft) {  // a chain: up to the first that has no token or is refused
            int e0, e1;
            const uint32_t q0 = parts(qx[0], e0), q1 = parts(qx[1], e1);
            const bool s0 = tok[0] >= 0 && below(u[0], q0, e0, px[0]);
            const bool s1 = tok[1] >= 0 && below(u[1], q1, e1, px[1]);
            const uint64_t stop = both(lane > 0 && !s0, !s1);  // nodes from T on have no token
            const uint64_t there = both(tok[0] >= 0, tok[1] >= 0);
            const int n = stop ? __ffsll((long long)stop) - 1 : MAXT;
            path = n < 64 ? (1ull << n) - 1 : ~0ull;
            end = n - 1;
            minus = n < 64 && ((there >> n) & 1);
        } else {
            // What each node is held against, all nodes at once: 1 less what its earlier
            // brothers had, each token once.
            uint64_t mine[2] = {fixed(__float_as_uint(px[0])), fixed(__float_as_uint(px[1]))};
            uint64_t left[2] = {1ull << 58, 1ull << 58};
            if (p.tree && T <= 32) {
                // brothers by one vote, and as many rounds as a node has earlier ones
                const uint32_t lower = (1u << lane) - 1u, with = __ballot_sync(0xffffffffu, tok[0] >= 0);
                uint32_t same = __match_any_sync(0xffffffffu, par[0]) & with & lower;
                const uint32_t twin = __match_any_sync(0xffffffffu, (unsigned long long)(uint32_t)par[0] << 32 | (uint32_t)tok[0]) & lower;
                if (tok[0] < 0) same = 0;
                if (tok[0] >= 0 && twin) {  // gone already
                    mine[0] = 0;
                    px[0] = 0.f;
                }
                while (__any_sync(0xffffffffu, same != 0)) {
                    const uint64_t mj = shuffle64(mine[0], same ? __ffs(same) - 1 : 0);
                    if (same) left[0] -= min(left[0], mj);
                    same &= same - 1;
                }
            } else if (p.tree) {
                auto of = [&](int x0, int x1, int j) { return __shfl_sync(0xffffffffu, j < 32 ? x0 : x1, j & 31); };
#pragma unroll 1
                for (int j = 1; j < T; ++j) {
                    const int pj = of(par[0], par[1], j), tj = of(tok[0], tok[1], j);
                    if (tj < 0) continue;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (j < lane + 32 * k && par[k] == pj && tok[k] == tj) {  // gone already
                            mine[k] = 0;
                            px[k] = 0.f;
                        }
                }
#pragma unroll 1
                for (int j = 1; j < T; ++j) {
                    const int pj = of(par[0], par[1], j);
                    const uint64_t mj = shuffle64(j < 32 ? mine[0] : mine[1], j & 31);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (j < lane + 32 * k && par[k] == pj) left[k] -= min(left[k], mj);
                }
            }
            auto stays = [&](int k) { return tok[k] >= 0 && below(u[k], left[k], -58, px[k]); };
            const bool t0 = stays(0), t1 = stays(1);
            for (;;) {  // down the first of each node's children that stays
                const uint64_t kids = both(par[0] == end && t0, par[1] == end && t1);
                if (!kids) break;
                end = __ffsll((long long)kids) - 1;
                path |= 1ull << end;
            }
            const uint64_t out = both(par[0] == end && tok[0] >= 0, par[1] == end && tok[1] >= 0);
            ngone = __popcll(out);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if ((out >> (lane + 32 * k)) & 1) gone[__popcll(out & ((1ull << (lane + 32 * k)) - 1))] = tok[k];
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0 && rank == 0) atomicOr(p.err, HS_DEVERR_INDEX_RANGE);
        if (lane == 0) {
            s_path = path;
            s_row = end;
            s_minus = minus;
            s_gone = ngone;
        }
    }
    __syncthreads();
    const P *row = static_cast<const P *>(p.probs) + ((int64_t)b * T + s_row) * p.ld;
    const P *guess = p.draft && s_minus ? static_cast<const P *>(p.draft) + ((int64_t)b * (T - 1) + s_row) * p.draft_ld : nullptr;
    int ngone = s_gone;
    // this warp's run of the row's units
    const int64_t unit = (int64_t)BATCH * p.per, units = (V + unit - 1) / unit;
    const int me = rank * NW + warp, W = G * NW;
    const int first = (int)(units * me / W), n = (int)(units * (me + 1) / W) - first;
    const int64_t v_first = first * unit;

    for (int attempt = 0;; ++attempt) {
        uint64_t total_lane = 0;
        const int whole = (int)((V - v_first) / BATCH);  // batches that lie inside the row
        auto load = [&](uint32_t (&x)[8], const P *from, int j) {  // batch j of the run
            const P *at = from + v_first + (int64_t)j * BATCH + lane;
            if (j < whole) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = bits_at<P>(at, 32 * e);
            } else {
                const int64_t left = V - (v_first + (int64_t)j * BATCH) - lane;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 32 * e < left ? bits_at<P>(at, 32 * e) : 0u;
            }
        };
        auto leave_out = [&](uint32_t (&x)[8], int j) {  // the refused children's tokens
            const int64_t v0 = v_first + (int64_t)j * BATCH;
#pragma unroll 1
            for (int g = 0; g < ngone; ++g) {
                const int64_t at = gone[g] - v0;
                if (at >= 0 && at < BATCH && (at & 31) == lane) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = (at >> 5) == e ? 0u : x[e];
                }
            }
        };
        // the lane's, at most 8; the digits' signs differ, their sum has none
        auto sum_of = [&](uint64_t high, uint64_t middle, uint32_t low) {
            const int h = __float2int_rn(both_of(high) * 0x1p20f), m = __float2int_rn(both_of(middle) * 0x1p41f);
            return (uint64_t)(((int64_t)h << 38) + ((int64_t)m << 17) + (int32_t)low);
        };
        auto plain = [&](const uint32_t (&x)[8]) {
            uint64_t h = 0, m = 0;
            uint32_t l = 0u - 8u * C3;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const Digits d = digits_of(pair(within(__uint_as_float(x[e])), within(__uint_as_float(x[e + 1]))));
                h = plus(h, d.h);
                m = plus(m, d.m);
                l += steps_of(d.l);
            }
            return sum_of(h, m, l);
        };
        auto beside = [&](const uint32_t (&x)[8], const uint32_t (&y)[8]) {
            uint64_t h = 0, m = 0;
            uint32_t l = 0;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float x0 = within(__uint_as_float(x[e])), x1 = within(__uint_as_float(x[e + 1]));
                const Digits d = digits_of(pair(x0, x1));
                // where the draft's is the larger, nothing is left: the same digits
                const Digits f = digits_of(pair(fminf(within(__uint_as_float(y[e])), x0), fminf(within(__uint_as_float(y[e + 1])), x1)));
                h = less(plus(h, d.h), f.h);
                m = less(plus(m, d.m), f.m);
                l += steps_of(d.l) - steps_of(f.l);
            }
            return sum_of(h, m, l);
        };
        uint32_t x[8], y[8];
        auto keep = [&](int i, uint64_t sum) {
            sums[warp][i][lane] = sum;
            total_lane = add_sat(total_lane, sum);
        };
        if (guess || p.per > 1) {
            int j = 0;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                uint64_t sum = 0;
                int k = p.per;
#pragma unroll 1
                do {
                    load(x, row, j);
                    if (guess) {
                        load(y, guess, j);
                        sum = add_sat(sum, beside(x, y));
                    } else {
                        leave_out(x, j);
                        sum = add_sat(sum, plain(x));
                    }
                    ++j;
                } while (--k > 0);
                keep(i, sum);
            }
        } else {  // two batches at a time
#pragma unroll 1
            for (int i = 0; i < n; i += 2) {
                load(x, row, i);
                if (i + 1 < n) load(y, row, i + 1);
                leave_out(x, i);
                keep(i, plain(x));
                if (i + 1 == n) break;
                leave_out(y, i + 1);
                keep(i + 1, plain(y));
            }
        }
        uint64_t all = total_lane;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) all = add_sat(all, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)all, o));
        if (attempt == 0) hs::cluster_wait();
        if (lane < G) {
            const uint32_t at = hs::dsmem_map(&totals[me], lane);
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(all) : "memory");
        }
        hs::cluster_arrive();
        if (rank == 0 && warp == 1 && attempt == 0) {
            const uint64_t path = s_path;
            const int len = __popcll(path);
            for (int t = lane; t < T; t += 32) {
                if ((path >> t) & 1) p.index[(int64_t)b * T + __popcll(path & ((1ull << t) - 1))] = t;
                if (t >= len) p.index[(int64_t)b * T + t] = -1;
            }
            if (lane == 0) p.count[b] = len;
        }
        const float u0 = p.uniform[(int64_t)b * T];
        hs::cluster_wait();
        // sums of the cluster's warps, two a lane
        const uint64_t t0 = 2 * lane < W ? totals[2 * lane] : 0ull, t1 = 2 * lane + 1 < W ? totals[2 * lane + 1] : 0ull;
        const uint64_t some = sum_up(add_sat(t0, t1), lane), total = shuffle64(some, 31);
        if (total == 0 && attempt == 0 && (guess || ngone)) {
            // nothing is left beside the draft: by the row itself
            guess = nullptr;
            ngone = 0;
            hs::cluster_arrive();  // the totals are read before they are written again
            hs::cluster_wait();
            continue;
        }
        if (total == 0) {
            if (me == 0 && lane == 0) {
                p.next[b] = -1;
                atomicOr(p.err, HS_DEVERR_INDEX_RANGE);
            }
            return;
        }
        // Which warp's run, which of its units, which batch, which lane's values, which value:
        // each time the first whose inclusive sum passes the border.
        uint64_t rest = part_of(u0, total);
        auto locate = [&](uint64_t incl) {  // lane; rest becomes what is left in it
            const uint32_t past = __ballot_sync(0xffffffffu, incl > rest);
            const int l = past ? __ffs(past) - 1 : -1;
            if (l > 0) rest -= shuffle64(incl, l - 1);
            return l;
        };
        int l = locate(some);
        if (l < 0) return;  // cannot be: it is less than the total
        const uint64_t t_first = shuffle64(t0, l);
        const int w = 2 * l + (rest >= t_first);
        if (w != me) return;
        if (w & 1) rest -= t_first;
        uint64_t mine = 0;  // of unit lane / 2: its even or odd lanes' sums
        if (lane < 2 * n) {
#pragma unroll 8
            for (int k = 0; k < 32; k += 2) mine = add_sat(mine, sums[warp][lane >> 1][k + (lane & 1)]);
        }
        mine = add_sat(mine, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)mine, 1));
        l = locate(sum_up(lane & 1 ? 0ull : mine, lane)) >> 1;
        if (l < 0) return;
#pragma unroll 1
        for (int k = 0; k < p.per; ++k) {
            const int64_t v0 = v_first + l * unit + (int64_t)k * BATCH + 8 * lane;
            uint32_t x[8], y[8];
            uint64_t r[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t v = v0 + e;
                x[e] = v < V ? bits_at<P>(row, v) : 0u;
                y[e] = guess && v < V ? bits_at<P>(guess, v) : 0u;
            }
#pragma unroll 1
            for (int g = 0; g < ngone; ++g) {
                const int64_t at = gone[g] - v0;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = at == e ? 0u : x[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t a = clean(x[e]), c = clean(y[e]);
                r[e] = a > c ? fixed(a) - fixed(c) : 0ull;
                sum += r[e];
            }
            sum = sum_up(sum, lane);
            const int at = locate(sum);
            if (at < 0) {  // a later batch: all of this one lies before the border
                rest -= shuffle64(sum, 31);
                continue;
            }
            if (lane == at) {
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
    // a run has at most `UNITS` units: one less, and one for what the division leaves
    p.per = (int)((batches + (int64_t)G * NW * (UNITS - 1) - 1) / ((int64_t)G * NW * (UNITS - 1)));
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
