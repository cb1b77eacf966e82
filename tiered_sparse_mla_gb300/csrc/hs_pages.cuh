// hs_pages.cuh -- what the tensor-core kernels over whole pages share: arithmetic on pairs of
// f32, FP8 pools' queries as pairs of e4m3 codes, and the pool's rows as a tensor map of pages.
#pragma once

#include <cstdint>

#include "hs_internal.cuh"
#include "hs_tmap.cuh"

namespace {

__host__ __device__ __forceinline__ int pages_of(int tokens) {
    return tokens <= 0 ? 0 : (tokens - 1) / hs::kPage + 1;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two f32 operations in one instruction.
__device__ __forceinline__ void mul2(float &a, float &b, float c, float d) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float &a, float &b, float c, float d) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}

// FP8 pools: a query row times a power of two, which brings its largest to (224, 448], as sums of
// two e4m3 codes per value. Which power, from the bits of the row's largest magnitude as
// BF16; as a pair of BF16, NaN where the row is not finite; and its inverse.
__device__ __forceinline__ int query_exponent(uint32_t top) {
    return min(135 - (int)(top >> 7) - ((top & 0x7fu) > 0x60u), 126);
}
__device__ __forceinline__ uint32_t query_power(uint32_t top) {
    return top >= 0x7f80u ? 0x7fc07fc0u : (uint32_t)(query_exponent(top) + 127) * 0x00800080u;
}
__device__ __forceinline__ float query_back(uint32_t top) {
    return __uint_as_float((uint32_t)(127 - query_exponent(top)) << 23);
}
// Two BF16 values times 2^k (a pair of BF16; at most 448, or NaN) as the sums of two
// e4m3 codes each. F16 holds the products' eight bits down to 2^-17, the codes'
// smallest step is 2^-9.
__device__ __forceinline__ void e4m3_pieces(uint32_t w, uint32_t pow2, uint16_t &p, uint16_t &r) {
    uint32_t x, h;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w), "r"(pow2));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(__uint_as_float(x & 0xffff0000u)), "f"(__uint_as_float(x << 16)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(p) : "r"(x));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(p));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(h));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
}
__device__ __forceinline__ void bf16x4_to_e4m3(uint32_t w0, uint32_t w1, uint32_t pow2, uint32_t &p, uint32_t &r) {
    uint16_t p0, p1, r0, r1;
    e4m3_pieces(w0, pow2, p0, r0);
    e4m3_pieces(w1, pow2, p1, r1);
    asm("mov.b32 %0, {%1, %2};" : "=r"(p) : "h"(p0), "h"(p1));
    asm("mov.b32 %0, {%1, %2};" : "=r"(r) : "h"(r0), "h"(r1));
}

// [rows][9 chunks][64] seen as (element, row, chunk), boxes of 64 x one page x n
bool make_page_map(CUtensorMap *m, bool fp8, const void *rows, uint64_t n_rows, uint32_t nchunks, CUtensorMapSwizzle sw) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t rb = fp8 ? hs::kDim : 2 * hs::kDim;
    cuuint64_t dims[3] = {64, n_rows, 9};
    cuuint64_t strides[2] = {rb, rb / 9};
    cuuint32_t box[3] = {64, (cuuint32_t)hs::kPage, nchunks};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void *>(rows), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              sw, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
