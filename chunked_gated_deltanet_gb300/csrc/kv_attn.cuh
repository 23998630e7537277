// Device helpers shared by the attention kernels over the 8-bit key/value cache.
#pragma once

#include <cuda_fp16.h>

#include "kv.cuh"
#include "umma.cuh"

namespace gdn {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 4 int8 -> 4 fp16, exact: 0x6400 | (b ^ 0x80) reads 1152 + b, and 1152 is taken away. (Keys fed as 1152 + b, with 1152
// times the sum of the query taken from the scores, spare these subtractions, but the scores' fp32 sums then carry a term
// that grows with the query's sum: 6 times the error bound for queries of mean 10.)
__device__ __forceinline__ uint2 i8_to_f16x4(uint32_t x) {
    x ^= 0x80808080u;
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const uint32_t off = 0x64806480u;
    const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&off));
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&b), *reinterpret_cast<const __half2 *>(&off));
    return make_uint2(*reinterpret_cast<const uint32_t *>(&c), *reinterpret_cast<const uint32_t *>(&d));
}

__device__ __forceinline__ void b8_to_f(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// The power of two that brings x > 0 into [2^14, 2^15), and its inverse; 1 for 0 and what is not finite, at most 2^100.
__device__ __forceinline__ float pow2_to_2_15(float x, float &back) {
    int e = 14 + 127 - (int)(__float_as_uint(x) >> 23);   // x >= 0
    if (x == 0.f || !(x <= 3.4e38f)) e = 0;
    e = min(e, 100);
    back = __uint_as_float((uint32_t)(127 - e) << 23);
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// Zeroes the bf16 of a vector that are not finite; whether there was one.
__device__ __forceinline__ bool drop_not_finite(uint4 &u) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool any = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if ((w[k] & 0x7F80u) == 0x7F80u) { w[k] &= 0xFFFF0000u; any = true; }
        if ((w[k] & 0x7F800000u) == 0x7F800000u) { w[k] &= 0xFFFFu; any = true; }
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
    return any;
}

// ---- the unit of the summed values ----
// The bf16 kernels sum 2^{x - m} v over a row's keys with the weights in fp16 and the int8 of a complete block as they
// are, so its value scale vs has to sit in the weight: 2^{x + log2 vs - lref - m}, where what is summed is in units of
// 2^lref. fp16 has few exponents, so the unit follows the scales: it moves to a block whose scale is further than
// 2^kUnitSpan from it, and what was summed moves along. Inside the span (blocks of like values, the usual case) nothing
// moves. A unit is a power of two, so a move is exact and leaves no trace in rows that do not see the block.
constexpr float kUnitSpan = 4.f;

// 2^e of a whole e in [-126, 127]
__device__ __forceinline__ float pow2_of(float e) {
    return __uint_as_float((uint32_t)(127 + (int)fminf(fmaxf(e, -126.f), 127.f)) << 23);
}
// log2 of a block's value scale; +inf of an all-zero block, whose values are at home in any unit
__device__ __forceinline__ float kv_log2_scale(float vs) { return vs != 0.f ? log2f(vs) : INFINITY; }
// That over the unit, which moves if it has to; `move` (1 before) becomes the power of two that the sums take along
__device__ __forceinline__ float kv_unit(float lvs, float &lref, float &move) {
    float dv = lvs - lref;
    if (!(fabsf(dv) <= kUnitSpan)) {
        dv = 0.f;
        if (lvs != INFINITY) {
            const float to = rintf(lvs);
            move = pow2_of(lref - to);
            lref = to;
            dv = lvs - to;
        }
    }
    return dv;
}

}  // namespace gdn
