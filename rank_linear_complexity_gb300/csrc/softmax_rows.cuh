// The softmax of a row a thread, whose scores stand in tensor memory (128 columns a block of keys).
#pragma once

#include <cmath>

#include "sm100_ptx.cuh"
#include "softmax_attn.cuh"

namespace linformer {
namespace sattn {

using namespace ptx;

// 2^(s sl + off) of 32 scores, summed and packed.
__device__ __forceinline__ void exp_chunk(const uint32_t (&v)[32], uint32_t (&o)[16], float sl, float off,
                                          float2 &sum0, float2 &sum1) {
    const float2 sl2 = make_float2(sl, sl), off2 = make_float2(off, off);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float2 y = ffma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sl2, off2);
        y.x = ex2_approx(y.x);
        y.y = ex2_approx(y.y);
        if (e & 2) sum1 = fadd2(sum1, y);
        else sum0 = fadd2(sum0, y);
        o[e / 2] = pack2(y.x, y.y);
    }
}
// Columns outside [a, a + w) become -inf.
__device__ __forceinline__ void mask_chunk(uint32_t (&v)[32], int a, int w) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if ((unsigned)(e - a) >= (unsigned)w) v[e] = 0xff800000u;
}
// Both out of line, away from the code of the common block.
// The masked scores of a block of 128 become -inf in tensor memory.
static __device__ __noinline__ void mask_block(uint32_t t, int a, int w) {
#pragma unroll 1
    for (int c = 0; c < kTile; c += 32) {
        uint32_t v[32];
        tmem_ld32(t + c, v);
        mask_chunk(v, a - c, w);
        tmem_st32(t + c, v);
    }
}
// O times f, eight columns at a time (the caller's scores are in registers).
static __device__ __noinline__ void rescale_output(uint32_t t, int columns, float f) {
#pragma unroll 1
    for (int c = 0; c < columns; c += 8) {
        uint32_t q[8];
        tmem_ld8(t + c, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(__uint_as_float(q[e]) * f);
        tmem_st8_async(t + c, q);
    }
    tmem_wait_st();
}
__device__ __forceinline__ float max_chunk(const uint32_t (&v)[32]) {
    float m0 = __uint_as_float(v[0]), m1 = __uint_as_float(v[1]);
#pragma unroll
    for (int e = 2; e < 30; e += 4) {
        m0 = max3(m0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        m1 = max3(m1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
    }
    return fmaxf(max3(m0, __uint_as_float(v[30]), __uint_as_float(v[31])), m1);
}

}  // namespace sattn
}  // namespace linformer
