// Declarations of the rotary positions (rotary.cu), and the turn itself for other kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "internal.cuh"

namespace linformer {
namespace rotary {

// One call's arguments, already validated: up to two tensors [b][heads][n][d].
struct Call {
    const void *x[2];
    void *y[2];
    Strides sx[2], sy[2];
    int heads[2];
    const uint64_t *phase;
    const int32_t *positions;
    int start, b, n, d, rot, interleaved, inverse, dtype;
    float amplitude;
    cudaStream_t stream;
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// Cosine and sine of position pos of a pair with `phase` turns per position: the product wraps
// modulo one turn by itself.
__device__ __forceinline__ void turn_of(uint64_t phase, int pos, float &c, float &s) {
    const uint64_t turns = phase * (uint64_t)(int64_t)pos;
    float sn, cs;
    // the top 32 bits of a turn as the nearest quarter and a signed rest of at most an
    // eighth, which a float holds to 2^-27 half turns (the whole turn: to 2^-25)
    const uint32_t t = (uint32_t)(turns >> 32), quarter = (t + 0x20000000u) >> 30;
    sincospif((float)(int32_t)(t - (quarter << 30)) * 0x1p-31f, &sn, &cs);
    const float c0 = quarter & 1 ? -sn : cs, s0 = quarter & 1 ? cs : sn;
    c = quarter & 2 ? -c0 : c0;
    s = quarter & 2 ? -s0 : s0;
}

int turn(const Call &c);
int phase_table(uint64_t *phase, int rot, double base, int scaling, double factor, int original,
                double beta_fast, double beta_slow, cudaStream_t s);

}  // namespace rotary
}  // namespace linformer
