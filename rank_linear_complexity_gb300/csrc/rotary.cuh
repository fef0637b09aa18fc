// Declarations of the rotary positions (rotary.cu).
#pragma once

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

int turn(const Call &c);
int phase_table(uint64_t *phase, int rot, double base, int scaling, double factor, int original,
                double beta_fast, double beta_slow, cudaStream_t s);

}  // namespace rotary
}  // namespace linformer
