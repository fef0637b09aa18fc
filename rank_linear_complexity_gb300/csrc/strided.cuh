// Strides of the [b][heads][n][d] tensors that an entry point takes (host).
#pragma once

#include "internal.cuh"

namespace linformer {

// The strides as given, or dense [b][heads][n][d].
inline Strides strides_of(const int64_t *s, int heads, int n, int d) {
    if (s) return Strides{s[0], s[1], s[2]};
    return Strides{(int64_t)heads * n * d, (int64_t)n * d, d};
}

// A dimension of more than one entry has a positive stride (bounded so that no offset
// overflows) that keeps 16-byte pieces aligned; rows of an output do not overlap.
inline int check_strides(const Strides &s, int b, int heads, int n, int d, int multiple, bool output) {
    const int64_t limit = 1LL << 38;
    const int64_t st[3] = {s.b, s.h, s.n};
    const int count[3] = {b, heads, n};
    for (int i = 0; i < 3; ++i) {
        if (count[i] <= 1) continue;
        if (st[i] < 1 || st[i] > limit) return LINFORMER_ERR_VALUE;
        if (output && st[i] < d) return LINFORMER_ERR_VALUE;
        if (st[i] % multiple) return LINFORMER_ERR_ALIGN;
    }
    return LINFORMER_OK;
}

}  // namespace linformer
