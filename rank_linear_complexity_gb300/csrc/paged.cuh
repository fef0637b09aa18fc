// Declarations of the paged key/value cache: appending and keeping rows (paged_cache.cu),
// attention over the pages (paged_attn.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "internal.cuh"

namespace linformer {
namespace paged {

// Codes in the device status word: a table entry that is needed and names no page, a row beyond
// the table, an accepted node before its place, a parent that is not before its node.
constexpr int kBadPage = 200, kBadRow = 201, kBadPath = 202, kBadParent = 203;

// Keys and values of all sequences, [pages][hk][page][d] each by strides (b: a page's), and which
// page holds rows [page x, page (x + 1)) of sequence beta: table[beta][x].
struct Cache {
    void *k, *v;
    Strides sk, sv;
    const int32_t *table;  // [b][width]
    int pages, page, width;
    int shift;  // page = 2^shift
};

// The page and the row within it of row `at` of a sequence; false where there is none.
__device__ __forceinline__ bool find_row(const Cache &c, int b, int64_t at, int *status, int &page, int &row) {
    const int64_t entry = at >> c.shift;
    row = (int)at & (c.page - 1);
    page = at >= 0 && entry < c.width ? __ldg(c.table + (int64_t)b * c.width + entry) : -1;
    if ((unsigned)page < (unsigned)c.pages) return true;
    if (status) atomicExch(status, at >= 0 && entry < c.width ? kBadPage : kBadRow);
    return false;
}

struct AppendCall {
    Cache cache;
    const void *x[3];  // queries (none: null), keys, values: [b][hq or hk][n][d]
    Strides sx[3];
    void *y;           // turned queries
    Strides sy;
    const int32_t *starts, *counts, *positions;
    const uint64_t *phase;
    int b, hq, hk, n, d, rot, interleaved, dtype;
    float amplitude;
    cudaStream_t stream;
};

struct KeepCall {
    Cache cache;
    const int32_t *starts, *path, *counts;
    int b, hk, m, d, dtype;
    cudaStream_t stream;
};

struct AttnCall {
    Cache cache;
    const void *q;
    void *out;
    Strides sq, so;
    float *lse;
    const int32_t *q_lengths, *k_lengths;
    const uint64_t *mask;  // trees: [b][nq][words]; null otherwise
    int words;
    int b, hq, hk, nq, d, causal, window;
    float scale;
    cudaStream_t stream;
};

int append(const AppendCall &c);
int keep(const KeepCall &c);
int tree_mask(const int32_t *parents, uint64_t *mask, int b, int n, cudaStream_t s);
int attention(const AttnCall &c);

}  // namespace paged
}  // namespace linformer
