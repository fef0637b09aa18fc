// Declarations shared by the exact softmax attention kernels (forward and backward).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "internal.cuh"

namespace linformer {
namespace sattn {

constexpr int kTile = 128;  // rows of a query tile, keys of a key block
constexpr int64_t kMaxItems = 1 << 30;  // work items of a launch (counted in 32 bits)

// One call's arguments, already validated.
struct Call {
    const void *Q, *K, *V, *O, *dO;
    void *out, *dQ, *dK, *dV;
    Strides sQ, sK, sV, sO, sdO, sdQ, sdK, sdV;
    float *lse;
    const int32_t *q_lengths, *k_lengths;
    int b, hq, hk, nq, nk, d, causal, window;
    float scale;
    cudaStream_t stream;
};

// Which keys the queries of one sequence see: query i of Lq stands at position
// i + (Lk - Lq) (the valid parts end together) and sees keys [first, end).
struct Span {
    int Lq, Lk, causal, window;
    __device__ __forceinline__ int end(int i) const {
        return causal ? min(Lk, i + Lk - Lq + 1) : Lk;
    }
    __device__ __forceinline__ int first(int i) const {
        return window ? max(0, i + Lk - Lq + 1 - window) : 0;
    }
};

// Order of the work items (`ranks` tiles of each of `units` heads): a few heads at a time, `some`
// of them, whose streamed tensors stay in L2 until all their tiles have gone through them;
// within those tile by tile, so that neighbours are about equally long.
// (Out of line: every role does this for every item, and most calls have one set.)
static __device__ __noinline__ int2 place_in_sets(int idx, int ranks, int units, int some) {
    const int set = idx / (ranks * some), base = set * some;
    idx -= base * ranks;
    units = min(some, units - base);
    const int rank = idx / units;
    return make_int2(rank, base + idx - rank * units);
}
template <bool kSets>
__device__ __forceinline__ void place(int idx, int ranks, int units, int some, int &rank, int &unit) {
    if (kSets && some < units) {
        const int2 at = place_in_sets(idx, ranks, units, some);
        rank = at.x;
        unit = at.y;
    } else {
        rank = idx / units;
        unit = idx - rank * units;
    }
}
// Heads at a time: as many as stream 32 MB; all of them where nothing is read twice, or all
// together stream little enough to stay in L2 without (`bytes` a head).  Measured, forward and
// backward, in sets and all at once: b h = 192, n = 4096, d = 64 (201 MB) 741 and 801, 2310 and
// 2686 us: less DRAM traffic, and less of the power that bounds them (sets of 16 and 64 MB: 739
// and 760, 2307 and 2351); 76 heads (80 MB) 288 and 299, 871 and 906.  With few tiles a head
// (480 heads of 512, 63 MB) the tail of each set costs more: 56 and 51, 157 and 151.
// Tiles under a causal mask are unequal, and all heads' longest go first where they come all at
// once: in sets from 128 MB on (backward of 19 heads of 8191, d = 128, 80 MB: 830 and 780; 100 heads
// of 4096, d = 64, 105 MB: 696 and 665), and only where a set holds two items an SM, so that its
// short ones fill its end (32 heads over 8, sets of one key/value head of 64 to 128 blocks: 8193
// rows 1617 and 1314, 12288 rows 3328 and 2886, 16384 rows 5618 and 5086; 256 heads of 2048, sets of
// 512 items: 853 and 941; of 4096, of 480: 2950 and 3230).
inline int units_at_once(int ranks, int units, int64_t bytes, bool causal, int sms) {
    constexpr int64_t kStreamed = 32 << 20;
    const int64_t held = causal || ranks < 16 ? 128 << 20 : 48 << 20;
    if (ranks <= 1 || bytes * units <= held) return units;
    const int64_t some = std::max<int64_t>(1, std::min<int64_t>(units, kStreamed / bytes));
    return causal && some * ranks < 2 * sms ? units : (int)some;
}

__device__ __forceinline__ int clamp_length(const int32_t *lengths, int batch, int n) {
    if (!lengths) return n;
    const int L = __ldg(lengths + batch);
    return L < 0 ? 0 : (L > n ? n : L);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}

// Whether every 16 columns of a tensor are 32 aligned bytes (strides of dimensions of size one
// do not count, but are harmless when they say no).
inline int wide_stores(const void *p, const Strides &s, int d) {
    return (reinterpret_cast<uintptr_t>(p) % 32 == 0 && d % 16 == 0 && s.b % 16 == 0 && s.h % 16 == 0 &&
            s.n % 16 == 0)
               ? 1
               : 0;
}
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Zeroes rows [row0, kRows) of a tile of DP / 64 column halves (each kRows rows of 128 bytes;
// whole rows, so the swizzle does not matter), shared by `count` threads.
template <int DP, int kRows>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int row0, int idx, int count) {
#pragma unroll
    for (int h = 0; h < DP / 64; ++h) {
        uint4 *p = reinterpret_cast<uint4 *>(tile + h * kRows * 128 + row0 * 128);
        for (int i = idx; i < (kRows - row0) * 8; i += count) p[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Host helpers (softmax_attn_fwd.cu).
// Map of a [b][heads][n][d] bf16 tensor for boxes of 64 columns x `rows` rows x `hrows`
// heads of a group of `group`: coordinates (column, row, head in group, group, batch).  promotion: what
// L2 fetches at a time.
bool encode_rows(CUtensorMap *m, const void *base, const Strides &s, int b, int heads, int group,
                 int n, int d, int rows, int hrows,
                 CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
int allow_smem(const void *kernel, uint32_t bytes, int slot);

int forward(const Call &c);
int backward(const Call &c);

}  // namespace sattn
}  // namespace linformer
