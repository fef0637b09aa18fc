// Rows on their way into a paged key/value cache, and within it.
//
// append: the new rows of each sequence go to the rows of the cache that follow its `start`,
// keys turned to their positions, and the queries that stand at the same positions are turned
// beside them (the turn of rotary.cu, formed in fp32 and rounded once).  Bound by memory: every
// element read and written once (8 x 4096 ragged rows of 32 + 8 + 8 heads of 128, bf16: 122 us, 5.9
// TB/s).  A thread keeps the sines of its pairs and goes through several heads with them.
//
// keep: of a tree of drafted tokens, the rows of the accepted ones move up behind the sequence's
// start.  A thread moves one piece of every row, in order, so that no other thread's store can
// reach what it has yet to read; path[i] >= i, so neither can its own.
//
// tree_mask: which nodes each node of a tree sees, itself and its ancestors.
#include <algorithm>
#include <cstring>
#include <cuda_bf16.h>

#include "internal.cuh"
#include "paged.cuh"
#include "rotary.cuh"
#include "sm100_ptx.cuh"

namespace linformer {
namespace paged {
namespace {

using rotary::from_float;
using rotary::to_float;
using rotary::Vec;

constexpr int kThreads = 128;
// Heads of a thread in flight, and blocks of an SM: registers for 32 warps (8 x 4096 ragged rows of 32 + 8
// + 8 heads of 128, before the stores past L1: 129 us; one head 155, four heads and the registers that they
// take 158, in 80 registers 212; 40 warps 160).
constexpr int kBatch = 2, kBlocks = 8;
constexpr int kMaxHeads = 16;  // heads of one thread

struct AppendParams {
    Cache cache;
    const void *x[3];
    Strides sx[3];
    void *y;
    Strides sy;
    const int32_t *starts, *counts, *positions;
    const uint64_t *phase;
    int hq, hk, heads, n, rot, chunks, rot_chunks, per_thread, splits;
    int64_t threads;
    float amplitude;
    int *status;
};

// A piece as one access of 16 bytes, stores past L1 (8 x 4096 ragged rows as above: 131 us with plain ones,
// 122 so, 123 with stores that L2 is to drop first).
template <typename Piece>
__device__ __forceinline__ Piece load_piece(const void *from) {
    if constexpr (sizeof(Piece) != 16) return *static_cast<const Piece *>(from);
    else {
        const uint4 w = *static_cast<const uint4 *>(from);
        Piece x;
        memcpy(&x, &w, sizeof x);
        return x;
    }
}
template <typename Piece>
__device__ __forceinline__ void store_piece(void *to, const Piece &x) {
    if constexpr (sizeof(Piece) != 16) *static_cast<Piece *>(to) = x;
    else {
        uint4 w;
        memcpy(&w, &x, sizeof w);
        __stcg(static_cast<uint4 *>(to), w);
    }
}

// V pairs a thread (V = 1: any strides and sizes; otherwise 16-byte pieces).
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocks) append_kernel(const AppendParams p) {
    using Piece = Vec<T, V>;
    ptx::launch_dependents();  // (here and below: the attention after it is set up meanwhile, and waits)
    const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (tid >= p.threads) return;
    const int c = (int)(tid % p.chunks);
    const int64_t r = tid / p.chunks;
    const int i = (int)(r % p.n);
    const int64_t r2 = r / p.n;
    const int split = (int)(r2 % p.splits), b = (int)(r2 / p.splits);
    const int h0 = split * p.per_thread, h1 = min(h0 + p.per_thread, p.heads);
    const int start = __ldg(p.starts + b);
    // rows behind the sequence's last, and those without a page, leave the cache as it was
    int page = 0, row = 0;
    bool kept = h1 > p.hq && (!p.counts || i < __ldg(p.counts + b));
    if (kept) kept = find_row(p.cache, b, (int64_t)start + i, p.status, page, row);
    const bool turn = c < p.rot_chunks;
    // the two pieces of the thread's pairs (of the copied rest: one)
    const int at0 = turn ? (kInterleaved ? 2 * V * c : V * c) : p.rot + V * (c - p.rot_chunks);
    const int at1 = turn ? (kInterleaved ? at0 + V : at0 + p.rot / 2) : at0;
    float cs[V], sn[V];
    if (turn && h0 < p.hq + p.hk) {
        const int pos = p.positions ? __ldg(p.positions + (int64_t)b * p.n + i) : (int)((unsigned)start + (unsigned)i);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            rotary::turn_of(__ldg(p.phase + V * c + v), pos, cs[v], sn[v]);
            cs[v] *= p.amplitude;
            sn[v] *= p.amplitude;
        }
    }
    // The thread's heads among `heads` of one tensor, the first of which is head `base` of all.
    auto move = [&](const void *from, const Strides &sx, void *to, const Strides &sy, int64_t at_y, int base, int heads,
                    bool turned) {
        const int first = max(h0 - base, 0), last = min(h1 - base, heads);
        const T *x = static_cast<const T *>(from) + b * sx.b + i * sx.n + first * sx.h;
        T *y = static_cast<T *>(to) + at_y + first * sy.h;
        for (int h = first; h < last; h += kBatch, x += kBatch * sx.h, y += kBatch * sy.h) {
            Piece u0[kBatch], u1[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (h + k >= last) continue;
                u0[k] = load_piece<Piece>(x + k * sx.h + at0);
                if (turn) u1[k] = load_piece<Piece>(x + k * sx.h + at1);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (h + k >= last) continue;
                if (turn) {
                    if (turned) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            // interleaved: elements 2 v and 2 v + 1 of the two pieces in a row
                            T &a = kInterleaved ? (2 * v < V ? u0[k].e[(2 * v) % V] : u1[k].e[(2 * v) % V]) : u0[k].e[v];
                            T &z = kInterleaved ? (2 * v + 1 < V ? u0[k].e[(2 * v + 1) % V] : u1[k].e[(2 * v + 1) % V])
                                                : u1[k].e[v];
                            const float fa = to_float(a), fz = to_float(z);
                            a = from_float<T>(fa * cs[v] - fz * sn[v]);
                            z = from_float<T>(fz * cs[v] + fa * sn[v]);
                        }
                    }
                    store_piece(y + k * sy.h + at1, u1[k]);
                }
                store_piece(y + k * sy.h + at0, u0[k]);
            }
        }
    };
    if (h0 < p.hq) move(p.x[0], p.sx[0], p.y, p.sy, b * p.sy.b + i * p.sy.n, 0, p.hq, true);
    if (kept) {
        const Cache &c = p.cache;
        if (h0 < p.hq + p.hk) move(p.x[1], p.sx[1], c.k, c.sk, page * c.sk.b + row * c.sk.n, p.hq, p.hk, true);
        move(p.x[2], p.sx[2], c.v, c.sv, page * c.sv.b + row * c.sv.n, p.hq + p.hk, p.hk, false);
    }
}

struct KeepParams {
    Cache cache;
    const int32_t *starts, *path, *counts;
    int hk, m, chunks;
    int64_t threads;
    int *status;
};

// One piece of every accepted row of one head of one sequence, of the keys or of the values.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) keep_kernel(const KeepParams p) {
    using Piece = Vec<T, V>;
    ptx::launch_dependents();
    const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (tid >= p.threads) return;
    const int c = (int)(tid % p.chunks);
    int64_t r = tid / p.chunks;
    const int head = (int)(r % p.hk);
    r /= p.hk;
    const bool value = r & 1;
    const int b = (int)(r >> 1);
    const Strides s = value ? p.cache.sv : p.cache.sk;
    T *base = static_cast<T *>(value ? p.cache.v : p.cache.k) + head * s.h + V * c;
    const int64_t start = __ldg(p.starts + b);
    const int count = p.counts ? min(max(__ldg(p.counts + b), 0), p.m) : p.m;
    const int32_t *path = p.path + (int64_t)b * p.m;
    // Rows in flight, each step for all of them before the next, so that a batch waits once for the
    // path, the table and the rows (64 sequences, 8 heads of 128, up to 16 rows: 7.6 us row by row).
    // Sources of later rows lie behind all targets before them.
    constexpr int kRows = 8;
    const int32_t *table = p.cache.table + (int64_t)b * p.cache.width;
    int bad = 0;
    for (int i = 0; i < count; i += kRows) {
        Piece u[kRows];
        int node[kRows], from[kRows], to[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) node[k] = i + k < count ? __ldg(path + i + k) : i + k;
        auto page_at = [&](int64_t at, bool wanted) {
            const int64_t entry = at >> p.cache.shift;
            const bool inside = at >= 0 && entry < p.cache.width;
            if (wanted && !inside) bad = kBadRow;
            return wanted && inside ? __ldg(table + entry) : -1;
        };
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const bool moves = node[k] > i + k;  // (a node in its place stays)
            from[k] = page_at(start + node[k], moves);
            to[k] = page_at(start + i + k, moves);
            if (node[k] < i + k) bad = kBadPath;
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const bool there = (unsigned)from[k] < (unsigned)p.cache.pages && (unsigned)to[k] < (unsigned)p.cache.pages;
            if (!there) {
                if (node[k] > i + k && !bad) bad = kBadPage;  // (whatever the entry: the table may hold any)
                to[k] = -1;
                continue;
            }
            u[k] = *reinterpret_cast<const Piece *>(base + from[k] * s.b + ((int)(start + node[k]) & (p.cache.page - 1)) * s.n);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (to[k] >= 0)
                *reinterpret_cast<Piece *>(base + to[k] * s.b + ((int)(start + i + k) & (p.cache.page - 1)) * s.n) = u[k];
    }
    if (bad && p.status) atomicExch(p.status, bad);
}

// A sequence a block, a node a thread: its ancestors come in falling order, so their bits are
// gathered a word at a time.
__global__ void __launch_bounds__(1024) tree_mask_kernel(const int32_t *parents, uint64_t *mask, int n, int words,
                                                         int *status) {
    __shared__ int parent[1024];
    ptx::launch_dependents();
    const int i = threadIdx.x;
    const int64_t b = blockIdx.x;
    if (i < n) {
        int x = __ldg(parents + b * n + i);
        if (x < -1 || x >= i) {
            if (status) atomicExch(status, kBadParent);
            x = -1;
        }
        parent[i] = x;
    }
    __syncthreads();
    if (i >= n) return;
    uint64_t *row = mask + (b * n + i) * words;
    int at = i;
    for (int w = words - 1; w >= 0; --w) {
        uint64_t bits = 0;
        for (; at >= 64 * w; at = parent[at]) bits |= 1ull << (at & 63);  // (-1 is below every word)
        row[w] = bits;
    }
}

template <typename T, int V>
int launch_append(const AppendParams &p, bool interleaved, cudaStream_t s) {
    const int64_t blocks = (p.threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return LINFORMER_ERR_SIZE;
    KernelScope scope(LINFORMER_KERNEL_CACHE, s);
    if (interleaved) append_kernel<T, V, true><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    else append_kernel<T, V, false><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? LINFORMER_OK : LINFORMER_ERR_LAUNCH;
}

template <typename T, int V>
int launch_keep(const KeepParams &p, cudaStream_t s) {
    const int64_t blocks = (p.threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return LINFORMER_ERR_SIZE;
    KernelScope scope(LINFORMER_KERNEL_CACHE, s);
    keep_kernel<T, V><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? LINFORMER_OK : LINFORMER_ERR_LAUNCH;
}

// Whether 16-byte pieces of V elements stay aligned over the dimensions of more than one entry.
bool pieces(const Strides &s, int b, int heads, int n, int V) {
    return (b == 1 || s.b % V == 0) && (heads == 1 || s.h % V == 0) && (n == 1 || s.n % V == 0);
}
bool pieces(const Cache &c, int hk, int V) {
    return pieces(c.sk, c.pages, hk, c.page, V) && pieces(c.sv, c.pages, hk, c.page, V);
}

}  // namespace

int append(const AppendCall &c) {
    AppendParams p{};
    const int V = c.dtype == LINFORMER_F32 ? 4 : 8;
    bool wide = c.d % V == 0 && c.rot % (2 * V) == 0 && pieces(c.cache, c.hk, V);
    for (int w = 0; w < 3; ++w) {
        p.x[w] = c.x[w];
        p.sx[w] = c.sx[w];
        if (w || c.hq) wide = wide && pieces(c.sx[w], c.b, w ? c.hk : c.hq, c.n, V);
    }
    if (c.hq) wide = wide && pieces(c.sy, c.b, c.hq, c.n, V);
    const int v = wide ? V : 1;
    p.cache = c.cache;
    p.y = c.y;
    p.sy = c.sy;
    p.starts = c.starts;
    p.counts = c.counts;
    p.positions = c.positions;
    p.phase = c.phase;
    p.hq = c.hq;
    p.hk = c.hk;
    p.heads = c.hq + 2 * c.hk;
    p.n = c.n;
    p.rot = c.rot;
    p.rot_chunks = c.rot / 2 / v;
    p.chunks = p.rot_chunks + (c.d - c.rot) / v;
    p.amplitude = c.amplitude;
    p.status = device_status_ptr();
    // Heads a thread: as in rotary.cu, as many as leave two full waves of threads.
    const int64_t rows = (int64_t)c.b * c.n * p.chunks;
    constexpr int64_t kSmThreads = 2048;
    const int64_t per = rows * p.heads / (2 * device_sms() * kSmThreads);
    p.per_thread = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(p.heads, kMaxHeads), per));
    p.splits = (p.heads + p.per_thread - 1) / p.per_thread;
    p.threads = rows * p.splits;
    if (c.dtype == LINFORMER_F32)
        return wide ? launch_append<float, 4>(p, c.interleaved, c.stream)
                    : launch_append<float, 1>(p, c.interleaved, c.stream);
    return wide ? launch_append<__nv_bfloat16, 8>(p, c.interleaved, c.stream)
                : launch_append<__nv_bfloat16, 1>(p, c.interleaved, c.stream);
}

int keep(const KeepCall &c) {
    KeepParams p{};
    const int V = c.dtype == LINFORMER_F32 ? 4 : 8;
    const bool wide = c.d % V == 0 && pieces(c.cache, c.hk, V);
    p.cache = c.cache;
    p.starts = c.starts;
    p.path = c.path;
    p.counts = c.counts;
    p.hk = c.hk;
    p.m = c.m;
    p.chunks = wide ? c.d / V : c.d;
    p.threads = (int64_t)c.b * 2 * c.hk * p.chunks;
    p.status = device_status_ptr();
    if (c.dtype == LINFORMER_F32) return wide ? launch_keep<float, 4>(p, c.stream) : launch_keep<float, 1>(p, c.stream);
    return wide ? launch_keep<__nv_bfloat16, 8>(p, c.stream) : launch_keep<__nv_bfloat16, 1>(p, c.stream);
}

int tree_mask(const int32_t *parents, uint64_t *mask, int b, int n, cudaStream_t s) {
    KernelScope scope(LINFORMER_KERNEL_CACHE, s);
    tree_mask_kernel<<<b, (n + 31) / 32 * 32, 0, s>>>(parents, mask, n, (n + 63) / 64, device_status_ptr());
    return cudaGetLastError() == cudaSuccess ? LINFORMER_OK : LINFORMER_ERR_LAUNCH;
}

}  // namespace paged
}  // namespace linformer
