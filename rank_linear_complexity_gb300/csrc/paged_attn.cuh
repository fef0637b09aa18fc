// What the kernels of the attention over pages share (paged_attn.cu, paged_attn_wide.cu): the list of
// key blocks, the runs of it that CTAs take, pages of a block.
#pragma once

#include <algorithm>

#include "paged.cuh"
#include "sm100_ptx.cuh"
#include "softmax_attn.cuh"

namespace linformer {
namespace paged {

using namespace ptx;
using sattn::kTile;  // keys of a block
using sattn::pack2;
using sattn::Span;

constexpr int kMaxSeqs = 512;  // sequences of a launch
constexpr float kOutgrown = 16.f, kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnParams {
    const int32_t *q_lengths, *k_lengths, *table;
    const uint64_t *mask;
    __nv_bfloat16 *out;
    Strides so;
    float *lse;
    float *part_o, *part_lse;  // [2 per CTA][per][N][DP], [2 per CTA][per][N]
    int4 *cuts;                // a CTA's: see join_kernel
    int words, b, hq, hk, group, nq, d, causal, window;
    // tiles of qbox positions of hbox heads (nch tiles to a group), `per` of them to a unit of work;
    // N: rows of a tile in the workspace
    int qbox, hbox, nch, ntiles, per, units, N, ctas;
    int whole;   // no unit is cut
    int direct;  // and each has a CTA of its own, by number
    int pages, page, width, shift, box, nbox;  // nbox boxes of `box` rows make a block of keys
    float scale, scale_log2;
    int wide_stores;
    int *status;
};

// The rows of a tile.
struct Rows {
    int q0, h0;
    __device__ __forceinline__ Rows(const AttnParams &p, int tile) {
        const int qt = p.nch > 1 ? tile / p.nch : tile;
        q0 = qt * p.qbox;
        h0 = (tile - qt * p.nch) * p.hbox;
    }
};

// The key blocks that a tile's rows see.
__device__ __forceinline__ void blocks_of(const AttnParams &p, const Span &sp, int q0, int &lo, int &hi) {
    lo = hi = 0;
    const int last = min(q0 + p.qbox, sp.Lq) - 1;
    if (last < q0) return;
    const int e = sp.end(last), f = sp.first(q0);
    if (e <= f) return;
    lo = f / kTile;
    hi = (e + kTile - 1) / kTile;
}
// Those of a unit's tiles together.
__device__ __forceinline__ void blocks_of_unit(const AttnParams &p, const Span &sp, int unit, int &lo, int &hi) {
    blocks_of(p, sp, Rows(p, unit * p.per).q0, lo, hi);
    if (p.per == 2 && 2 * unit + 1 < p.ntiles) {
        int a, z;
        blocks_of(p, sp, Rows(p, 2 * unit + 1).q0, a, z);
        if (z > a) {
            lo = hi > lo ? min(lo, a) : a;
            hi = max(hi, z);
        }
    }
}
// A sequence's length (not by __ldg: a load of what is taken to be constant may be moved up, past the
// wait for the kernel that writes it).
__device__ __forceinline__ int read_length(const int32_t *lengths, int seq, int most) {
    if (!lengths) return most;
    int x;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(lengths + seq) : "memory");
    return min(max(x, 0), most);
}
// The lengths and the list's marks, in shared memory.
struct Marks {
    int2 length[kMaxSeqs];    // queries, cache rows
    int first[kMaxSeqs + 1];  // where the blocks of each sequence begin in the list
    bool empty[kMaxSeqs];     // some unit has none
    __device__ __forceinline__ Span span(const AttnParams &p, int seq) const {
        return Span{length[seq].x, length[seq].y, p.causal, p.window};
    }
};
__device__ __forceinline__ int run_begin(int total, int cta, int ctas) {
    const int each = total / ctas;
    return each * cta + min(cta, total - each * ctas);
}
__device__ __forceinline__ int runs(const AttnParams &p, int total) {
    return min(p.ctas, max(1, total));
}

// Fills the marks, by a whole CTA (it has one of the CTA's barriers; one has to follow).
__device__ __forceinline__ void fill(const AttnParams &p, Marks &marks, int tid, int threads) {
    int *first = marks.first;
    for (int s = tid; s < p.b; s += threads) {
        marks.length[s] = make_int2(read_length(p.q_lengths, s, p.nq), read_length(p.k_lengths, s, p.width * p.page));
        const Span sp = marks.span(p, s);
        int sum = 0;
        bool empty = false;
        for (int u = 0; u < p.units; ++u) {
            int lo, hi;
            blocks_of_unit(p, sp, u, lo, hi);
            sum += (hi - lo) * p.hk;
            empty |= hi <= lo;
        }
        marks.empty[s] = empty;
        first[s + 1] = sum;
    }
    __syncthreads();
    if (tid < 32) {
        const int each = (p.b + 31) / 32, s0 = min(tid * each, p.b), s1 = min(s0 + each, p.b);
        int sum = 0;
        for (int s = s0; s < s1; ++s) sum += first[s + 1];
        int run = sum;
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, run, o);
            if (tid >= o) run += x;
        }
        run -= sum;
        for (int s = s0; s < s1; ++s) first[s + 1] = run += first[s + 1];
        if (tid == 0) first[0] = 0;
    }
}

// A CTA's part of the list, unit by unit: sequence-major, then unit, then key/value head.
struct Item {
    int seq, unit, kvh, lo, hi;  // blocks [lo, hi) of it
    Span sp;
    int slot;  // where its partial result goes; -1: the unit is whole
};
struct Walk {
    int at = 0, end = 0;
    int seq, unit, kvh, blk, lo, hi, slot;
    Span sp;
    Walk() = default;
    // A unit a CTA.
    __device__ __forceinline__ explicit Walk(const AttnParams &p) {
        seq = blockIdx.x / (p.units * p.hk);
        const int r = blockIdx.x - seq * (p.units * p.hk);
        unit = r / p.hk;
        kvh = r - unit * p.hk;
        sp = Span{read_length(p.q_lengths, seq, p.nq), read_length(p.k_lengths, seq, p.width * p.page), p.causal,
                  p.window};
        blocks_of_unit(p, sp, unit, lo, hi);
        blk = 0;
        end = hi > lo ? 1 : 0;
    }
    __device__ __forceinline__ Walk(const AttnParams &p, const Marks &marks, int cta) {
        const int *first = marks.first;
        const int total = first[p.b], n = runs(p, total);
        if (cta >= n) return;
        at = run_begin(total, cta, n);
        end = run_begin(total, cta + 1, n);
        if (at >= end) return;
        int a = 0, z = p.b;  // first[a] <= at < first[z]
        while (z - a > 1) {
            const int m = (a + z) / 2;
            if (first[m] <= at) a = m;
            else z = m;
        }
        seq = a;
        sp = marks.span(p, seq);
        int off = at - first[seq];
        for (unit = 0;; ++unit) {
            blocks_of_unit(p, sp, unit, lo, hi);
            const int c = (hi - lo) * p.hk;
            if (off < c) break;
            off -= c;
        }
        kvh = off / (hi - lo);
        blk = off - kvh * (hi - lo);
        slot = 2 * cta;
        if (p.whole && blk > 0) {  // the CTA before this one takes all of that unit
            at += hi - lo - blk;
            blk = 0;
            advance(p, marks);
        }
    }
    // To the unit at `at`, the one after this.
    __device__ __forceinline__ void advance(const AttnParams &p, const Marks &marks) {
        if (at < end && ++kvh == p.hk) {
            kvh = 0;
            do {
                if (++unit == p.units) {
                    unit = 0;
                    ++seq;
                    sp = marks.span(p, seq);
                }
                blocks_of_unit(p, sp, unit, lo, hi);
            } while (hi <= lo);
        }
    }
    // The next item, while there is one.
    __device__ __forceinline__ bool next(const AttnParams &p, const Marks &marks, Item &it) {
        if (at >= end) return false;
        const int n = p.whole ? hi - lo : min(hi - lo - blk, end - at);
        it.seq = seq;
        it.unit = unit;
        it.kvh = kvh;
        it.lo = lo + blk;
        it.hi = it.lo + n;
        it.sp = sp;
        it.slot = blk == 0 && it.hi == hi ? -1 : blk ? slot : slot + 1;
        at += n;
        blk = 0;
        advance(p, marks);
        return true;
    }
};

// What the join has to know of a CTA, by one thread of it, from its walk's start: the unit whose last
// part the CTA does, and the CTA that does the first; x = -1 where it ends no cut unit.
__device__ __forceinline__ void write_cut(const AttnParams &p, const Walk &w, const Marks &marks) {
    if (p.whole) return;
    const int total = marks.first[p.b];
    int4 cut = make_int4(-1, 0, 0, 0);
    if (w.at < w.end && w.blk > 0 && w.end - w.at >= w.hi - w.lo - w.blk) {
        const int n = runs(p, total);
        int c0 = blockIdx.x - 1;
        while (run_begin(total, c0, n) > w.at - w.blk) --c0;
        cut = make_int4(w.seq, w.unit, w.kvh, c0);
    }
    p.cuts[blockIdx.x] = cut;
}

// For a CTA that has to leave without its work (all its threads do): recorded, and the join, which reads
// every CTA's cut, is told that this one ends no unit.
__device__ __forceinline__ void leave(const AttnParams &p, int code) {
    if (threadIdx.x != 0) return;
    if (p.status) atomicExch(p.status, code);
    wait_prerequisites();  // (the workspace may be an earlier kernel's until then)
    if (!p.whole) p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
}

// Units without blocks: O = 0, lse = -inf.  A unit a CTA in turn, by `warps` warps of it, 16 bytes a thread;
// own: of a unit a CTA.
__device__ __forceinline__ void write_empty(const AttnParams &p, const Marks &marks, const Walk *own, int warp, int warps,
                                            int lane) {
    const int tile_rows = p.qbox * p.hbox, pieces = p.d / 8, all = p.per * tile_rows * pieces;
    auto write = [&](int seq, int kvh, int unit) {
#pragma unroll 2
        for (int e = warp * 32 + lane; e < all; e += warps * 32) {
            const int r = e / pieces, piece = e - r * pieces, t = r >= tile_rows ? 1 : 0, y = r - t * tile_rows,
                      tile = unit * p.per + t;
            const Rows at(p, tile);
            const int i = at.q0 + (y & (p.qbox - 1)), hg = at.h0 + y / p.qbox;
            if (tile >= p.ntiles || hg >= p.group || i >= p.nq) continue;
            const int64_t h = (int64_t)kvh * p.group + hg;
            *reinterpret_cast<uint4 *>(p.out + seq * p.so.b + h * p.so.h + (int64_t)i * p.so.n + 8 * piece) =
                make_uint4(0u, 0u, 0u, 0u);
            if (piece == 0) p.lse[(seq * (int64_t)p.hq + h) * p.nq + i] = -INFINITY;
        }
    };
    if (own) {
        if (own->hi <= own->lo) write(own->seq, own->kvh, own->unit);
        return;
    }
    const int ctas = gridDim.x;
    int turn = 0;  // the CTA whose turn the next unit is
    for (int s0 = 0; s0 < p.b; s0 += 32) {
        unsigned some = __ballot_sync(0xffffffffu, s0 + lane < p.b && marks.empty[min(s0 + lane, p.b - 1)]);
        for (; some; some &= some - 1) {
            const int seq = s0 + __ffs(some) - 1;
            const Span sp = marks.span(p, seq);
            for (int u0 = 0; u0 < p.units; u0 += 32) {
                int lo = 0, hi = 1;
                if (u0 + lane < p.units) blocks_of_unit(p, sp, u0 + lane, lo, hi);
                unsigned none = __ballot_sync(0xffffffffu, hi <= lo);
                for (; none; none &= none - 1) {
                    const int ahead = blockIdx.x - turn, first = ahead < 0 ? ahead + ctas : ahead;
                    for (int kvh = first; kvh < p.hk; kvh += ctas) write(seq, kvh, u0 + __ffs(none) - 1);
                    turn = (turn + p.hk) % ctas;
                }
            }
        }
    }
}

// The page of rows `row` on of key block j of a sequence; p.pages, which lies outside the tensor map
// and comes as zeros, where there is none, or where every row is hidden: behind the length, or before
// `low`, where the window of the unit's first query begins (such pages may long be another sequence's).
__device__ __forceinline__ int page_of(const AttnParams &p, const int32_t *table, int j, int row, int low, int Lk) {
    const int at = j * kTile + row;
    if (at >= Lk || at + p.box <= low) return p.pages;
    const int x = __ldg(table + (at >> p.shift));
    if ((unsigned)x < (unsigned)p.pages) return x;
    if (p.status) atomicExch(p.status, kBadPage);
    return p.pages;
}

// Host side (paged_attn.cu).
// Launches a kernel for rows of `dp` elements (p.N, p.per, p.ctas set), and the join after it.
using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, AttnParams);
int launch_with_join(Kernel kernel, int threads, uint32_t smem, int slot, const AttnCall &c, AttnParams &p, int dp);

// Tiles of 128 rows in pairs (paged_attn_wide.cu).
int launch_wide(const AttnCall &c, AttnParams &p);

}  // namespace paged
}  // namespace linformer
