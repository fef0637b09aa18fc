// Exact softmax attention, forward: for every query row i of every head
//
//     O_i = sum_j p_ij V_j,   p_ij = exp(scale Q_i.K_j - lse_i),
//     lse_i = log sum_j exp(scale Q_i.K_j)
//
// over the keys that the row sees (valid length, causal, sliding window), in one pass
// over the keys: a running reference m and sum l per row, P = exp(s - m) in bf16 for the
// second product.  Any m near the maximum serves (bf16 and fp32 keep their relative
// precision; P is rounded to bf16 because the tensor cores take it so, at most 2^-8 of each term),
// so m is the maximum of the row's first block and taken anew, with O and l rescaled, only when a
// later block's maximum outgrows it by 2^kOutgrown.
// The n x n scores never leave the SM.
//
// Persistent CTAs take work items one after another: a pair of 128-row query tiles of
// one key/value head, and (with few items) one part of the keys, whose partial result a
// second kernel joins.  A tile's 128 rows are 128 positions of one query head, or, when
// there are fewer positions, several heads of the group that shares the key/value head:
// single-token decoding reads each key block once for the whole group.
//   warps 0-3, 4-7  softmax of tile 0 and tile 1: one thread a row, S out of TMEM, P back
//   warp 8          lane 0: TMA loads (Q per item; K and V blocks through a ring);
//                   lanes 1-31: zero the rows of V past the valid length (P is 0 there,
//                   but 0 x NaN is not)
//   warps 9, 10     one thread each issues a tile's S = Q.K^T (both from shared memory) and
//                   O += P.V (P from TMEM); a thread of its own per tile, since a product
//                   takes about 350 cycles more from issue to notice than it computes, and
//                   one thread would spend them waiting while the other tile is ready
// Tensor memory: head dimension up to 64: S0 S1 (128 columns each), P0 P1 (64), O0 O1
// (64): S of the next block is computed while this block's exponentials are taken.  Up to
// 128: S0 S1 with P over the first half of S, O0 O1 (128): the next S waits for P.V.
//
// Bound by the chain product -> exponentials -> product and, back to back, by the board's
// power: b h = 192, n = 4096, d = 64: 740 us, 1.11 PFLOP/s (special-function unit and tensor pipe
// 50 % busy each); 64 causal heads of 8192, d = 128: 782 us, 1.40 PFLOP/s.  One
// token over 8192 keys, d = 128: bound by memory, 82 % of its peak (keys split six ways an SM).
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "softmax_attn.cuh"
#include "sm100_ptx.cuh"
#include "work_queue.cuh"

namespace linformer {
namespace sattn {
namespace {

using namespace ptx;

// Twelve warps (one idle), 168 registers each at launch; the two warpgroups that do the
// arithmetic take registers from the third: 2 x 208 + 88 = 3 x 168.
constexpr int kThreads = 384;
constexpr uint32_t kMathRegs = 208, kIssueRegs = 88;
static_assert(2 * kMathRegs + kIssueRegs == 3 * 168, "register split");
constexpr int kLoadWarp = 8, kMmaWarp = 9;
// log2 of the growth of the maximum that is left unscaled: sums reach 2^16 times the keys times
// the largest value (2^8 instead: causal 8192, d = 128, 3 % slower; 2^40: the same as 2^16)
constexpr float kOutgrown = 16.f;
constexpr float kLog2e = 1.4426950408889634f;

struct FwdParams {
    const int32_t *q_lengths, *k_lengths;
    __nv_bfloat16 *out;
    Strides so;
    float *lse;
    float *part_o, *part_lse;  // with splits: [split][b][hq][nq][DP] and [split][b][hq][nq]
    int b, hq, hk, group, nq, nk, d, causal, window;
    int qbox, hbox, nch, ntiles, npairs, nsplit, units, some, order;
    int items;
    float scale, scale_log2;
    int wide;  // O takes 32-byte stores
    int *queue;  // items taken so far beyond each CTA's first
    int *status;
};

// How a CTA comes by its items: in turn, in turn and in sets of heads, from a counter.
enum { kInTurn, kInSets, kFromQueue };

template <int DP>
struct Layout {
    static constexpr bool kSep = DP == 64;  // P beside S, not over it
    static constexpr int kStages = DP == 64 ? 10 : 4;
    static constexpr uint32_t kTileBytes = kTile * DP * 2;
    static constexpr uint32_t kS = 0, kP = kSep ? 256 : 0, kPStep = kSep ? 64 : 128;
    static constexpr uint32_t kO = kSep ? 384 : 256;
    static constexpr uint32_t kSmem = 1024 + (2 + kStages) * kTileBytes + 512;
};

// One query tile of an item.
struct Tile {
    int q0, h0;      // first position, first query head in the group
    int lo, hi;      // key blocks
    bool live;       // exists (it has outputs to write)
};
struct Item {
    int batch, kvh, split;
    Span sp;
    Tile t[2];
    int lo, hi;  // union of the tiles' blocks
};

// kSets: the heads come in sets (a variant of its own: without them every role's code is shorter,
// 16 causal heads of 8192, d = 128: 878 us against 898).
template <bool kSets>
__device__ __forceinline__ Item load_item(const FwdParams &p, int idx) {
    Item it;
    // (32-bit divisions, and none where the divisor is often one: every role does this for
    // every item)
    int rank, u;
    place<kSets>(idx, p.npairs * p.nsplit, p.units, p.some, rank, u);
    it.split = 0;
    if (p.nsplit > 1) {
        const int r = rank;
        rank = r / p.nsplit;
        it.split = r - rank * p.nsplit;
    }
    // causal rows further down see more keys: the longest items first
    const int pair = p.causal ? p.npairs - 1 - rank : rank;
    it.batch = u / p.hk;
    it.kvh = u - it.batch * p.hk;
    it.sp = Span{clamp_length(p.q_lengths, it.batch, p.nq),
                 clamp_length(p.k_lengths, it.batch, p.nk), p.causal, p.window};
    it.lo = 1 << 30;
    it.hi = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int lin = 2 * pair + t;
        Tile &x = it.t[t];
        x.live = lin < p.ntiles;
        const int qt = p.nch > 1 ? lin / p.nch : lin;
        x.q0 = qt * p.qbox;
        x.h0 = (lin - qt * p.nch) * p.hbox;
        x.lo = x.hi = 0;
        const int last = min(x.q0 + p.qbox, it.sp.Lq) - 1;
        if (x.live && last >= x.q0) {
            const int e = it.sp.end(last), f = it.sp.first(x.q0);
            if (e > f) {
                x.lo = f / kTile;
                x.hi = (e + kTile - 1) / kTile;
                it.lo = min(it.lo, x.lo);
                it.hi = max(it.hi, x.hi);
            }
        }
    }
    if (it.hi > it.lo && p.nsplit > 1) {  // this item's share of the blocks
        const int per = (it.hi - it.lo + p.nsplit - 1) / p.nsplit;
        const int a = it.lo + it.split * per, z = min(it.hi, a + per);
        it.lo = a;
        it.hi = max(a, z);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            it.t[t].lo = max(it.t[t].lo, a);
            it.t[t].hi = min(it.t[t].hi, z);
        }
    }
    return it;
}

// Whether the item's last block holds rows past the valid length that are in memory (rows
// past the tensor's end come in as zero).
__device__ __forceinline__ bool ragged_end(const Item &it, int nk) {
    return it.hi > it.lo && it.sp.Lk < nk && it.hi * kTile > it.sp.Lk;
}

struct Barriers {
    uint64_t q_full[2], q_free[2], s_full[2], s_free[2], p_full[2], p_half[2], pv_done[2], o_free[2];
    // fix_wanted takes an arrival from both issuing threads: the next fix then waits until both
    // have passed their wait on the last one, and neither is ever two phases behind a single bit
    // of parity, however far a tile without keys runs ahead.  (A barrier per V stage instead:
    // causal 8192, d = 128: 820 us against 786.)
    uint64_t fix_wanted, fixed, drain[2];
    uint64_t full[10], empty[10];
    Queue queue;
    uint32_t tmem;
    int abort;
};

static_assert(sizeof(Barriers) <= 512, "room for the barriers");

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
__device__ __noinline__ void mask_block(uint32_t t, int a, int w) {
#pragma unroll 1
    for (int c = 0; c < kTile; c += 32) {
        uint32_t v[32];
        tmem_ld32(t + c, v);
        mask_chunk(v, a - c, w);
        tmem_st32(t + c, v);
    }
}
// O times f, eight columns at a time (the caller's scores are in registers).
__device__ __noinline__ void rescale_output(uint32_t t, int columns, float f) {
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

template <int DP, int kOrder>
__global__ void __launch_bounds__(kThreads, 1)
softmax_attn_fwd_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                        const __grid_constant__ CUtensorMap tV, const FwdParams p) {
    using C = Layout<DP>;
    constexpr bool kQueue = kOrder == kFromQueue, kSets = kOrder == kInSets || (kQueue && DP == 128);
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sKV = smem + 2 * C::kTileBytes;
    Barriers *bar = reinterpret_cast<Barriers *>(sKV + C::kStages * C::kTileBytes);
    volatile int *abort_flag = &bar->abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar->q_full[t], 1);
            mbar_init(&bar->q_free[t], 1);
            mbar_init(&bar->s_full[t], 1);
            mbar_init(&bar->s_free[t], 4);
            mbar_init(&bar->p_full[t], 4);
            mbar_init(&bar->p_half[t], 4);
            mbar_init(&bar->pv_done[t], 1);
            mbar_init(&bar->o_free[t], 4);
        }
        mbar_init(&bar->fix_wanted, 2);
        mbar_init(&bar->fixed, 31);
        mbar_init(&bar->drain[0], 1);
        mbar_init(&bar->drain[1], 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 2);  // one arrival from each tile's products
        }
        if (kQueue) init_queue(bar->queue, 31 + 2 + 8);  // zeroing lanes, issuing threads, warps
        bar->abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tQ);
        prefetch_tmap(&tK);
        prefetch_tmap(&tV);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bar->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    // a single thread's next item
    auto advance = [&](int &idx, int &turn) {
        if (kQueue) return thread_next(bar->queue, turn, idx, p.status, abort_flag);
        idx += gridDim.x;
        return true;
    };
    if (p.nsplit > 1 && tid == 0) launch_dependents();  // the join, which waits for this grid's end

    if (warp >= kLoadWarp) {
        setmaxnreg_dec<kIssueRegs>();
        if (warp == kLoadWarp) {
            if (lane == 0) {  // ---------------- loads
                if (kQueue) wait_prerequisites();  // the counter
                int ring = 0, nq[2] = {0, 0}, turn = 0;
                bool ok = true;
                for (int idx = blockIdx.x; idx < p.items && ok;) {
                    const int following = gridDim.x + (kQueue ? atomicAdd(p.queue, 1) : idx);
                    const Item it = load_item<kSets>(p, idx);
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (it.t[t].hi <= it.t[t].lo) continue;
                        if (nq[t] > 0 && !thread_spin(&bar->q_free[t], (nq[t] - 1) & 1, p.status, 70, abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bar->q_full[t], (uint32_t)(p.qbox * p.hbox * DP * 2));
                        for (int h = 0; h < DP / 64; ++h)
                            tma_load_5d(sQ + t * C::kTileBytes + h * 16384, &tQ, &bar->q_full[t], h * 64,
                                        it.t[t].q0, it.t[t].h0, it.kvh, it.batch);
                        ++nq[t];
                    }
                    for (int j = it.lo; j < it.hi && ok; ++j)
                        for (int kv = 0; kv < 2; ++kv, ++ring) {
                            const int s = ring % C::kStages;
                            if (ring >= C::kStages &&
                                !thread_spin(&bar->empty[s], (ring / C::kStages - 1) & 1, p.status, 71, abort_flag)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(&bar->full[s], C::kTileBytes);
                            for (int h = 0; h < DP / 64; ++h)
                                tma_load_5d(sKV + s * C::kTileBytes + h * 16384, kv ? &tV : &tK, &bar->full[s],
                                            h * 64, j * kTile, 0, it.kvh, it.batch);
                        }
                    if (kQueue) ok = ok && tell(bar->queue, turn, following, p.status, abort_flag);
                    idx = following;
                }
                // no copy outlives the CTA
                for (int t = 0; t < 2; ++t)
                    if (nq[t] > 0) mbar_wait_drain(&bar->q_full[t], (nq[t] - 1) & 1);
                for (int i = max(0, ring - C::kStages); i < ring; ++i)
                    mbar_wait_drain(&bar->full[i % C::kStages], (i / C::kStages) & 1);
            } else {  // ---------------- V rows past the valid length
                int ring = 0, nfix = 0;
                bool ok = true;
                for (int idx = blockIdx.x, turn = 0; idx < p.items && ok; ok = advance(idx, turn)) {
                    const Item it = load_item<kSets>(p, idx);
                    const int blocks = max(0, it.hi - it.lo);
                    ring += 2 * blocks;
                    if (!ragged_end(it, p.nk)) continue;
                    // the issuing threads have seen the block land
                    if (!thread_spin(&bar->fix_wanted, nfix & 1, p.status, 72, abort_flag)) break;
                    ++nfix;
                    const int s = (ring - 1) % C::kStages;
                    zero_rows<DP, kTile>(sKV + s * C::kTileBytes, it.sp.Lk - (it.hi - 1) * kTile, lane - 1, 31);
                    fence_proxy_async_smem();
                    mbar_arrive(&bar->fixed);
                }
            }
            __syncwarp();
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            const int t = warp - kMmaWarp;
            if (elect_one()) {  // ---------------- products of tile t
                const uint32_t idesc_s = idesc_f16(128, 128, 1, 0, 0), idesc_o = idesc_f16(128, DP, 1, 0, 1);
                const uint64_t dq = sdesc(smem_u32(sQ + t * C::kTileBytes), 16, 1024, kSwizzle128B);
                const uint32_t tS = tmem + C::kS + 128 * t, tP = tmem + C::kP + C::kPStep * t,
                               tO = tmem + C::kO + DP * t;
                // The ring's entries in pairs, K and V of a block: where the next K and the next V
                // stand (counted up, not divided out: this thread's own instructions are on the
                // path from one product to the next).
                constexpr int kPairs = C::kStages / 2;
                struct At {
                    int s = 0;
                    uint32_t parity = 0;
                    __device__ __forceinline__ void next() {
                        if (++s == kPairs) {
                            s = 0;
                            parity ^= 1u;
                        }
                    }
                } ak, av;
                const uint64_t dk0 = sdesc(smem_u32(sKV), 16, 1024, kSwizzle128B),
                               dv0 = sdesc(smem_u32(sKV) + C::kTileBytes, 16384, 1024, kSwizzle128B);
                int n = 0, items = 0;  // the tile's blocks and items
                int nfix = 0;
                bool ok = true;
                for (int idx = blockIdx.x, turn = 0; idx < p.items && ok; ok = ok && advance(idx, turn)) {
                    const Item it = load_item<kSets>(p, idx);
                    const int lo = t ? it.t[1].lo : it.t[0].lo, hi = t ? it.t[1].hi : it.t[0].hi;
                    const bool fix = ragged_end(it, p.nk);
                    int ns = n;  // blocks of the tile whose S has been issued
                    // S of block j: once the last S has been read and, with P over S, its product
                    // is done
                    auto score = [&](int j) {
                        uint64_t *full = &bar->full[2 * ak.s], *empty = &bar->empty[2 * ak.s];
                        if (!thread_spin(full, ak.parity, p.status, 73, abort_flag)) return false;
                        const uint64_t k = dk0 + (uint64_t)(ak.s * (int)(2 * C::kTileBytes >> 4));
                        ak.next();
                        if (j < lo || j >= hi) {
                            mbar_arrive(empty);
                            return true;
                        }
                        if (j == lo && !thread_spin(&bar->q_full[t], items & 1, p.status, 74, abort_flag)) return false;
                        if (ns > 0 && !thread_spin(C::kSep ? &bar->s_free[t] : &bar->pv_done[t], (ns - 1) & 1,
                                                   p.status, 75, abort_flag))
                            return false;
                        ++ns;
                        tc_fence_after();
    #pragma unroll
                        for (int x = 0; x < DP / 16; ++x) {
                            const uint64_t off = (uint64_t)((x >> 2) * 1024 + (x & 3) * 2);
                            mma_ss(tS, dq + off, k + off, idesc_s, x > 0 ? 1u : 0u);
                        }
                        mma_commit(&bar->s_full[t]);
                        mma_commit(empty);
                        if (j == hi - 1) mma_commit(&bar->q_free[t]);
                        return true;
                    };
                    // O += P.V of block j
                    auto output = [&](int j) {
                        uint64_t *full = &bar->full[2 * av.s + 1], *empty = &bar->empty[2 * av.s + 1];
                        if (!thread_spin(full, av.parity, p.status, 76, abort_flag)) return false;
                        const uint64_t v = dv0 + (uint64_t)(av.s * (int)(2 * C::kTileBytes >> 4));
                        if (fix && j == it.hi - 1) {
                            mbar_arrive(&bar->fix_wanted);
                            if (!thread_spin(&bar->fixed, nfix++ & 1, p.status, 77, abort_flag)) return false;
                        }
                        av.next();
                        if (j < lo || j >= hi) {
                            mbar_arrive(empty);
                            return true;
                        }
                        // P over S comes in halves of 64 keys: the first half's products run while
                        // the other is in its exponentials
                        if (!thread_spin(C::kSep ? &bar->p_full[t] : &bar->p_half[t], n & 1, p.status, 78, abort_flag))
                            return false;
                        if (j == lo && items > 0 &&
                            !thread_spin(&bar->o_free[t], (items - 1) & 1, p.status, 79, abort_flag))
                            return false;
                        tc_fence_after();
    #pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma_ts(tO, tP + 8 * x, v + (uint64_t)(128 * x), idesc_o, (j > lo || x > 0) ? 1u : 0u);
                        if (!C::kSep) {
                            if (!thread_spin(&bar->p_full[t], n & 1, p.status, 68, abort_flag)) return false;
                            tc_fence_after();
                        }
                        ++n;
    #pragma unroll
                        for (int x = 4; x < 8; ++x) mma_ts(tO, tP + 8 * x, v + (uint64_t)(128 * x), idesc_o, 1u);
                        mma_commit(&bar->pv_done[t]);
                        mma_commit(empty);
                        return true;
                    };
                    // P beside S: S(j + 1) before O(j); P over S: after it
                    if (C::kSep && it.hi > it.lo) ok = score(it.lo);
                    for (int j = it.lo; j < it.hi && ok; ++j) {
                        if (C::kSep) ok = (j + 1 >= it.hi || score(j + 1)) && output(j);
                        else ok = score(j) && output(j);
                    }
                    if (hi > lo) ++items;
                }
                mma_commit(&bar->drain[t]);
                mbar_wait_drain(&bar->drain[t], 0);
            }
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<kMathRegs>();  // ---------------- softmax of one tile, one thread a row
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + C::kS + 128 * t + lanes, tP = tmem + C::kP + C::kPStep * t + lanes,
                       tO = tmem + C::kO + DP * t + lanes;
        const float sl = p.scale_log2;
        const int qi = row % p.qbox, hi_ = row / p.qbox;  // position and head within the tile
        int n = 0;
        bool ok = true;
        // P.V of the tile's block before this one is done: P may be written over, O rescaled
        auto last_product = [&](bool any) {
            if (any) {
                ok = warp_spin(&bar->pv_done[t], (n - 1) & 1, p.status, 81, abort_flag);
                tc_fence_after();
            }
            return ok;
        };
        // What the thread's row does in an item, worked out while the item before it ends.
        struct Row {
            int lo, hi, first, end;
            bool live, valid, warp_valid;
        };
        auto row_of = [&](int idx) {
            const Item it = load_item<kSets>(p, min(idx, p.items - 1));
            const Tile x = t ? it.t[1] : it.t[0];
            const int i = x.q0 + qi;
            Row r;
            r.live = x.live;
            r.lo = x.lo;
            r.hi = x.hi;
            r.valid = x.live && hi_ < p.hbox && x.h0 + hi_ < p.group && i < it.sp.Lq;
            r.first = r.valid ? it.sp.first(i) : 0;
            r.end = r.valid ? it.sp.end(i) : (1 << 30);
            r.warp_valid = __any_sync(0xffffffffu, r.valid);
            return r;
        };
        Row next = row_of(blockIdx.x);
        // a warp's next item
        auto following = [&](int idx, int &turn) {
            if (kQueue) ok = warp_next(bar->queue, turn, idx, p.status, abort_flag);
            else idx += gridDim.x;
            return idx;
        };
        for (int idx = blockIdx.x, turn = 0; idx < p.items && ok;) {
            const Row now = next;
            if (!now.live) {
                idx = following(idx, turn);
                next = row_of(idx);
                continue;
            }
            const int lo = now.lo, hi = now.hi, first = now.first, end = now.end;
            const bool valid = now.valid, warp_valid = now.warp_valid;
            float m = -INFINITY, l = 0.f;  // maximum (of the raw scores), sum of 2^((s - m) sl)
            for (int j = lo; j < hi; ++j, ++n) {
                if (!warp_spin(&bar->s_full[t], n & 1, p.status, 80, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!warp_valid) {  // only takes part in the barriers
                    __syncwarp();
                    if (C::kSep && lane == 0) mbar_arrive(&bar->s_free[t]);
                    // no second arrival on p_full before the other warps' first
                    if (C::kSep && !last_product(j > lo)) break;
                    __syncwarp();
                    if (!C::kSep && lane == 0) mbar_arrive(&bar->p_half[t]);
                    if (lane == 0) mbar_arrive(&bar->p_full[t]);
                    continue;
                }
                // Masked keys (whatever they hold) become -inf in place, in a rolled loop: the
                // few blocks at a mask's edge must not widen the code of the others.
                const int k0 = j * kTile;
                if (__any_sync(0xffffffffu, first > k0 || end < k0 + kTile)) {
                    mask_block(tS, first - k0, first < end ? end - first : 0);
                }
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_async(tS + 32 * c, v[c]);
                tmem_wait_ld(v[0]);
                tie32(v[1]);
                tie32(v[2]);
                tie32(v[3]);
                if (C::kSep) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->s_free[t]);
                }
                const float mx = fmaxf(fmaxf(max_chunk(v[0]), max_chunk(v[1])),
                                       fmaxf(max_chunk(v[2]), max_chunk(v[3])));
                if (__any_sync(0xffffffffu, valid && (mx - m) * sl > kOutgrown)) {
                    if (!last_product(j > lo)) break;
                    const float mn = fmaxf(m, mx);
                    const float f = mn == -INFINITY ? 1.f : ex2_approx((m - mn) * sl);
                    l *= f;
                    m = mn;
                    if (j > lo) rescale_output(tO, DP, f);
                }
                const float off = m == -INFINITY ? 0.f : -m * sl;
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                if (C::kSep) {
                    // P beside S is written at the end: until then the last block's is in use
                    uint32_t o[4][16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) exp_chunk(v[c], o[c], sl, off, sum0, sum1);
                    if (!last_product(j > lo)) break;
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_st16_async(tP + 16 * c, o[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[16];
                        exp_chunk(v[c], o, sl, off, sum0, sum1);
                        tmem_st16_async(tP + 16 * c, o);
                        if (c == 1) {
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar->p_half[t]);
                        }
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->p_full[t]);
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
            }
            if (!ok) break;
            // O / l out of TMEM; rows without keys give O = 0 and lse = -inf
            const bool some = hi > lo;
            // (derived again: kept through the loop, it would cost registers there)
            int again = idx;
            asm volatile("" : "+r"(again));
            const Item it = load_item<kSets>(p, again);
            const Tile x = t ? it.t[1] : it.t[0];
            const int i = x.q0 + qi, hg = x.h0 + hi_;
            const bool exists = hi_ < p.hbox && hg < p.group && i < p.nq;
            idx = following(idx, turn);
            if (!ok) break;
            next = row_of(idx);
            const bool dead = !valid || l == 0.f;
            const float inv = dead ? 0.f : 1.f / l;
            const float lse = dead ? -INFINITY : m * p.scale + logf(l);
            const int64_t head = (int64_t)it.kvh * p.group + hg;
            const int64_t r = ((int64_t)it.batch * p.hq + head) * p.nq + i;
            const int64_t pr = (int64_t)it.split * p.b * p.hq * p.nq + r;
            __nv_bfloat16 *dst = p.out + it.batch * p.so.b + head * p.so.h + (int64_t)i * p.so.n;
            if (some) {
                if (!warp_spin(&bar->pv_done[t], (n - 1) & 1, p.status, 82, abort_flag)) break;
                tc_fence_after();
                if (warp_valid) {
                    uint32_t o[DP / 32][32];
#pragma unroll
                    for (int c = 0; c < DP / 32; ++c) tmem_ld32_async(tO + 32 * c, o[c]);
                    tmem_wait_ld(o[0]);
#pragma unroll
                    for (int c = 1; c < DP / 32; ++c) tie32(o[c]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->o_free[t]);
#pragma unroll
                    for (int c = 0; c < DP; c += 16) {
                        float y[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = dead ? 0.f : __uint_as_float(o[c / 32][c % 32 + e]) * inv;
                        if (p.nsplit > 1) {
                            if (dead) continue;
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<float4 *>(p.part_o + pr * DP + c + e) =
                                    make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                        } else if (exists && c < p.d) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = pack2(y[2 * e], y[2 * e + 1]);
                            // one store of 32 bytes where the tensor allows it: a warp's store
                            // touches 32 rows, and each row's line costs a cycle of the
                            // load/store unit
                            if (p.wide) {
                                store32(dst + c, w);
                            } else {
                                *reinterpret_cast<uint4 *>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
                                if (c + 8 < p.d) *reinterpret_cast<uint4 *>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    }
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->o_free[t]);
                }
            }
            if (!(some && warp_valid) && exists && p.nsplit == 1)
#pragma unroll 1
                for (int c = 0; c < p.d; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
            if (exists) (p.nsplit > 1 ? p.part_lse[pr] : p.lse[r]) = lse;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the parts of a row: lse = log sum_s exp(lse_s), O = sum_s exp(lse_s - lse) O_s.
// One warp a row.
template <int DP>
__global__ void __launch_bounds__(128) join_kernel(const FwdParams p) {
    const int64_t rows = (int64_t)p.b * p.hq * p.nq;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    wait_prerequisites();
    float m = -INFINITY;
    for (int s = lane; s < p.nsplit; s += 32) m = fmaxf(m, p.part_lse[s * rows + r]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int i = (int)(r % p.nq), h = (int)(r / p.nq % p.hq), b = (int)(r / ((int64_t)p.nq * p.hq));
    __nv_bfloat16 *dst = p.out + b * p.so.b + h * p.so.h + (int64_t)i * p.so.n;
    constexpr int E = DP / 32;
    float acc[E] = {}, sum = 0.f;
    if (m != -INFINITY) {
        for (int s = 0; s < p.nsplit; ++s) {
            const float w = __expf(p.part_lse[s * rows + r] - m);
            if (w == 0.f) continue;  // a part without keys wrote no O
            sum += w;
            const float *src = p.part_o + (s * rows + r) * DP + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += w * src[e];
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    if (lane * E < p.d) {
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t *>(dst + lane * E + e) = pack2(acc[e] * inv, acc[e + 1] * inv);
    }
    if (lane == 0) p.lse[r] = m == -INFINITY ? -INFINITY : m + logf(sum);
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

constexpr int kMaxDev = 64;

__global__ void zero_queue_kernel(int *queue) {
    launch_dependents();
    *queue = 0;
}

template <int DP>
int launch(const Call &c, FwdParams &p) {
    using C = Layout<DP>;
    CUtensorMap tQ, tK, tV;
    if (!encode_rows(&tQ, c.Q, c.sQ, c.b, c.hq, p.group, c.nq, c.d, p.qbox, p.hbox) ||
        !encode_rows(&tK, c.K, c.sK, c.b, c.hk, 1, c.nk, c.d, kTile, 1) ||
        !encode_rows(&tV, c.V, c.sV, c.b, c.hk, 1, c.nk, c.d, kTile, 1))
        return LINFORMER_ERR_LAUNCH;
    char *ws = nullptr;
    const size_t parts = p.nsplit > 1 ? (size_t)c.b * c.hq * c.nq * p.nsplit : 0;
    const bool queue = p.order == kFromQueue;
    if ((parts || queue) &&
        workspace_alloc(reinterpret_cast<void **>(&ws), (parts * (DP + 1) + (queue ? 1 : 0)) * sizeof(float), c.stream) !=
            LINFORMER_OK)
        return LINFORMER_ERR_ALLOC;
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_lse = p.part_o + parts * DP;
    p.queue = reinterpret_cast<int *>(p.part_lse + parts);
    const auto kernel = queue ? softmax_attn_fwd_kernel<DP, kFromQueue>
                        : p.order == kInSets ? softmax_attn_fwd_kernel<DP, kInSets>
                                             : softmax_attn_fwd_kernel<DP, kInTurn>;
    int st = allow_smem(reinterpret_cast<const void *>(kernel), C::kSmem, (DP == 64 ? 4 : 7) + p.order);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = c.stream;
    cfg.attrs = attr;
    if (!st && queue) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX, c.stream);
        zero_queue_kernel<<<1, 1, 0, c.stream>>>(p.queue);
        if (cudaGetLastError() != cudaSuccess) st = LINFORMER_ERR_LAUNCH;
    }
    if (!st) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX, c.stream);
        cfg.gridDim = dim3((unsigned)std::min(p.items, device_sms()));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cfg.numAttrs = queue ? 1 : 0;  // set up beside the kernel that zeroes the counter
        if (cudaLaunchKernelEx(&cfg, kernel, tQ, tK, tV, p) != cudaSuccess) {
            cudaGetLastError();
            st = LINFORMER_ERR_LAUNCH;
        }
    }
    if (!st && p.nsplit > 1) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX, c.stream);
        const int64_t rows = (int64_t)c.b * c.hq * c.nq;
        // set up while the parts are computed; it waits for them before it reads
        cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
        cfg.blockDim = dim3(128);
        cfg.dynamicSmemBytes = 0;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, join_kernel<DP>, p) != cudaSuccess) {
            cudaGetLastError();
            st = LINFORMER_ERR_LAUNCH;
        }
    }
    if (ws) workspace_free(ws, c.stream);
    return st;
}

}  // namespace

bool encode_rows(CUtensorMap *m, const void *base, const Strides &s, int b, int heads, int group,
                 int n, int d, int rows, int hrows) {
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (!g_encode) return false;
    // the stride of a dimension of size one is never used, but has to be a legal one
    auto bytes = [](int64_t stride, int64_t count) { return (cuuint64_t)(count > 1 ? stride * 2 : 16); };
    cuuint64_t dims[5] = {(cuuint64_t)d, (cuuint64_t)n, (cuuint64_t)group, (cuuint64_t)(heads / group),
                          (cuuint64_t)b};
    cuuint64_t strides[4] = {bytes(s.n, n), bytes(s.h, group), bytes(s.h * group, heads / group),
                             bytes(s.b, b)};
    cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)hrows, 1, 1};
    cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box,
                    one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel's shared memory, allowed once per device (slot: one per kernel).
int allow_smem(const void *kernel, uint32_t bytes, int slot) {
    static std::atomic<uint8_t> done[kMaxDev][10];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < kMaxDev && done[dev][slot].load(std::memory_order_acquire)) return LINFORMER_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return LINFORMER_ERR_LAUNCH;
    }
    if (dev >= 0 && dev < kMaxDev) done[dev][slot].store(1, std::memory_order_release);
    return LINFORMER_OK;
}

int forward(const Call &c) {
    FwdParams p{};
    p.q_lengths = c.q_lengths;
    p.k_lengths = c.k_lengths;
    p.out = static_cast<__nv_bfloat16 *>(c.out);
    p.so = c.sO;
    p.lse = c.lse;
    p.b = c.b;
    p.hq = c.hq;
    p.hk = c.hk;
    p.group = c.hq / c.hk;
    p.nq = c.nq;
    p.nk = c.nk;
    p.d = c.d;
    p.causal = c.causal;
    p.window = c.window;
    p.scale = c.scale;
    p.scale_log2 = c.scale * kLog2e;
    p.wide = wide_stores(c.out, c.sO, c.d);
    p.status = device_status_ptr();
    // Rows of a tile: 128 positions of one head, or the smallest power of two that holds
    // all positions times as many heads of the group as fit.
    p.qbox = kTile;
    while (p.qbox > 1 && p.qbox / 2 >= c.nq) p.qbox /= 2;
    p.hbox = std::min(kTile / p.qbox, p.group);
    p.nch = (p.group + p.hbox - 1) / p.hbox;
    p.ntiles = (c.nq + p.qbox - 1) / p.qbox * p.nch;
    p.npairs = (p.ntiles + 1) / 2;
    p.units = c.b * c.hk;
    const int64_t whole = (int64_t)p.units * p.npairs;
    if (whole > kMaxItems) return LINFORMER_ERR_SIZE;
    const int sms = device_sms();
    // The keys are split where whole rows give fewer items than SMs; and where a tile has so
    // few rows that a part's result is small beside the keys it reads, down to kWaves items an
    // SM, so that sequences of differing lengths even out.  At least kMinBlocks blocks a part
    // (from 12 blocks on: the second launch costs what a block or two takes).
    constexpr int kMinBlocks = 4, kFirst = 12, kFewRows = 16, kWaves = 6;
    const int reach = c.window ? std::min(c.nk, c.window + kTile) : c.nk;
    const int blocks = (reach + kTile - 1) / kTile;
    const int64_t wanted = p.qbox * p.hbox <= kFewRows ? (kWaves * (int64_t)sms + whole - 1) / whole : sms / whole;
    p.nsplit = blocks < kFirst ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(wanted, blocks / kMinBlocks));
    p.items = (int)whole * p.nsplit;
    // Causal calls take all heads at once (in sets: 2 x 8192 with 32 heads over 8, d = 128, 801 us
    // against 767, 8 x 4096 885 against 824), and so do ragged ones with heads of up to 64 (384
    // heads of 4096: 845 against 760; d = 128: 1226 against 1264).
    const bool uneven = c.k_lengths || c.q_lengths || c.causal;
    p.some = c.causal || (uneven && c.d <= 64)
                 ? p.units
                 : units_at_once(p.npairs, p.units, (int64_t)c.nk * c.d * 4, false, sms);
    // Masked and ragged items differ in length and come from a counter, in calls long enough for
    // the launch that zeroes it.
    p.order = uneven && p.items > 2 * sms ? kFromQueue : p.some < p.units ? kInSets : kInTurn;
    return c.d <= 64 ? launch<64>(c, p) : launch<128>(c, p);
}

}  // namespace sattn
}  // namespace linformer
