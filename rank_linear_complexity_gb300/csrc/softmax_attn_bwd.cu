// Exact softmax attention, backward.  With P_ij = exp(scale Q_i.K_j - lse_i) recomputed
// from the forward's lse, delta_i = dO_i.O_i and
//
//     dP = dO V^T,   dS_ij = P_ij (dP_ij - delta_i),
//     dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K,
//
// two kernels after a small one, each a sum that one CTA owns, so that no gradient is added up
// by atomics and every result repeats bit for bit (where there are few of them they are split
// into parts, which a fourth kernel adds up in their order):
//   rows_kernel  -lse log2(e) and -delta of every query row, for the other two.
//   dq_kernel    a 128-row query tile against its keys: S, dP, then dQ += dS.K.
//   dkv_kernel   a 128-key block against the queries of every head of its group:
//                S^T = K.Q^T and dP^T = V.dO^T, then dV += P^T.dO and dK += dS^T.Q.  With
//                keys as the rows, P^T and dS^T leave the registers of the thread that made
//                them for the tensor memory of the next product: no transpose, no shared
//                memory.
// Seven products instead of five: S and dP are formed twice, which costs less than adding
// partial dQ through memory in a fixed order.  P and dS are rounded to bf16 as operands, since
// the tensor cores take them at the rate of Q's and K's type only so (at most 2^-8 of each term; fp32
// operands would cost several products for one), and delta takes the O that the forward rounded,
// which is what its caller has.  Sums are fp32 in tensor memory.
//
// Both are chains of product -> arithmetic -> product, about 350 cycles from a product's last
// cycle to the arithmetic, so they go in steps of 64 columns with several in flight: tensor
// memory holds, beside the sums, as many slots as fit (64 columns of S and 64 of dP each; two
// or three), and every slot has a warpgroup of its own, one thread a row, 64 columns a thread.
// Whole steps of 128 columns, one in flight and half a step a warpgroup, took 1.25 times as long
// (d = 64).  The last warpgroup issues: warp 0 of it loads (lane 0) and zeroes rows past the
// valid length (lanes 1-31, where 0 x NaN would reach a sum); one thread each of the other
// three issues S, dP and the sums, since such a thread takes about 300 cycles from one product
// to the next (short code that runs now and then, fetched anew each time) and the tensor cores
// would wait for a single one.
// Measured (b h = 76, n = 4096, each launch alone): d = 64: rows 16 us (5.2 TB/s), dQ 373 us
// (1.31 PFLOP/s of its three products), dK and dV 460 to 485 us (1.35 to 1.42 PFLOP/s of four,
// tensor pipe 59 %); d = 128: 30, 664 (1.47, 62 %) and 788 us (1.66, 71 %).  Back to back they draw
// the board's full power and the clock settles at 1650 to 1950 MHz of 2070.
#include <algorithm>
#include <cmath>

#include "softmax_attn.cuh"
#include "sm100_ptx.cuh"
#include "work_queue.cuh"

namespace linformer {
namespace sattn {
namespace {

using namespace ptx;

constexpr int kHalf = 64;  // columns of a step: queries (dK, dV) or keys (dQ)
// G warpgroups do the arithmetic and a last one loads and issues; it hands registers to the
// others, whose shares add up to the launch's.
constexpr int threads_of(int G) { return 128 * (G + 1); }
__host__ __device__ constexpr uint32_t math_regs(int G) { return G == 3 ? 144 : 208; }
__host__ __device__ constexpr uint32_t issue_regs(int G) { return G == 3 ? 80 : 88; }
constexpr uint32_t launch_regs(int G) { return 65536 / threads_of(G) / 8 * 8; }
static_assert(3 * math_regs(3) + issue_regs(3) == 4 * launch_regs(3), "register split");
static_assert(2 * math_regs(2) + issue_regs(2) == 3 * launch_regs(2), "register split");
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
    const int32_t *q_lengths, *k_lengths;
    const __nv_bfloat16 *O, *dO;
    Strides sO, sdO;
    __nv_bfloat16 *dQ, *dK, *dV;
    Strides sdQ, sdK, sdV;
    const float *lse;
    // [b][hq][2 query tiles][2][64]: -lse log2(e) and -delta, as they are added; -inf and 0 for
    // rows that are past the length or see no key
    float *rows;
    int b, hq, hk, group, nq, nk, d, causal, window;
    int qtiles, kblocks;
    int wide;  // bits: dQ, dK, dV take 32-byte stores
    // parts of the steps that an item is split into, and the parts' sums, fp32 [part][b][heads][n][DP]
    int qsplit, ksplit;
    int qsome, ksome;  // heads at a time
    int *queue;        // items taken so far beyond each CTA's first: of the dQ kernel, of the other
    float *part_q, *part_k, *part_v;
    int items;
    float scale, scale_log2;
    int *status;
};

// Columns outside [a, a + w) of 64 in tensor memory become -inf: for the few steps at a
// mask's edge, out of line, away from the code of the others.
constexpr uint32_t kMinusInf = 0xff800000u;
__device__ __noinline__ void hide_outside(uint32_t t, int a, unsigned w) {
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        uint32_t u[32];
        tmem_ld32(t + c, u);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if ((unsigned)(c + e - a) >= w) u[e] = kMinusInf;
        tmem_st32(t + c, u);
    }
}
__device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// Products of two pairs of bf16, added in fp32.
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b) {
    return __uint_as_float(a << 16) * __uint_as_float(b << 16) +
           __uint_as_float(a & 0xffff0000u) * __uint_as_float(b & 0xffff0000u);
}
// 32 columns of a row, scaled and rounded (columns from d on do not exist): 32-byte stores where
// the tensor allows them (a warp's store touches 32 rows, and each row's line costs a cycle of
// the load/store unit), else two of 16 bytes for each.
__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, const uint32_t (&o)[32], int c, int d,
                                          float f, bool zero, bool wide) {
#pragma unroll
    for (int x = 0; x < 32; x += 16) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = zero ? 0u : pack2(__uint_as_float(o[x + 2 * e]) * f, __uint_as_float(o[x + 2 * e + 1]) * f);
        if (wide) {
            if (c + x < d) store32(dst + c + x, w);
        } else {
            if (c + x < d) *reinterpret_cast<uint4 *>(dst + c + x) = make_uint4(w[0], w[1], w[2], w[3]);
            if (c + x + 8 < d) *reinterpret_cast<uint4 *>(dst + c + x + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}
// The same into a part's sums.
__device__ __forceinline__ void store_part(float *dst, const uint32_t (&o)[32], bool zero) {
#pragma unroll
    for (int x = 0; x < 32; x += 8) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = zero ? 0u : o[x + e];
        store32(dst + x, w);
    }
}
// The first d columns of a row as zero.
__device__ __forceinline__ void zero_row(__nv_bfloat16 *dst, int d) {
#pragma unroll 1
    for (int c = 0; c < d; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void zero_part(float *dst, int d) {
#pragma unroll 1
    for (int c = 0; c < d; c += 4) *reinterpret_cast<float4 *>(dst + c) = make_float4(0.f, 0.f, 0.f, 0.f);
}
// 32 N columns of tensor memory, one wait for all.
template <int N>
__device__ __forceinline__ void load_columns(uint32_t t, uint32_t (&o)[N][32]) {
#pragma unroll
    for (int c = 0; c < N; ++c) tmem_ld32_async(t + 32 * c, o[c]);
    tmem_wait_ld(o[0]);
#pragma unroll
    for (int c = 1; c < N; ++c) tie32(o[c]);
}

// D (128 x 64) = A (128 rows of DP) . B (64 rows of DP)^T, both in shared memory.
template <int DP>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b) {
    const uint32_t idesc = idesc_f16(128, kHalf, 1, 0, 0);
    const uint64_t da = sdesc(a, 16, 1024, kSwizzle128B), db = sdesc(b, 16, 1024, kSwizzle128B);
#pragma unroll
    for (int x = 0; x < DP / 16; ++x)
        mma_ss(d, da + (uint64_t)((x >> 2) * 1024 + (x & 3) * 2), db + (uint64_t)((x >> 2) * 512 + (x & 3) * 2),
               idesc, x > 0 ? 1u : 0u);
}
// D (128 x DP) += A (128 x 64, packed in 32 columns of tensor memory) . B (64 rows of DP).
template <int DP>
__device__ __forceinline__ void mma_sum(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    const uint32_t idesc = idesc_f16(128, DP, 1, 0, 1);
    const uint64_t db = sdesc(b, 8192, 1024, kSwizzle128B);
#pragma unroll
    for (int x = 0; x < kHalf / 16; ++x)
        mma_ts(d, a + 8 * x, db + (uint64_t)(128 * x), idesc, (acc || x > 0) ? 1u : 0u);
}

// 64 N rows of DP columns, each 64 columns a tile of its own (maps have boxes of 64 x 64).
template <int DP, int N>
__device__ __forceinline__ void load_rows(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int row,
                                          int head, int group, int batch) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
#pragma unroll
        for (int r = 0; r < N; ++r)
            tma_load_5d(dst + (c * N + r) * 8192, m, bar, c * 64, row + 64 * r, head, group, batch);
}

// Where a step stands in a ring of N = some times G positions: the position (its stage and its
// barriers of every kind), the ring's phase, and the slot.
template <int G, int N>
struct Ring {
    uint32_t pos = 0, phase = 0, slot = 0;
    // the step G before: the slot's last user (its phase; the first G steps find a fresh
    // barrier, whose phase -1 counts as over)
    __device__ __forceinline__ uint32_t before() const { return pos >= G ? pos - G : pos + N - G; }
    __device__ __forceinline__ uint32_t phase_before() const { return pos >= G ? phase : phase ^ 1u; }
    __device__ __forceinline__ void next() {
        ++pos;
        slot = slot == G - 1 ? 0 : slot + 1;
        if (pos == N) pos = 0, phase ^= 1u;
    }
};

// ---------------------------------------------------------------- row values
// -lse log2(e) and -delta = -dO.O of a query tile's 128 rows, eight warps of sixteen rows; a row
// is read by DP / 8 lanes, 16 bytes each.  Bound by memory: O and dO once.
constexpr int kRowsThreads = 256;
template <int DP>
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const BwdParams p) {
    launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x < 2) p.queue[threadIdx.x] = 0;
    constexpr int kLanes = DP / 8, kAtOnce = 32 / kLanes, kTurns = 16 / kAtOnce;
    const int unit = blockIdx.x / p.qtiles, tile = blockIdx.x - unit * p.qtiles;
    const int batch = unit / p.hq, head = unit - batch * p.hq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane % kLanes * 8;
    const int Lq = clamp_length(p.q_lengths, batch, p.nq);
    const int r0 = tile * kTile + 16 * warp + lane / kLanes;  // the lane's row of the first turn
    const __nv_bfloat16 *o = p.O + batch * p.sO.b + head * p.sO.h + col;
    const __nv_bfloat16 *g = p.dO + batch * p.sdO.b + head * p.sdO.h + col;
    uint4 a[kTurns], b[kTurns];
    float x[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const int i = r0 + t * kAtOnce;
        a[t] = b[t] = make_uint4(0u, 0u, 0u, 0u);
        x[t] = -INFINITY;
        if (i < Lq) {
            if (col < p.d) {
                a[t] = __ldg(reinterpret_cast<const uint4 *>(o + (int64_t)i * p.sO.n));
                b[t] = __ldg(reinterpret_cast<const uint4 *>(g + (int64_t)i * p.sdO.n));
            }
            x[t] = __ldg(p.lse + (int64_t)unit * p.nq + i);
        }
    }
    float *dst = p.rows + (int64_t)blockIdx.x * 256 + (warp >> 2) * 128 + 16 * (warp & 3) + lane / kLanes;
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        float y = (dot2(a[t].x, b[t].x) + dot2(a[t].y, b[t].y)) + (dot2(a[t].z, b[t].z) + dot2(a[t].w, b[t].w));
#pragma unroll
        for (int k = kLanes / 2; k; k >>= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
        if (lane % kLanes == 0) {
            dst[t * kAtOnce] = x[t] == -INFINITY ? -INFINITY : -x[t] * kLog2e;
            dst[t * kAtOnce + 64] = x[t] == -INFINITY ? 0.f : -y;
        }
    }
}

// ---------------------------------------------------------------- dQ
template <int DP>
struct DqLayout {
    // slots, one of each warpgroup: S in 64 columns, dP in 64
    static constexpr int G = DP == 64 ? 3 : 2;
    static constexpr uint32_t kTileBytes = kTile * DP * 2, kStepBytes = kHalf * DP * 2;
    static constexpr int kStages = DP == 64 ? 9 : 4;  // of a step's K and V
    // Items whose Q, dO and dQ are held: with two the next one starts while dQ of the last one is
    // formed and written (384 heads of 512: 48 us against 58).  No room at DP = 128.
    static constexpr int kItems = DP == 64 ? 2 : 1;
    static constexpr uint32_t kDq = 128 * G;
    static constexpr uint32_t kSmem = 1024 + kItems * 2 * kTileBytes + kStages * 2 * kStepBytes + 2048 + 1024;
};
// Part i of n of the steps [lo, hi).
__device__ __forceinline__ void take_part(int &lo, int &hi, int i, int n) {
    const int steps = hi - lo;
    hi = lo + steps * (i + 1) / n;
    lo += steps * i / n;
}
struct DqItem {
    int batch, head, q0, lo, hi, part;  // steps [lo, hi) of 64 keys
    Span sp;
};
__device__ __forceinline__ DqItem dq_item(const BwdParams &p, int idx) {
    DqItem it;
    const int units = p.b * p.hq;
    int rank, u;
    place<true>(idx, p.qtiles * p.qsplit, units, p.qsome, rank, u);
    it.part = 0;
    if (p.qsplit > 1) {
        const int x = rank;
        rank = x / p.qsplit;
        it.part = x - rank * p.qsplit;
    }
    const int tile = p.causal ? p.qtiles - 1 - rank : rank;  // longest first
    it.batch = u / p.hq;
    it.head = u - it.batch * p.hq;
    it.q0 = tile * kTile;
    it.sp = Span{clamp_length(p.q_lengths, it.batch, p.nq), clamp_length(p.k_lengths, it.batch, p.nk),
                 p.causal, p.window};
    it.lo = it.hi = 0;
    const int last = min(it.q0 + kTile, it.sp.Lq) - 1;
    if (last >= it.q0) {
        const int e = it.sp.end(last), f = it.sp.first(it.q0);
        if (e > f) {
            it.lo = f / kHalf;
            it.hi = (e + kHalf - 1) / kHalf;
            if (p.qsplit > 1) take_part(it.lo, it.hi, it.part, p.qsplit);
        }
    }
    return it;
}

// Barriers of steps: one of each kind for every position of the ring.
struct DqBarriers {
    uint64_t k_full[9], v_full[9], s_full[9], s_free[9], dp_full[9], ds_full[9], dq_done[9];
    uint64_t q_full[2], q_free[2], acc_full[2], acc_free[2], fix_wanted, fixed_k, fixed_v, drain[3];
    Queue queue;
    uint32_t tmem;
    int abort;
    alignas(16) float rows[2][2 * kTile];  // an item's rows, loaded with its Q and dO
};

static_assert(sizeof(DqBarriers) <= 2048 + 1024, "room for the barriers");

template <int DP>
__global__ void __launch_bounds__(threads_of(DqLayout<DP>::G), 1)
softmax_attn_dq_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                       const __grid_constant__ CUtensorMap tV, const __grid_constant__ CUtensorMap tdO,
                       const BwdParams p) {
    using C = DqLayout<DP>;
    constexpr int G = C::G, kLoadWarp = 4 * G, kMmaWarp = 4 * G + 1;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    // Q and dO of an item at smem + (item % kItems) 2 tiles
    uint8_t *sQ = smem, *sdO = smem + C::kTileBytes, *sKV = smem + C::kItems * 2 * C::kTileBytes;
    DqBarriers *bar = reinterpret_cast<DqBarriers *>(sKV + C::kStages * 2 * C::kStepBytes);  // [K, V] a stage
    volatile int *abort_flag = &bar->abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bar->k_full[i], 1);
            mbar_init(&bar->v_full[i], 1);
            mbar_init(&bar->s_full[i], 1);
            mbar_init(&bar->s_free[i], 4);
            mbar_init(&bar->dp_full[i], 1);
            mbar_init(&bar->ds_full[i], 4);
            mbar_init(&bar->dq_done[i], 1);
        }
        for (int i = 0; i < C::kItems; ++i) {
            mbar_init(&bar->q_full[i], 1);
            mbar_init(&bar->q_free[i], 2 + 4 * G);  // the products, and the rows read
            mbar_init(&bar->acc_full[i], 1);
            mbar_init(&bar->acc_free[i], 8);
        }
        mbar_init(&bar->fix_wanted, 2);
        mbar_init(&bar->fixed_k, 31);
        mbar_init(&bar->fixed_v, 31);
        for (int i = 0; i < 3; ++i) mbar_init(&bar->drain[i], 1);
        init_queue(bar->queue, (p.k_lengths ? 31 : 0) + 3 + 4 * G);  // zeroing lanes, issuing threads, warps
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bar->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    if (warp >= kLoadWarp) {
        setmaxnreg_dec<issue_regs(G)>();
        if (warp == kLoadWarp) {
            if (lane == 0) {
                wait_prerequisites();  // the row values; and only then may the third kernel start
                launch_dependents();
                int steps = 0, nq = 0, t = 0;
                Ring<G, C::kStages> at;
                bool ok = true;
                for (int idx = blockIdx.x; idx < p.items && ok;) {
                    const int following = gridDim.x + atomicAdd(p.queue, 1);
                    const DqItem it = dq_item(p, idx);
                    if (it.hi > it.lo) {
                        const int qb = nq % C::kItems;
                        if (nq >= C::kItems &&
                            !thread_spin(&bar->q_free[qb], (nq / C::kItems - 1) & 1, p.status, 83, abort_flag))
                            break;
                        uint64_t *q_full = &bar->q_full[qb];
                        mbar_arrive_expect_tx(q_full, 2 * C::kTileBytes + 1024);
                        const int g = it.head % p.group, kvh = it.head / p.group;
                        bulk_load(bar->rows[qb], p.rows + (((int64_t)it.batch * p.hq + it.head) * p.qtiles + it.q0 / kTile) * 256,
                                  1024, q_full);
                        load_rows<DP, 2>(sQ + qb * 2 * C::kTileBytes, &tQ, q_full, it.q0, g, kvh, it.batch);
                        load_rows<DP, 2>(sdO + qb * 2 * C::kTileBytes, &tdO, q_full, it.q0, g, kvh, it.batch);
                        ++nq;
                        for (int j = it.lo; j < it.hi; ++j, ++steps, at.next()) {
                            uint8_t *st = sKV + at.pos * 2 * C::kStepBytes;
                            // (dQ comes last: with it all products of a step have been formed)
                            ok = thread_spin(&bar->dq_done[at.pos], at.phase ^ 1, p.status, 84, abort_flag);
                            if (!ok) break;
                            mbar_arrive_expect_tx(&bar->k_full[at.pos], C::kStepBytes);
                            load_rows<DP, 1>(st, &tK, &bar->k_full[at.pos], j * kHalf, 0, kvh, it.batch);
                            mbar_arrive_expect_tx(&bar->v_full[at.pos], C::kStepBytes);
                            load_rows<DP, 1>(st + C::kStepBytes, &tV, &bar->v_full[at.pos], j * kHalf, 0, kvh, it.batch);
                        }
                    }
                    ok = ok && tell(bar->queue, t, following, p.status, abort_flag);
                    idx = following;
                }
                for (int i = max(0, nq - C::kItems); i < nq; ++i)
                    mbar_wait_drain(&bar->q_full[i % C::kItems], (i / C::kItems) & 1);
                for (int i = max(0, steps - C::kStages); i < steps; ++i) {
                    mbar_wait_drain(&bar->k_full[i % C::kStages], (i / C::kStages) & 1);
                    mbar_wait_drain(&bar->v_full[i % C::kStages], (i / C::kStages) & 1);
                }
            } else if (p.k_lengths) {  // K and V rows past the valid length: P and dS are 0 there, but 0 x NaN is not
                int ring = 0, nfix = 0;
                bool ok = true;
                for (int idx = blockIdx.x, t = 0; idx < p.items && ok;
                     ok = ok && thread_next(bar->queue, t, idx, p.status, abort_flag)) {
                    const DqItem it = dq_item(p, idx);
                    if (it.hi <= it.lo) continue;
                    ring += it.hi - it.lo;
                    if (it.sp.Lk >= p.nk || it.hi * kHalf <= it.sp.Lk) continue;
                    if (!thread_spin(&bar->fix_wanted, nfix & 1, p.status, 85, abort_flag)) break;
                    ++nfix;
                    const int row0 = it.sp.Lk - (it.hi - 1) * kHalf;
                    uint8_t *st = sKV + (ring - 1) % C::kStages * 2 * C::kStepBytes;
                    zero_rows<DP, kHalf>(st, row0, lane - 1, 31);
                    zero_rows<DP, kHalf>(st + C::kStepBytes, row0, lane - 1, 31);
                    fence_proxy_async_smem();
                    mbar_arrive(&bar->fixed_k);
                    mbar_arrive(&bar->fixed_v);
                }
            }
            __syncwarp();
        } else if (warp <= kMmaWarp + 1) {
            const bool first = warp == kMmaWarp;  // S = Q K^T; the other thread: dP = dO V^T
            if (elect_one()) {
                int items = 0;
                uint32_t nfix = 0;
                Ring<G, C::kStages> at;
                bool ok = true;
                const uint32_t a0 = smem_u32(first ? sQ : sdO), b = smem_u32(sKV) + (first ? 0 : C::kStepBytes),
                               slots = tmem + (first ? 0 : 64), loaded = smem_u32(first ? bar->k_full : bar->v_full),
                               free = smem_u32(first ? bar->s_free : bar->dq_done),
                               out = smem_u32(first ? bar->s_full : bar->dp_full),
                               fixed = smem_u32(first ? &bar->fixed_k : &bar->fixed_v);
                for (int idx = blockIdx.x, t = 0; idx < p.items && ok;
                     ok = ok && thread_next(bar->queue, t, idx, p.status, abort_flag)) {
                    const DqItem it = dq_item(p, idx);
                    const int steps = it.hi - it.lo;
                    if (steps <= 0) continue;
                    const bool fix = it.sp.Lk < p.nk && it.hi * kHalf > it.sp.Lk;
                    const int qb = items % C::kItems;
                    const uint32_t a = a0 + qb * 2 * C::kTileBytes;
                    ok = thread_spin(&bar->q_full[qb], (items / C::kItems) & 1, p.status, 91, abort_flag);
                    for (int j = steps; j > 0 && ok; --j, at.next()) {
                        ok = thread_spin(loaded + 8 * at.pos, at.phase, p.status, 86, abort_flag) &&
                             thread_spin(free + 8 * at.before(), at.phase_before(), p.status, 88, abort_flag);
                        if (ok && fix && j == 1) {
                            mbar_arrive(&bar->fix_wanted);
                            ok = thread_spin(fixed, nfix++ & 1, p.status, 87, abort_flag);
                        }
                        if (!ok) break;
                        tc_fence_after();
                        mma_scores<DP>(slots + 128 * at.slot, a, b + at.pos * (2 * C::kStepBytes));
                        mma_commit(out + 8 * at.pos);
                    }
                    mma_commit(&bar->q_free[qb]);
                    ++items;
                }
                mma_commit(&bar->drain[first ? 0 : 1]);
                mbar_wait_drain(&bar->drain[first ? 0 : 1], 0);
            }
            __syncwarp();
        } else {
            if (elect_one()) {  // dQ += dS K
                int items = 0;
                Ring<G, C::kStages> at;
                bool ok = true;
                const uint32_t b = smem_u32(sKV), ready = smem_u32(bar->ds_full), done = smem_u32(bar->dq_done);
                for (int idx = blockIdx.x, t = 0; idx < p.items && ok;
                     ok = ok && thread_next(bar->queue, t, idx, p.status, abort_flag)) {
                    const DqItem it = dq_item(p, idx);
                    const int steps = it.hi - it.lo;
                    if (steps <= 0) continue;
                    const int ab = items % C::kItems;
                    const uint32_t acc = tmem + C::kDq + ab * DP;
                    if (items >= C::kItems)
                        ok = thread_spin(&bar->acc_free[ab], (items / C::kItems - 1) & 1, p.status, 93, abort_flag);
                    for (int j = 0; j < steps && ok; ++j, at.next()) {
                        // (dS says that S has been formed, so the block of K has landed)
                        ok = thread_spin(ready + 8 * at.pos, at.phase, p.status, 92, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        mma_sum<DP>(acc, tmem + 128 * at.slot + 64, b + at.pos * (2 * C::kStepBytes), j > 0 ? 1u : 0u);
                        mma_commit(done + 8 * at.pos);
                    }
                    mma_commit(&bar->acc_full[ab]);
                    ++items;
                }
                mma_commit(&bar->drain[2]);
                mbar_wait_drain(&bar->drain[2], 0);
            }
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<math_regs(G)>();
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + 128 * w + lanes, tD = tS + 64;
        const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
        const uint32_t s_full = smem_u32(bar->s_full), s_free = smem_u32(bar->s_free), dp_full = smem_u32(bar->dp_full),
                       ds_full = smem_u32(bar->ds_full);
        int n = 0, items = 0;
        uint32_t pos = w, phase = 0;  // in the ring; the warpgroup's steps are at w, w + G and so on
        // writes dQ of an item, the nth with steps
        auto finish = [&](const DqItem &x, int nth) {
            const int i = x.q0 + row;
            const bool exists = i < p.nq, valid = i < x.sp.Lq;
            __nv_bfloat16 *dst = p.dQ + x.batch * p.sdQ.b + x.head * p.sdQ.h + (int64_t)i * p.sdQ.n;
            float *part = p.part_q + ((((int64_t)x.part * p.b + x.batch) * p.hq + x.head) * p.nq + i) * DP;
            if (w < 2 && x.hi > x.lo) {  // half of the columns each
                const int ab = (nth - 1) % C::kItems;
                if (!warp_spin(&bar->acc_full[ab], ((nth - 1) / C::kItems) & 1, p.status, 96, abort_flag)) return false;
                tc_fence_after();
                uint32_t o[DP / 64][32];
                load_columns(tmem + C::kDq + ab * DP + w * (DP / 2) + lanes, o);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->acc_free[ab]);
                if (exists)
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c) {
                        const int at = w * (DP / 2) + 32 * c;
                        if (p.qsplit > 1) store_part(part + at, o[c], !valid);
                        else store_row(dst, o[c], at, p.d, p.scale, !valid, p.wide & 1);
                    }
            } else if (w == 0 && exists) {
                if (p.qsplit > 1) zero_part(part, DP);
                else zero_row(dst, p.d);
            }
            return true;
        };
        DqItem it = dq_item(p, min((int)blockIdx.x, p.items - 1));
        DqItem last = it;
        int held = -1;
        bool ok = true;
        for (int idx = blockIdx.x, t = 0; idx < p.items;) {
            const int steps = max(0, it.hi - it.lo);
            float nl = 0.f, nd = 0.f;
            if (steps) {  // the row values come with Q and dO
                const int qb = items % C::kItems;
                if (!warp_spin(&bar->q_full[qb], (items / C::kItems) & 1, p.status, 97, abort_flag)) break;
                nl = bar->rows[qb][(row >> 6) * 128 + (row & 63)];
                nd = bar->rows[qb][(row >> 6) * 128 + 64 + (row & 63)];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->q_free[qb]);
                ++items;
            }
            const bool seen = it.q0 + row < it.sp.Lq;
            const int first = seen ? it.sp.first(it.q0 + row) : 0, end = seen ? it.sp.end(it.q0 + row) : 0;
            const unsigned width = end > first ? (unsigned)(end - first) : 0u;
            const int skip = (w + G - n % G) % G;
            for (int j = skip; j < steps; j += G) {
                if (!warp_spin(s_full + 8 * pos, phase, p.status, 94, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // keys that take no part: P = 0 whatever S holds (and rows past the length are
                // zeros in shared memory, so dP is finite)
                const int k0 = (it.lo + j) * kHalf;
                if (__any_sync(0xffffffffu, first > k0 || end < k0 + kHalf)) hide_outside(tS, first - k0, width);
                uint32_t v[2][32];
                load_columns(tS, v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + 8 * pos);
                const float2 off2 = make_float2(nl, nl);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = ffma2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])),
                                               sl2, off2);
                        v[c][e] = __float_as_uint(ex2_approx(y.x));
                        v[c][e + 1] = __float_as_uint(ex2_approx(y.y));
                    }
                if (!warp_spin(dp_full + 8 * pos, phase, p.status, 95, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float2 nd2 = make_float2(nd, nd);
                // 32 columns at a time; dS takes the columns that have been read
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t u[32], o[16];
                    tmem_ld32(tD + 32 * c, u);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = fadd2(make_float2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])), nd2);
                        const float2 z = fmul2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), y);
                        o[e / 2] = pack2(z.x, z.y);
                    }
                    tmem_st16_async(tD + 16 * c, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full + 8 * pos);
                pos += G;
                if (pos >= C::kStages) pos = w, phase ^= 1u;
            }
            n += steps;
            if (!ok) break;
            int following = 0;
            if (!warp_next(bar->queue, t, following, p.status, abort_flag)) break;
            const DqItem next = dq_item(p, min(following, p.items - 1));  // while dQ ends
            // with two items held, the last one's dQ is written after this one's steps: its
            // sums have ended by then
            if (C::kItems == 1) ok = finish(it, items);
            else if (held >= 0) ok = finish(last, held);
            if (!ok) break;
            last = it;
            held = items;
            it = next;
            idx = following;
        }
        if (C::kItems > 1 && ok && held >= 0) finish(last, held);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dK, dV
template <int DP>
struct DkvLayout {
    // slots, one of each warpgroup: S in 64 columns, dP in 64 (as many as fit beside dV and dK)
    static constexpr int G = DP == 64 ? 3 : 2;
    static constexpr uint32_t kTileBytes = kTile * DP * 2, kStepBytes = kHalf * DP * 2;
    static constexpr int kStages = DP == 64 ? 9 : 4;  // steps: Q, dO, lse and delta
    static constexpr int kKv = DP == 64 ? 2 : 1;  // items whose K and V are held
    static constexpr uint32_t kDv = 128 * G, kDk = kDv + DP;
    static constexpr uint32_t kSmem = 1024 + kKv * 2 * kTileBytes + kStages * (2 * kStepBytes + 512) + 1024;
};
struct DkvItem {
    int batch, kvh, k0, part, lo, hi;  // steps [lo, hi) of 64 queries of each head of the group
    Span sp;
};
__device__ __forceinline__ DkvItem dkv_item(const BwdParams &p, int idx) {
    DkvItem it;
    const int units = p.b * p.hk;
    int block, u;
    place<true>(idx, p.kblocks * p.ksplit, units, p.ksome, block, u);
    it.part = 0;
    if (p.ksplit > 1) {
        const int x = block;
        block = x / p.ksplit;
        it.part = x - block * p.ksplit;
    }
    it.k0 = block * kTile;  // causal: early keys are seen by the most queries
    it.batch = u / p.hk;
    it.kvh = u - it.batch * p.hk;
    it.sp = Span{clamp_length(p.q_lengths, it.batch, p.nq), clamp_length(p.k_lengths, it.batch, p.nk),
                 p.causal, p.window};
    it.lo = it.hi = 0;
    const int last = min(it.k0 + kTile, it.sp.Lk) - 1, off = it.sp.Lk - it.sp.Lq;
    if (last >= it.k0) {
        const int a = p.causal ? max(0, it.k0 - off) : 0;
        const int z = p.window ? min((long long)it.sp.Lq, (long long)last - off + p.window) : it.sp.Lq;
        if (z > a) {
            it.lo = a / kHalf;
            it.hi = (z + kHalf - 1) / kHalf;
            if (p.ksplit > 1) take_part(it.lo, it.hi, it.part, p.ksplit);
        }
    }
    return it;
}

struct DkvBarriers {
    uint64_t full[9], fixed[9], s_full[9], p_full[9], pv_done[9], dp_full[9], ds_full[9], ds_done[9];
    uint64_t kv_full[2], kv_free[2], acc_full, acc_free, fix_wanted, drain[3];
    Queue queue;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(DkvBarriers) <= 1024, "room for the barriers");

template <int DP>
__global__ void __launch_bounds__(threads_of(DkvLayout<DP>::G), 1)
softmax_attn_dkv_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                        const __grid_constant__ CUtensorMap tV, const __grid_constant__ CUtensorMap tdO,
                        const BwdParams p) {
    using C = DkvLayout<DP>;
    constexpr int G = C::G, kLoadWarp = 4 * G, kMmaWarp = 4 * G + 1;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    // K and V of an item at sK + (item % kKv) 2 tiles
    uint8_t *sK = smem, *sT = smem + C::kKv * 2 * C::kTileBytes;
    // stage s: the step's Q and dO, then (after all of them) its 512 bytes of row values
    uint8_t *sR = sT + C::kStages * 2 * C::kStepBytes;
    DkvBarriers *bar = reinterpret_cast<DkvBarriers *>(sR + C::kStages * 512);
    volatile int *abort_flag = &bar->abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar->kv_full[i], 1);
            mbar_init(&bar->kv_free[i], 2);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&bar->drain[i], 1);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bar->full[i], 1);
            mbar_init(&bar->fixed[i], 31);
            mbar_init(&bar->s_full[i], 1);
            mbar_init(&bar->p_full[i], 4);
            mbar_init(&bar->pv_done[i], 1);
            mbar_init(&bar->dp_full[i], 1);
            mbar_init(&bar->ds_full[i], 4);
            mbar_init(&bar->ds_done[i], 1);
        }
        mbar_init(&bar->acc_full, 1);
        mbar_init(&bar->acc_free, 8);
        mbar_init(&bar->fix_wanted, 1);
        init_queue(bar->queue, (p.q_lengths ? 31 : 0) + 3 + 4 * G);  // zeroing lanes, issuing threads, warps
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bar->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;

    if (warp >= kLoadWarp) {
        setmaxnreg_dec<issue_regs(G)>();
        if (warp == kLoadWarp) {
            if (lane == 0) {
                int ring = 0, items = 0, t = 0;
                Ring<G, C::kStages> at;
                bool ok = true;
                for (int idx = blockIdx.x; idx < p.items && ok;) {
                    const int following = gridDim.x + atomicAdd(p.queue + 1, 1);
                    const DkvItem it = dkv_item(p, idx);
                    if (it.hi > it.lo) {
                        const int kb = items % C::kKv;
                        if (items >= C::kKv &&
                            !thread_spin(&bar->kv_free[kb], (items / C::kKv - 1) & 1, p.status, 100, abort_flag))
                            break;
                        uint8_t *kv = sK + kb * 2 * C::kTileBytes;
                        mbar_arrive_expect_tx(&bar->kv_full[kb], 2 * C::kTileBytes);
                        load_rows<DP, 2>(kv, &tK, &bar->kv_full[kb], it.k0, 0, it.kvh, it.batch);
                        load_rows<DP, 2>(kv + C::kTileBytes, &tV, &bar->kv_full[kb], it.k0, 0, it.kvh, it.batch);
                        ++items;
                        for (int g = 0; g < p.group && ok; ++g)
                            for (int j = it.lo; j < it.hi; ++j, ++ring, at.next()) {
                                const int s = at.pos;
                                // (dK comes last: with it all products of a step have been formed)
                                if (!thread_spin(&bar->ds_done[s], at.phase ^ 1, p.status, 101, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                uint8_t *st = sT + s * 2 * C::kStepBytes;
                                mbar_arrive_expect_tx(&bar->full[s], 2 * C::kStepBytes + 512);
                                load_rows<DP, 1>(st, &tQ, &bar->full[s], j * kHalf, g, it.kvh, it.batch);
                                load_rows<DP, 1>(st + C::kStepBytes, &tdO, &bar->full[s], j * kHalf, g, it.kvh, it.batch);
                                const int64_t head = (int64_t)it.batch * p.hq + it.kvh * p.group + g;
                                bulk_load(sR + s * 512, p.rows + (head * 2 * p.qtiles + j) * 128, 512, &bar->full[s]);
                            }
                    }
                    ok = ok && tell(bar->queue, t, following, p.status, abort_flag);
                    idx = following;
                }
                for (int i = max(0, items - C::kKv); i < items; ++i)
                    mbar_wait_drain(&bar->kv_full[i % C::kKv], (i / C::kKv) & 1);
                for (int i = max(0, ring - C::kStages); i < ring; ++i)
                    mbar_wait_drain(&bar->full[i % C::kStages], (i / C::kStages) & 1);
            } else if (p.q_lengths) {  // Q and dO rows past the valid length: P and dS are 0 there, but 0 x NaN is not
                int ring = 0, nfix = 0;
                bool ok = true;
                for (int idx = blockIdx.x, t = 0; idx < p.items && ok;
                     ok = ok && thread_next(bar->queue, t, idx, p.status, abort_flag)) {
                    const DkvItem it = dkv_item(p, idx);
                    if (it.hi <= it.lo) continue;
                    if (it.sp.Lq >= p.nq || it.hi * kHalf <= it.sp.Lq) {
                        ring += p.group * (it.hi - it.lo);
                        continue;
                    }
                    for (int g = 0; g < p.group; ++g) {
                        ring += it.hi - it.lo;
                        if (!thread_spin(&bar->fix_wanted, nfix & 1, p.status, 102, abort_flag)) {
                            ok = false;
                            break;
                        }
                        ++nfix;
                        const int s = (ring - 1) % C::kStages, row0 = it.sp.Lq - (it.hi - 1) * kHalf;
                        uint8_t *st = sT + s * 2 * C::kStepBytes;
                        zero_rows<DP, kHalf>(st, row0, lane - 1, 31);
                        zero_rows<DP, kHalf>(st + C::kStepBytes, row0, lane - 1, 31);
                        fence_proxy_async_smem();
                        mbar_arrive(&bar->fixed[s]);
                    }
                }
            }
            __syncwarp();
        } else if (warp <= kMmaWarp + 1) {
            const bool first = warp == kMmaWarp;  // S = K Q^T; the other thread: dP = V dO^T
            if (elect_one()) {
                int items = 0;
                uint32_t fixes = 0;  // bit s: parity of stage s's next fix
                Ring<G, C::kStages> at;
                bool ok = true;
                const uint32_t a0 = smem_u32(sK) + (first ? 0 : C::kTileBytes), b = smem_u32(sT) + (first ? 0 : C::kStepBytes),
                               slots = tmem + (first ? 0 : 64), loaded = smem_u32(bar->full),
                               done = smem_u32(first ? bar->pv_done : bar->ds_done),
                               out = smem_u32(first ? bar->s_full : bar->dp_full), fixed = smem_u32(bar->fixed);
                for (int idx = blockIdx.x, t = 0; idx < p.items && ok;
                     ok = ok && thread_next(bar->queue, t, idx, p.status, abort_flag)) {
                    const DkvItem it = dkv_item(p, idx);
                    const int per = it.hi - it.lo;
                    if (per <= 0) continue;
                    const bool fix = it.sp.Lq < p.nq && it.hi * kHalf > it.sp.Lq;
                    const int kb = items % C::kKv;
                    const uint32_t a = a0 + kb * 2 * C::kTileBytes;
                    int in_head = per;
                    ok = thread_spin(&bar->kv_full[kb], (items / C::kKv) & 1, p.status, 107, abort_flag);
                    for (int j = per * p.group; j > 0 && ok; --j, at.next()) {
                        ok = thread_spin(loaded + 8 * at.pos, at.phase, p.status, 103, abort_flag) &&
                             thread_spin(done + 8 * at.before(), at.phase_before(), p.status, 105, abort_flag);
                        if (ok && fix && --in_head == 0) {
                            in_head = per;
                            if (first) mbar_arrive(&bar->fix_wanted);
                            ok = thread_spin(fixed + 8 * at.pos, fixes >> at.pos & 1, p.status, 104, abort_flag);
                            fixes ^= 1u << at.pos;
                        }
                        if (!ok) break;
                        tc_fence_after();
                        mma_scores<DP>(slots + 128 * at.slot, a, b + at.pos * (2 * C::kStepBytes));
                        mma_commit(out + 8 * at.pos);
                    }
                    mma_commit(&bar->kv_free[kb]);
                    ++items;
                }
                mma_commit(&bar->drain[first ? 0 : 1]);
                mbar_wait_drain(&bar->drain[first ? 0 : 1], 0);
            }
            __syncwarp();
        } else {
            if (elect_one()) {  // dV += P^T dO of each step, then dK += dS^T Q, with three slots of the step before
                constexpr int kLag = G - 2;
                int items = 0;
                Ring<G, C::kStages> av, ak;
                bool ok = true;
                const uint32_t b = smem_u32(sT), p_full = smem_u32(bar->p_full), ds_full = smem_u32(bar->ds_full),
                               pv_done = smem_u32(bar->pv_done), ds_done = smem_u32(bar->ds_done);
                for (int idx = blockIdx.x, t = 0; idx < p.items && ok;
                     ok = ok && thread_next(bar->queue, t, idx, p.status, abort_flag)) {
                    const DkvItem it = dkv_item(p, idx);
                    const int steps = (it.hi - it.lo) * p.group;
                    if (steps <= 0) continue;
                    if (items > 0) ok = thread_spin(&bar->acc_free, (items - 1) & 1, p.status, 109, abort_flag);
                    for (int j = 0; j < steps + kLag && ok; ++j) {
                        if (j < steps) {
                            ok = thread_spin(p_full + 8 * av.pos, av.phase, p.status, 106, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            mma_sum<DP>(tmem + C::kDv, tmem + 128 * av.slot, b + av.pos * (2 * C::kStepBytes) + C::kStepBytes,
                                        j > 0 ? 1u : 0u);
                            mma_commit(pv_done + 8 * av.pos);
                            av.next();
                        }
                        if (j >= kLag) {
                            ok = thread_spin(ds_full + 8 * ak.pos, ak.phase, p.status, 108, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            mma_sum<DP>(tmem + C::kDk, tmem + 128 * ak.slot + 64, b + ak.pos * (2 * C::kStepBytes),
                                        j > kLag ? 1u : 0u);
                            mma_commit(ds_done + 8 * ak.pos);
                            ak.next();
                        }
                    }
                    mma_commit(&bar->acc_full);
                    ++items;
                }
                mma_commit(&bar->drain[2]);
                mbar_wait_drain(&bar->drain[2], 0);
            }
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<math_regs(G)>();
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + 128 * w + lanes, tD = tS + 64;
        const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
        const uint32_t s_full = smem_u32(bar->s_full), p_full = smem_u32(bar->p_full), dp_full = smem_u32(bar->dp_full),
                       ds_full = smem_u32(bar->ds_full), loaded = smem_u32(bar->full), rows = smem_u32(sR);
        int n = 0, items = 0;
        uint32_t pos = w, phase = 0;  // in the ring; the warpgroup's steps are at w, w + G and so on
        bool ok = true;
        DkvItem it = dkv_item(p, min((int)blockIdx.x, p.items - 1));
        for (int idx = blockIdx.x, t = 0; idx < p.items && ok;) {
            const int key = it.k0 + row, off = it.sp.Lk - it.sp.Lq, hi = it.hi, per = max(0, hi - it.lo),
                      steps = per * p.group;
            // queries [first, end) see this key (the rows past the length need no mask: their
            // -lse is -inf)
            const int first = p.causal ? max(0, key - off) : 0;
            const int end = p.window ? (int)min((long long)it.sp.Lq, (long long)key - off + p.window) : 1 << 30;
            const unsigned width = end > first ? (unsigned)(end - first) : 0u;
            int h = n + (w + G - n % G) % G, j = it.lo + h - n;
            n += steps;
            for (; h < n; h += G, j += G) {
                while (j >= hi) j -= per;  // the next head
                const uint32_t aR = rows + pos * 512;  // -lse and, 256 on, -delta
                if (!warp_spin(s_full + 8 * pos, phase, p.status, 112, abort_flag) ||
                    !warp_spin(loaded + 8 * pos, phase, p.status, 111, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int q0 = j * kHalf;
                if (__any_sync(0xffffffffu, first > q0 || end < q0 + kHalf)) hide_outside(tS, first - q0, width);
                uint32_t v[2][32];
                load_columns(tS, v);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 l = lds4(aR + 4 * (32 * c + e));
                        const float2 y0 = ffma2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])),
                                                sl2, make_float2(l.x, l.y));
                        const float2 y1 = ffma2(make_float2(__uint_as_float(v[c][e + 2]), __uint_as_float(v[c][e + 3])),
                                                sl2, make_float2(l.z, l.w));
                        v[c][e] = __float_as_uint(ex2_approx(y0.x));
                        v[c][e + 1] = __float_as_uint(ex2_approx(y0.y));
                        v[c][e + 2] = __float_as_uint(ex2_approx(y1.x));
                        v[c][e + 3] = __float_as_uint(ex2_approx(y1.y));
                        o[e / 2] = pack2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                        o[e / 2 + 1] = pack2(__uint_as_float(v[c][e + 2]), __uint_as_float(v[c][e + 3]));
                    }
                    tmem_st16_async(tS + 16 * c, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * pos);
                if (!warp_spin(dp_full + 8 * pos, phase, p.status, 113, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // 32 columns at a time; dS takes the columns that have been read
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t u[32], o[16];
                    tmem_ld32(tD + 32 * c, u);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 dl = lds4(aR + 256 + 4 * (32 * c + e));
                        const float2 y0 = fadd2(make_float2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])),
                                                make_float2(dl.x, dl.y));
                        const float2 y1 = fadd2(make_float2(__uint_as_float(u[e + 2]), __uint_as_float(u[e + 3])),
                                                make_float2(dl.z, dl.w));
                        const float2 z0 = fmul2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), y0);
                        const float2 z1 = fmul2(make_float2(__uint_as_float(v[c][e + 2]), __uint_as_float(v[c][e + 3])), y1);
                        o[e / 2] = pack2(z0.x, z0.y);
                        o[e / 2 + 1] = pack2(z1.x, z1.y);
                    }
                    tmem_st16_async(tD + 16 * c, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full + 8 * pos);
                pos += G;
                if (pos >= C::kStages) pos = w, phase ^= 1u;
            }
            if (!ok) break;
            int following = 0;
            if (!warp_next(bar->queue, t, following, p.status, abort_flag)) break;
            const DkvItem next = dkv_item(p, min(following, p.items - 1));  // while the sums end
            const bool exists = key < p.nk, valid = key < it.sp.Lk;
            // the first two warpgroups write dV and dK
            __nv_bfloat16 *dst =
                w ? p.dK + it.batch * p.sdK.b + it.kvh * p.sdK.h + (int64_t)key * p.sdK.n
                  : p.dV + it.batch * p.sdV.b + it.kvh * p.sdV.h + (int64_t)key * p.sdV.n;
            float *part = (w ? p.part_k : p.part_v) +
                          ((((int64_t)it.part * p.b + it.batch) * p.hk + it.kvh) * p.nk + key) * DP;
            if (w < 2 && steps) {
                if (!warp_spin(&bar->acc_full, items & 1, p.status, 114, abort_flag)) break;
                tc_fence_after();
                ++items;
                uint32_t o[DP / 32][32];
                load_columns(tmem + (w ? C::kDk : C::kDv) + lanes, o);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->acc_free);
                if (exists)
#pragma unroll
                    for (int c = 0; c < DP / 32; ++c) {
                        if (p.ksplit > 1) store_part(part + 32 * c, o[c], !valid);
                        else store_row(dst, o[c], 32 * c, p.d, w ? p.scale : 1.f, !valid, p.wide >> (w ? 1 : 2) & 1);
                    }
            } else if (w < 2 && exists) {
                if (p.ksplit > 1) zero_part(part, DP);
                else zero_row(dst, p.d);
            }
            it = next;
            idx = following;
        }
    }
    if (warp == kLoadWarp) wait_prerequisites();  // no later kernel before the second one has ended
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Adds up the parts of dQ, dK and dV (blockIdx.y) in their order, four columns a thread.
constexpr int kJoinThreads = 128;
template <int DP>
__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(const BwdParams p) {
    const int which = blockIdx.y, parts = which ? p.ksplit : p.qsplit;
    if (parts <= 1) return;
    const int heads = which ? p.hk : p.hq, n = which ? p.nk : p.nq;
    const int64_t rows = (int64_t)p.b * heads * n, t = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
    const int64_t r = t / (DP / 4);
    const int col = (int)(t % (DP / 4)) * 4;
    if (r >= rows || col >= p.d) return;
    const float *src = (which == 0 ? p.part_q : which == 1 ? p.part_k : p.part_v) + r * DP + col;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < parts; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(src + i * rows * DP);
        sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
    }
    const int row = (int)(r % n), head = (int)(r / n % heads), batch = (int)(r / ((int64_t)n * heads));
    const Strides &st = which == 0 ? p.sdQ : which == 1 ? p.sdK : p.sdV;
    __nv_bfloat16 *dst = (which == 0 ? p.dQ : which == 1 ? p.dK : p.dV) + batch * st.b + head * st.h + row * st.n + col;
    const float f = which < 2 ? p.scale : 1.f;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(sum.x * f, sum.y * f), pack2(sum.z * f, sum.w * f));
}

// Parts of an item of `steps` steps where `items` leave SMs idle: at least kMinSteps each, and
// only where an item gets shorter by kGain steps, about what the launch that joins costs.  (8
// items, whole and in parts: d = 64: 16 steps 19.4 and 21.9 us, 32 steps 23.1 and 21.4, 64 steps
// 39.8 and 24.8; d = 128: 20.6 and 21.6, 30.6 and 26.5, 55.4 and 29.3 us; in parts of 16 steps
// 30.7 and 31.0 at 32 and 64.  64 items of up to 32 steps: 25.1 whole, 29.0 halved.)
int parts_of(int64_t items, int64_t steps, int sms) {
    constexpr int kMinSteps = 8, kGain = 24;
    const int64_t n = std::min<int64_t>(sms / items, steps / kMinSteps);
    return n > 1 && steps - steps / n >= kGain ? (int)n : 1;
}

template <int DP>
int launch(const Call &c, BwdParams &p) {
    using Cq = DqLayout<DP>;
    using Ck = DkvLayout<DP>;
    CUtensorMap tQ, tK, tV, tdO;
    if (!encode_rows(&tQ, c.Q, c.sQ, c.b, c.hq, p.group, c.nq, c.d, kHalf, 1) ||
        !encode_rows(&tdO, c.dO, c.sdO, c.b, c.hq, p.group, c.nq, c.d, kHalf, 1) ||
        !encode_rows(&tK, c.K, c.sK, c.b, c.hk, 1, c.nk, c.d, kHalf, 1) ||
        !encode_rows(&tV, c.V, c.sV, c.b, c.hk, 1, c.nk, c.d, kHalf, 1))
        return LINFORMER_ERR_LAUNCH;
    int st = allow_smem(reinterpret_cast<const void *>(softmax_attn_dq_kernel<DP>), Cq::kSmem, DP == 64 ? 0 : 1);
    if (!st) st = allow_smem(reinterpret_cast<const void *>(softmax_attn_dkv_kernel<DP>), Ck::kSmem, DP == 64 ? 2 : 3);
    if (st) return st;
    void *ws = nullptr;
    const int64_t qitems = (int64_t)c.b * c.hq * p.qtiles, kitems = (int64_t)c.b * c.hk * p.kblocks;
    if (qitems > kMaxItems || kitems > kMaxItems) return LINFORMER_ERR_SIZE;
    const int sms = device_sms();
    auto reach = [&](int n) { return c.window ? std::min(n, c.window + kTile) : n; };
    auto steps_of = [&](int n) { return (reach(n) + kHalf - 1) / kHalf; };
    p.qsplit = parts_of(qitems, steps_of(c.nk), sms);
    p.ksplit = std::min(parts_of(kitems, (int64_t)steps_of(c.nq) * p.group, sms), steps_of(c.nq));
    p.qsome = units_at_once(p.qtiles, c.b * c.hq, ((int64_t)reach(c.nk) * c.d * 4 + p.group - 1) / p.group, c.causal, sms);
    p.ksome = units_at_once(p.kblocks, c.b * c.hk, (int64_t)p.group * reach(c.nq) * c.d * 4, c.causal, sms);
    const int64_t qrows = (int64_t)c.b * c.hq * c.nq, krows = (int64_t)c.b * c.hk * c.nk;
    const int64_t qparts = p.qsplit > 1 ? p.qsplit * qrows * DP : 0, kparts = p.ksplit > 1 ? p.ksplit * krows * DP : 0;
    if (workspace_alloc(&ws, (size_t)(qitems * 256 + qparts + 2 * kparts + 2) * sizeof(float), c.stream) != LINFORMER_OK)
        return LINFORMER_ERR_ALLOC;
    p.rows = static_cast<float *>(ws);
    p.part_q = p.rows + qitems * 256;
    p.part_k = p.part_q + qparts;
    p.part_v = p.part_k + kparts;
    p.queue = reinterpret_cast<int *>(p.part_v + kparts);
    {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX_BWD, c.stream);
        rows_kernel<DP><<<(unsigned)qitems, kRowsThreads, 0, c.stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) st = LINFORMER_ERR_LAUNCH;
    }
    // The other two as programmatic dependents: the second is set up while the first ends, and
    // the third, which needs only the first one's rows, takes over SMs as the second leaves
    // them (and ends after it).
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!st) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX_BWD, c.stream);
        p.items = (int)qitems * p.qsplit;
        cfg.gridDim = dim3((unsigned)std::min(p.items, sms));
        cfg.blockDim = dim3(threads_of(Cq::G));
        cfg.dynamicSmemBytes = Cq::kSmem;
        if (cudaLaunchKernelEx(&cfg, softmax_attn_dq_kernel<DP>, tQ, tK, tV, tdO, p) != cudaSuccess)
            st = LINFORMER_ERR_LAUNCH;
    }
    if (!st) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX_BWD, c.stream);
        p.items = (int)kitems * p.ksplit;
        cfg.gridDim = dim3((unsigned)std::min(p.items, sms));
        cfg.blockDim = dim3(threads_of(Ck::G));
        cfg.dynamicSmemBytes = Ck::kSmem;
        if (cudaLaunchKernelEx(&cfg, softmax_attn_dkv_kernel<DP>, tQ, tK, tV, tdO, p) != cudaSuccess)
            st = LINFORMER_ERR_LAUNCH;
    }
    if (!st && (p.qsplit > 1 || p.ksplit > 1)) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX_BWD, c.stream);
        const int64_t rows = std::max(p.qsplit > 1 ? qrows : 0, p.ksplit > 1 ? krows : 0);
        const unsigned blocks = (unsigned)((rows * (DP / 4) + kJoinThreads - 1) / kJoinThreads);
        join_parts_kernel<DP><<<dim3(blocks, 3), kJoinThreads, 0, c.stream>>>(p);
        if (cudaPeekAtLastError() != cudaSuccess) st = LINFORMER_ERR_LAUNCH;
    }
    if (st) cudaGetLastError();
    workspace_free(ws, c.stream);
    return st;
}

}  // namespace

int backward(const Call &c) {
    BwdParams p{};
    p.q_lengths = c.q_lengths;
    p.k_lengths = c.k_lengths;
    p.O = static_cast<const __nv_bfloat16 *>(c.O);
    p.dO = static_cast<const __nv_bfloat16 *>(c.dO);
    p.sO = c.sO;
    p.sdO = c.sdO;
    p.dQ = static_cast<__nv_bfloat16 *>(c.dQ);
    p.dK = static_cast<__nv_bfloat16 *>(c.dK);
    p.dV = static_cast<__nv_bfloat16 *>(c.dV);
    p.sdQ = c.sdQ;
    p.sdK = c.sdK;
    p.sdV = c.sdV;
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
    p.qtiles = (c.nq + kTile - 1) / kTile;
    p.kblocks = (c.nk + kTile - 1) / kTile;
    p.scale = c.scale;
    p.scale_log2 = c.scale * kLog2e;
    p.wide = wide_stores(c.dQ, c.sdQ, c.d) | wide_stores(c.dK, c.sdK, c.d) << 1 | wide_stores(c.dV, c.sdV, c.d) << 2;
    p.status = device_status_ptr();
    return c.d <= 64 ? launch<64>(c, p) : launch<128>(c, p);
}

}  // namespace sattn
}  // namespace linformer
