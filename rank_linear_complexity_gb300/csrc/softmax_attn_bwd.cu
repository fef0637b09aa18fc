// Exact softmax attention, backward.  With P_ij = exp(scale Q_i.K_j - lse_i) recomputed
// from the forward's lse, delta_i = dO_i.O_i and
//
//     dP = dO V^T,   dS_ij = P_ij (dP_ij - delta_i),
//     dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K,
//
// two kernels after a small one, each a sum that one CTA owns, so that no gradient is added up by atomics
// and every result repeats bit for bit:
//   rows_kernel  -lse log2(e) and -delta of every query row, for the other two.
//   dq_kernel   a 128-row query tile against its key blocks: S, dP, then dQ += dS.K.
//   dkv_kernel  a 128-key block against the query tiles of every head of its group:
//               S^T = K.Q^T and dP^T = V.dO^T, then dV += P^T.dO and dK += dS^T.Q.  With
//               keys as the rows, P^T and dS^T leave the registers of the thread that made
//               them for the tensor memory of the next product: no transpose, no shared
//               memory.
// Seven products instead of five: S and dP are formed twice, which costs less than adding
// partial dQ through memory in a fixed order.  P and dS are rounded to bf16 as operands
// (relative 2^-9, in sums of many terms); sums are fp32 in tensor memory.
//
// Roles, both kernels: warps 0-3 and 4-7 do the arithmetic of the two halves (64 columns) of
// every step, one thread a row; each half's P or dS is multiplied as soon as it is there;
// warp 8 loads (lane 0) and zeroes rows past the valid length (lanes 1-31, where 0 x NaN
// would reach a sum); one thread each of warps 9 and 10 issues products, so that a chain of
// products that waits for arithmetic does not hold up the other one.
#include <algorithm>
#include <cmath>

#include "softmax_attn.cuh"
#include "sm100_ptx.cuh"

namespace linformer {
namespace sattn {
namespace {

using namespace ptx;

// Twelve warps (one idle), 168 registers each at launch; the two warpgroups that do the
// arithmetic take registers from the third: 2 x 208 + 88 = 3 x 168.
constexpr int kThreads = 384;
constexpr uint32_t kMathRegs = 208, kIssueRegs = 88;
static_assert(2 * kMathRegs + kIssueRegs == 3 * 168, "register split");
constexpr int kMathWarps = 8, kHalfWarps = 4, kLoadWarp = 8, kMmaWarp = 9;
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
    const int32_t *q_lengths, *k_lengths;
    const __nv_bfloat16 *O, *dO;
    Strides sO, sdO;
    __nv_bfloat16 *dQ, *dK, *dV;
    Strides sdQ, sdK, sdV;
    const float *lse;
    // [b][hq][query tiles][2][128]: -lse log2(e) and -delta, as they are added; -inf and 0 for
    // rows that are past the length or see no key
    float *rows;
    int b, hq, hk, group, nq, nk, d, causal, window;
    int qtiles, kblocks;
    int wide;  // bits: dQ, dK, dV take 32-byte stores
    int items;
    float scale, scale_log2;
    int *status;
};

// Columns outside [a, a + w) of 64 in tensor memory become `value`: for the few blocks at a
// mask's edge, out of line, away from the code of the others.
__device__ __noinline__ void fill_outside(uint32_t t, int a, unsigned w, uint32_t value) {
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        uint32_t u[32];
        tmem_ld32(t + c, u);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if ((unsigned)(c + e - a) >= w) u[e] = value;
        tmem_st32(t + c, u);
    }
}
constexpr uint32_t kMinusInf = 0xff800000u;
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
// 32 N columns of an accumulator, one wait for all.
// The first d columns of a row as zero.
__device__ __forceinline__ void zero_row(__nv_bfloat16 *dst, int d) {
#pragma unroll 1
    for (int c = 0; c < d; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
}
template <int N>
__device__ __forceinline__ void load_columns(uint32_t t, uint32_t (&o)[N][32]) {
#pragma unroll
    for (int c = 0; c < N; ++c) tmem_ld32_async(t + 32 * c, o[c]);
    tmem_wait_ld(o[0]);
#pragma unroll
    for (int c = 1; c < N; ++c) tie32(o[c]);
}

template <int DP>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b) {
    const uint32_t idesc = idesc_f16(128, 128, 1, 0, 0);
    const uint64_t da = sdesc(a, 16, 1024, kSwizzle128B), db = sdesc(b, 16, 1024, kSwizzle128B);
#pragma unroll
    for (int x = 0; x < DP / 16; ++x) {
        const uint64_t off = (uint64_t)((x >> 2) * 1024 + (x & 3) * 2);
        mma_ss(d, da + off, db + off, idesc, x > 0 ? 1u : 0u);
    }
}
// D (128 x DP) += A (128 x 64, packed in 32 columns of tensor memory) . B (64 rows of DP): half
// of a step's sum, issued as soon as that half of P or dS is there.
template <int DP>
__device__ __forceinline__ void mma_sum_half(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    const uint32_t idesc = idesc_f16(128, DP, 1, 0, 1);
    const uint64_t db = sdesc(b, 16384, 1024, kSwizzle128B);
#pragma unroll
    for (int x = 0; x < 4; ++x)
        mma_ts(d, a + 8 * x, db + (uint64_t)(128 * x), idesc, (acc || x > 0) ? 1u : 0u);
}

template <int DP>
__device__ __forceinline__ void load_rows(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int row,
                                          int head, int group, int batch) {
#pragma unroll
    for (int h = 0; h < DP / 64; ++h) tma_load_5d(dst + h * 16384, m, bar, h * 64, row, head, group, batch);
}

// ---------------------------------------------------------------- row values
// -lse log2(e) and -delta = -dO.O of a query tile's 128 rows, eight warps of sixteen rows; a row
// is read by DP / 8 lanes, 16 bytes each.  Bound by memory: O and dO once.
constexpr int kRowsThreads = 256;
template <int DP>
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const BwdParams p) {
    launch_dependents();
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
    float *dst = p.rows + (int64_t)blockIdx.x * 256 + 16 * warp + lane / kLanes;
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        float y = (dot2(a[t].x, b[t].x) + dot2(a[t].y, b[t].y)) + (dot2(a[t].z, b[t].z) + dot2(a[t].w, b[t].w));
#pragma unroll
        for (int k = kLanes / 2; k; k >>= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
        if (lane % kLanes == 0) {
            dst[t * kAtOnce] = x[t] == -INFINITY ? -INFINITY : -x[t] * kLog2e;
            dst[t * kAtOnce + 128] = x[t] == -INFINITY ? 0.f : -y;
        }
    }
}

// ---------------------------------------------------------------- dQ
template <int DP>
struct DqLayout {
    static constexpr uint32_t kTileBytes = kTile * DP * 2;
    static constexpr int kStages = DP == 64 ? 8 : 5;
    static constexpr uint32_t kS = 0, kDp = 128, kDq = 384;
    static constexpr uint32_t kSmem = 1024 + (2 + kStages) * kTileBytes + 512 + 1024;
};
struct DqItem {
    int batch, head, q0, lo, hi;
    Span sp;
};
__device__ __forceinline__ DqItem dq_item(const BwdParams &p, int idx) {
    DqItem it;
    const int units = p.b * p.hq;
    const int rank = idx / units, u = idx - rank * units;
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
            it.lo = f / kTile;
            it.hi = (e + kTile - 1) / kTile;
        }
    }
    return it;
}

struct DqBarriers {
    // (pairs: even and odd blocks)
    uint64_t q_full, q_free, s_full[2], s_free, dp_full[2], ds_full[2][2], dq_done[2];
    uint64_t acc_full, acc_free;
    uint64_t fix_wanted, fixed, drain[2];
    uint64_t full[8], empty[8];
    uint32_t tmem;
    int abort;
    alignas(16) float rows[2 * kTile];  // the item's rows, loaded with Q and dO
};

static_assert(sizeof(DqBarriers) <= 512 + 1024, "room for the barriers");

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
softmax_attn_dq_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                       const __grid_constant__ CUtensorMap tV, const __grid_constant__ CUtensorMap tdO,
                       const BwdParams p) {
    using C = DqLayout<DP>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sdO = smem + C::kTileBytes, *sKV = smem + 2 * C::kTileBytes;
    DqBarriers *bar = reinterpret_cast<DqBarriers *>(sKV + C::kStages * C::kTileBytes);
    volatile int *abort_flag = &bar->abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        mbar_init(&bar->q_full, 1);
        mbar_init(&bar->q_free, 1 + kMathWarps);  // the products, and the rows read
        mbar_init(&bar->s_free, kMathWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar->s_full[i], 1);
            mbar_init(&bar->dp_full[i], 1);
            mbar_init(&bar->ds_full[i][0], kHalfWarps);  // halves of 64 columns
            mbar_init(&bar->ds_full[i][1], kHalfWarps);
            mbar_init(&bar->dq_done[i], 1);
        }
        mbar_init(&bar->acc_full, 1);
        mbar_init(&bar->acc_free, kMathWarps);
        mbar_init(&bar->fix_wanted, 1);
        mbar_init(&bar->fixed, 31);
        mbar_init(&bar->drain[0], 1);
        mbar_init(&bar->drain[1], 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
        }
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
    // ring entry 2 j + kv of an item: K (kv = 0) and V of its j-th block
    if (warp >= kLoadWarp) {
    setmaxnreg_dec<kIssueRegs>();
    if (warp == kLoadWarp) {
        if (lane == 0) {
            wait_prerequisites();  // the row values; and only then may the third kernel start
            launch_dependents();
            int ring = 0, nq = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < p.items && ok; idx += gridDim.x) {
                const DqItem it = dq_item(p, idx);
                if (it.hi <= it.lo) continue;
                if (nq > 0 && !thread_spin(&bar->q_free, (nq - 1) & 1, p.status, 83, abort_flag)) break;
                mbar_arrive_expect_tx(&bar->q_full, 2 * C::kTileBytes + 1024);
                const int g = it.head % p.group, kvh = it.head / p.group;
                bulk_load(bar->rows, p.rows + (((int64_t)it.batch * p.hq + it.head) * p.qtiles + it.q0 / kTile) * 256,
                          1024, &bar->q_full);
                load_rows<DP>(sQ, &tQ, &bar->q_full, it.q0, g, kvh, it.batch);
                load_rows<DP>(sdO, &tdO, &bar->q_full, it.q0, g, kvh, it.batch);
                ++nq;
                for (int j = it.lo; j < it.hi && ok; ++j)
                    for (int kv = 0; kv < 2; ++kv, ++ring) {
                        const int s = ring % C::kStages;
                        if (ring >= C::kStages &&
                            !thread_spin(&bar->empty[s], (ring / C::kStages - 1) & 1, p.status, 84, abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bar->full[s], C::kTileBytes);
                        load_rows<DP>(sKV + s * C::kTileBytes, kv ? &tV : &tK, &bar->full[s], j * kTile, 0,
                                      kvh, it.batch);
                    }
            }
            if (nq > 0) mbar_wait_drain(&bar->q_full, (nq - 1) & 1);
            for (int i = max(0, ring - C::kStages); i < ring; ++i)
                mbar_wait_drain(&bar->full[i % C::kStages], (i / C::kStages) & 1);
        } else {  // K rows past the valid length: dS is 0 there, but 0 x NaN is not
            int ring = 0, nfix = 0;
            for (int idx = blockIdx.x; idx < p.items; idx += gridDim.x) {
                const DqItem it = dq_item(p, idx);
                if (it.hi <= it.lo) continue;
                ring += 2 * (it.hi - it.lo);
                if (it.sp.Lk >= p.nk || it.hi * kTile <= it.sp.Lk) continue;
                if (!thread_spin(&bar->fix_wanted, nfix & 1, p.status, 85, abort_flag)) break;
                ++nfix;
                zero_rows<DP>(sKV + (ring - 2) % C::kStages * C::kTileBytes,
                              it.sp.Lk - (it.hi - 1) * kTile, lane - 1, 31);
                fence_proxy_async_smem();
                mbar_arrive(&bar->fixed);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (elect_one()) {  // S and dP
            int ring = 0, items = 0, n = 0, nfix = 0;
            bool ok = true;
            const uint32_t aQ = smem_u32(sQ), adO = smem_u32(sdO), aKV = smem_u32(sKV);
            for (int idx = blockIdx.x; idx < p.items && ok; idx += gridDim.x) {
                const DqItem it = dq_item(p, idx);
                const int blocks = it.hi - it.lo;
                if (blocks <= 0) continue;
                const bool fix = it.sp.Lk < p.nk && it.hi * kTile > it.sp.Lk;
                ok = thread_spin(&bar->q_full, items & 1, p.status, 91, abort_flag);
                for (int j = 0; j < blocks && ok; ++j, ++n, ring += 2) {
                    int s = ring % C::kStages;
                    ok = thread_spin(&bar->full[s], (ring / C::kStages) & 1, p.status, 86, abort_flag);
                    if (ok && fix && j == blocks - 1) {
                        mbar_arrive(&bar->fix_wanted);
                        ok = thread_spin(&bar->fixed, nfix++ & 1, p.status, 87, abort_flag);
                    }
                    ok = ok && (n == 0 || thread_spin(&bar->s_free, (n - 1) & 1, p.status, 88, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    mma_scores<DP>(tmem + C::kS, aQ, aKV + s * C::kTileBytes);
                    mma_commit(&bar->s_full[n & 1]);
                    s = (ring + 1) % C::kStages;
                    ok = thread_spin(&bar->full[s], ((ring + 1) / C::kStages) & 1, p.status, 89, abort_flag) &&
                         (n < 2 || thread_spin(&bar->dq_done[n & 1], ((n >> 1) - 1) & 1, p.status, 90, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    mma_scores<DP>(tmem + C::kDp + 128 * (n & 1), adO, aKV + s * C::kTileBytes);
                    mma_commit(&bar->dp_full[n & 1]);
                    mma_commit(&bar->empty[s]);
                }
                mma_commit(&bar->q_free);
                ++items;
            }
            mma_commit(&bar->drain[0]);
            mbar_wait_drain(&bar->drain[0], 0);
        }
        __syncwarp();
    } else if (warp == kMmaWarp + 1) {
        if (elect_one()) {  // dQ
            int ring = 0, items = 0, n = 0;
            bool ok = true;
            const uint32_t aKV = smem_u32(sKV);
            for (int idx = blockIdx.x; idx < p.items && ok; idx += gridDim.x) {
                const DqItem it = dq_item(p, idx);
                const int blocks = it.hi - it.lo;
                if (blocks <= 0) continue;
                for (int j = 0; j < blocks && ok; ++j, ++n, ring += 2) {
                    // (dS says that S has been formed, so the block of K has landed)
                    const int s = ring % C::kStages;
                    const uint32_t ds = tmem + C::kDp + 128 * (n & 1), k = aKV + s * C::kTileBytes;
                    ok = thread_spin(&bar->ds_full[n & 1][0], (n >> 1) & 1, p.status, 92, abort_flag) &&
                         (j > 0 || items == 0 ||
                          thread_spin(&bar->acc_free, (items - 1) & 1, p.status, 93, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    mma_sum_half<DP>(tmem + C::kDq, ds, k, j > 0 ? 1u : 0u);
                    ok = thread_spin(&bar->ds_full[n & 1][1], (n >> 1) & 1, p.status, 92, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    mma_sum_half<DP>(tmem + C::kDq, ds + 64, k + 8192, 1u);
                    mma_commit(&bar->dq_done[n & 1]);
                    mma_commit(&bar->empty[s]);
                }
                mma_commit(&bar->acc_full);
                ++items;
            }
            mma_commit(&bar->drain[1]);
            mbar_wait_drain(&bar->drain[1], 0);
        }
        __syncwarp();
    }
    } else {
        setmaxnreg_inc<kMathRegs>();
        const int half = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float sl = p.scale_log2;
        int n = 0, items = 0;
        DqItem it = dq_item(p, min((int)blockIdx.x, p.items - 1));
        for (int idx = blockIdx.x; idx < p.items; idx += gridDim.x) {
            const int lo = it.lo, hi = it.hi;
            float nl = 0.f, nd = 0.f;
            if (hi > lo) {  // the row values come with Q and dO
                if (!warp_spin(&bar->q_full, items & 1, p.status, 97, abort_flag)) break;
                nl = bar->rows[row];
                nd = bar->rows[128 + row];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->q_free);
                ++items;
            }
            const bool seen = it.q0 + row < it.sp.Lq;
            const int first = seen ? it.sp.first(it.q0 + row) : 0, end = seen ? it.sp.end(it.q0 + row) : 0;
            const unsigned width = end > first ? (unsigned)(end - first) : 0u;
            bool ok = true;
            for (int j = lo, g = n; j < hi; ++j, ++g) {
                if (!warp_spin(&bar->s_full[g & 1], (g >> 1) & 1, p.status, 94, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // keys that take no part: P = 0 whatever S holds, and dP = 0 below whatever it holds
                const int k0 = j * kTile + 64 * half;
                const bool masked = __any_sync(0xffffffffu, first > k0 || end < k0 + 64);
                const uint32_t tS = tmem + C::kS + 64 * half + lanes;
                if (masked) fill_outside(tS, first - k0, width, kMinusInf);
                uint32_t v[2][32];
                load_columns(tS, v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->s_free);
                const float2 sl2 = make_float2(sl, sl), off2 = make_float2(nl, nl);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = ffma2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])),
                                               sl2, off2);
                        v[c][e] = __float_as_uint(ex2_approx(y.x));
                        v[c][e + 1] = __float_as_uint(ex2_approx(y.y));
                    }
                const uint32_t tD = tmem + C::kDp + 128 * (g & 1) + 64 * half + lanes;
                if (!warp_spin(&bar->dp_full[g & 1], (g >> 1) & 1, p.status, 95, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (masked) fill_outside(tD, first - k0, width, 0u);
                const float2 nd2 = make_float2(nd, nd);
                uint32_t u[2][32], o[32];
                load_columns(tD, u);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = fadd2(make_float2(__uint_as_float(u[c][e]), __uint_as_float(u[c][e + 1])), nd2);
                        const float2 z = fmul2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), y);
                        o[16 * c + e / 2] = pack2(z.x, z.y);
                    }
                tmem_st32(tD, o);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->ds_full[g & 1][half]);
            }
            n += max(0, hi - lo);
            if (!ok) break;
            const bool some = hi > lo;
            const DqItem next = dq_item(p, min(idx + (int)gridDim.x, p.items - 1));  // while dQ ends
            const int i = it.q0 + row;
            const bool exists = i < p.nq, valid = i < it.sp.Lq;
            __nv_bfloat16 *dst = p.dQ + it.batch * p.sdQ.b + it.head * p.sdQ.h + (int64_t)i * p.sdQ.n;
            if (some) {
                if (!warp_spin(&bar->acc_full, (items - 1) & 1, p.status, 96, abort_flag)) break;
                tc_fence_after();
                uint32_t o[DP / 64][32];  // half of the columns
                load_columns(tmem + C::kDq + half * (DP / 2) + lanes, o);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->acc_free);
                if (exists)
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c)
                        store_row(dst, o[c], half * (DP / 2) + 32 * c, p.d, p.scale, !valid, p.wide & 1);
            } else if (exists && half == 0) {
                zero_row(dst, p.d);
            }
            it = next;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dK, dV
template <int DP>
struct DkvLayout {
    static constexpr uint32_t kTileBytes = kTile * DP * 2;
    static constexpr int kStages = DP == 64 ? 4 : 2;
    static constexpr uint32_t kStageBytes = 2 * kTileBytes + 1024;  // Q, dO, lse and delta
    static constexpr int kKv = DP == 64 ? 2 : 1;  // items whose K and V are held
    // S and dP of the steps in turn take kBufs buffers of 128 columns: S of step g buffer
    // 2 g, dP buffer 2 g + 1, modulo kBufs.  Each lives from its product over the arithmetic
    // to the product that takes its P or dS.
    static constexpr int kBufs = DP == 64 ? 3 : 2;
    static constexpr uint32_t kDv = 128 * kBufs, kDk = kDv + DP;
    static constexpr uint32_t kSmem = 1024 + kKv * 2 * kTileBytes + kStages * kStageBytes + 512;
};
struct DkvItem {
    int batch, kvh, k0, lo, hi;  // query tiles [lo, hi) of each head of the group
    Span sp;
};
__device__ __forceinline__ DkvItem dkv_item(const BwdParams &p, int idx) {
    DkvItem it;
    const int units = p.b * p.hk;
    const int block = idx / units, u = idx - block * units;
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
            it.lo = a / kTile;
            it.hi = (z + kTile - 1) / kTile;
        }
    }
    return it;
}

// Barriers of steps come in pairs, for even and odd steps: a waiter that falls behind by one
// step still finds its own phase.
struct DkvBarriers {
    uint64_t kv_full[2], kv_free[2], s_full[2], p_full[2][2], pv_done[2], dp_full[2], ds_full[2][2], ds_done[2];
    uint64_t acc_full, acc_free, fix_wanted, fixed[2], drain[2];
    uint64_t full[4], empty[4];
    uint32_t tmem;
    int abort;
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
softmax_attn_dkv_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                        const __grid_constant__ CUtensorMap tV, const __grid_constant__ CUtensorMap tdO,
                        const BwdParams p) {
    using C = DkvLayout<DP>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    // K and V of an item at sK + (item % kKv) 2 tiles
    uint8_t *sK = smem, *sT = smem + C::kKv * 2 * C::kTileBytes;
    // stage s: Q and dO tiles, then (after all tiles) its 1 KB of row values
    uint8_t *sR = sT + C::kStages * 2 * C::kTileBytes;
    DkvBarriers *bar = reinterpret_cast<DkvBarriers *>(sR + C::kStages * 1024);
    volatile int *abort_flag = &bar->abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar->kv_full[i], 1);
            mbar_init(&bar->kv_free[i], 2);
            mbar_init(&bar->s_full[i], 1);
            for (int h = 0; h < 2; ++h) {  // halves of 64 columns
                mbar_init(&bar->p_full[i][h], kHalfWarps);
                mbar_init(&bar->ds_full[i][h], kHalfWarps);
            }
            mbar_init(&bar->pv_done[i], 1);
            mbar_init(&bar->dp_full[i], 1);
            mbar_init(&bar->ds_done[i], 1);
            mbar_init(&bar->drain[i], 1);
            mbar_init(&bar->fixed[i], 31);
        }
        mbar_init(&bar->acc_full, 2);
        mbar_init(&bar->acc_free, kMathWarps);
        mbar_init(&bar->fix_wanted, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 2);  // both issuing threads
        }
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
    setmaxnreg_dec<kIssueRegs>();
    if (warp == kLoadWarp) {
        if (lane == 0) {
            int ring = 0, items = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < p.items && ok; idx += gridDim.x) {
                const DkvItem it = dkv_item(p, idx);
                if (it.hi <= it.lo) continue;
                const int kb = items % C::kKv;
                if (items >= C::kKv &&
                    !thread_spin(&bar->kv_free[kb], (items / C::kKv - 1) & 1, p.status, 100, abort_flag))
                    break;
                uint8_t *kv = sK + kb * 2 * C::kTileBytes;
                mbar_arrive_expect_tx(&bar->kv_full[kb], 2 * C::kTileBytes);
                load_rows<DP>(kv, &tK, &bar->kv_full[kb], it.k0, 0, it.kvh, it.batch);
                load_rows<DP>(kv + C::kTileBytes, &tV, &bar->kv_full[kb], it.k0, 0, it.kvh, it.batch);
                ++items;
                for (int g = 0; g < p.group && ok; ++g)
                    for (int j = it.lo; j < it.hi; ++j, ++ring) {
                        const int s = ring % C::kStages;
                        if (ring >= C::kStages &&
                            !thread_spin(&bar->empty[s], (ring / C::kStages - 1) & 1, p.status, 101, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint8_t *st = sT + s * 2 * C::kTileBytes;
                        mbar_arrive_expect_tx(&bar->full[s], 2 * C::kTileBytes + 1024);
                        load_rows<DP>(st, &tQ, &bar->full[s], j * kTile, g, it.kvh, it.batch);
                        load_rows<DP>(st + C::kTileBytes, &tdO, &bar->full[s], j * kTile, g, it.kvh, it.batch);
                        const int64_t head = (int64_t)it.batch * p.hq + it.kvh * p.group + g;
                        bulk_load(sR + s * 1024, p.rows + (head * p.qtiles + j) * 256, 1024, &bar->full[s]);
                    }
            }
            for (int i = max(0, items - C::kKv); i < items; ++i)
                mbar_wait_drain(&bar->kv_full[i % C::kKv], (i / C::kKv) & 1);
            for (int i = max(0, ring - C::kStages); i < ring; ++i)
                mbar_wait_drain(&bar->full[i % C::kStages], (i / C::kStages) & 1);
        } else {  // Q and dO rows past the valid length: P and dS are 0 there, but 0 x NaN is not
            int ring = 0, nfix = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < p.items && ok; idx += gridDim.x) {
                const DkvItem it = dkv_item(p, idx);
                if (it.hi <= it.lo) continue;
                if (it.sp.Lq >= p.nq || it.hi * kTile <= it.sp.Lq) {
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
                    uint8_t *st = sT + (ring - 1) % C::kStages * 2 * C::kTileBytes;
                    zero_rows<DP>(st, it.sp.Lq - (it.hi - 1) * kTile, lane - 1, 31);
                    zero_rows<DP>(st + C::kTileBytes, it.sp.Lq - (it.hi - 1) * kTile, lane - 1, 31);
                    fence_proxy_async_smem();
                    mbar_arrive(&bar->fixed[(nfix - 1) & 1]);
                }
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        const bool first = warp == kMmaWarp;  // S and dV; the other thread: dP and dK
        if (elect_one()) {
            int n = 0, items = 0, nfix = 0;
            bool ok = true;
            const uint32_t aKV0 = smem_u32(sK) + (first ? 0 : C::kTileBytes), aT = smem_u32(sT);
            uint64_t *done = first ? bar->pv_done : bar->ds_done, *full = first ? bar->s_full : bar->dp_full,
                     (*ready)[2] = first ? bar->p_full : bar->ds_full;
            auto phase = [](int g) { return (uint32_t)(g >> 1) & 1u; };
            auto buffer = [&](int g) { return tmem + 128 * ((2 * g + (first ? 0 : 1)) % C::kBufs); };
            for (int idx = blockIdx.x; idx < p.items && ok; idx += gridDim.x) {
                const DkvItem it = dkv_item(p, idx);
                const int per = it.hi - it.lo;
                if (per <= 0) continue;
                const int steps = per * p.group, end = n + steps;
                const bool fix = it.sp.Lq < p.nq && it.hi * kTile > it.sp.Lq;
                const int kb = items % C::kKv;
                const uint32_t aKV = aKV0 + kb * 2 * C::kTileBytes;
                int in_head = 0;  // tile of the next score step within its head
                // S = K Q^T (or dP = V dO^T) of step g, into the buffer that step g - 1 or g - 2
                // has left
                auto score = [&](int g) {
                    const int s = g % C::kStages;
                    if (!thread_spin(&bar->full[s], (g / C::kStages) & 1, p.status, 103, abort_flag)) return false;
                    if (++in_head == per) {
                        in_head = 0;
                        if (fix) {
                            if (first) mbar_arrive(&bar->fix_wanted);
                            if (!thread_spin(&bar->fixed[nfix & 1], phase(nfix), p.status, 104, abort_flag)) return false;
                            ++nfix;
                        }
                    }
                    if (C::kBufs == 2) {  // its own kind of the step before
                        if (g >= 1 && !thread_spin(&done[(g - 1) & 1], phase(g - 1), p.status, 105, abort_flag))
                            return false;
                    } else if (first) {  // S follows dP of step g - 2
                        if (g >= 2 && !thread_spin(&bar->ds_done[g & 1], phase(g - 2), p.status, 105, abort_flag))
                            return false;
                    } else {  // dP follows S of step g - 1
                        if (g >= 1 && !thread_spin(&bar->pv_done[(g - 1) & 1], phase(g - 1), p.status, 106, abort_flag))
                            return false;
                    }
                    tc_fence_after();
                    mma_scores<DP>(buffer(g), aKV, aT + s * 2 * C::kTileBytes + (first ? 0 : C::kTileBytes));
                    mma_commit(&full[g & 1]);
                    return true;
                };
                // dV += P^T dO (or dK += dS^T Q) of step g
                auto sum = [&](int g) {
                    const int s = g % C::kStages;
                    const uint32_t d = tmem + (first ? C::kDv : C::kDk), m = buffer(g),
                                   t = aT + s * 2 * C::kTileBytes + (first ? C::kTileBytes : 0);
                    if (!thread_spin(&ready[g & 1][0], phase(g), p.status, 108, abort_flag)) return false;
                    if (g == n && items > 0 &&
                        !thread_spin(&bar->acc_free, (items - 1) & 1, p.status, 109, abort_flag))
                        return false;
                    tc_fence_after();
                    mma_sum_half<DP>(d, m, t, g > n ? 1u : 0u);
                    if (!thread_spin(&ready[g & 1][1], phase(g), p.status, 108, abort_flag)) return false;
                    tc_fence_after();
                    mma_sum_half<DP>(d, m + 64, t + 8192, 1u);
                    mma_commit(&done[g & 1]);
                    mma_commit(&bar->empty[s]);
                    return true;
                };
                ok = thread_spin(&bar->kv_full[kb], (items / C::kKv) & 1, p.status, 107, abort_flag) && score(n);
                if (C::kBufs == 3 && first && steps > 1) ok = ok && score(n + 1);
                for (int g = n; g < end && ok; ++g) {
                    if (C::kBufs == 2) ok = sum(g) && (g + 1 >= end || score(g + 1));
                    else if (first) ok = sum(g) && (g + 2 >= end || score(g + 2));
                    else ok = (g + 1 >= end || score(g + 1)) && sum(g);
                }
                if (!ok) break;
                mma_commit(&bar->kv_free[kb]);
                mma_commit(&bar->acc_full);
                n = end;
                ++items;
            }
            mma_commit(&bar->drain[first ? 0 : 1]);
            mbar_wait_drain(&bar->drain[first ? 0 : 1], 0);
        }
        __syncwarp();
    }
    } else {
        setmaxnreg_inc<kMathRegs>();
        const int half = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float sl = p.scale_log2;
        const float2 sl2 = make_float2(sl, sl);
        int n = 0, items = 0;
        bool ok = true;
        DkvItem it = dkv_item(p, min((int)blockIdx.x, p.items - 1));
        for (int idx = blockIdx.x; idx < p.items && ok; idx += gridDim.x) {
            const int key = it.k0 + row, off = it.sp.Lk - it.sp.Lq, lo = it.lo, hi = it.hi,
                      steps = (hi - lo) * p.group;
            // queries [first, end) see this key (the rows past the length need no mask: their
            // -lse is -inf)
            const int first = p.causal ? max(0, key - off) : 0;
            const int end = p.window ? (int)min((long long)it.sp.Lq, (long long)key - off + p.window) : 1 << 30;
            const unsigned width = end > first ? (unsigned)(end - first) : 0u;
            int j = lo;
            for (int g = n; g < n + steps; ++g) {
                const int s = g % C::kStages;
                const uint32_t tS = tmem + 128 * (2 * g % C::kBufs) + 64 * half + lanes,
                               tD = tmem + 128 * ((2 * g + 1) % C::kBufs) + 64 * half + lanes;
                const uint32_t aR = smem_u32(sR) + s * 1024 + 256 * half;  // -lse and, 512 on, -delta
                const uint32_t parity = (uint32_t)(g >> 1) & 1u;
                if (!warp_spin(&bar->full[s], (g / C::kStages) & 1, p.status, 111, abort_flag) ||
                    !warp_spin(&bar->s_full[g & 1], parity, p.status, 112, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int q0 = j * kTile + 64 * half;
                if (__any_sync(0xffffffffu, first > q0 || end < q0 + 64))
                    fill_outside(tS, first - q0, width, kMinusInf);
                uint32_t v[2][32], o[32];
                load_columns(tS, v);
#pragma unroll
                for (int c = 0; c < 2; ++c)
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
                        o[16 * c + e / 2] = pack2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                        o[16 * c + e / 2 + 1] = pack2(__uint_as_float(v[c][e + 2]), __uint_as_float(v[c][e + 3]));
                    }
                tmem_st32(tS, o);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->p_full[g & 1][half]);
                if (!warp_spin(&bar->dp_full[g & 1], parity, p.status, 113, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t u[2][32];
                load_columns(tD, u);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 dl = lds4(aR + 512 + 4 * (32 * c + e));
                        const float2 y0 = fadd2(make_float2(__uint_as_float(u[c][e]), __uint_as_float(u[c][e + 1])),
                                                make_float2(dl.x, dl.y));
                        const float2 y1 = fadd2(make_float2(__uint_as_float(u[c][e + 2]), __uint_as_float(u[c][e + 3])),
                                                make_float2(dl.z, dl.w));
                        const float2 z0 = fmul2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), y0);
                        const float2 z1 = fmul2(make_float2(__uint_as_float(v[c][e + 2]), __uint_as_float(v[c][e + 3])), y1);
                        o[16 * c + e / 2] = pack2(z0.x, z0.y);
                        o[16 * c + e / 2 + 1] = pack2(z1.x, z1.y);
                    }
                tmem_st32(tD, o);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->ds_full[g & 1][half]);
                if (++j == hi) j = lo;
            }
            n += max(0, steps);
            if (!ok) break;
            const bool some = steps > 0;
            const DkvItem next = dkv_item(p, min(idx + (int)gridDim.x, p.items - 1));  // while the sums end
            const bool exists = key < p.nk, valid = key < it.sp.Lk;
            // warps 0-3 write dV, warps 4-7 dK
            __nv_bfloat16 *dst =
                half ? p.dK + it.batch * p.sdK.b + it.kvh * p.sdK.h + (int64_t)key * p.sdK.n
                      : p.dV + it.batch * p.sdV.b + it.kvh * p.sdV.h + (int64_t)key * p.sdV.n;
            if (some) {
                if (!warp_spin(&bar->acc_full, items & 1, p.status, 114, abort_flag)) break;
                tc_fence_after();
                ++items;
                uint32_t o[DP / 32][32];
                load_columns(tmem + (half ? C::kDk : C::kDv) + lanes, o);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->acc_free);
                if (exists)
#pragma unroll
                    for (int c = 0; c < DP / 32; ++c)
                        store_row(dst, o[c], 32 * c, p.d, half ? p.scale : 1.f, !valid, p.wide >> (half ? 1 : 2) & 1);
            } else if (exists) {
                zero_row(dst, p.d);
            }
            it = next;
        }
    }
    if (warp == kLoadWarp) wait_prerequisites();  // no later kernel before the second one has ended
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int DP>
int launch(const Call &c, BwdParams &p) {
    using Cq = DqLayout<DP>;
    using Ck = DkvLayout<DP>;
    CUtensorMap tQ, tK, tV, tdO;
    if (!encode_rows(&tQ, c.Q, c.sQ, c.b, c.hq, p.group, c.nq, c.d, kTile, 1) ||
        !encode_rows(&tdO, c.dO, c.sdO, c.b, c.hq, p.group, c.nq, c.d, kTile, 1) ||
        !encode_rows(&tK, c.K, c.sK, c.b, c.hk, 1, c.nk, c.d, kTile, 1) ||
        !encode_rows(&tV, c.V, c.sV, c.b, c.hk, 1, c.nk, c.d, kTile, 1))
        return LINFORMER_ERR_LAUNCH;
    int st = allow_smem(reinterpret_cast<const void *>(softmax_attn_dq_kernel<DP>), Cq::kSmem, DP == 64 ? 2 : 3);
    if (!st) st = allow_smem(reinterpret_cast<const void *>(softmax_attn_dkv_kernel<DP>), Ck::kSmem, DP == 64 ? 4 : 5);
    if (st) return st;
    void *ws = nullptr;
    const int64_t qitems = (int64_t)c.b * c.hq * p.qtiles, kitems = (int64_t)c.b * c.hk * p.kblocks;
    if (qitems > kMaxItems || kitems > kMaxItems) return LINFORMER_ERR_SIZE;
    if (workspace_alloc(&ws, (size_t)qitems * 1024, c.stream) != LINFORMER_OK) return LINFORMER_ERR_ALLOC;
    p.rows = static_cast<float *>(ws);
    const int sms = device_sms();
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
    cfg.blockDim = dim3(kThreads);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!st) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX_BWD, c.stream);
        p.items = (int)qitems;
        cfg.gridDim = dim3((unsigned)std::min<int64_t>(qitems, sms));
        cfg.dynamicSmemBytes = Cq::kSmem;
        if (cudaLaunchKernelEx(&cfg, softmax_attn_dq_kernel<DP>, tQ, tK, tV, tdO, p) != cudaSuccess)
            st = LINFORMER_ERR_LAUNCH;
    }
    if (!st) {
        KernelScope scope(LINFORMER_KERNEL_SOFTMAX_BWD, c.stream);
        p.items = (int)kitems;
        cfg.gridDim = dim3((unsigned)std::min<int64_t>(kitems, sms));
        cfg.dynamicSmemBytes = Ck::kSmem;
        if (cudaLaunchKernelEx(&cfg, softmax_attn_dkv_kernel<DP>, tQ, tK, tV, tdO, p) != cudaSuccess)
            st = LINFORMER_ERR_LAUNCH;
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
