// Exact softmax attention of new tokens over a paged cache, with trees of drafted tokens: for
// every query row i of every head
//
//     O_i = sum_j p_ij V_j,   p_ij = exp(scale Q_i.K_j - lse_i),   lse_i = log sum_j exp(scale Q_i.K_j)
//
// over the cache rows j that the row sees, in one pass over the pages.
//
// New tokens are few beside the rows that they look at, so the products are turned round: keys
// take the 128 rows of a product and queries its columns, of which there can be as few as 16,
//
//     S^T = K Q^T   (128 keys x N rows),   O^T += V^T P^T   (d x N rows),
//
// and a thread has one key and N / 2 queries: what a length or a page hides is a thread's own
// business, sums over keys stay in the thread until a row ends, and only a maximum that outgrows
// its reference by 2^kOutgrown makes threads exchange anything but a vote (the reference is any m
// near the maximum; P = 2^(s - m) goes to the tensor cores as bf16, in two parts where that is cheap,
// else rounded, at most 2^-8 of each term; sums and statistics are fp32).  Tiles of 128 keys come by
// TMA, a box a page, through a ring in shared memory.
//
// The blocks of 128 keys of all rows form one long list, sequence by sequence, and each CTA takes an
// equal run of it, so that differing lengths cost nothing; a row whose run is cut is joined from
// its parts, in order, by a second kernel.  Where tables or windows are short nothing is cut, and where
// units are few each CTA has its own without a list.
//
// Bound by memory: one token over 62 ragged caches of up to 8192 rows, 32 over 8 heads of 128, pages of
// 16: 228 us, 5.9 TB/s, 6.5 while all CTAs stream (a ring of four tiles of 32 KB is as good as five, of
// three 270 us).  Short calls are bound by their start (two short sequences: 7.9 us, of which 3.6 until the
// first keys are there, 0.7 to 0.9 a block, 1.1 to the end).  64 rows a head: 1.1 us a block, 0.7 of it
// softmax.  More than 64 rows go to paged_attn_wide.cu, whose threads have a row each (128 columns here: the
// chunk of that file 1533 us).
//   warps 0-7   softmax: two groups of four warps, each half of the columns
//   warp 8      loads: looks the pages up and issues a box a lane
//   warp 9      one thread issues the products
//   warps 10 11 rows without keys: O = 0, lse = -inf
#include <algorithm>
#include <cmath>

#include "paged_attn.cuh"

namespace linformer {
namespace paged {
namespace {

constexpr int kThreads = 384, kLoadWarp = 8, kMmaWarp = 9, kEmptyWarp = 10;

template <int DP, int N>
struct Layout {
    static constexpr uint32_t kTileBytes = kTile * DP * 2;
    // DP = 64: K and V of a block share an entry of the ring, V first (the product takes 128 rows of
    // V^T, of which the second half falls on K and is not used)
    static constexpr bool kPair = DP == 64;
    static constexpr int kEntries = 5;
    static constexpr uint32_t kEntryBytes = kPair ? 2 * kTileBytes : kTileBytes;
    // P in two parts of bf16 each, the rounded and the rest, as columns beside each other, where the
    // products cost next to nothing (N = 16, 32: 1 % more time, and the result is off by its own rounding
    // alone, 1.7e-3 against 2.3e-3; N = 64: 4 %, left at one).
    static constexpr bool kSplit = N < 64;
    static constexpr int kCols = kSplit ? 2 * N : N;  // of P and of O
    static_assert(kCols <= 64, "a row of P is 128 bytes");
    static constexpr int kPBufs = 2;
    static constexpr uint32_t kPBytes = kTile * 128;
    static constexpr uint32_t kQHalf = N * 128, kQBytes = kQHalf * (DP / 64);
    static constexpr uint32_t kP = kEntries * kEntryBytes, kQ = kP + kPBufs * kPBytes, kEnd = kQ + kQBytes;
    static constexpr uint32_t kS = 0, kO = 2 * N;  // tensor memory: S, S, O
};

struct Shared {
    uint64_t full[5], empty[5], q_full, q_free, s_full[2], s_free[2], p_full[2], pv_done[2], o_free, drain;
    uint32_t tmem;
    int abort;
    // of each column: the reference (log2; -infinity where no key has been seen), what is added to the
    // scores for it, what the reference moves by, and what l and O take for that, or 1 / l
    alignas(16) float m[64];
    alignas(16) float off[64];
    alignas(16) float up[64];
    alignas(16) float f[64];
    float part[2][4][32];  // a value a column, by warp of each group
    alignas(16) int64_t row[64];  // where a column's row of O begins, -1: nowhere
    Marks marks;
};

template <int C>
__device__ __forceinline__ void tmem_load(uint32_t t, uint32_t (&v)[C]) {
    if constexpr (C == 8) tmem_ld8(t, v);
    else if constexpr (C == 16) tmem_ld16(t, v);
    else tmem_ld32(t, v);
}

// Reduces C columns over the 32 lanes of a warp; column(lane) of lane's result.  Each exchange
// halves the columns that a lane still holds.
template <int C, typename F>
__device__ __forceinline__ float reduce_columns(float (&v)[C], int lane, F f) {
    static_assert(C <= 32, "a column a lane");
    int w = 16;
#pragma unroll
    for (int c = C / 2; c >= 1; c /= 2, w /= 2) {
        const bool upper = lane & w;
#pragma unroll
        for (int i = 0; i < c; ++i) {
            const float send = upper ? v[i] : v[i + c], keep = upper ? v[i + c] : v[i];
            v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, w));
        }
    }
    float r = v[0];
    for (; w >= 1; w /= 2) r = f(r, __shfl_xor_sync(0xffffffffu, r, w));
    return r;
}
// Over a warp, into part[0 .. C).
template <int C, typename F>
__device__ __forceinline__ void reduce_to(const float (&v)[C], float *part, int lane, F f) {
    constexpr int H = C < 16 ? C : 16;
#pragma unroll
    for (int h = 0; h < C; h += H) {
        float x[H];
#pragma unroll
        for (int i = 0; i < H; ++i) x[i] = v[h + i];
        const float r = reduce_columns(x, lane, f);
        if (lane % (32 / H) == 0) part[h + lane / (32 / H)] = r;
    }
}

// Which of `positions` rows from q0 on see node `node` of a tree, a bit a row.
__device__ __noinline__ uint64_t tree_bits(const uint64_t *mask, int words, int node, int q0, int positions, int Lq) {
    uint64_t see = 0;
    mask += (int64_t)q0 * words + (node >> 6);
#pragma unroll 8
    for (int x = 0; x < positions; ++x)
        if (q0 + x < Lq) see |= (__ldg(mask + (int64_t)x * words) >> (node & 63) & 1) << x;
    return see;
}

template <int DP, int N>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                  const __grid_constant__ CUtensorMap tV, const __grid_constant__ AttnParams p) {
    using L = Layout<DP, N>;
    constexpr int C = N / 2;  // columns of a thread
    // (addresses in it are constants then, and take no registers)
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        leave(p, 133);
        return;
    }
    Shared *sh = reinterpret_cast<Shared *>(smem + L::kEnd);
    volatile int *abort_flag = &sh->abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 32) {
        for (int s = 0; s < L::kEntries; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        mbar_init(&sh->q_full, 1);
        mbar_init(&sh->q_free, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh->s_full[s], 1);
            mbar_init(&sh->s_free[s], 8);
            mbar_init(&sh->p_full[s], 8);
            mbar_init(&sh->pv_done[s], 1);
        }
        mbar_init(&sh->o_free, 8);
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tQ);
        prefetch_tmap(&tK);
        prefetch_tmap(&tV);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh->tmem, 512);
        tmem_relinquish();
    }
    // rows of Q that no box fills
    for (uint32_t x = tid * 16; x < L::kQBytes; x += kThreads * 16)
        *reinterpret_cast<uint4 *>(smem + L::kQ + x) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    tc_fence_before();
    wait_prerequisites();
    if (tid == 0) launch_dependents();  // the join, which waits for this grid's end
    Walk walk = p.direct ? Walk(p) : Walk();
    if (!p.direct) fill(p, sh->marks, tid, kThreads);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    if (!p.direct) walk = Walk(p, sh->marks, blockIdx.x);
    Item it;

    if (warp == kLoadWarp) {  // ---------------- loads
        // a lane's box of a tile: `box` rows of a page, 64 columns
        const int bi = lane / (DP / 64), half = lane % (DP / 64);
        const bool mine = bi < p.nbox;
        const int row = bi * p.box;
        const uint32_t dst = half * 16384u + row * 128u;
        int ring = 0, nq = 0;
        bool ok = true;
        while (ok && walk.next(p, sh->marks, it)) {
            const Rows r(p, it.unit);
            const int32_t *table = p.table + (int64_t)it.seq * p.width;
            const int low = it.sp.first(r.q0);
            auto look = [&](int j) { return mine ? page_of(p, table, j, row, low, it.sp.Lk) : 0; };
            int page = look(it.lo);
            // (one token over 62 caches: 228 us; Q after the next item's first keys, which then do not wait for
            // the last scores, 232; Q in two buffers 229)
            if (nq > 0 && !warp_spin(&sh->q_free, (nq - 1) & 1, p.status, 120, abort_flag)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sh->q_full, (uint32_t)(p.qbox * p.hbox * DP * 2));
                for (int h = 0; h < DP / 64; ++h)
                    tma_load_5d(smem + L::kQ + h * L::kQHalf, &tQ, &sh->q_full, h * 64, r.q0, r.h0, it.kvh, it.seq);
            }
            ++nq;
            for (int j = it.lo; j < it.hi; ++j) {
                const int now = page, at = (j * kTile + row) & (p.page - 1);
                if (j + 1 < it.hi) page = look(j + 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int e = ring % L::kEntries;
                    if (!L::kPair || kv == 0) {
                        if (ring >= L::kEntries &&
                            !warp_spin(&sh->empty[e], (ring / L::kEntries - 1) & 1, p.status, 121, abort_flag)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&sh->full[e], L::kEntryBytes);
                        __syncwarp();
                    }
                    if (mine)
                        tma_load_5d(smem + e * L::kEntryBytes + (L::kPair && kv == 0 ? L::kTileBytes : 0) + dst,
                                    kv ? &tV : &tK, &sh->full[e], half * 64, at, 0, it.kvh, now);
                    if (!L::kPair || kv == 1) ++ring;
                }
                if (!ok) break;
            }
        }
        // no copy outlives the CTA
        if (lane == 0) {
            if (nq > 0) mbar_wait_drain(&sh->q_full, (nq - 1) & 1);
            for (int i = max(0, ring - L::kEntries); i < ring; ++i)
                mbar_wait_drain(&sh->full[i % L::kEntries], (i / L::kEntries) & 1);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (elect_one()) {  // ---------------- products
            const uint32_t idesc_s = idesc_f16(128, N, 1, 0, 0), idesc_o = idesc_f16(128, L::kCols, 1, 1, 1);
            const uint64_t dq = sdesc(smem_u32(smem + L::kQ), 16, 1024, kSwizzle128B);
            int ns = 0, no = 0, items = 0;  // blocks whose S, whose O has been issued
            bool ok = true;
            while (ok && walk.next(p, sh->marks, it)) {
                auto score = [&](int j) {
                    const int r = L::kPair ? ns : 2 * ns, e = r % L::kEntries, s = ns & 1;
                    if (!thread_spin(&sh->full[e], (r / L::kEntries) & 1, p.status, 122, abort_flag)) return false;
                    if (j == it.lo && !thread_spin(&sh->q_full, items & 1, p.status, 123, abort_flag)) return false;
                    if (ns > 1 && !thread_spin(&sh->s_free[s], ((ns >> 1) - 1) & 1, p.status, 124, abort_flag)) return false;
                    tc_fence_after();
                    const uint64_t dk = sdesc(smem_u32(smem + e * L::kEntryBytes + (L::kPair ? L::kTileBytes : 0)), 16, 1024,
                                              kSwizzle128B);
#pragma unroll
                    for (int x = 0; x < DP / 16; ++x)
                        mma_ss(tmem + L::kS + N * s, dk + (uint64_t)((x >> 2) * 1024 + (x & 3) * 2),
                               dq + (uint64_t)((x >> 2) * (L::kQHalf >> 4) + (x & 3) * 2), idesc_s, x > 0 ? 1u : 0u);
                    mma_commit(&sh->s_full[s]);
                    if (!L::kPair) mma_commit(&sh->empty[e]);
                    if (j == it.hi - 1) mma_commit(&sh->q_free);
                    ++ns;
                    return true;
                };
                auto output = [&](int j) {
                    const int r = L::kPair ? no : 2 * no + 1, e = r % L::kEntries, b = no % L::kPBufs;
                    if (!L::kPair && !thread_spin(&sh->full[e], (r / L::kEntries) & 1, p.status, 125, abort_flag)) return false;
                    if (!thread_spin(&sh->p_full[b], (no / L::kPBufs) & 1, p.status, 126, abort_flag)) return false;
                    if (j == it.lo && items > 0 && !thread_spin(&sh->o_free, (items - 1) & 1, p.status, 127, abort_flag))
                        return false;
                    tc_fence_after();
                    const uint64_t dv = sdesc(smem_u32(smem + e * L::kEntryBytes), 16384, 1024, kSwizzle128B);
                    const uint64_t dp = sdesc(smem_u32(smem + L::kP + b * L::kPBytes), 16384, 1024, kSwizzle128B);
#pragma unroll
                    for (int x = 0; x < kTile / 16; ++x)
                        mma_ss(tmem + L::kO, dv + (uint64_t)(128 * x), dp + (uint64_t)(128 * x), idesc_o,
                               (j > it.lo || x > 0) ? 1u : 0u);
                    mma_commit(&sh->pv_done[b]);
                    mma_commit(&sh->empty[e]);
                    ++no;
                    return true;
                };
                ok = score(it.lo);
                for (int j = it.lo; j < it.hi && ok; ++j) ok = (j + 1 >= it.hi || score(j + 1)) && output(j);
                ++items;
            }
            mma_commit(&sh->drain);
            mbar_wait_drain(&sh->drain, 0);
        }
        __syncwarp();
    } else if (warp >= kEmptyWarp) {  // ---------------- rows without keys
        if (warp == kEmptyWarp && lane == 0) write_cut(p, walk, sh->marks);
        __syncwarp();
        write_empty(p, sh->marks, p.direct ? &walk : nullptr, warp - kEmptyWarp, kThreads / 32 - kEmptyWarp, lane);
    } else {  // ---------------- softmax: one key a thread, C of the rows
        const int w = warp >> 2, key0 = tid & 127, c0 = w * C;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tO = tmem + L::kO + c0 + lanes;
        const float sl = p.scale_log2;
        float *part = sh->part[w][warp & 3];
        int n = 0;
        bool ok = true;
        // the product of block x and P is done; with a barrier a buffer of P, no waiting warp is ever two
        // phases behind: the next product from a buffer waits for every warp's P
        auto product = [&](int x, int code) {
            return warp_spin(&sh->pv_done[x % L::kPBufs], (x / L::kPBufs) & 1, p.status, code, abort_flag);
        };
        // The group's warps leave together: what a wait of one came to is ANDed at a barrier.
        auto agree = [&] { return ok = named_barrier_and(1 + w, 128, ok); };
        while (walk.next(p, sh->marks, it)) {
            float l[C];
#pragma unroll
            for (int c = 0; c < C; ++c) l[c] = 0.f;
            bool unset = true;  // some row has seen no key yet: its first one is its reference, however small
            if (key0 < C) sh->off[c0 + key0] = 0.f;
            named_barrier_sync(1 + w, 128);
            const Rows r(p, it.unit);
            const int before = it.sp.Lk - it.sp.Lq;
            const uint64_t *mask = p.mask ? p.mask + (int64_t)it.seq * p.nq * p.words : nullptr;
            for (int j = it.lo; j < it.hi; ++j, ++n) {
                const int s = n & 1, b = n % L::kPBufs, k0 = j * kTile, key = k0 + key0;
                const uint32_t tS = tmem + L::kS + N * s + c0 + lanes;
                ok = ok && warp_spin(&sh->s_full[s], (n >> 1) & 1, p.status, 128, abort_flag);
                tc_fence_after();
                float y[C];  // log2 of p, from the reference
                {
                    uint32_t v[C];
                    tmem_load(tS, v);
#pragma unroll
                    for (int c = 0; c < C; c += 4) {
                        const float4 off = *reinterpret_cast<const float4 *>(&sh->off[c0 + c]);
                        const float2 a = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                               make_float2(sl, sl), make_float2(off.x, off.y));
                        const float2 z = ffma2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                                               make_float2(sl, sl), make_float2(off.z, off.w));
                        y[c] = a.x, y[c + 1] = a.y, y[c + 2] = z.x, y[c + 3] = z.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->s_free[s]);
                // which columns see the key, a bit each: rows [key, key + window) of the new tokens, or
                // those whose masks have the node
                const bool ragged = k0 + kTile > it.sp.Lk;
                const bool edge = p.mask ? k0 + kTile > before
                                         : p.causal && (it.sp.end(r.q0) < min(k0 + kTile, it.sp.Lk) ||
                                                        k0 < it.sp.first(min(r.q0 + p.qbox, it.sp.Lq) - 1));
                if (ragged || edge) {
                    uint32_t see = key < it.sp.Lk ? 0xffffffffu : 0u;
                    if (edge) {
                        uint64_t rows = ~0ull;  // of the tile's positions
                        const int at = key - before - r.q0;
                        if (p.mask) {
                            if (key >= before && key < it.sp.Lk)
                                rows = tree_bits(mask, p.words, key - before, r.q0, p.qbox, it.sp.Lq);
                        } else {
                            if (at > 0) rows = at < 64 ? rows << at : 0;
                            const int z = p.window ? at + p.window : 64;  // (at + window fits: both are below 2^30)
                            if (z < 64) rows = z > 0 ? rows & ~(~0ull << z) : 0;
                        }
                        // the positions come again for each head
                        see &= p.qbox >= C ? (uint32_t)(rows >> (c0 & (p.qbox - 1)))
                                           : ((uint32_t)rows & ((1u << p.qbox) - 1)) * (0xffffffffu / ((1u << p.qbox) - 1));
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (!(see >> c & 1)) y[c] = -INFINITY;  // (whatever it was)
                }
                float top = y[0];
#pragma unroll
                for (int c = 1; c < C; ++c) top = fmaxf(top, y[c]);
                if (named_barrier_or(1 + w, 128, unset || top > kOutgrown || !ok)) {
                    // references move up by the columns' maxima (where there is none yet, to it); y, l and O
                    // with them
                    if (!agree()) break;
                    reduce_to(y, part, lane, [](float a, float z) { return fmaxf(a, z); });
                    if (j > it.lo) ok = product(n - 1, 129);
                    if (!agree()) break;
                    bool none = false;
                    if (key0 < C) {
                        const int c = c0 + key0;
                        float up = sh->part[w][0][key0];
                        for (int x = 1; x < 4; ++x) up = fmaxf(up, sh->part[w][x][key0]);
                        // A padded query gets a reference that no score outgrows: what stands there has no vote on
                        // when references move, on which the last bits of all results depend.  (Columns that no
                        // box fills are zeros, alike in every call.)
                        if (it.sp.Lq < p.nq && r.q0 + (c & (p.qbox - 1)) >= it.sp.Lq) up = INFINITY;
                        const float m = j > it.lo ? sh->m[c] : -INFINITY;
                        none = m == -INFINITY && up == -INFINITY;
                        // (a reference of 0 stands for none)
                        if (m != -INFINITY) up = fmaxf(up, 0.f);
                        if (!none) {
                            const float mn = m == -INFINITY ? up : m + up;
                            sh->m[c] = mn;
                            sh->off[c] = -mn;
                        } else {
                            sh->m[c] = -INFINITY;
                            up = 0.f;
                        }
                        sh->up[c] = up;
                        sh->f[c] = m == -INFINITY ? 1.f : ex2_approx(-up);  // (l and O are 0 where there was none)
                        none = none && c < p.qbox * p.hbox && r.h0 + c / p.qbox < p.group &&
                               r.q0 + (c & (p.qbox - 1)) < it.sp.Lq;
                    }
                    unset = named_barrier_or(1 + w, 128, none);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        y[c] -= sh->up[c0 + c];
                        l[c] *= sh->f[c0 + c];
                    }
                    if (j > it.lo) {
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < (L::kSplit ? 2 : 1) * C; x += 8) {
                            const int c = x % C;
                            const uint32_t at = tO + c + (x < C ? 0 : N);
                            uint32_t q[8];
                            tmem_ld8(at, q);
#pragma unroll
                            for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(__uint_as_float(q[e]) * sh->f[c0 + c + e]);
                            tmem_st8_async(at, q);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                }
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    y[c] = ex2_approx(y[c]);
                    l[c] += y[c];
                }
                // the buffer's last product is done
                if (ok && n >= L::kPBufs) ok = product(n - L::kPBufs, 130);
                uint8_t *row = smem + L::kP + b * L::kPBytes + key0 * 128;
#pragma unroll
                for (int c = 0; c < C; c += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = y[c + 2 * e], z = y[c + 2 * e + 1];
                        hi[e] = pack2(a, z);
                        lo[e] = pack2(a - __uint_as_float(hi[e] << 16), z - __uint_as_float(hi[e] & 0xffff0000u));
                    }
                    auto at = [&](int col) { return row + ((col / 8 ^ (key0 & 7)) * 16); };
                    *reinterpret_cast<uint4 *>(at(c0 + c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if (L::kSplit) *reinterpret_cast<uint4 *>(at(N + c0 + c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (ragged && w == 0) {
                    // rows of V past the length may hold anything: P is 0 there, but 0 x NaN is not
                    const int rr = L::kPair ? n : 2 * n + 1, e = rr % L::kEntries;
                    ok = ok && warp_spin(&sh->full[e], (rr / L::kEntries) & 1, p.status, 131, abort_flag);
                    if (ok && key >= it.sp.Lk) {
                        uint8_t *at = smem + e * L::kEntryBytes + key0 * 128;
#pragma unroll
                        for (int x = 0; x < DP / 8; ++x)
                            *reinterpret_cast<uint4 *>(at + (x / 8) * 16384 + (x % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[b]);
            }
            // O / l out of tensor memory, where a thread has an element of every row, and through the
            // buffers of P, a row a warp, to memory (in a short loop: at a CTA's end its instructions come
            // from far, and a store a column in line took 2.6 us)
            reduce_to(l, part, lane, [](float a, float z) { return a + z; });
            ok = ok && product(n - 1, 132);
            // (both groups: each stores over what the other may still write as P)
            if (!(ok = named_barrier_and(3, 256, ok))) break;
            tc_fence_after();
            uint32_t o[C];
            tmem_load(tO, o);
            if (L::kSplit) {
                uint32_t rest[C];
                tmem_load(tO + N, rest);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(rest[c]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->o_free);
            float *stage = reinterpret_cast<float *>(smem + L::kP) + c0 * DP;
            if (key0 < DP)
#pragma unroll
                for (int c = 0; c < C; ++c) stage[c * DP + key0] = __uint_as_float(o[c]);
            if (key0 < C) {
                const int c = c0 + key0, i = r.q0 + (c & (p.qbox - 1)), hg = r.h0 + c / p.qbox;
                float sum = 0.f;
                for (int x = 0; x < 4; ++x) sum += sh->part[w][x][key0];
                const bool dead = i >= it.sp.Lq || sum == 0.f;
                const float lse = dead ? -INFINITY : sh->m[c] * kLn2 + logf(sum);
                const int64_t h = (int64_t)it.kvh * p.group + hg;
                const bool exists = c < p.qbox * p.hbox && hg < p.group && i < p.nq;
                sh->f[c] = dead ? 0.f : 1.f / sum;
                sh->row[c] = !exists ? -1 : it.slot >= 0 ? ((int64_t)it.slot * N + c) * DP
                                                         : it.seq * p.so.b + h * p.so.h + (int64_t)i * p.so.n;
                if (it.slot >= 0) p.part_lse[(int64_t)it.slot * N + c] = lse;
                else if (exists) p.lse[(it.seq * (int64_t)p.hq + h) * p.nq + i] = lse;
            }
            named_barrier_sync(1 + w, 128);
            constexpr int E = DP / 32;  // elements of a lane
#pragma unroll 1
            for (int x = warp & 3; x < C; x += 4) {
                const int64_t at = sh->row[c0 + x];
                if (at < 0 || lane * E >= p.d) continue;
                const float f = sh->f[c0 + x];
                float y[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    y[e] = stage[x * DP + lane * E + e];
                    y[e] = f == 0.f ? 0.f : y[e] * f;
                }
                if (it.slot >= 0) {
#pragma unroll
                    for (int e = 0; e < E; e += 2)
                        *reinterpret_cast<float2 *>(p.part_o + at + lane * E + e) = make_float2(y[e], y[e + 1]);
                } else {
#pragma unroll
                    for (int e = 0; e < E; e += 2)
                        *reinterpret_cast<uint32_t *>(p.out + at + lane * E + e) = pack2(y[e], y[e + 1]);
                }
            }
            named_barrier_sync(3, 256);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the parts of the rows whose run of blocks was cut: lse = log sum_s exp(lse_s), O = sum_s
// exp(lse_s - lse) O_s, in the parts' order.  Bound by latency: each block lists the cut units, the rows of
// all of them are dealt out evenly, and a row's parts come kAtOnce at a time, weights and values together
// (a block a unit and 32nd of its rows, weights before values: 884 tokens of 8 heads of 40, window 5470, 45 us
// in all and 38 so; 16 x 5 tokens over 6001 rows, window 4095, 26.3 and 24.9; trees of 64 97.3 and 95.0.  Eight
// at a time: 37, 24.5, 99; 2 blocks an SM of eight at a time: trees 106).
// DP / 4 lanes a row; kEach warps a row where units are few and their parts many (4 units of 1024 blocks,
// 38 parts each).
constexpr int kJoinWarps = 8, kJoinThreads = kJoinWarps * 32, kJoinBlocks = 8;  // blocks an SM
template <int DP, int kEach>
__global__ void __launch_bounds__(kJoinThreads, 4) join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int kLanes = DP / 4, kRows = 32 / kLanes * kJoinWarps / kEach, kAtOnce = 4;
    __shared__ int4 units[kJoinThreads];
    __shared__ int last[kJoinThreads], counts[kJoinWarps];
    __shared__ float shared[kEach > 1 ? kJoinWarps : 1][6][32];
    launch_dependents();
    wait_prerequisites();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, mine = warp % kEach;
    const int4 cut = tid < p.ctas ? p.cuts[tid] : make_int4(-1, 0, 0, 0);
    const unsigned some = __ballot_sync(0xffffffffu, cut.x >= 0);
    if (lane == 0) counts[warp] = __popc(some);
    __syncthreads();
    int n = 0, before = 0;
    for (int w = 0; w < kJoinWarps; ++w) {
        before += w < warp ? counts[w] : 0;
        n += counts[w];
    }
    if (cut.x >= 0) {
        const int at = before + __popc(some & ((1u << lane) - 1));
        units[at] = cut;
        last[at] = tid;
    }
    __syncthreads();
    const int rows = p.qbox * p.hbox, all = p.per * rows, total = n * all, col = lane % kLanes * 4;
    for (int first = blockIdx.x * kRows; first < total; first += gridDim.x * kRows) {  // (a block's warps alike)
        const int row = first + warp / kEach * (32 / kLanes) + lane / kLanes, u = min(row, total - 1) / all,
                  y = min(row, total - 1) - u * all, t = y / rows, x = y - t * rows;
        const int4 unit = units[u];
        const int c0 = unit.w, c1 = last[u], tile = unit.y * p.per + t;
        const Rows r(p, tile);
        const int i = r.q0 + (x & (p.qbox - 1)), hg = r.h0 + x / p.qbox;
        const bool exists = row < total && tile < p.ntiles && hg < p.group && i < p.nq;
        // a row is cut at the end of its first CTA's run, and goes on at the start of the others'
        auto slot = [&](int c) { return ((int64_t)(2 * c + (c == c0 ? 1 : 0)) * p.per + t) * p.N + x; };
        const int each = (c1 + 1 - c0 + kEach - 1) / kEach, from = c0 + mine * each, to = exists ? min(c1 + 1, from + each) : 0;
        float m = -INFINITY, sum = 0.f, acc[4] = {};
        for (int c = from; c < to; c += kAtOnce) {
            float ls[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (c + k >= to) {
                    ls[k] = -INFINITY;
                    continue;
                }
                const int64_t at = slot(c + k);
                ls[k] = p.part_lse[at];
                v[k] = *reinterpret_cast<const float4 *>(p.part_o + at * DP + col);
            }
            float mn = m;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) mn = fmaxf(mn, ls[k]);
            // (fmaxf drops a NaN, its weight does not)
            const float f = m == mn ? 1.f : __expf(m - mn);
            m = mn;
            sum *= f;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] *= f;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (ls[k] == -INFINITY) continue;  // (a part without keys wrote no O)
                const float w = __expf(ls[k] - m);
                sum += w;
                acc[0] += w * v[k].x, acc[1] += w * v[k].y, acc[2] += w * v[k].z, acc[3] += w * v[k].w;
            }
        }
        if constexpr (kEach > 1) {
            shared[warp][0][lane] = m;
            shared[warp][1][lane] = sum;
#pragma unroll
            for (int e = 0; e < 4; ++e) shared[warp][2 + e][lane] = acc[e];
            __syncthreads();
            if (mine == 0) {
                float top = m;
                for (int o = 1; o < kEach; ++o) top = fmaxf(top, shared[warp + o][0][lane]);
                sum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = 0.f;
                for (int o = 0; o < kEach; ++o) {
                    const float mo = shared[warp + o][0][lane], f = mo == top ? 1.f : __expf(mo - top);
                    sum += f * shared[warp + o][1][lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] += f * shared[warp + o][2 + e][lane];
                }
                m = top;
            }
        }
        if (mine == 0 && exists) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int64_t h = (int64_t)unit.z * p.group + hg;
            __nv_bfloat16 *dst = p.out + unit.x * p.so.b + h * p.so.h + (int64_t)i * p.so.n;
            if (col < p.d)
                *reinterpret_cast<uint2 *>(dst + col) =
                    make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
            if (col == 0) p.lse[(unit.x * (int64_t)p.hq + h) * p.nq + i] = sum == 0.f ? -INFINITY : m + logf(sum);
        }
        if (kEach > 1) __syncthreads();  // `shared` again
    }
}

template <int DP, int N>
int launch(const AttnCall &c, AttnParams &p) {
    constexpr uint32_t kSmem = Layout<DP, N>::kEnd + sizeof(Shared);
    static_assert(kSmem <= 227 * 1024, "shared memory");
    constexpr int kSlot = 10 + (DP == 128 ? 3 : 0) + (N == 16 ? 0 : N == 32 ? 1 : 2);
    p.N = N;
    return launch_with_join(paged_attn_kernel<DP, N>, kThreads, kSmem, kSlot, c, p, DP);
}

template <int DP>
int launch_rows(const AttnCall &c, AttnParams &p) {
    const int rows = p.qbox * p.hbox;
    if (rows <= 16) return launch<DP, 16>(c, p);
    if (rows <= 32) return launch<DP, 32>(c, p);
    return launch<DP, 64>(c, p);
}

}  // namespace

int launch_with_join(Kernel kernel, int threads, uint32_t smem, int slot, const AttnCall &c, AttnParams &p, int dp) {
    CUtensorMap q, k, v;
    const Cache &cache = c.cache;
    // Rows of the caches are fetched 64 bytes at a time, not 256: what lies behind a short row is another
    // head's, or comes with its own box (one token, rows of 64 elements side by side with 11 other heads: 104
    // us and 84; of 40 with 7: 204 and 143, with 128 bytes 176; of 96 with 2: 72 and 62; of 128: 231 both).
    constexpr CUtensorMapL2promotion kFetch = CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    if (!sattn::encode_rows(&q, c.q, c.sq, c.b, c.hq, p.group, c.nq, c.d, p.qbox, p.hbox) ||
        !sattn::encode_rows(&k, cache.k, cache.sk, cache.pages, c.hk, 1, cache.page, c.d, p.box, 1, kFetch) ||
        !sattn::encode_rows(&v, cache.v, cache.sv, cache.pages, c.hk, 1, cache.page, c.d, p.box, 1, kFetch))
        return LINFORMER_ERR_LAUNCH;
    char *ws = nullptr;
    if (!p.whole) {
        const size_t head = (p.ctas * sizeof(int4) + 31) / 32 * 32;  // (parts are written 32 bytes at a time)
        const size_t parts = (size_t)2 * p.ctas * p.per * p.N;
        if (workspace_alloc(reinterpret_cast<void **>(&ws), head + parts * (dp + 1) * sizeof(float), c.stream) !=
            LINFORMER_OK)
            return LINFORMER_ERR_ALLOC;
        p.cuts = reinterpret_cast<int4 *>(ws);
        p.part_o = reinterpret_cast<float *>(ws + head);
        p.part_lse = p.part_o + parts * dp;
    }
    // each kernel is set up while the one before it ends, and waits for that before it reads
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int st = sattn::allow_smem(reinterpret_cast<const void *>(kernel), smem, slot);
    if (!st) {
        KernelScope scope(LINFORMER_KERNEL_PAGED, c.stream);
        cfg.gridDim = dim3((unsigned)p.ctas);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        if (cudaLaunchKernelEx(&cfg, kernel, q, k, v, p) != cudaSuccess) {
            cudaGetLastError();
            st = LINFORMER_ERR_LAUNCH;
        }
    }
    if (!st && !p.whole) {
        KernelScope scope(LINFORMER_KERNEL_PAGED, c.stream);
        // many parts where a unit's blocks, all units alike, would fill sixteen runs
        const int64_t units = std::min<int64_t>((int64_t)p.b * p.units * p.hk, p.ctas);
        const bool many = units * 16 <= p.ctas;
        const int64_t at_once = (dp == 64 ? 2 : 1) * (many ? kJoinWarps / 4 : kJoinWarps);
        cfg.gridDim = dim3((unsigned)std::min<int64_t>((int64_t)device_sms() * kJoinBlocks,
                                                       (units * p.per * p.qbox * p.hbox + at_once - 1) / at_once));
        cfg.blockDim = dim3(kJoinThreads);
        cfg.dynamicSmemBytes = 0;
        const auto join = dp == 64 ? (many ? join_kernel<64, 4> : join_kernel<64, 1>)
                                   : (many ? join_kernel<128, 4> : join_kernel<128, 1>);
        if (cudaLaunchKernelEx(&cfg, join, p) != cudaSuccess) {
            cudaGetLastError();
            st = LINFORMER_ERR_LAUNCH;
        }
    }
    if (ws) workspace_free(ws, c.stream);
    return st;
}

int attention(const AttnCall &call) {
    AttnParams p{};
    p.words = call.words;
    p.hq = call.hq;
    p.hk = call.hk;
    p.group = call.hq / call.hk;
    p.nq = call.nq;
    p.d = call.d;
    p.causal = call.causal;
    p.window = call.window;
    p.scale = call.scale;
    p.scale_log2 = call.scale * kLog2e;
    p.so = call.so;
    p.wide_stores = sattn::wide_stores(call.out, call.so, call.d);
    p.status = device_status_ptr();
    p.pages = call.cache.pages;
    p.page = call.cache.page;
    p.width = call.cache.width;
    p.shift = call.cache.shift;
    p.box = std::min(call.cache.page, kTile);
    p.nbox = kTile / p.box;
    // Rows of a tile: 128 positions of one head, or the smallest power of two that holds all
    // positions times as many heads of the group as fit.
    p.qbox = kTile;
    while (p.qbox > 1 && p.qbox / 2 >= call.nq) p.qbox /= 2;
    p.hbox = std::min(kTile / p.qbox, p.group);
    p.nch = (p.group + p.hbox - 1) / p.hbox;
    const int64_t ntiles = ((int64_t)call.nq + p.qbox - 1) / p.qbox * p.nch;
    const bool wide = p.qbox * p.hbox > 64;
    p.per = wide ? 2 : 1;
    const int64_t units = (ntiles + p.per - 1) / p.per;
    // the list of blocks is counted in 32 bits: at most kMaxSeqs sequences a launch, fewer where they
    // are huge
    const int64_t most = units * call.hk * (((int64_t)p.width * p.page + kTile - 1) / kTile);
    if (most > 0x7fffffffLL) return LINFORMER_ERR_SIZE;
    // Units of a few blocks at most stay whole: no workspace, no second kernel, 2.7 us less on the host.  Whole
    // and cut, in a graph, us: one token, 12 heads of 64 of two sequences, 512 rows 7.6 and 9.5, 1000 rows 11.6
    // and 11.1, 1500 rows 15.3 and 12.0; 40 tokens of four, 1000 rows 13.1 and 16.8; 256 tokens of two, 8 groups of
    // heads of 128, 1000 rows 22.4 and 32.8.  One token, 8 groups of heads of 128, where a block takes
    // longer: 512 rows 9.2 and 9.6, 768 rows 12.2 and 10.2, 1000 rows 15.6 and 10.9; of eight sequences 9.5 and
    // 11.4, 12.5 and 12.7, 16.0 and 14.7.
    // Wide units take 10 to 25 us more cut than whole (ends, partial sums, join), so those that fit a CTA each
    // also stay whole where that leaves CTAs idle for no more than eight blocks' time: 1100 tokens of 18 units a
    // head, 8 heads of 128, over 1500 rows 29.9 and 55.6, 3000 rows 50.4 and 73.1; 16 trees of 64 over 32 over 8
    // heads, 2000 rows 39.2 and 60.8, ragged 37.6 and 50.8, 3000 rows ragged 52.8 and 60.2; four of them, 1500 rows 29.1
    // and 24.3.  Of several sequences, one may be long and the others short, which only cut units even out, so
    // then up to 24 blocks.
    const int64_t whole_blocks = call.d > 64 && !wide ? 6 : 8, all = units * call.hk * call.b, sms = device_sms();
    int64_t blocks = ((int64_t)p.width * p.page + kTile - 1) / kTile;  // of a unit at most
    // (rows of `per` tiles of positions and their window, which need not begin with a block: one token, window of
    // 100 in tables of 16000 rows, 32 over 8 heads of 128, 8.2 us by the table and 5.4 so; four tokens of eight
    // sequences, window of 500, 14.2 and 9.3)
    if (p.window) blocks = std::min(blocks, ((int64_t)p.window + p.per * p.qbox + kTile - 2) / kTile + 1);
    // Under a causal mask the units of a prompt's first tokens have fewer blocks than its last, and a CTA idles
    // for `less` blocks on average: cut where that is more than 32 with a head to a unit, 64 with two, whose
    // units cost more cut.  Whole and cut, d = 128, prompts without rows before them: 6 heads of 6400 tokens 87
    // and 85, 8 of 4608 66 and 70, 4 of 9600 129 and 113, 3 of 12800 165 and 131, one of 38000 465 and 312; two on
    // one of 19200 243 and 231, three of 12800 165 and 190, four of 9600 126 and 167.  Windows even units out:
    // two heads of 19200, window of 6000, 83 and 118.
    int64_t less = 0;
    if (call.causal) {
        // the positions before each of which a query sees fewer rows than the last one
        const int64_t rows = (int64_t)p.width * p.page, before = std::max<int64_t>(rows - call.nq, 0);
        const int64_t growing = std::max<int64_t>((p.window ? std::min<int64_t>(p.window, rows) : rows) - before, 0);
        less = growing * growing / (2LL * kTile * call.nq);
    }
    p.whole = blocks <= whole_blocks ||
              (wide && all <= sms && (call.b == 1 || blocks <= 24) && blocks * (sms - all) <= 8 * sms &&
               less <= (p.nch > 1 ? 64 : 32));
    p.direct = p.whole && all <= sms;
    const int seqs = (int)std::min<int64_t>(kMaxSeqs, 0x7fffffffLL / most);
    p.ntiles = (int)ntiles;
    p.units = (int)units;
    int st = LINFORMER_OK;
    for (int b0 = 0; b0 < call.b && !st; b0 += seqs) {
        AttnCall c = call;
        c.b = p.b = std::min(call.b - b0, seqs);
        c.q = static_cast<const __nv_bfloat16 *>(call.q) + b0 * call.sq.b;
        p.out = static_cast<__nv_bfloat16 *>(call.out) + b0 * call.so.b;
        p.lse = call.lse + (int64_t)b0 * call.hq * call.nq;
        p.table = call.cache.table + (int64_t)b0 * call.cache.width;
        p.k_lengths = call.k_lengths + b0;
        p.q_lengths = call.q_lengths ? call.q_lengths + b0 : nullptr;
        p.mask = call.mask ? call.mask + (int64_t)b0 * call.nq * call.words : nullptr;
        p.ctas = (int)(p.direct ? units * call.hk * c.b : std::min<int64_t>(std::min(device_sms(), kJoinThreads), most * c.b));
        if (wide) st = launch_wide(c, p);
        else st = call.d <= 64 ? launch_rows<64>(c, p) : launch_rows<128>(c, p);
    }
    return st;
}

}  // namespace paged
}  // namespace linformer
