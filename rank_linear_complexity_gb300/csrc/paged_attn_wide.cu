// Attention over pages where a key/value head's new tokens fill more than 64 rows: trees and chunks
// of prompts.  The products are those of softmax_attn_fwd.cu, queries as the 128 rows of a product
// and a thread a row, two tiles of rows to a unit of work, which share the key blocks in shared
// memory; blocks come page by page, and CTAs take equal runs of the list of blocks (paged_attn.cuh).
//
// A block of 128 keys is two steps of 64.  P stands over its own scores, and the other step's scores
// are computed meanwhile; the chain product, softmax, product of one step hides behind the other's and
// the other tile's.  A chunk of 2048 tokens over 2 x 16384, 32 over 8 heads of 128: 697 to 757 us in a graph, 1.36
// to 1.48 PFLOP/s, at the power limit, and 780 by the call; trees of 64 nodes over 16 caches of up to 8192, 94 to
// 95 in a graph.  (In blocks of 128 the next scores wait for the last product: by the call, in earlier states,
// 770 us against 726 so, trees 101 and 99.)  The tensor pipe's arithmetic takes 2048 of the about 3300 cycles
// of a block of two tiles; scores of 64 columns load their query operand twice as often as scores of 128.
// P goes to the tensor cores as one bf16, rounded by at most 2^-8 of each term (error of O 2.3e-3, 1.7e-3 of it
// the result's own rounding): two parts would double the products from P, which bound chunks.  Two threads a row instead of one: 874 us (the scores do not fit in
// the registers of sixteen warps and are read twice).
//   warps 0-3, 4-7  softmax of tile 0 and tile 1: S out of tensor memory, P back
//   warp 8          loads: goes through the CTA's run, tells the others each item, looks the pages up
//                   and issues a box a lane (one thread issuing all: tree, pages of 16, 116 us against 105)
//   warps 9, 10     one thread each issues a tile's S = Q.K^T and O += P.V
//   warp 11         rows without keys: O = 0, lse = -inf
#include <cmath>

#include "paged_attn.cuh"
#include "softmax_rows.cuh"

namespace linformer {
namespace paged {
namespace {

constexpr int kThreads = 384, kLoadWarp = 8, kMmaWarp = 9, kEmptyWarp = 11;
constexpr int kStep = kTile / 2;  // keys of a step
// Tensor memory: of each tile S of two steps (64 columns each), P over its own S, then O.
template <int DP>
struct Layout {
    static constexpr int kStages = DP == 64 ? 8 : 4;
    static constexpr uint32_t kTileBytes = kTile * DP * 2;
    static constexpr uint32_t kO = 256;
    static constexpr uint32_t kEnd = (2 + kStages) * kTileBytes;
};

constexpr int kAhead = 4;        // items told ahead
constexpr int kReaders = 2 + 8;  // issuing threads, softmax warps

struct Shared {
    uint64_t full[8], empty[8], q_full[2], q_free[2], s_full[2][2], p_full[2][2], pv_done[2][2], o_free[2],
        drain[2], told[kAhead], taken[kAhead];
    struct Told : Item {
        int before;  // blocks of the items before it
    } items[kAhead];  // (in shared memory: the softmax has no registers to spare for a walk)
    uint32_t tmem;
    int abort;
    Marks marks;
};

// A tile's part of an item.
struct Part {
    int q0, h0, lo, hi;
    bool live;
    __device__ __forceinline__ Part(const AttnParams &p, const Item &it, int t) {
        const int tile = 2 * it.unit + t;
        live = tile < p.ntiles;
        const Rows r(p, tile);
        q0 = r.q0;
        h0 = r.h0;
        lo = hi = 0;
        if (live) blocks_of(p, it.sp, q0, lo, hi);
        lo = max(lo, it.lo);
        hi = max(lo, min(hi, it.hi));
    }
};

// Which of 64 nodes from `node` on (below 0: rows before the tree) a row's mask leaves.
__device__ __forceinline__ uint64_t nodes_seen(const uint64_t *mask, int words, int node) {
    auto word = [&](int w) { return w < 0 ? ~0ull : w < words ? __ldg(mask + w) : 0ull; };
    const int w = node >> 6, off = node & 63;
    return word(w) >> off | (off ? word(w + 1) << (64 - off) : 0ull);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
paged_wide_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                  const __grid_constant__ CUtensorMap tV, const __grid_constant__ AttnParams p) {
    using L = Layout<DP>;
    // (addresses in it are constants then, and take no registers)
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        leave(p, 157);
        return;
    }
    uint8_t *sQ = smem, *sKV = smem + 2 * L::kTileBytes;
    Shared *sh = reinterpret_cast<Shared *>(smem + L::kEnd);
    volatile int *abort_flag = &sh->abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 32) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh->q_full[t], 1);
            mbar_init(&sh->q_free[t], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sh->s_full[t][h], 1);
                mbar_init(&sh->p_full[t][h], 4);
                mbar_init(&sh->pv_done[t][h], 1);
            }
            mbar_init(&sh->o_free[t], 4);
            mbar_init(&sh->drain[t], 1);
        }
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 2);  // one arrival from each tile's products
        }
        for (int s = 0; s < kAhead; ++s) {
            mbar_init(&sh->told[s], 1);
            mbar_init(&sh->taken[s], kReaders);
        }
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
    tc_fence_before();
    wait_prerequisites();
    if (tid == 0) launch_dependents();  // the join, which waits for this grid's end
    const Walk own = p.direct ? Walk(p) : Walk();
    if (!p.direct) fill(p, sh->marks, tid, kThreads);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;

    if (warp >= kLoadWarp) {
        if (warp == kLoadWarp) {  // ---------------- loads
            // a lane's box of a tile: `box` rows of a page, 64 columns
            const int bi = lane / (DP / 64), half = lane % (DP / 64);
            const bool mine = bi < p.nbox;
            const int row = bi * p.box;
            const uint32_t dst = half * 16384u + row * 128u;
            int ring = 0, nq[2] = {0, 0};
            bool ok = true;
            auto spin = [&](uint64_t *bar, uint32_t parity, int code) {
                return warp_spin(bar, parity, p.status, code, abort_flag);
            };
            Walk walk = p.direct ? own : Walk(p, sh->marks, blockIdx.x);
            const Walk begin = walk;
            Shared::Told it;
            it.before = 0;
            for (int k = 0; ok; ++k) {
                const int slot = k % kAhead;
                const bool more = walk.next(p, sh->marks, it);
                const int low = more ? it.sp.first(Rows(p, 2 * it.unit).q0) : 0;
                int page = more && mine ? page_of(p, p.table + (int64_t)it.seq * p.width, it.lo, row, low, it.sp.Lk) : 0;
                if (!more) it.seq = -1;
                ok = k < kAhead || spin(&sh->taken[slot], (k / kAhead - 1) & 1, 153);
                if (!ok) break;
                if (lane == 0) {
                    sh->items[slot] = it;
                    mbar_arrive(&sh->told[slot]);
                    if (!more && k == 0) write_cut(p, begin, sh->marks);
                }
                __syncwarp();
                if (!more) break;
                // The first item's Q before its keys, the others' after their first block's: the last
                // item's scores may still need theirs, and the keys are not to wait for that.
                auto load_q = [&] {
                    for (int t = 0; t < 2 && ok; ++t) {
                        const Part x(p, it, t);
                        if (x.hi <= x.lo) continue;
                        ok = nq[t] == 0 || spin(&sh->q_free[t], (nq[t] - 1) & 1, 140);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&sh->q_full[t], (uint32_t)(p.qbox * p.hbox * DP * 2));
                            for (int h = 0; h < DP / 64; ++h)
                                tma_load_5d(sQ + t * L::kTileBytes + h * 16384, &tQ, &sh->q_full[t], h * 64, x.q0, x.h0,
                                            it.kvh, it.seq);
                        }
                        ++nq[t];
                    }
                };
                const int32_t *table = p.table + (int64_t)it.seq * p.width;
                const int lo = it.lo, hi = it.hi, kvh = it.kvh, Lk = it.sp.Lk;
                if (k == 0) load_q();
                for (int j = lo; j < hi && ok; ++j) {
                    const int now = page, at = (j * kTile + row) & (p.page - 1);
                    if (j + 1 < hi && mine) page = page_of(p, table, j + 1, row, low, Lk);
                    for (int kv = 0; kv < 2 && ok; ++kv, ++ring) {
                        const int s = ring % L::kStages;
                        if (ring >= L::kStages) ok = spin(&sh->empty[s], (ring / L::kStages - 1) & 1, 141);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&sh->full[s], L::kTileBytes);
                        __syncwarp();
                        if (mine)
                            tma_load_5d(sKV + s * L::kTileBytes + dst, kv ? &tV : &tK, &sh->full[s], half * 64, at, 0,
                                        kvh, now);
                    }
                    if (ok && j == lo && k > 0) load_q();
                }
                if (k == 0 && lane == 0) write_cut(p, begin, sh->marks);
                it.before += hi - lo;
            }
            // no copy outlives the CTA
            if (lane == 0) {
                for (int t = 0; t < 2; ++t)
                    if (nq[t] > 0) mbar_wait_drain(&sh->q_full[t], (nq[t] - 1) & 1);
                for (int i = max(0, ring - L::kStages); i < ring; ++i)
                    mbar_wait_drain(&sh->full[i % L::kStages], (i / L::kStages) & 1);
            }
            __syncwarp();
        } else if (warp == kEmptyWarp) {
            write_empty(p, sh->marks, p.direct ? &own : nullptr, 0, 1, lane);
        } else if (elect_one()) {  // ---------------- products of tile t
            const int t = warp - kMmaWarp;
            const uint32_t idesc_s = idesc_f16(128, kStep, 1, 0, 0), idesc_o = idesc_f16(128, DP, 1, 0, 1);
            const uint64_t dq = sdesc(smem_u32(sQ + t * L::kTileBytes), 16, 1024, kSwizzle128B);
            const uint32_t tS = tmem + 128 * t, tO = tmem + L::kO + DP * t;
            // the next K and the next V of the ring, whose entries come in pairs
            constexpr int kPairs = L::kStages / 2;
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
                           dv0 = sdesc(smem_u32(sKV) + L::kTileBytes, 16384, 1024, kSwizzle128B);
            int nb = 0, mb = 0, items = 0;  // the tile's blocks with S, with O, and its items
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int slot = k % kAhead;
                if (!thread_spin(&sh->told[slot], (k / kAhead) & 1, p.status, 154, abort_flag)) break;
                const Item it = sh->items[slot];
                mbar_arrive(&sh->taken[slot]);
                if (it.seq < 0) break;
                const Part x(p, it, t);
                const int lo = x.lo, hi = x.hi;
                // S of half h of block j, once the last product from that half's P is done
                auto score = [&](int j, int h) {
                    if (h == 0 && !thread_spin(&sh->full[2 * ak.s], ak.parity, p.status, 142, abort_flag)) return false;
                    if (h == 0 && j == lo && !thread_spin(&sh->q_full[t], items & 1, p.status, 143, abort_flag)) return false;
                    if (nb > 0 && !thread_spin(&sh->pv_done[t][h], (nb - 1) & 1, p.status, 144, abort_flag)) return false;
                    tc_fence_after();
                    const uint64_t key = dk0 + (uint64_t)(ak.s * (int)(2 * L::kTileBytes >> 4) + h * (kStep * 128 >> 4));
#pragma unroll
                    for (int y = 0; y < DP / 16; ++y) {
                        const uint64_t off = (uint64_t)((y >> 2) * 1024 + (y & 3) * 2);
                        mma_ss(tS + kStep * h, dq + off, key + off, idesc_s, y > 0 ? 1u : 0u);
                    }
                    mma_commit(&sh->s_full[t][h]);
                    if (h == 1) {
                        mma_commit(&sh->empty[2 * ak.s]);
                        if (j == hi - 1) mma_commit(&sh->q_free[t]);
                        ak.next();
                        ++nb;
                    }
                    return true;
                };
                // O += P.V of half h of block j
                auto output = [&](int j, int h) {
                    if (h == 0 && !thread_spin(&sh->full[2 * av.s + 1], av.parity, p.status, 145, abort_flag)) return false;
                    if (!thread_spin(&sh->p_full[t][h], mb & 1, p.status, 146, abort_flag)) return false;
                    if (h == 0 && j == lo && items > 0 &&
                        !thread_spin(&sh->o_free[t], (items - 1) & 1, p.status, 147, abort_flag))
                        return false;
                    tc_fence_after();
                    const uint64_t v = dv0 + (uint64_t)(av.s * (int)(2 * L::kTileBytes >> 4) + h * (kStep * 128 >> 4));
#pragma unroll
                    for (int y = 0; y < kStep / 16; ++y)
                        mma_ts(tO, tS + kStep * h + 8 * y, v + (uint64_t)(128 * y), idesc_o, (j > lo || h > 0 || y > 0) ? 1u : 0u);
                    mma_commit(&sh->pv_done[t][h]);
                    if (h == 1) {
                        mma_commit(&sh->empty[2 * av.s + 1]);
                        av.next();
                        ++mb;
                    }
                    return true;
                };
                // blocks that only the other tile sees
                auto skip = [&](int from, int to) {
                    for (int j = from; j < to; ++j) {
                        if (!thread_spin(&sh->full[2 * ak.s], ak.parity, p.status, 148, abort_flag)) return false;
                        mbar_arrive(&sh->empty[2 * ak.s]);
                        ak.next();
                        if (!thread_spin(&sh->full[2 * av.s + 1], av.parity, p.status, 158, abort_flag)) return false;
                        mbar_arrive(&sh->empty[2 * av.s + 1]);
                        av.next();
                    }
                    return true;
                };
                if (hi <= lo) {
                    ok = skip(it.lo, it.hi);
                    continue;
                }
                ok = skip(it.lo, lo) && score(lo, 0);
                for (int j = lo; j < hi && ok; ++j)
                    ok = score(j, 1) && output(j, 0) && (j + 1 >= hi || score(j + 1, 0)) && output(j, 1);
                ok = ok && skip(hi, it.hi);
                ++items;
            }
            mma_commit(&sh->drain[t]);
            mbar_wait_drain(&sh->drain[t], 0);
        }
        __syncwarp();
    } else {
        // ---------------- softmax of one tile, one thread a row
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + 128 * t + lanes, tO = tmem + L::kO + DP * t + lanes;
        const float sl = p.scale_log2;
        // The row's position and head within the tile, worked out where they are needed (kept through the
        // loop they would cost registers there).
        auto place = [&](int &qi, int &head) {
            int r = row;
            asm volatile("" : "+r"(r));
            qi = r & (p.qbox - 1);
            head = r / p.qbox;
        };
        int n = 0;  // the tile's steps: two a block
        bool ok = true;
        // the product of the step before this one is done, and with it all of O so far
        auto last_product = [&](int code) {
            ok = warp_spin(&sh->pv_done[t][(n - 1) & 1], ((n - 1) >> 1) & 1, p.status, code, abort_flag);
            tc_fence_after();
            return ok;
        };
        for (int k = 0;; ++k) {
            if (!warp_spin(&sh->told[k % kAhead], (k / kAhead) & 1, p.status, 155, abort_flag)) break;
            const auto &it = sh->items[k % kAhead];
            if (it.seq < 0) break;
            // [clean_lo, clean_hi): blocks that every row of the tile sees all of
            int xlo, xhi, clean_lo, clean_hi;
            bool valid, warp_valid;
            {
                const Part x(p, it, t);
                int qi, head;
                place(qi, head);
                const int i = x.q0 + qi;
                xlo = x.lo;
                xhi = x.hi;
                valid = x.live && head < p.hbox && x.h0 + head < p.group && i < it.sp.Lq;
                warp_valid = __any_sync(0xffffffffu, valid);
                const int end = min(it.sp.end(x.q0), p.mask ? it.sp.Lk - it.sp.Lq : it.sp.Lk);
                clean_hi = max(end, 0) / kTile;
                clean_lo = (it.sp.first(max(min(x.q0 + p.qbox, it.sp.Lq) - 1, 0)) + kTile - 1) / kTile;
            }
            // reference (of the raw scores; one that no score outgrows where there is no query, so that what
            // stands there has no vote on when the references move), sum of 2^((s - m) sl)
            float m = valid ? -INFINITY : INFINITY, l = 0.f;
            for (int u = 2 * xlo; u < 2 * xhi; ++u, ++n) {
                const int j = u >> 1, h = u & 1;
                if (!warp_spin(&sh->s_full[t][h], (n >> 1) & 1, p.status, 150, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool clean = j >= clean_lo && j < clean_hi;
                if (!clean && h == 0 && (j + 1) * kTile > it.sp.Lk) {
                    // rows of V past the length may hold anything: P is 0 there, but 0 x NaN is not
                    // (both tiles' threads write the zeros; a product that reads them by then needs
                    // no others)
                    const int v = 2 * (it.before + j - it.lo) + 1, s = v % L::kStages;
                    if (!warp_spin(&sh->full[s], (v / L::kStages) & 1, p.status, 151, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (j * kTile + row >= it.sp.Lk) {
                        uint8_t *at = sKV + s * L::kTileBytes + row * 128;
#pragma unroll 1
                        for (int y = 0; y < DP / 8; ++y)
                            *reinterpret_cast<uint4 *>(at + (y / 8) * 16384 + (y % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (warp_valid) {
                    uint32_t va[32], vb[32];
                    tmem_ld32_async(tS + kStep * h, va);
                    tmem_ld32_async(tS + kStep * h + 32, vb);
                    tmem_wait_ld(va);
                    tie32(vb);
                    if (!clean) {
                        const Part x(p, it, t);
                        int qi, head;
                        place(qi, head);
                        const int k0 = u * kStep, i = x.q0 + qi;
                        if (head < p.hbox && x.h0 + head < p.group && i < it.sp.Lq) {
                            const int a = it.sp.first(i) - k0, z = it.sp.end(i) - k0;
                            uint64_t see = a <= 0 ? ~0ull : a < 64 ? ~0ull << a : 0ull;
                            if (z < 64) see &= z > 0 ? ~(~0ull << z) : 0ull;
                            if (p.mask)
                                see &= nodes_seen(p.mask + ((int64_t)it.seq * p.nq + i) * p.words, p.words,
                                                  k0 - (it.sp.Lk - it.sp.Lq));
                            const uint32_t sa = (uint32_t)see, sb = (uint32_t)(see >> 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {  // (whatever they hold)
                                if (!(sa >> e & 1)) va[e] = 0xff800000u;
                                if (!(sb >> e & 1)) vb[e] = 0xff800000u;
                            }
                        }
                    }
                    const float mx = fmaxf(sattn::max_chunk(va), sattn::max_chunk(vb));
                    if (__any_sync(0xffffffffu, (mx - m) * sl > kOutgrown)) {
                        const bool any = u > 2 * xlo;
                        if (any && !last_product(149)) break;
                        const float mn = fmaxf(m, mx);
                        const float f = mn == -INFINITY ? 1.f : ex2_approx((m - mn) * sl);
                        l *= f;
                        m = mn;
                        if (any) sattn::rescale_output(tO, DP, f);
                    }
                    const float off = m == -INFINITY ? 0.f : -m * sl;
                    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                    uint32_t o[16];
                    sattn::exp_chunk(va, o, sl, off, sum0, sum1);
                    tmem_st16_async(tS + kStep * h, o);
                    sattn::exp_chunk(vb, o, sl, off, sum0, sum1);
                    tmem_st16_async(tS + kStep * h + 16, o);
                    tmem_wait_st();
                    l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[t][h]);
            }
            if (!ok) break;
            // O / l out of tensor memory; rows without keys give O = 0 and lse = -inf
            const Part x(p, it, t);
            int qi, head;
            place(qi, head);
            const int i = x.q0 + qi, hg = x.h0 + head;
            const bool exists = x.live && head < p.hbox && hg < p.group && i < p.nq;
            const bool dead = !exists || i >= it.sp.Lq || l == 0.f, some = xhi > xlo, whole = it.slot < 0;
            const float inv = dead ? 0.f : 1.f / l;
            const int64_t h = (int64_t)it.kvh * p.group + hg, pr = ((int64_t)it.slot * 2 + t) * kTile + row;
            __nv_bfloat16 *dst = p.out + it.seq * p.so.b + h * p.so.h + (int64_t)i * p.so.n;
            if (some) {
                if (!last_product(152)) break;
#pragma unroll 1
                for (int c = 0; c < DP && warp_valid; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(dead ? 0.f : __uint_as_float(o[e]) * inv);
                    if (!whole) {
                        if (dead) continue;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            const uint32_t w[8] = {o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7]};
                            sattn::store32(p.part_o + pr * DP + c + e, w);
                        }
                    } else if (exists) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            if (c + e >= p.d) continue;
                            uint32_t w[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                w[y] = pack2(__uint_as_float(o[e + 2 * y]), __uint_as_float(o[e + 2 * y + 1]));
                            if (p.wide_stores) {
                                sattn::store32(dst + c + e, w);
                            } else {
                                *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                                if (c + e + 8 < p.d)
                                    *reinterpret_cast<uint4 *>(dst + c + e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->o_free[t]);
            }
            if (whole && exists && !(some && warp_valid))
#pragma unroll 1
                for (int c = 0; c < p.d; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
            const float lse = dead ? -INFINITY : m * p.scale + logf(l);
            if (!whole) p.part_lse[pr] = lse;
            else if (exists) p.lse[((int64_t)it.seq * p.hq + h) * p.nq + i] = lse;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->taken[k % kAhead]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int DP>
int launch(const AttnCall &c, AttnParams &p) {
    constexpr uint32_t kSmem = Layout<DP>::kEnd + sizeof(Shared);
    static_assert(kSmem <= 227 * 1024, "shared memory");
    p.N = kTile;
    return launch_with_join(paged_wide_kernel<DP>, kThreads, kSmem, DP == 64 ? 16 : 17, c, p, DP);
}

}  // namespace

int launch_wide(const AttnCall &c, AttnParams &p) { return c.d <= 64 ? launch<64>(c, p) : launch<128>(c, p); }

}  // namespace paged
}  // namespace linformer
