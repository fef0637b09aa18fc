// Exact softmax attention of new tokens over a paged cache, with trees of drafted tokens: the
// sums of softmax_attn_fwd.cu over the rows that the table leads to.
#include <cmath>
#include <cuda_bf16.h>

#include "internal.cuh"
#include "paged.cuh"
#include "softmax_attn.cuh"

namespace linformer {
namespace paged {
namespace {

constexpr int kMaxD = 128;

struct AttnParams {
    Cache cache;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    Strides sq, so;
    float *lse;
    const int32_t *q_lengths, *k_lengths;
    const uint64_t *mask;
    int words, b, hq, hk, nq, d, causal, window;
    float scale;
    int *status;
};

// A warp a query row: the running maximum m and sum l of the softmax, and the output so far, a
// lane holding every 32nd element.
__global__ void __launch_bounds__(128) paged_attn_kernel(const AttnParams p) {
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= (int64_t)p.b * p.hq * p.nq) return;
    const int i = (int)(r % p.nq), h = (int)(r / p.nq % p.hq), b = (int)(r / ((int64_t)p.nq * p.hq));
    const int kvh = h / (p.hq / p.hk);
    const int Lq = sattn::clamp_length(p.q_lengths, b, p.nq);
    const int Lk = sattn::clamp_length(p.k_lengths, b, p.cache.width * p.cache.page);
    const sattn::Span sp{Lq, Lk, p.causal, p.window};
    constexpr int E = kMaxD / 32;
    float q[E], o[E] = {};
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int x = lane + 32 * e;
        q[e] = x < p.d && i < Lq ? __bfloat162float(p.q[b * p.sq.b + h * p.sq.h + i * p.sq.n + x]) : 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int end = i < Lq ? sp.end(i) : 0;
    for (int j = i < Lq ? sp.first(i) : 0; j < end; ++j) {
        const int node = j - (Lk - Lq);
        if (p.mask && node >= 0 && !(p.mask[((int64_t)b * p.nq + i) * p.words + node / 64] >> (node % 64) & 1)) continue;
        int page, row;
        const bool there = find_row(p.cache, b, j, p.status, page, row);
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(p.cache.k) + page * p.cache.sk.b +
                                 kvh * p.cache.sk.h + row * p.cache.sk.n;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.cache.v) + page * p.cache.sv.b +
                                 kvh * p.cache.sv.h + row * p.cache.sv.n;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (there && lane + 32 * e < p.d) s += q[e] * __bfloat162float(k[lane + 32 * e]);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale;
        const float mn = fmaxf(m, s), f = expf(m - mn), w = expf(s - mn);
        l = l * f + w;
        m = mn;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * f + (there && lane + 32 * e < p.d ? w * __bfloat162float(v[lane + 32 * e]) : 0.f);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (lane + 32 * e < p.d)
            p.out[b * p.so.b + h * p.so.h + i * p.so.n + lane + 32 * e] = __float2bfloat16_rn(l > 0.f ? o[e] / l : 0.f);
    if (lane == 0) p.lse[r] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

int attention(const AttnCall &c) {
    AttnParams p{};
    p.cache = c.cache;
    p.q = static_cast<const __nv_bfloat16 *>(c.q);
    p.out = static_cast<__nv_bfloat16 *>(c.out);
    p.sq = c.sq;
    p.so = c.so;
    p.lse = c.lse;
    p.q_lengths = c.q_lengths;
    p.k_lengths = c.k_lengths;
    p.mask = c.mask;
    p.words = c.words;
    p.b = c.b, p.hq = c.hq, p.hk = c.hk, p.nq = c.nq, p.d = c.d;
    p.causal = c.causal;
    p.window = c.window;
    p.scale = c.scale;
    p.status = device_status_ptr();
    const int64_t blocks = ((int64_t)c.b * c.hq * c.nq + 3) / 4;
    if (blocks > 0x7fffffffLL) return LINFORMER_ERR_SIZE;
    KernelScope scope(LINFORMER_KERNEL_PAGED, c.stream);
    paged_attn_kernel<<<(unsigned)blocks, 128, 0, c.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? LINFORMER_OK : LINFORMER_ERR_LAUNCH;
}

}  // namespace paged
}  // namespace linformer
