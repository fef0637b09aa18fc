// Entry points of the exact softmax attention and the rotary positions: argument checks
// (all on the host, before anything is launched) and the tensors' strides.
#include <cmath>

#include "internal.cuh"
#include "rotary.cuh"
#include "softmax_attn.cuh"

namespace linformer {
namespace {

// The strides as given, or dense [b][heads][n][d].
Strides strides_of(const int64_t *s, int heads, int n, int d) {
    if (s) return Strides{s[0], s[1], s[2]};
    return Strides{(int64_t)heads * n * d, (int64_t)n * d, d};
}

// A dimension of more than one entry has a positive stride (bounded so that no offset
// overflows) that keeps 16-byte pieces aligned; rows of an output do not overlap.
int check_strides(const Strides &s, int b, int heads, int n, int d, int multiple, bool output) {
    const int64_t limit = 1LL << 38;
    const int64_t st[3] = {s.b, s.h, s.n};
    const int count[3] = {b, heads, n};
    for (int i = 0; i < 3; ++i) {
        if (count[i] <= 1) continue;
        if (st[i] < 1 || st[i] > limit) return LINFORMER_ERR_VALUE;
        if (output && st[i] < d) return LINFORMER_ERR_VALUE;
        if (st[i] % multiple) return LINFORMER_ERR_ALIGN;
    }
    return LINFORMER_OK;
}

struct View {
    const void *p;
    const int64_t *strides;
    int heads, n;
    bool output;
    Strides *to;
};

int check_attention(int b, int hq, int hk, int nq, int nk, int d, float scale, int causal, int window,
                    int dtype, const float *lse, const int32_t *q_lengths, const int32_t *k_lengths,
                    const View *views, int count) {
    if (!lse) return LINFORMER_ERR_NULL;
    for (int i = 0; i < count; ++i)
        if (!views[i].p) return LINFORMER_ERR_NULL;
    if (b < 1 || hq < 1 || hk < 1 || nq < 1 || nk < 1 || d < 1 || hq % hk) return LINFORMER_ERR_SIZE;
    if (nq > (1 << 29) || nk > (1 << 29) || (int64_t)b * hq > (1 << 29)) return LINFORMER_ERR_SIZE;
    if (dtype < LINFORMER_F32 || dtype > LINFORMER_BF16_F32OUT) return LINFORMER_ERR_ENUM;
    if (dtype != LINFORMER_BF16 || d > 128 || d % 8) return LINFORMER_ERR_UNSUPPORTED;
    // (the scale is multiplied by log2(e) for the exponentials)
    if (!std::isfinite(scale * 1.5f) || scale <= 0.f || window < 0 || (window && !causal) || causal < 0 ||
        causal > 1)
        return LINFORMER_ERR_VALUE;
    const void *words[] = {lse, q_lengths, k_lengths};
    for (const void *p : words)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return LINFORMER_ERR_ALIGN;
    for (int i = 0; i < count; ++i) {
        const View &v = views[i];
        if (!aligned16(v.p)) return LINFORMER_ERR_ALIGN;
        *v.to = strides_of(v.strides, v.heads, v.n, d);
        const int st = check_strides(*v.to, b, v.heads, v.n, d, 8, v.output);
        if (st) return st;
    }
    // an output that starts where another tensor does overlaps it
    for (int i = 0; i < count; ++i)
        for (int k = 0; views[i].output && k < count; ++k)
            if (k != i && views[k].p == views[i].p) return LINFORMER_ERR_VALUE;
    return LINFORMER_OK;
}

}  // namespace
}  // namespace linformer

using namespace linformer;

extern "C" int linformer_softmax_attn_fwd(
    const void *Q, const int64_t *Q_strides, const void *K, const int64_t *K_strides, const void *V,
    const int64_t *V_strides, void *O, const int64_t *O_strides, float *lse, const int32_t *q_lengths,
    const int32_t *k_lengths, int b, int hq, int hk, int nq, int nk, int d, float scale, int causal,
    int window, int dtype, void *stream) {
    sattn::Call c{};
    const View views[] = {{Q, Q_strides, hq, nq, false, &c.sQ},
                          {K, K_strides, hk, nk, false, &c.sK},
                          {V, V_strides, hk, nk, false, &c.sV},
                          {O, O_strides, hq, nq, true, &c.sO}};
    const int st = check_attention(b, hq, hk, nq, nk, d, scale, causal, window, dtype, lse, q_lengths,
                                   k_lengths, views, 4);
    if (st) return st;
    c.Q = Q;
    c.K = K;
    c.V = V;
    c.out = O;
    c.lse = lse;
    c.q_lengths = q_lengths;
    c.k_lengths = k_lengths;
    c.b = b, c.hq = hq, c.hk = hk, c.nq = nq, c.nk = nk, c.d = d;
    c.causal = causal;
    c.window = window >= nk ? 0 : window;  // no query looks further back than nk keys
    c.scale = scale;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return sattn::forward(c);
}

extern "C" int linformer_softmax_attn_bwd(
    const void *Q, const int64_t *Q_strides, const void *K, const int64_t *K_strides, const void *V,
    const int64_t *V_strides, const void *O, const int64_t *O_strides, const void *dO,
    const int64_t *dO_strides, const float *lse, void *dQ, const int64_t *dQ_strides, void *dK,
    const int64_t *dK_strides, void *dV, const int64_t *dV_strides, const int32_t *q_lengths,
    const int32_t *k_lengths, int b, int hq, int hk, int nq, int nk, int d, float scale, int causal,
    int window, int dtype, void *stream) {
    sattn::Call c{};
    const View views[] = {{Q, Q_strides, hq, nq, false, &c.sQ},
                          {K, K_strides, hk, nk, false, &c.sK},
                          {V, V_strides, hk, nk, false, &c.sV},
                          {O, O_strides, hq, nq, false, &c.sO},
                          {dO, dO_strides, hq, nq, false, &c.sdO},
                          {dQ, dQ_strides, hq, nq, true, &c.sdQ},
                          {dK, dK_strides, hk, nk, true, &c.sdK},
                          {dV, dV_strides, hk, nk, true, &c.sdV}};
    const int st = check_attention(b, hq, hk, nq, nk, d, scale, causal, window, dtype, lse, q_lengths,
                                   k_lengths, views, 8);
    if (st) return st;
    c.Q = Q;
    c.K = K;
    c.V = V;
    c.O = O;
    c.dO = dO;
    c.dQ = dQ;
    c.dK = dK;
    c.dV = dV;
    c.lse = const_cast<float *>(lse);
    c.q_lengths = q_lengths;
    c.k_lengths = k_lengths;
    c.b = b, c.hq = hq, c.hk = hk, c.nq = nq, c.nk = nk, c.d = d;
    c.causal = causal;
    c.window = window >= nk ? 0 : window;
    c.scale = scale;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return sattn::backward(c);
}

extern "C" int linformer_rotary(const void *X, const int64_t *X_strides, void *Y, const int64_t *Y_strides,
                                int hx, const void *X2, const int64_t *X2_strides, void *Y2,
                                const int64_t *Y2_strides, int hx2, const uint64_t *phase,
                                const int32_t *positions, int start, int b, int n, int d, int rot,
                                int layout, float amplitude, int inverse, int dtype, void *stream) {
    if (!X || !Y || !phase || (hx2 > 0 && (!X2 || !Y2))) return LINFORMER_ERR_NULL;
    if (b < 1 || hx < 1 || hx2 < 0 || n < 1 || d < 1) return LINFORMER_ERR_SIZE;
    if ((int64_t)b * ((int64_t)hx + hx2) > (1 << 29) || (int64_t)b * n > (1LL << 33) || d > (1 << 20) ||
        hx > (1 << 20) || hx2 > (1 << 20))
        return LINFORMER_ERR_SIZE;
    if (layout < LINFORMER_ROTARY_HALVES || layout > LINFORMER_ROTARY_INTERLEAVED) return LINFORMER_ERR_ENUM;
    if (dtype != LINFORMER_F32 && dtype != LINFORMER_BF16)
        return dtype == LINFORMER_BF16_F32OUT ? LINFORMER_ERR_UNSUPPORTED : LINFORMER_ERR_ENUM;
    if (rot < 2 || rot > d || rot % 2 || !std::isfinite(amplitude) || inverse < 0 || inverse > 1 ||
        (int64_t)start + n > (1LL << 31))
        return LINFORMER_ERR_VALUE;
    rotary::Call c{};
    const void *xs[] = {X, hx2 ? X2 : nullptr};
    void *ys[] = {Y, hx2 ? Y2 : nullptr};
    const int64_t *sx[] = {X_strides, X2_strides}, *sy[] = {Y_strides, Y2_strides};
    const int heads[] = {hx, hx2};
    if ((reinterpret_cast<uintptr_t>(phase) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
        return LINFORMER_ERR_ALIGN;
    for (int w = 0; w < 2; ++w) {
        c.x[w] = xs[w];
        c.y[w] = ys[w];
        c.heads[w] = heads[w];
        if (!heads[w]) continue;
        if (!aligned16(xs[w]) || !aligned16(ys[w])) return LINFORMER_ERR_ALIGN;
        c.sx[w] = strides_of(sx[w], heads[w], n, d);
        c.sy[w] = strides_of(sy[w], heads[w], n, d);
        int st = check_strides(c.sx[w], b, heads[w], n, d, 1, false);
        if (!st) st = check_strides(c.sy[w], b, heads[w], n, d, 1, true);
        if (st) return st;
        // in place means the same elements in the same places
        if (xs[w] == ys[w] && ((b > 1 && c.sx[w].b != c.sy[w].b) || (heads[w] > 1 && c.sx[w].h != c.sy[w].h) ||
                               (n > 1 && c.sx[w].n != c.sy[w].n)))
            return LINFORMER_ERR_VALUE;
    }
    if (hx2 && (Y == Y2 || Y == X2 || Y2 == X)) return LINFORMER_ERR_VALUE;  // overlapping outputs
    c.phase = phase;
    c.positions = positions;
    c.start = start;
    c.b = b, c.n = n, c.d = d, c.rot = rot;
    c.interleaved = layout == LINFORMER_ROTARY_INTERLEAVED;
    c.inverse = inverse;
    c.dtype = dtype;
    c.amplitude = amplitude;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return rotary::turn(c);
}

extern "C" int linformer_rotary_phase(uint64_t *phase, int rot, double base, int scaling, double factor,
                                      int original_length, double beta_fast, double beta_slow,
                                      void *stream) {
    if (!phase) return LINFORMER_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(phase) & 7u) return LINFORMER_ERR_ALIGN;
    if (scaling < LINFORMER_ROTARY_PLAIN || scaling > LINFORMER_ROTARY_BY_PARTS) return LINFORMER_ERR_ENUM;
    if (rot < 2 || rot % 2 || rot > (1 << 20)) return LINFORMER_ERR_SIZE;
    if (!std::isfinite(base) || base <= 0 || !std::isfinite(factor) || factor <= 0) return LINFORMER_ERR_VALUE;
    if (scaling == LINFORMER_ROTARY_BY_PARTS &&
        (original_length < 1 || !std::isfinite(beta_fast) || !std::isfinite(beta_slow) ||
         beta_fast <= beta_slow))
        return LINFORMER_ERR_VALUE;
    return rotary::phase_table(phase, rot, base, scaling, factor, original_length, beta_fast, beta_slow,
                               reinterpret_cast<cudaStream_t>(stream));
}
