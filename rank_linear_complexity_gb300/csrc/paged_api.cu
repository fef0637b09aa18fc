// Entry points of the paged key/value cache: argument checks, all on the host, before anything
// is launched.
#include <cmath>
#include <cstring>

#include "internal.cuh"
#include "paged.cuh"
#include "strided.cuh"

namespace linformer {
namespace {

constexpr int kMinPage = 8, kMaxPage = 1 << 16;
constexpr int kMaxRows = 1 << 29;  // of one sequence's table

bool unaligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// `multiple`: of the strides, in elements.
int check_cache(paged::Cache &c, const void *K, const int64_t *sk, const void *V, const int64_t *sv,
                const int32_t *table, int b, int hk, int d, int pages, int page, int width, int multiple) {
    if (!K || !V || !table) return LINFORMER_ERR_NULL;
    if (b < 1 || hk < 1 || d < 1 || pages < 1 || width < 1) return LINFORMER_ERR_SIZE;
    if (page < kMinPage || page > kMaxPage || (page & (page - 1)) || (int64_t)width * page > kMaxRows)
        return LINFORMER_ERR_SIZE;
    if (!aligned16(K) || !aligned16(V) || unaligned(table, 4)) return LINFORMER_ERR_ALIGN;
    if (K == V) return LINFORMER_ERR_VALUE;
    c.k = const_cast<void *>(K);
    c.v = const_cast<void *>(V);
    c.sk = strides_of(sk, hk, page, d);
    c.sv = strides_of(sv, hk, page, d);
    c.table = table;
    c.pages = pages;
    c.page = page;
    c.width = width;
    for (c.shift = 0; (1 << c.shift) < page;) ++c.shift;
    const int st = check_strides(c.sk, pages, hk, page, d, multiple, true);
    return st ? st : check_strides(c.sv, pages, hk, page, d, multiple, true);
}

int check_attention(paged::AttnCall &c, const void *Q, const int64_t *Q_strides, const void *K,
                    const int64_t *K_strides, const void *V, const int64_t *V_strides, void *O,
                    const int64_t *O_strides, float *lse, const int32_t *table, const int32_t *k_lengths,
                    const int32_t *q_lengths, int b, int hq, int hk, int nq, int d, int pages, int page, int width,
                    float scale, int dtype) {
    if (!Q || !O || !lse || !k_lengths || !K || !V || !table) return LINFORMER_ERR_NULL;
    if (b < 1 || hq < 1 || hk < 1 || nq < 1 || d < 1 || hq % hk) return LINFORMER_ERR_SIZE;
    if (nq > kMaxRows || (int64_t)b * hq > (1 << 29)) return LINFORMER_ERR_SIZE;
    if (dtype < LINFORMER_F32 || dtype > LINFORMER_BF16_F32OUT) return LINFORMER_ERR_ENUM;
    if (dtype != LINFORMER_BF16 || d > 128 || d % 8) return LINFORMER_ERR_UNSUPPORTED;
    // (the scale is multiplied by log2(e) for the exponentials)
    if (!std::isfinite(scale * 1.5f) || scale <= 0.f) return LINFORMER_ERR_VALUE;
    if (unaligned(lse, 4) || unaligned(k_lengths, 4) || unaligned(q_lengths, 4) || !aligned16(Q) || !aligned16(O))
        return LINFORMER_ERR_ALIGN;
    int st = check_cache(c.cache, K, K_strides, V, V_strides, table, b, hk, d, pages, page, width, 8);
    if (st) return st;
    c.sq = strides_of(Q_strides, hq, nq, d);
    c.so = strides_of(O_strides, hq, nq, d);
    st = check_strides(c.sq, b, hq, nq, d, 8, false);
    if (!st) st = check_strides(c.so, b, hq, nq, d, 8, true);
    if (st) return st;
    if (O == Q || O == K || O == V) return LINFORMER_ERR_VALUE;
    c.q = Q;
    c.out = O;
    c.lse = lse;
    c.q_lengths = q_lengths;
    c.k_lengths = k_lengths;
    c.b = b, c.hq = hq, c.hk = hk, c.nq = nq, c.d = d;
    c.scale = scale;
    return LINFORMER_OK;
}

// A block of arguments, one after the other.
struct Words {
    int64_t w[64];
    int at = 0;
    bool fits = true;  // every integer so far fits an int

    template <typename T>
    T *pointer() { return reinterpret_cast<T *>((uintptr_t)w[at++]); }
    const int64_t *strides() { return w + (at += 3) - 3; }
    int integer() {
        const int64_t x = w[at++];
        fits = fits && x >= INT32_MIN && x <= INT32_MAX;
        return (int)x;
    }
    float real() {
        double x;
        std::memcpy(&x, w + at++, sizeof x);
        return (float)x;
    }
};

}  // namespace
}  // namespace linformer

using namespace linformer;

extern "C" int linformer_cache_append(const void *K, const int64_t *K_strides, const void *V,
                                      const int64_t *V_strides, void *K_pages, const int64_t *K_pages_strides,
                                      void *V_pages, const int64_t *V_pages_strides, const void *Q,
                                      const int64_t *Q_strides, void *Y, const int64_t *Y_strides,
                                      const int32_t *table, const int32_t *starts, const int32_t *counts,
                                      const uint64_t *phase, const int32_t *positions, int b, int hq, int hk,
                                      int n, int d, int pages, int page, int width, int rot, int layout,
                                      float amplitude, int dtype, void *stream) {
    if (!K || !V || !K_pages || !V_pages || !table || !starts || (hq > 0 && (!Q || !Y || !phase)))
        return LINFORMER_ERR_NULL;
    if (b < 1 || hq < 0 || hk < 1 || n < 1 || d < 1) return LINFORMER_ERR_SIZE;
    if ((int64_t)b * ((int64_t)hq + 2LL * hk) > (1 << 29) || (int64_t)b * n > (1LL << 33) || n > kMaxRows ||
        d > (1 << 20) || hq > (1 << 20) || hk > (1 << 20))
        return LINFORMER_ERR_SIZE;
    if (layout < LINFORMER_ROTARY_HALVES || layout > LINFORMER_ROTARY_INTERLEAVED) return LINFORMER_ERR_ENUM;
    if (dtype != LINFORMER_F32 && dtype != LINFORMER_BF16)
        return dtype == LINFORMER_BF16_F32OUT ? LINFORMER_ERR_UNSUPPORTED : LINFORMER_ERR_ENUM;
    if (phase && (rot < 2 || rot > d || rot % 2 || !std::isfinite(amplitude))) return LINFORMER_ERR_VALUE;
    if (unaligned(phase, 8) || unaligned(positions, 4) || unaligned(starts, 4) || unaligned(counts, 4))
        return LINFORMER_ERR_ALIGN;
    paged::AppendCall c{};
    int st = check_cache(c.cache, K_pages, K_pages_strides, V_pages, V_pages_strides, table, b, hk, d, pages, page,
                         width, 1);
    if (st) return st;
    const void *xs[] = {hq ? Q : nullptr, K, V};
    const int64_t *sx[] = {Q_strides, K_strides, V_strides};
    for (int w = 0; w < 3; ++w) {
        const int heads = w ? hk : hq;
        c.x[w] = xs[w];
        if (!heads) continue;
        if (!aligned16(xs[w])) return LINFORMER_ERR_ALIGN;
        c.sx[w] = strides_of(sx[w], heads, n, d);
        st = check_strides(c.sx[w], b, heads, n, d, 1, false);
        if (st) return st;
        if (xs[w] == K_pages || xs[w] == V_pages) return LINFORMER_ERR_VALUE;  // overlapping outputs
    }
    if (hq) {
        if (!aligned16(Y)) return LINFORMER_ERR_ALIGN;
        c.sy = strides_of(Y_strides, hq, n, d);
        st = check_strides(c.sy, b, hq, n, d, 1, true);
        if (st) return st;
        if (Y == K || Y == V || Y == K_pages || Y == V_pages) return LINFORMER_ERR_VALUE;
        // in place means the same elements in the same places
        if (Y == Q && ((b > 1 && c.sy.b != c.sx[0].b) || (hq > 1 && c.sy.h != c.sx[0].h) ||
                       (n > 1 && c.sy.n != c.sx[0].n)))
            return LINFORMER_ERR_VALUE;
        c.y = Y;
    }
    c.starts = starts;
    c.counts = counts;
    c.positions = positions;
    c.phase = phase;
    c.b = b, c.hq = hq, c.hk = hk, c.n = n, c.d = d;
    c.rot = phase ? rot : 0;
    c.interleaved = layout == LINFORMER_ROTARY_INTERLEAVED;
    c.dtype = dtype;
    c.amplitude = amplitude;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return paged::append(c);
}

extern "C" int linformer_cache_keep(void *K_pages, const int64_t *K_pages_strides, void *V_pages,
                                    const int64_t *V_pages_strides, const int32_t *table, const int32_t *starts,
                                    const int32_t *path, const int32_t *counts, int b, int hk, int m, int d,
                                    int pages, int page, int width, int dtype, void *stream) {
    if (!K_pages || !V_pages || !table || !starts || !path) return LINFORMER_ERR_NULL;
    if (b < 1 || hk < 1 || m < 1 || d < 1) return LINFORMER_ERR_SIZE;
    if ((int64_t)b * hk > (1 << 28) || m > kMaxRows || d > (1 << 20)) return LINFORMER_ERR_SIZE;
    if (dtype != LINFORMER_F32 && dtype != LINFORMER_BF16)
        return dtype == LINFORMER_BF16_F32OUT ? LINFORMER_ERR_UNSUPPORTED : LINFORMER_ERR_ENUM;
    if (unaligned(starts, 4) || unaligned(path, 4) || unaligned(counts, 4)) return LINFORMER_ERR_ALIGN;
    paged::KeepCall c{};
    const int st = check_cache(c.cache, K_pages, K_pages_strides, V_pages, V_pages_strides, table, b, hk, d, pages,
                               page, width, 1);
    if (st) return st;
    c.starts = starts;
    c.path = path;
    c.counts = counts;
    c.b = b, c.hk = hk, c.m = m, c.d = d;
    c.dtype = dtype;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return paged::keep(c);
}

extern "C" int linformer_paged_attn_fwd(const void *Q, const int64_t *Q_strides, const void *K_pages,
                                        const int64_t *K_pages_strides, const void *V_pages,
                                        const int64_t *V_pages_strides, void *O, const int64_t *O_strides, float *lse,
                                        const int32_t *table, const int32_t *k_lengths, const int32_t *q_lengths,
                                        int b, int hq, int hk, int nq, int d, int pages, int page, int width,
                                        float scale, int causal, int window, int dtype, void *stream) {
    paged::AttnCall c{};
    const int st = check_attention(c, Q, Q_strides, K_pages, K_pages_strides, V_pages, V_pages_strides, O, O_strides,
                                   lse, table, k_lengths, q_lengths, b, hq, hk, nq, d, pages, page, width, scale,
                                   dtype);
    if (st) return st;
    if (window < 0 || (window && !causal) || causal < 0 || causal > 1) return LINFORMER_ERR_VALUE;
    c.causal = causal;
    c.window = window >= width * page ? 0 : window;  // no query looks further back than its rows
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return paged::attention(c);
}

extern "C" int linformer_tree_attn_fwd(const void *Q, const int64_t *Q_strides, const void *K_pages,
                                       const int64_t *K_pages_strides, const void *V_pages,
                                       const int64_t *V_pages_strides, void *O, const int64_t *O_strides, float *lse,
                                       const int32_t *table, const int32_t *k_lengths, const int32_t *q_lengths,
                                       const uint64_t *mask, int b, int hq, int hk, int nq, int d, int pages,
                                       int page, int width, float scale, int dtype, void *stream) {
    if (!mask) return LINFORMER_ERR_NULL;
    paged::AttnCall c{};
    const int st = check_attention(c, Q, Q_strides, K_pages, K_pages_strides, V_pages, V_pages_strides, O, O_strides,
                                   lse, table, k_lengths, q_lengths, b, hq, hk, nq, d, pages, page, width, scale,
                                   dtype);
    if (st) return st;
    if (nq > LINFORMER_TREE_NODES) return LINFORMER_ERR_SIZE;
    if (unaligned(mask, 8)) return LINFORMER_ERR_ALIGN;
    c.mask = mask;
    c.words = (nq + 63) / 64;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return paged::attention(c);
}

extern "C" int linformer_tree_mask(const int32_t *parents, uint64_t *mask, int b, int n, void *stream) {
    if (!parents || !mask) return LINFORMER_ERR_NULL;
    if (b < 1 || n < 1 || n > LINFORMER_TREE_NODES) return LINFORMER_ERR_SIZE;
    if (unaligned(parents, 4) || unaligned(mask, 8)) return LINFORMER_ERR_ALIGN;
    return paged::tree_mask(parents, mask, b, n, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int linformer_cache_packed(int call, const void *words, int count) {
    if (!words) return LINFORMER_ERR_NULL;
    static constexpr int kCount[] = {42, 21, 33, 32};
    if (call < LINFORMER_PACKED_APPEND || call > LINFORMER_PACKED_TREE) return LINFORMER_ERR_ENUM;
    if (count != kCount[call]) return LINFORMER_ERR_VALUE;
    Words a;
    std::memcpy(a.w, words, count * sizeof(int64_t));
    if (call == LINFORMER_PACKED_APPEND) {
        void *x[6];
        const int64_t *sx[6];
        for (int i = 0; i < 6; ++i) {  // K, V, K_pages, V_pages, Q, Y
            x[i] = a.pointer<void>();
            sx[i] = a.strides();
        }
        const auto table = a.pointer<int32_t>(), starts = a.pointer<int32_t>(), counts = a.pointer<int32_t>();
        const auto phase = a.pointer<uint64_t>();
        const auto positions = a.pointer<int32_t>();
        int n[10];  // b, hq, hk, n, d, pages, page, width, rot, layout
        for (int &y : n) y = a.integer();
        const float amplitude = a.real();
        const int dtype = a.integer();
        const auto stream = a.pointer<void>();
        if (!a.fits) return LINFORMER_ERR_SIZE;
        return linformer_cache_append(x[0], sx[0], x[1], sx[1], x[2], sx[2], x[3], sx[3], x[4], sx[4], x[5], sx[5],
                                      table, starts, counts, phase, positions, n[0], n[1], n[2], n[3], n[4], n[5],
                                      n[6], n[7], n[8], n[9], amplitude, dtype, stream);
    }
    if (call == LINFORMER_PACKED_KEEP) {
        const auto K = a.pointer<void>();
        const auto sK = a.strides();
        const auto V = a.pointer<void>();
        const auto sV = a.strides();
        const auto table = a.pointer<int32_t>(), starts = a.pointer<int32_t>(), path = a.pointer<int32_t>(),
                   counts = a.pointer<int32_t>();
        int n[8];  // b, hk, m, d, pages, page, width, dtype
        for (int &y : n) y = a.integer();
        const auto stream = a.pointer<void>();
        if (!a.fits) return LINFORMER_ERR_SIZE;
        return linformer_cache_keep(K, sK, V, sV, table, starts, path, counts, n[0], n[1], n[2], n[3], n[4], n[5],
                                    n[6], n[7], stream);
    }
    const bool tree = call == LINFORMER_PACKED_TREE;
    void *x[4];
    const int64_t *sx[4];
    for (int i = 0; i < 4; ++i) {  // Q, K_pages, V_pages, O
        x[i] = a.pointer<void>();
        sx[i] = a.strides();
    }
    const auto lse = a.pointer<float>();
    const auto table = a.pointer<int32_t>(), k_lengths = a.pointer<int32_t>(), q_lengths = a.pointer<int32_t>();
    const auto mask = tree ? a.pointer<uint64_t>() : nullptr;
    int n[8];  // b, hq, hk, nq, d, pages, page, width
    for (int &y : n) y = a.integer();
    const float scale = a.real();
    const int causal = tree ? 0 : a.integer(), window = tree ? 0 : a.integer();
    const int dtype = a.integer();
    const auto stream = a.pointer<void>();
    if (!a.fits) return LINFORMER_ERR_SIZE;
    if (tree)
        return linformer_tree_attn_fwd(x[0], sx[0], x[1], sx[1], x[2], sx[2], x[3], sx[3], lse, table, k_lengths,
                                       q_lengths, mask, n[0], n[1], n[2], n[3], n[4], n[5], n[6], n[7], scale, dtype,
                                       stream);
    return linformer_paged_attn_fwd(x[0], sx[0], x[1], sx[1], x[2], sx[2], x[3], sx[3], lse, table, k_lengths,
                                    q_lengths, n[0], n[1], n[2], n[3], n[4], n[5], n[6], n[7], scale, causal, window,
                                    dtype, stream);
}
