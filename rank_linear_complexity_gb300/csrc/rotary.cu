// Rotary positions: the pairs of the first `rot` elements of every head are turned by an
// angle proportional to the position,
//
//     (y_a, y_b) = amplitude (x_a cos t - x_b sin t, x_b cos t + x_a sin t),  t = pos f_i,
//
// pair i being elements (i, i + rot/2) or (2 i, 2 i + 1); the gradient is the same turn
// backwards.  The frequencies come as fractions of a full turn per position in 64-bit fixed
// point: pos x step wraps modulo one turn by itself, so the angle of position 2^31 is as
// exact as that of position 1, without 64-bit floating point.
//
// Bound by memory: every element read and written once (bf16, 4 x 16384 rows of 32 heads of 64:
// 95 us, 5.7 TB/s; sines shared by a block in shared memory instead: 123 us, the barrier and
// the second phase cost more than the sines).  A thread keeps the 8 (bf16) or 4
// (fp32) sines and cosines of its pairs in registers and goes through several heads of both
// tensors with them, 16-byte pieces at a time.
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>

#include "internal.cuh"
#include "rotary.cuh"

namespace linformer {
namespace rotary {
namespace {

constexpr int kThreads = 64;
constexpr int kMaxHeads = 16; // heads of one thread

struct Params {
    const void *x[2];
    void *y[2];
    Strides sx[2], sy[2];
    int heads[2];
    const uint64_t *phase;
    const int32_t *positions;
    int start, b, n, d, rot, chunks, rot_chunks, per_thread, splits;
    int64_t threads;
    float amplitude, sign;
};

// V pairs a thread (V = 1: any strides and sizes; otherwise 16-byte pieces).
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const Params p) {
    using Piece = Vec<T, V>;
    const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (tid >= p.threads) return;
    const int c = (int)(tid % p.chunks);
    const int64_t r = tid / p.chunks;
    const int i = (int)(r % p.n);
    const int64_t r2 = r / p.n;
    const int split = (int)(r2 % p.splits), b = (int)(r2 / p.splits);
    const int h0 = split * p.per_thread, h1 = min(h0 + p.per_thread, p.heads[0] + p.heads[1]);
    const bool turn = c < p.rot_chunks;
    float cs[V], sn[V];
    // the two pieces of the thread's pairs (of the copied rest: one)
    const int at0 = turn ? (kInterleaved ? 2 * V * c : V * c) : p.rot + V * (c - p.rot_chunks);
    const int at1 = turn ? (kInterleaved ? at0 + V : at0 + p.rot / 2) : at0;
    if (turn) {
        const int pos = p.positions ? __ldg(p.positions + (int64_t)b * p.n + i) : p.start + i;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float c0, s0;
            turn_of(__ldg(p.phase + V * c + v), pos, c0, s0);
            cs[v] = c0 * p.amplitude;
            sn[v] = s0 * p.sign;
        }
    }
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const int w = h >= p.heads[0] ? 1 : 0, hh = h - (w ? p.heads[0] : 0);
        const T *x = static_cast<const T *>(p.x[w]) + b * p.sx[w].b + hh * p.sx[w].h + i * p.sx[w].n;
        T *y = static_cast<T *>(p.y[w]) + b * p.sy[w].b + hh * p.sy[w].h + i * p.sy[w].n;
        Piece u0 = *reinterpret_cast<const Piece *>(x + at0);
        if (turn) {
            Piece u1 = *reinterpret_cast<const Piece *>(x + at1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                // interleaved: elements 2 v and 2 v + 1 of the two pieces in a row
                T &a = kInterleaved ? (2 * v < V ? u0.e[(2 * v) % V] : u1.e[(2 * v) % V]) : u0.e[v];
                T &z = kInterleaved ? (2 * v + 1 < V ? u0.e[(2 * v + 1) % V] : u1.e[(2 * v + 1) % V]) : u1.e[v];
                const float fa = to_float(a), fz = to_float(z);
                a = from_float<T>(fa * cs[v] - fz * sn[v]);
                z = from_float<T>(fz * cs[v] + fa * sn[v]);
            }
            *reinterpret_cast<Piece *>(y + at1) = u1;
        }
        *reinterpret_cast<Piece *>(y + at0) = u0;
    }
}

// Sums of two doubles (Dekker's and Knuth's error-free sums and products), relative precision
// about 2^-102: a double alone keeps 53 of a phase word's 64 bits, and position 2^31 would be off
// by 2^-22 turns.
struct Pair {
    double hi, lo;
};
__device__ __forceinline__ Pair add_exact(double a, double b) {
    const double s = a + b, c = s - a;
    return {s, (a - (s - c)) + (b - c)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const Pair s = add_exact(a.hi, b.hi);
    return add_exact(s.hi, s.lo + (a.lo + b.lo));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    const double p = __dmul_rn(a.hi, b.hi);  // (not to be merged into the sum below)
    return add_exact(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
__device__ __forceinline__ Pair div(Pair a, Pair b) {
    const double q = a.hi / b.hi;
    const Pair r = add(a, mul({-q, 0.0}, b));
    return add_exact(q, r.hi / b.hi);
}
__device__ Pair power(Pair x, int n) {
    Pair y{1.0, 0.0};
    for (; n; n >>= 1) {
        if (n & 1) y = mul(y, x);
        if (n > 1) x = mul(x, x);
    }
    return y;
}
// base^(-1 / n): Newton steps from the double's value, each of which squares its error.
__device__ Pair inverse_root(double base, int n) {
    Pair r{pow(base, -1.0 / n), 0.0};
    for (int i = 0; i < 2; ++i) {
        const Pair e = add(mul(power(r, n), {base, 0.0}), {-1.0, 0.0});
        if (!isfinite(e.hi)) break;  // a base next to the ends of a double's range
        r = add(r, mul({-r.hi / n, 0.0}, e));
    }
    return r;
}

// One thread a pair: f_i = base^(-2 i / rot), scaled, as a 64-bit fraction of a turn.
__global__ void phase_kernel(uint64_t *phase, int pairs, double base, int scaling, double factor,
                             double original, double beta_fast, double beta_slow) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= pairs) return;
    const Pair per_radian{0.15915494309189535, -9.839338337591243e-18};  // 1 / (2 pi)
    Pair turns = mul(power(inverse_root(base, pairs), i), per_radian);
    // the base times factor^(rot / (rot - 2)), to the power -2 i / rot
    if (scaling == LINFORMER_ROTARY_BASE && pairs > 1) turns = mul(turns, power(inverse_root(factor, pairs - 1), i));
    if (scaling == LINFORMER_ROTARY_LINEAR) turns = div(turns, {factor, 0.0});
    if (scaling == LINFORMER_ROTARY_BY_PARTS) {
        Pair keep = div(add(mul(turns, {original, 0.0}), {-beta_slow, 0.0}), add_exact(beta_fast, -beta_slow));
        if (keep.hi < 0.0) keep = {0.0, 0.0};
        if (keep.hi > 1.0 || (keep.hi == 1.0 && keep.lo > 0.0)) keep = {1.0, 0.0};
        const Pair rest = div(add({1.0, 0.0}, {-keep.hi, -keep.lo}), {factor, 0.0});
        turns = mul(turns, add(keep, rest));
    }
    // the fraction of both parts in units of 2^-64, modulo 2^64
    const double units = ldexp(turns.hi - floor(turns.hi), 64), whole = floor(units);
    const double low = ldexp(turns.lo - rint(turns.lo), 64);
    phase[i] = (uint64_t)whole + (uint64_t)(int64_t)rint((units - whole) + low);
}

template <typename T, int V>
int launch(const Params &p, bool interleaved, cudaStream_t s) {
    const int64_t blocks = (p.threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return LINFORMER_ERR_SIZE;
    KernelScope scope(LINFORMER_KERNEL_ROTARY, s);
    if (interleaved) rotary_kernel<T, V, true><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    else rotary_kernel<T, V, false><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? LINFORMER_OK : LINFORMER_ERR_LAUNCH;
}

}  // namespace

int turn(const Call &c) {
    Params p{};
    const int V = c.dtype == LINFORMER_F32 ? 4 : 8;
    bool wide = c.d % V == 0 && c.rot % (2 * V) == 0;
    for (int w = 0; w < 2; ++w) {
        p.x[w] = c.x[w];
        p.y[w] = c.y[w];
        p.sx[w] = c.sx[w];
        p.sy[w] = c.sy[w];
        p.heads[w] = c.heads[w];
        if (!c.heads[w]) continue;
        for (const Strides *s : {&c.sx[w], &c.sy[w]})
            wide = wide && (c.b == 1 || s->b % V == 0) && (c.heads[w] == 1 || s->h % V == 0) &&
                   (c.n == 1 || s->n % V == 0);
    }
    const int v = wide ? V : 1;
    p.phase = c.phase;
    p.positions = c.positions;
    p.start = c.start;
    p.b = c.b;
    p.n = c.n;
    p.d = c.d;
    p.rot = c.rot;
    p.amplitude = c.amplitude;
    p.sign = c.inverse ? -c.amplitude : c.amplitude;
    p.rot_chunks = c.rot / 2 / v;
    // in place the rest of the head stays where it is
    const bool in_place = c.x[0] == c.y[0] && (!c.heads[1] || c.x[1] == c.y[1]);
    p.chunks = p.rot_chunks + (in_place ? 0 : (c.d - c.rot) / v);
    // Heads per thread: the sines cost about as much as the work on three heads, so as many
    // heads as leave two full waves of threads, at most kMaxHeads.
    const int heads = c.heads[0] + c.heads[1];
    const int64_t rows = (int64_t)c.b * c.n * p.chunks;
    constexpr int64_t kSmThreads = 2048;
    const int64_t per = rows * heads / (2 * device_sms() * kSmThreads);
    p.per_thread = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(heads, kMaxHeads), per));
    p.splits = (heads + p.per_thread - 1) / p.per_thread;
    p.threads = rows * p.splits;
    if (c.dtype == LINFORMER_F32)
        return wide ? launch<float, 4>(p, c.interleaved, c.stream) : launch<float, 1>(p, c.interleaved, c.stream);
    return wide ? launch<__nv_bfloat16, 8>(p, c.interleaved, c.stream)
                : launch<__nv_bfloat16, 1>(p, c.interleaved, c.stream);
}

int phase_table(uint64_t *phase, int rot, double base, int scaling, double factor, int original,
                double beta_fast, double beta_slow, cudaStream_t s) {
    KernelScope scope(LINFORMER_KERNEL_ROTARY, s);
    const int pairs = rot / 2;
    phase_kernel<<<(pairs + 127) / 128, 128, 0, s>>>(phase, pairs, base, scaling, factor, original,
                                                     beta_fast, beta_slow);
    return cudaGetLastError() == cudaSuccess ? LINFORMER_OK : LINFORMER_ERR_LAUNCH;
}

}  // namespace rotary
}  // namespace linformer
