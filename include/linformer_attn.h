/*
 * linformer_attn.h -- C ABI of the GB300 (sm_103a) Linformer attention forward.
 *
 * The operation ("Linformer(Self-Attention with Linear Complexity) 요약 설명",
 * section Model; "Linformer: Self-Attention with Linear Complexity - 中文验证版",
 * section 方法适配): for every batch index beta < b and head eta < h (a "unit"),
 *
 *     Kbar = Ehat . K[beta][eta]        (k x n) . (n x d) -> k x d
 *     Vbar = Fhat . V[beta][eta]        (k x n) . (n x d) -> k x d
 *     O[beta][eta] = softmax(Q[beta][eta] . Kbar^T / sqrt(d)) . Vbar   -> n x d
 *
 * E and F project the sequence axis (length n) down to k positions; the queries
 * are not compressed, so O has one row per input position and the n x k score
 * matrix never leaves the chip.  The scale 1/sqrt(d) is the scaled dot product
 * of the PaperWeekly efficient-Transformer survey, section 2.1.
 *
 * Sharing modes (中文验证版, section 方法适配; 요약 설명, section Additional
 * Efficiency Techniques):
 *   LINFORMER_SHARE_PER_HEAD  E, F: [h][k][n], each head its own pair
 *   LINFORMER_SHARE_KV        E:    [h][k][n], F = E (F must be NULL or == E)
 *   LINFORMER_SHARE_HEADWISE  E, F: [k][n], one pair for all heads
 *   LINFORMER_SHARE_LAYERWISE E:    [k][n], one projection for all heads and for
 *                                   keys and values (F must be NULL or == E)
 * In every mode E and F are shared across the batch (they are parameters).
 *
 * Padding (요약 설명, section Model, padding paragraph): pad_lengths[beta] is the
 * valid length L of batch entry beta (clamped to [0, n] on the device).  Rows
 * t >= L of K and V count as zero before the projection, whatever they hold,
 * and query rows i >= L get O = 0.  NULL means L = n for every entry.
 *
 * Layouts: every tensor is dense and row-major, but for the calls that take strides (see
 * there).  Q, K, V, O: [b][h][n][d].
 * E, F: as listed above ([k][n] rows of length n).
 *
 * Number types (dtype):
 *   LINFORMER_F32          Q, K, V, E, F, O in fp32; all arithmetic in fp32.
 *   LINFORMER_BF16         Q, K, V, E, F, O in bf16; fp32 accumulation.
 *   LINFORMER_BF16_F32OUT  inputs in bf16, O in fp32.
 *
 * Ownership: the caller owns every buffer.  All pointers of linformer_attn_fwd
 * and linformer_project_fwd are device pointers of the current CUDA device, 16-byte
 * aligned.  The library writes only O (or Kbar/Vbar) and a stream-ordered
 * workspace that it allocates and frees on `stream` (cudaMallocFromPoolAsync /
 * cudaFreeAsync) from a memory pool of its own per device, created on first use,
 * which keeps freed memory mapped for the next call until the process exits (as much
 * as the largest call in flight needed).  Calls are asynchronous on `stream` (a cudaStream_t; NULL is
 * the legacy default stream): inputs must stay unchanged until the stream has
 * passed the call.  Calls on different streams may run concurrently.  The forward's
 * first kernel is launched with programmatic stream serialisation and waits for the
 * kernel before it (griddepcontrol.wait) before it reads or writes memory; its last
 * kernel lets the next kernel in the stream launch early, so a caller's kernel that
 * is itself launched with programmatic stream serialisation after a call must wait
 * for its prerequisite grid (cudaGridDependencySynchronize) before it reads O, as
 * CUDA requires of any such kernel.  Kernels launched without that attribute are
 * ordered as usual.
 *
 * Errors: every function returns LINFORMER_OK (0) or a negative status; no call
 * traps or aborts.  Argument errors are detected on the host before anything is
 * launched.  Device-side failures (a bounded wait that ran out; a page, path or tree
 * that the device found wrong) set a device status word that linformer_debug_read_device_status() reads and clears.
 */
#ifndef LINFORMER_ATTN_H
#define LINFORMER_ATTN_H

#include <stdint.h>

/* Exported symbols (the library is built with hidden default visibility). */
#if defined(__GNUC__)
#define LINFORMER_API __attribute__((visibility("default")))
#else
#define LINFORMER_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LINFORMER_F32 = 0,
    LINFORMER_BF16 = 1,
    LINFORMER_BF16_F32OUT = 2
} linformer_dtype;

typedef enum {
    LINFORMER_SHARE_PER_HEAD = 0,
    LINFORMER_SHARE_KV = 1,
    LINFORMER_SHARE_HEADWISE = 2,
    LINFORMER_SHARE_LAYERWISE = 3
} linformer_share_mode;

typedef enum {
    LINFORMER_OK = 0,
    LINFORMER_ERR_NULL = -1,        /* a required pointer is NULL */
    LINFORMER_ERR_SIZE = -2,        /* b, h, n, d or k < 1, or a size overflows */
    LINFORMER_ERR_UNSUPPORTED = -3, /* d > 128 or k > 1024 */
    LINFORMER_ERR_ENUM = -4,        /* bad share_mode or dtype */
    LINFORMER_ERR_ALIGN = -5,       /* a pointer is not 16-byte aligned */
    LINFORMER_ERR_F_MODE = -6,      /* F given (and != E) in KV / LAYERWISE mode, or
                                       missing in PER_HEAD / HEADWISE mode */
    LINFORMER_ERR_ALLOC = -7,       /* workspace allocation failed */
    LINFORMER_ERR_LAUNCH = -8,      /* a CUDA call or kernel launch failed */
    LINFORMER_ERR_DEVICE = -9,      /* a device-side bounded wait ran out, or a table, path or
                                       tree on the device named what is not there */
    LINFORMER_ERR_VALUE = -10       /* a parameter or a stride is out of its range */
} linformer_status;

/* Which kernels a call uses. */
typedef enum {
    LINFORMER_PATH_SIMT = 0,        /* fp32 FFMA kernels: any supported shape */
    LINFORMER_PATH_TENSOR = 1       /* tcgen05/TMA kernels: bf16 inputs, d = 64,
                                       k <= 256, n a multiple of 8 */
} linformer_path_kind;

/* Kernel identifiers for the profiling counters. */
typedef enum {
    LINFORMER_KERNEL_PROJECT_TC = 0,
    LINFORMER_KERNEL_ATTEND_TC = 1,
    LINFORMER_KERNEL_PROJECT_SIMT = 2,
    LINFORMER_KERNEL_ATTEND_SIMT = 3,
    LINFORMER_KERNEL_WINDOW = 4,    /* linformer_window_projection */
    LINFORMER_KERNEL_BACKWARD = 5,  /* the kernels of linformer_attn_bwd */
    LINFORMER_KERNEL_DENSE = 6,     /* the kernels of linformer_dense_attn_fwd */
    LINFORMER_KERNEL_ROTARY = 7,    /* the kernels of linformer_rotary */
    LINFORMER_KERNEL_SOFTMAX = 8,   /* the kernels of linformer_softmax_attn_fwd */
    LINFORMER_KERNEL_SOFTMAX_BWD = 9, /* the kernels of linformer_softmax_attn_bwd */
    LINFORMER_KERNEL_CACHE = 10,    /* the kernels of linformer_cache_append, _keep and
                                       linformer_tree_mask */
    LINFORMER_KERNEL_PAGED = 11,    /* the kernels of linformer_paged_attn_fwd and
                                       linformer_tree_attn_fwd */
    LINFORMER_KERNEL_COUNT = 12
} linformer_kernel_id;

/*
 * The whole Linformer attention forward (all steps above) for b*h units.
 * Q, K, V: [b][h][n][d] (dtype in); E, F: see the sharing modes; pad_lengths:
 * device int32[b] or NULL; O: [b][h][n][d] (dtype out).  Supported: d <= 128,
 * k <= 1024 (the tensor-core path takes bf16 inputs with d = 64, k <= 256 and
 * n % 8 == 0; other shapes run on the fp32 SIMT kernels).
 */
LINFORMER_API int linformer_attn_fwd(const void *Q, const void *K, const void *V,
                       const void *E, const void *F,
                       const int32_t *pad_lengths, void *O,
                       int b, int h, int n, int d, int k,
                       int share_mode, int dtype, void *stream);

/*
 * The projection step alone: Kbar = Ehat . K and Vbar = Fhat . V over the valid
 * rows (요약 설명, section Model), written as fp32 [b][h][k][d] into the
 * caller's device buffers Kbar and Vbar.  Same argument rules as above.  On the
 * tensor-core path Kbar and Vbar are the exact sums of the on-chip split
 * representation the attention step consumes.
 */
LINFORMER_API int linformer_project_fwd(const void *K, const void *V, const void *E, const void *F,
                          const int32_t *pad_lengths, float *Kbar, float *Vbar,
                          int b, int h, int n, int d, int k,
                          int share_mode, int dtype, void *stream);

/*
 * Same operation as linformer_attn_fwd, for callers whose data is in HOST memory
 * (page-locked memory gives the fastest copies).  Q, K, V, E, F, pad_lengths and
 * O are host pointers.  The call allocates device buffers on `stream`, copies
 * the inputs in, runs the forward, copies O back and synchronises `stream`
 * before returning, so O is complete on return.
 */
LINFORMER_API int linformer_attn_fwd_host(const void *Q, const void *K, const void *V,
                            const void *E, const void *F,
                            const int32_t *pad_lengths, void *O,
                            int b, int h, int n, int d, int k,
                            int share_mode, int dtype, void *stream);

/*
 * linformer_attn_fwd_noalloc: the same operation, arguments and device buffers as
 * linformer_attn_fwd, for callers that must not allocate device memory while they
 * run it -- for example a server that reserved its whole memory budget at start-up,
 * a plugin whose host framework owns every device allocation, code called from an
 * allocator or out-of-memory handler, or a setup without stream-ordered memory
 * pools.  It allocates nothing: its workspace is one fixed 32 MiB array in device
 * memory that every GPU loading this library holds until the process exits.
 *   - Problems whose workspace does not fit in 32 MiB even without splitting the
 *     sequence (about b*h*k_pad*512 bytes, k_pad = k rounded up to 16) return
 *     LINFORMER_ERR_SIZE before anything is launched.
 *   - Only tensor-core configurations (bf16 inputs, d = 64, k <= 256, n % 8 == 0)
 *     are served; others return LINFORMER_ERR_UNSUPPORTED.
 *   - The first call on a device looks up the array's address on that device;
 *     make it before any stream capture starts.
 *   - Every call reuses the same array and clears its per-unit counters itself;
 *     calls that overlap on the GPU (other streams, other host threads) race on
 *     the array and must be serialised by the caller.
 * The pages describe no counterpart: this is a deployment variant, not part of the
 * method.
 */
LINFORMER_API int linformer_attn_fwd_noalloc(const void *Q, const void *K, const void *V,
                                             const void *E, const void *F,
                                             const int32_t *pad_lengths, void *O,
                                             int b, int h, int n, int d, int k,
                                             int share_mode, int dtype, void *stream);

/*
 * The backward of linformer_attn_fwd: given dO = dLoss/dO, writes dQ, dK, dV
 * ([b][h][n][d]) and dE (shaped like E) and, in PER_HEAD and HEADWISE modes, dF
 * (shaped like F; in KV and LAYERWISE modes F is E and dE holds both terms, dF must be
 * NULL).  The chain rule through the forward's definition (요약 설명, section Model):
 * rows t >= L of K and V and query rows i >= L take no part (their gradients are
 * zero), and the gradient of a shared E or F sums the terms of every unit that shares
 * it.  fp32 only (LINFORMER_F32; other dtypes return LINFORMER_ERR_UNSUPPORTED),
 * d <= 128, k <= 1024, b*h <= 65535 (else LINFORMER_ERR_SIZE).  All pointers are
 * device pointers, 16-byte aligned; the caller owns every buffer; a stream-ordered
 * workspace of b*h*(2 n k + 12 k d) floats (8 k d of the 12 hold split partial sums;
 * the 2 n k, once P and dS are used, the partial sums of dE and dF) comes from the
 * library's pool and is returned to it in stream order.
 */
LINFORMER_API int linformer_attn_bwd(const void *Q, const void *K, const void *V,
                                     const void *E, const void *F, const int32_t *pad_lengths,
                                     const void *dO, void *dQ, void *dK, void *dV, void *dE,
                                     void *dF, int b, int h, int n, int d, int k,
                                     int share_mode, int dtype, void *stream);

/*
 * Dense softmax attention, the full-attention baseline that the pages' inference table
 * ("Linformer 요약 설명", section Inference-time Efficiency Results) compares the
 * method with: O = softmax(Q K^T / sqrt(d)) V per unit, Q, K, V, O [b][h][n][d] fp32.
 * With pad_lengths, keys t >= L take no part in the softmax and query rows i >= L are
 * written as zero.  The n x n scores of every unit live in a stream-ordered workspace
 * of b*h*n*n floats from the library's pool (the memory the standard form needs).
 * fp32 only (else LINFORMER_ERR_UNSUPPORTED); d <= 128; b*h <= 65535 and n <= 8388480
 * (else LINFORMER_ERR_SIZE); pointers device, 16-byte aligned; the caller owns them.
 */
LINFORMER_API int linformer_dense_attn_fwd(const void *Q, const void *K, const void *V,
                                           const int32_t *pad_lengths, void *O, int b, int h,
                                           int n, int d, int dtype, void *stream);

/*
 * Strided tensors.  The entry points below take, beside each tensor of shape
 * [b][heads][n][d], its element strides {batch, head, row} as int64_t[3] (host memory, read
 * during the call), or NULL for a dense tensor; the last dimension is contiguous.  A stride
 * of a dimension of size one is ignored; others are positive and at most 2^38.  An output's
 * strides are at least d, and its elements must not overlap each other or another tensor of the
 * call, except where a call says that it works in place (an output that starts where another
 * tensor does is refused with LINFORMER_ERR_VALUE).
 */

/*
 * Exact softmax attention without the n x n scores in memory, with what its backward pass
 * needs: for batch entry beta, query head eta and its key/value head eta / (hq / hk),
 *
 *     s_ij = scale Q_i . K_j,   lse_i = log sum_j exp(s_ij),
 *     O_i  = sum_j exp(s_ij - lse_i) V_j
 *
 * over the keys j < Lk that query i sees, Lq = q_lengths[beta], Lk = k_lengths[beta]
 * (device int32[b], clamped to [0, nq] and [0, nk]; NULL: nq, nk).  With causal != 0 the
 * valid parts end together: query i stands at position i + Lk - Lq and sees keys up to its
 * own position, with window > 0 only the last `window` of them (itself included).  A row
 * that sees no key, and rows i >= Lq, get O = 0 and lse = -infinity; rows of Q, K and V
 * past the lengths may hold anything.  Rows within the lengths have to be finite, also
 * those that a causal mask hides (0 x NaN would reach a sum).  Sums are fp32, in range while
 * |V| < 2^112 / nk and the terms of Q_i.K_j, also times scale log2(e), add up to less than 2^127.
 *
 * Q, O: [b][hq][nq][d]; K, V: [b][hk][nk][d], hq a multiple of hk; lse: dense fp32
 * [b][hq][nq].  dtype LINFORMER_BF16 (else LINFORMER_ERR_UNSUPPORTED), d a multiple of 8 up
 * to 128 (else LINFORMER_ERR_UNSUPPORTED), 0 < scale < 2^127, causal 0 or 1, window >= 0
 * and 0 unless causal (else LINFORMER_ERR_VALUE); nq, nk and b hq up to 2^29, and up to 2^30 tiles of 128 rows over
 * all heads (else LINFORMER_ERR_SIZE).  Pointers are
 * 16-byte aligned (lse and the lengths: 4) and strides multiples of 8.  A few query rows
 * (single tokens over a cache) are served by splitting the keys over the GPU; the parts are
 * joined in a stream-ordered workspace; long calls with masks or lengths keep a counter there.  The result of a call does not depend on timing.
 */
LINFORMER_API int linformer_softmax_attn_fwd(
    const void *Q, const int64_t *Q_strides, const void *K, const int64_t *K_strides,
    const void *V, const int64_t *V_strides, void *O, const int64_t *O_strides, float *lse,
    const int32_t *q_lengths, const int32_t *k_lengths, int b, int hq, int hk, int nq, int nk,
    int d, float scale, int causal, int window, int dtype, void *stream);

/*
 * The backward of linformer_softmax_attn_fwd: from its inputs, its O and lse, and dO =
 * dLoss/dO, writes
 *
 *     dV_j = sum_i p_ij dO_i,          p_ij = exp(s_ij - lse_i)  (recomputed),
 *     dQ_i = scale sum_j g_ij K_j,     g_ij = p_ij (dO_i . V_j - dO_i . O_i),
 *     dK_j = scale sum_i g_ij Q_i,
 *
 * dK and dV summed over the query heads that share the key/value head; rows past the
 * lengths get zero.  Same argument rules; dO and dQ are shaped like O, dK and dV like K.
 * Sums are formed in a fixed order (no atomics): repeated calls agree bit for bit.  The
 * workspace is 8 bytes per query row, rows rounded up to 128 per head, and where few tiles
 * have long sums, which are then split, fp32 partial sums (at most a tile of 128 rows an SM, of each gradient).
 */
LINFORMER_API int linformer_softmax_attn_bwd(
    const void *Q, const int64_t *Q_strides, const void *K, const int64_t *K_strides,
    const void *V, const int64_t *V_strides, const void *O, const int64_t *O_strides,
    const void *dO, const int64_t *dO_strides, const float *lse, void *dQ,
    const int64_t *dQ_strides, void *dK, const int64_t *dK_strides, void *dV,
    const int64_t *dV_strides, const int32_t *q_lengths, const int32_t *k_lengths, int b, int hq,
    int hk, int nq, int nk, int d, float scale, int causal, int window, int dtype, void *stream);

/* Which elements of a head form pair i of rot / 2. */
typedef enum {
    LINFORMER_ROTARY_HALVES = 0,      /* i and i + rot / 2 */
    LINFORMER_ROTARY_INTERLEAVED = 1  /* 2 i and 2 i + 1 */
} linformer_rotary_layout;

/* How a rotary frequency f_i = base^(-2 i / rot) is scaled for contexts longer than the
 * trained one. */
typedef enum {
    LINFORMER_ROTARY_PLAIN = 0,
    LINFORMER_ROTARY_LINEAR = 1,   /* f_i / factor: positions are compressed */
    LINFORMER_ROTARY_BASE = 2,     /* base factor^(rot / (rot - 2)): the slowest pair is
                                      slowed by factor, the fastest keeps its frequency */
    LINFORMER_ROTARY_BY_PARTS = 3  /* by the turns r_i = original_length f_i / 2 pi that a pair
                                      makes in the original context: f_i from beta_fast turns
                                      up, f_i / factor from beta_slow down, linear between */
} linformer_rotary_scaling;

/*
 * Rotary positions: pair i of the first rot elements of every head at position pos is turned
 * by the angle pos f_i and scaled by `amplitude`,
 *
 *     y_a = amplitude (x_a cos - x_z sin),   y_z = amplitude (x_z cos + x_a sin);
 *
 * elements from rot on are copied.  inverse = 1 turns backwards: with it the call maps the
 * gradient of Y to the gradient of X.  One call takes up to two tensors that stand at the
 * same positions (queries and keys): X [b][hx][n][d] -> Y, and, with hx2 > 0, X2 [b][hx2][n][d]
 * -> Y2.  Y may be X with the same strides (in place).
 *
 * positions: device int32 [b][n] (dense), or NULL for start + row.  phase: device, rot / 2
 * entries, each the pair's turns per position f_i / 2 pi modulo 1 as a 64-bit binary fraction
 * (linformer_rotary_phase fills it, to the last bit; it is kept and used again by the caller).
 * Angles are exact to fp32 at every int32 position.  dtype LINFORMER_F32 or LINFORMER_BF16 (the turn in
 * fp32, rounded once).  2 <= rot <= d, even; a finite amplitude; start + n <= 2^31 (else
 * LINFORMER_ERR_VALUE).  X, Y, X2, Y2 16-byte aligned, phase 8; any strides (multiples of 16
 * bytes, d and rot / 2 multiples of 16 bytes run fastest).
 */
LINFORMER_API int linformer_rotary(const void *X, const int64_t *X_strides, void *Y,
                                   const int64_t *Y_strides, int hx, const void *X2,
                                   const int64_t *X2_strides, void *Y2, const int64_t *Y2_strides,
                                   int hx2, const uint64_t *phase, const int32_t *positions,
                                   int start, int b, int n, int d, int rot, int layout,
                                   float amplitude, int inverse, int dtype, void *stream);

/* Fills phase (device, rot / 2 entries) for linformer_rotary, asynchronously on `stream`.
 * base > 0, factor > 0; BY_PARTS also needs original_length >= 1 and beta_fast > beta_slow. */
LINFORMER_API int linformer_rotary_phase(uint64_t *phase, int rot, double base, int scaling,
                                         double factor, int original_length, double beta_fast,
                                         double beta_slow, void *stream);

/*
 * Paged key/value cache.  The rows of b sequences stand in pages, K_pages and V_pages
 * [pages][hk][page][d], given with element strides {page, head, row} as int64_t[3] (NULL:
 * dense; a cache laid out [pages][page][hk][d], or with keys and values side by side, is the
 * same memory with other strides).  table (device int32, dense [b][width]) says which page holds
 * rows [x page, (x + 1) page) of a sequence: table[beta][x].  Entries behind the rows in use are
 * not read.  page is a power of two from 8 to 65536, and width page at most 2^29 (else
 * LINFORMER_ERR_SIZE).  Several sequences may share pages that a call only reads.
 *
 * An entry outside [0, pages) where a row is needed, or a row behind the table's end, records a
 * failure in the device status word; no memory outside the cache is touched.
 *
 * The kernels of these calls let the next kernel in the stream launch early, and the attention's are
 * launched with programmatic stream serialisation themselves; they wait before they read or write
 * anything (as the forward's do, see Ownership above).
 */

/*
 * Appends rows: row i < counts[beta] (device int32[b]; NULL: n) of K and V [b][hk][n][d] goes to
 * row starts[beta] + i (device int32[b]) of sequence beta.  With phase, keys are turned on the way
 * as linformer_rotary turns them (rot, layout, amplitude, to the position positions[beta][i],
 * device int32 dense [b][n], or starts[beta] + i where positions is NULL), and with hq > 0 the
 * queries Q [b][hq][n][d] that stand at the same positions, all n rows of them, to Y (which may be
 * Q, with the same strides).  Without phase the keys are copied, and hq has to be 0.
 *
 * Nothing else in the cache is written: not the rows behind counts, and a row that the table has
 * no page for is dropped (and recorded).  No two rows of a call may go to one place.  dtype of all
 * tensors LINFORMER_F32 or LINFORMER_BF16.  Pointers 16-byte aligned (phase 8; table, starts, counts and
 * positions 4); any strides (multiples of 16 bytes, d and rot / 2 multiples of 16 bytes run fastest).
 * fp32 serves caches that a program reads by itself; the attention below takes bf16.
 */
LINFORMER_API int linformer_cache_append(
    const void *K, const int64_t *K_strides, const void *V, const int64_t *V_strides, void *K_pages,
    const int64_t *K_pages_strides, void *V_pages, const int64_t *V_pages_strides, const void *Q,
    const int64_t *Q_strides, void *Y, const int64_t *Y_strides, const int32_t *table,
    const int32_t *starts, const int32_t *counts, const uint64_t *phase, const int32_t *positions,
    int b, int hq, int hk, int n, int d, int pages, int page, int width, int rot, int layout,
    float amplitude, int dtype, void *stream);

/*
 * Keeps the accepted rows of a tree of drafted tokens: row starts[beta] + path[beta][i] of the
 * cache moves to row starts[beta] + i, for i < counts[beta] (device int32[b], clamped to [0, m];
 * NULL: m), path device int32 dense [b][m] with path[beta][i] >= i (a path from a tree's root down,
 * nodes numbered before their children, is one).  Sources are read as they were before the call.
 * An entry below its place is skipped and recorded in the device status word.  dtype LINFORMER_F32 or LINFORMER_BF16.
 */
LINFORMER_API int linformer_cache_keep(void *K_pages, const int64_t *K_pages_strides, void *V_pages,
                                       const int64_t *V_pages_strides, const int32_t *table,
                                       const int32_t *starts, const int32_t *path,
                                       const int32_t *counts, int b, int hk, int m, int d, int pages,
                                       int page, int width, int dtype, void *stream);

/*
 * Exact softmax attention over a paged cache: linformer_softmax_attn_fwd with the keys and values
 * of sequence beta in its pages, Lk = k_lengths[beta] of them (device int32[b], clamped to
 * [0, width page]; the new tokens' rows among them), and Lq = q_lengths[beta] queries (NULL: nq).
 * Masks, rows without keys, rows past the lengths, sums and types are that call's: bf16, d a
 * multiple of 8 up to 128, strides multiples of 8.  Rows of the pages behind the length may hold
 * anything, and with a window so may whole pages before the first query's: their table entries are not
 * read.  A page that is not there (see above) counts as rows of zeros.  Work is cut by rows of
 * keys, not by sequences: units of work whose table holds more than 768 rows may be joined from parts
 * in a stream-ordered workspace.  The result of a call depends neither on timing nor, in any bit, on what
 * rows past the lengths hold.  Probabilities enter the products as two bf16 parts where a key/value head
 * has up to 32 rows (tokens, rounded up to a power of two, times query heads), rounded to one bf16
 * elsewhere: at most 2^-8 of each term, as in linformer_softmax_attn_fwd.  The blocks of 128
 * rows that the queries of one sequence go through, all tiles of queries and heads counted, have to be
 * fewer than 2^31 (else LINFORMER_ERR_SIZE).
 */
LINFORMER_API int linformer_paged_attn_fwd(
    const void *Q, const int64_t *Q_strides, const void *K_pages, const int64_t *K_pages_strides,
    const void *V_pages, const int64_t *V_pages_strides, void *O, const int64_t *O_strides, float *lse,
    const int32_t *table, const int32_t *k_lengths, const int32_t *q_lengths, int b, int hq, int hk,
    int nq, int d, int pages, int page, int width, float scale, int causal, int window, int dtype,
    void *stream);

/* Nodes of a tree of drafted tokens at most. */
#define LINFORMER_TREE_NODES 1024

/*
 * The same for a tree of drafted tokens, the sequence's last Lq rows: query i sees every row before
 * the tree, and node j of the tree where bit j % 64 of mask[beta][i][j / 64] is set (device, dense
 * [b][nq][ceil(nq / 64)]; bits from Lq on are ignored).  A node's mask holds its own bit and its
 * ancestors' as linformer_tree_mask makes it; any other mask serves as well, one that leaves a row
 * empty among them.  nq up to LINFORMER_TREE_NODES (else LINFORMER_ERR_SIZE).
 */
LINFORMER_API int linformer_tree_attn_fwd(
    const void *Q, const int64_t *Q_strides, const void *K_pages, const int64_t *K_pages_strides,
    const void *V_pages, const int64_t *V_pages_strides, void *O, const int64_t *O_strides, float *lse,
    const int32_t *table, const int32_t *k_lengths, const int32_t *q_lengths, const uint64_t *mask,
    int b, int hq, int hk, int nq, int d, int pages, int page, int width, float scale, int dtype,
    void *stream);

/* mask[beta][i] for linformer_tree_attn_fwd, of trees given by each node's parent: device int32
 * dense [b][n], -1 for a root (a tree may have several), else a node before it (an entry that is
 * neither counts as a root and is recorded in the device status word).  n up to LINFORMER_TREE_NODES. */
LINFORMER_API int linformer_tree_mask(const int32_t *parents, uint64_t *mask, int b, int n, void *stream);

/* Calls that linformer_cache_packed makes. */
typedef enum {
    LINFORMER_PACKED_APPEND = 0, /* linformer_cache_append: 42 words */
    LINFORMER_PACKED_KEEP = 1,   /* linformer_cache_keep: 21 words */
    LINFORMER_PACKED_ATTN = 2,   /* linformer_paged_attn_fwd: 33 words */
    LINFORMER_PACKED_TREE = 3    /* linformer_tree_attn_fwd: 32 words */
} linformer_packed_call;

/*
 * The same calls with their arguments in one block of 64-bit words, for bindings that pay by the
 * argument.  The words follow the call's own order: a pointer its address, strides three words behind
 * their tensor's (always given; those of an absent tensor are not read), an integer its value (one
 * that an int does not hold: LINFORMER_ERR_SIZE), amplitude and scale the bits of a double.  count:
 * words in the block (else LINFORMER_ERR_VALUE).  The block is read before the call returns.
 */
LINFORMER_API int linformer_cache_packed(int call, const void *words, int count);

/*
 * Largest number of bytes the library's workspace pool on the current device has had
 * in use at once since the pool was created or last reset; reset != 0 then sets the
 * mark back to the bytes in use now.  Returns -1 if the pool cannot be queried.
 */
LINFORMER_API int64_t linformer_pool_peak_bytes(int reset);

/*
 * Pooling or convolution instead of a learned projection (요약 설명, section
 * "Additional Efficiency Techniques").  With s = n / k (n % k == 0), writes into the
 * caller's device buffer P, [k][n] in the input dtype (bf16 for LINFORMER_BF16 and
 * LINFORMER_BF16_F32OUT, fp32 for LINFORMER_F32), the map whose row j averages or
 * convolves the window of positions [j s, (j + 1) s):
 *   weights == NULL: mean pooling, P[j][j s + t] = 1 / s (rounded to the dtype);
 *   weights: device float[s], a convolution with kernel size = stride = s,
 *            P[j][j s + t] = weights[t];
 * every other entry 0.  Pass P as E (and F) of linformer_attn_fwd with a shared mode
 * (LAYERWISE, HEADWISE), or fill one [k][n] slice per head for the per-head modes.
 * Asynchronous on `stream`; P is owned by the caller.  Errors: LINFORMER_ERR_NULL,
 * LINFORMER_ERR_SIZE (n % k != 0 or a size < 1), LINFORMER_ERR_ENUM, LINFORMER_ERR_LAUNCH.
 */
LINFORMER_API int linformer_window_projection(void *P, const float *weights, int n, int k,
                                              int dtype, void *stream);

/* Which path (linformer_path_kind) a call with these arguments takes, or a
 * negative status if the arguments are invalid.  Host only; launches nothing. */
LINFORMER_API int linformer_select_path(int b, int h, int n, int d, int k, int share_mode, int dtype);

/* Human-readable text for a status code (static storage). */
LINFORMER_API const char *linformer_status_string(int status);

/* Synchronises `stream`, returns LINFORMER_ERR_DEVICE if a kernel of this library
 * recorded a device-side failure on the current device since the last read (and
 * clears it), else LINFORMER_OK.  For tests and debugging. */
LINFORMER_API int linformer_debug_read_device_status(void *stream);

/* Test of the device-side failure path: launches one warp on `stream` that waits,
 * through the same bounded wait as the kernels, on a barrier nothing completes.  After
 * the wait limit (2 s) the warp records a failure in the device status word and exits;
 * no fault, trap or hang.  Returns LINFORMER_OK once launched;
 * linformer_debug_read_device_status() then reports LINFORMER_ERR_DEVICE, and the
 * library keeps working on the same context.  For tests and debugging. */
LINFORMER_API int linformer_debug_wait_probe(void *stream);

/* Number of products in the P.Vbar step of the tensor-core path: 0 = chosen per
 * unit on the device from max|Vbar| (default: 1 below 24, 2 below 40, else 3),
 * 1 = one product (fp16 P, fp16 Vbar), 2 = P times the hi/lo split of Vbar,
 * 3 = three products (hi/lo splits of P and Vbar).  Process-wide setting for
 * tests and tuning; returns the previous value, or LINFORMER_ERR_ENUM. */
LINFORMER_API int linformer_set_pv_terms(int terms);

/* Number of kernels this library has launched in this process (all devices). */
LINFORMER_API int64_t linformer_launch_count(void);

/* Profiling: while enabled, every kernel launch is bracketed by CUDA events on
 * its own stream.  linformer_profile_collect() synchronises those events, adds
 * each kernel's total milliseconds and launch count into ms[id] and launches[id]
 * (arrays of LINFORMER_KERNEL_COUNT entries), and clears the record. */
LINFORMER_API int linformer_profile_enable(int enable);
LINFORMER_API int linformer_profile_collect(double *ms, int64_t *launches);

/* Name of a linformer_kernel_id (static storage), or NULL. */
LINFORMER_API const char *linformer_kernel_name(int id);

#ifdef __cplusplus
}
#endif

#endif /* LINFORMER_ATTN_H */
