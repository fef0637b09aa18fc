// Work items of the exact attention's persistent kernels, taken from a counter.
#pragma once

#include "sm100_ptx.cuh"

namespace linformer {
namespace sattn {

using namespace ptx;

// A CTA begins with the item of its number; the loading thread takes each further one from a
// counter and tells the other roles, two items ahead at most.  Which CTA computes an item does
// not change its result.  (Items differ in length, under a causal mask and with ragged
// lengths.  Taken in turn instead, item i by CTA i modulo the CTAs: backward of 32 causal heads
// over 8 of 8191 1424 us against 1353, of 32 ragged entries of 12 heads of 512 120 against 115;
// forward of 64 causal heads of 8192 887 and 782 to 824, with a window of 2048 246 and 226, one
// token over 8192 ragged keys 147 and 139.)
struct Queue {
    uint64_t full[2], free[2];
    int next[2];
};
__device__ __forceinline__ void init_queue(Queue &q, int readers) {
    for (int i = 0; i < 2; ++i) {
        mbar_init(&q.full[i], 1);
        mbar_init(&q.free[i], readers);
    }
}
__device__ __forceinline__ bool tell(Queue &q, int &t, int idx, int *status, volatile int *abort) {
    const int s = t & 1;
    if (!thread_spin(&q.free[s], ((t >> 1) & 1) ^ 1, status, 65, abort)) return false;
    *(volatile int *)&q.next[s] = idx;
    mbar_arrive(&q.full[s]);
    ++t;
    return true;
}
// A single thread's next item, and a warp's.
__device__ __forceinline__ bool thread_next(Queue &q, int &t, int &idx, int *status, volatile int *abort) {
    const int s = t & 1;
    if (!thread_spin(&q.full[s], (t >> 1) & 1, status, 66, abort)) return false;
    idx = *(volatile int *)&q.next[s];
    mbar_arrive(&q.free[s]);
    ++t;
    return true;
}
__device__ __forceinline__ bool warp_next(Queue &q, int &t, int &idx, int *status, volatile int *abort) {
    const int s = t & 1;
    if (!warp_spin(&q.full[s], (t >> 1) & 1, status, 67, abort)) return false;
    idx = *(volatile int *)&q.next[s];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&q.free[s]);
    ++t;
    return true;
}

}  // namespace sattn
}  // namespace linformer
