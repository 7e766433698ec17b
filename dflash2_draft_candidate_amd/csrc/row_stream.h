// Streaming over the whole vectors of a row slice (row_slices.h), for the passes that read every
// logit of a row and keep what they need of it in registers.
#pragma once

#include "device_common.h"
#include "row_slices.h"

namespace dflash2 {

constexpr int kStreamVectors = 4;  // 16-byte vectors per thread and batch

// Runs over a thread's share of n vectors at p (tid, tid + nt, ...): batches of
// kStreamVectors vectors with the next batch's loads in flight (batch(vectors, index of the
// first); the others follow NT apart), then the rest one by one (single(vector, index)).
template <int NT, typename FB, typename FV>
__device__ __forceinline__ void stream(const u32x4 *p, int n, int tid, FB &&batch, FV &&single) {
    const int whole = n / (NT * kStreamVectors);
    u32x4 cur[kStreamVectors], nxt[kStreamVectors];
    if (whole > 0) {
#pragma unroll
        for (int u = 0; u < kStreamVectors; ++u) cur[u] = p[tid + u * NT];
    }
    for (int b = 0; b < whole; ++b) {
        const int base = (b + 1) * NT * kStreamVectors + tid;
        if (b + 1 < whole) {
#pragma unroll
            for (int u = 0; u < kStreamVectors; ++u) nxt[u] = p[base + u * NT];
        }
        batch(cur, base - NT * kStreamVectors);
#pragma unroll
        for (int u = 0; u < kStreamVectors; ++u) cur[u] = nxt[u];
    }
    // the rest: at most kStreamVectors vectors per thread, loaded together
    const int base = whole * NT * kStreamVectors + tid;
#pragma unroll
    for (int u = 0; u < kStreamVectors; ++u)
        if (base + u * NT < n) cur[u] = p[base + u * NT];
#pragma unroll
    for (int u = 0; u < kStreamVectors; ++u)
        if (base + u * NT < n) single(cur[u], base + u * NT);
}

// Ragged element `tid` of a unit (its row's ends outside whole vectors): index, or -1.
__device__ __forceinline__ int64_t ragged_element(const UnitRange &u, int tid) {
    const int nh = (int)(u.h1 - u.h0);
    if (tid < nh) return u.h0 + tid;
    if (tid - nh < (int)(u.t1 - u.t0)) return u.t0 + (tid - nh);
    return -1;
}

}  // namespace dflash2
