// Streaming over the whole vectors of a row slice (row_slices.h), for the passes that read every
// logit of a row and keep what they need of it in registers.
#pragma once

#include "device_common.h"
#include "row_slices.h"

namespace dflash2 {

constexpr int kStreamVectors = 4;  // 16-byte vectors per thread and batch

// Runs over a thread's share of n vectors at p (tid, tid + NT, ...): batches of kStreamVectors
// vectors (batch(vectors, index of the first); the others follow NT apart), then the rest one by
// one (single(vector, index)). Two sets of registers take turns, so that the next batch is in
// flight while one is worked on; no load is conditional (a wait at the join of two paths must assume
// that the later loads are missing, and then waits for the ones in flight).
template <int NT, typename FB, typename FV>
__device__ __forceinline__ void stream(const u32x4 *p, int n, int tid, FB &&batch, FV &&single) {
    constexpr int kStep = NT * kStreamVectors;
    const int whole = n / kStep;
    u32x4 a[kStreamVectors], c[kStreamVectors];
    auto load = [&](u32x4 *v, int b) {
#pragma unroll
        for (int u = 0; u < kStreamVectors; ++u) v[u] = p[b * kStep + tid + u * NT];
    };
    const int base = whole * kStep + tid;
    auto load_rest = [&](u32x4 *v) {
#pragma unroll
        for (int u = 0; u < kStreamVectors; ++u)
            if (base + u * NT < n) v[u] = p[base + u * NT];
    };
    auto rest = [&](const u32x4 *v) {
#pragma unroll
        for (int u = 0; u < kStreamVectors; ++u)
            if (base + u * NT < n) single(v[u], base + u * NT);
    };
    if (whole == 0) {
        load_rest(a);
        rest(a);
        return;
    }
    load(a, 0);
    int b = 0;
    for (; b + 2 < whole; b += 2) {
        load(c, b + 1);
        batch(a, b * kStep + tid);
        load(a, b + 2);
        batch(c, (b + 1) * kStep + tid);
    }
    if (b + 2 == whole) {
        load(c, b + 1);
        batch(a, b * kStep + tid);
        load_rest(a);
        batch(c, (b + 1) * kStep + tid);
        rest(a);
    } else {
        load_rest(c);
        batch(a, b * kStep + tid);
        rest(c);
    }
}

// Ragged element `tid` of a unit (its row's ends outside whole vectors): index, or -1.
__device__ __forceinline__ int64_t ragged_element(const UnitRange &u, int tid) {
    const int nh = (int)(u.h1 - u.h0);
    if (tid < nh) return u.h0 + tid;
    if (tid - nh < (int)(u.t1 - u.t0)) return u.t0 + (tid - nh);
    return -1;
}

}  // namespace dflash2
