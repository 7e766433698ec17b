// Distillation of a drafter from its target's top logits: the loss of each row, its gradient, and
// both in one pass.
//
// Student logits z [R, V]; per row K teacher entries (id_j, t_j), as the top-k pass keeps them. With
//   p_j = softmax_j(t_j / tau) over the row's entries with an id in [0, V),
//   q_v = softmax_v(z_v / tau) over the whole vocabulary,
// the row's loss is tau^2 KL(p || q) and its gradient, for the gradient g of the row's loss,
//   loss = tau^2 sum_j p_j (ln p_j - ln q_{id_j}),
//   dz_v = g tau (q_v - sum_{j: id_j = v} p_j).
// (d ln q_j / dz_v = ([v = id_j] - q_v) / tau and the p_j add up to 1.)
//
// What is kept of a row between the passes is its maximum m and Sigma = sum_v exp((z_v - m) / tau):
// relative to the maximum, a 32-bit Sigma carries q to 2^-24 at any size of the logits, where a
// 32-bit logsumexp of large logits would not.
//
// Arithmetic. The row's exponentials and their sums are fp32 (base 2: v_exp_f32 of
// z s - ref with s = log2(e) / tau in one fma); a thread keeps the reference ref = m s of the largest
// element it has seen, moved once per batch of loads. ref is whatever fp32 number m s rounds to:
// the sums of threads, waves and slices are joined in terms of the rounded references, and the
// last step multiplies by 2^(ref - m s) in fp64, so that rounding cancels. Everything that happens
// once per row or per teacher entry is fp64 (the loss is a difference of logarithms, and at the
// teacher's ids the gradient is a difference of probabilities).
// A row with |m s| >= 2^23 (nothing but masks of the type's lowest value, infinities) has no such
// reference; it is summed again with exp2((z - m) s), which is exact there too.
//
// What bounds it: the reading (and writing) of the logits where rows are many; a batch of loads is in
// flight while one is worked on (row_stream.h). Forward, 1024 rows x 151936 bf16: 57 us, 5.4 TB/s.
// Backward, 512 x 262144: 107 us, 5.0 TB/s read and written. Step, 1024 x 151936: 151 us, 4096 x 151936:
// 512 us, 4.1 and 4.9 TB/s; a copy reaches 4.8. Few rows: launches and the chain of a row (16 rows x
// 151936 forward: 12 us, 11 of them the kernel).
#include <float.h>

#include "device_common.h"
#include "kernels.h"
#include "row_stream.h"

namespace dflash2 {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kU = kStreamVectors;
constexpr float kMaxRef = 8388608.f;  // 2^23: references stay within this, so each is within 0.5
                                      // of m s and 2^(m s - ref) cannot overflow
constexpr float kNoRef = -kMaxRef;    // reference before the first element
constexpr int kBufferWord3 = 0x00020000;  // gfx9-family buffer descriptor word 3 (raw data)
constexpr int kHeldRows = 128;   // rows from which on a step always holds a row in registers
// Vectors up to which a step reads its row twice: one launch, and the second read hits the cache. (Held
// rows just above, 10000 logits bf16: 1024 rows 22 us, 20 read twice; 4096 rows 50, 69.)
constexpr int kShortRow = 1024;
constexpr int kUnitVectors = 2 * kThreads;  // a slice holds at least this many vectors

// ---- element output ------------------------------------------------------------------------

template <typename T> struct Pack;
template <> struct Pack<float> {
    static __device__ __forceinline__ u32x4 vec(const float *v) {
        return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3])};
    }
    static __device__ __forceinline__ void one(float *p, float v) { *p = v; }
};
template <> struct Pack<uint16_t> {  // round to nearest even, once
    static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 h = {(__bf16)lo, (__bf16)hi};
        return __builtin_bit_cast(uint32_t, h);
    }
    static __device__ __forceinline__ u32x4 vec(const float *v) {
        return u32x4{pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])};
    }
    static __device__ __forceinline__ void one(uint16_t *p, float v) {
        *p = __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};

// ---- wave reductions in fp64 -----------------------------------------------------------------

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ double wave_max64(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o));
    return v;
}

// ---- a row's teacher entries, one per lane of a wave --------------------------------------------

struct Teacher {
    int id;    // -1: no entry on this lane
    double p;  // the entry's share of the row's teacher mass
    double ln_p;
    bool any;  // wave-uniform: the row has teacher mass
};

// Entry `lane` of a row: its id (-1: none) and t / tau.
__device__ __forceinline__ int teacher_entry(const int32_t *ids, const float *logits, int64_t row,
                                             int K, int V, double inv_tau, int lane, double &a) {
    a = -INFINITY;
    if (lane >= K) return -1;
    const int id = ids[row * K + lane];
    if (id < 0 || id >= V) return -1;
    a = (double)logits[row * K + lane] * inv_tau;
    return id;
}

// Whether the row has teacher mass (wave-uniform): an entry above -inf, or a NaN.
__device__ __forceinline__ bool teacher_any(const int32_t *ids, const float *logits, int64_t row,
                                            int K, int V, double inv_tau, int lane) {
    double a;
    teacher_entry(ids, logits, row, K, V, inv_tau, lane, a);
    return __ballot(a != -INFINITY) != 0ull;
}

__device__ __forceinline__ Teacher teacher_row(const int32_t *ids, const float *logits,
                                               int64_t row, int K, int V, double inv_tau,
                                               int lane) {
    Teacher t;
    double a;
    t.id = teacher_entry(ids, logits, row, K, V, inv_tau, lane, a);
    const double top = wave_max64(a);  // (ignores NaN; a NaN entry makes the sum NaN)
    t.any = __ballot(a != -INFINITY) != 0ull;
    const double e = t.id < 0 || !t.any ? 0.0 : exp(a - top);
    const double sum = wave_sum64(e);
    t.p = t.any ? e / sum : 0.0;
    t.ln_p = a - top - log(sum);
    return t;
}

// The row's loss from its statistics (wave-wide; the same value in every lane).
template <typename T>
__device__ __forceinline__ double row_loss(const Teacher &t, const T *student, int64_t row, int V,
                                           double m, double sigma, double tau) {
    if (!t.any) return 0.0;
    double term = 0.0;
    if (t.id >= 0 && t.p != 0.0) {
        const double z = (double)Elem<T>::load(student, row * V + t.id);
        const double ln_q = (z - m) / tau - log(sigma);
        term = t.p * (t.ln_p - (sigma == 0.0 ? -INFINITY : ln_q));
    }
    return tau * tau * wave_sum64(term);
}

// ---- row statistics ------------------------------------------------------------------------

struct Stat {
    float m;    // largest element
    float ref;  // log2-domain reference: fl(m s)
    float sum;  // sum of 2^(z s - ref)
};

template <int N>
__device__ __forceinline__ void stat_add(Stat &st, const float *x, float s) {
    float c = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) c = fmaxf(c, x[i]);
    st.m = fmaxf(st.m, c);
    const float ref = __builtin_amdgcn_fmed3f(c * s, st.ref, kMaxRef);  // max(st.ref, c s), capped
    float a0 = st.sum * __builtin_amdgcn_exp2f(st.ref - ref), a1 = 0.f, a2 = 0.f, a3 = 0.f;
    st.ref = ref;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        a0 += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], s, -ref));
        if (i + 1 < N) a1 += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i + 1], s, -ref));
        if (i + 2 < N) a2 += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i + 2], s, -ref));
        if (i + 3 < N) a3 += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i + 3], s, -ref));
    }
    st.sum = (a0 + a1) + (a2 + a3);
}

__device__ __forceinline__ void stat_join(Stat &a, const Stat &b) {
    a.m = fmaxf(a.m, b.m);
    const float r = fmaxf(a.ref, b.ref);
    a.sum = a.sum * __builtin_amdgcn_exp2f(a.ref - r) + b.sum * __builtin_amdgcn_exp2f(b.ref - r);
    a.ref = r;
}

// (a fixed tree: lane l joins l ^ 32, l ^ 16, ...)
__device__ __forceinline__ Stat wave_stat(Stat st) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const Stat b{__shfl_xor(st.m, o), __shfl_xor(st.ref, o), __shfl_xor(st.sum, o)};
        stat_join(st, b);
    }
    return st;
}

// The threads' statistics joined, in every thread.
template <int NT>
__device__ __forceinline__ Stat group_stat(Stat st, Stat *sh, int tid) {
    st = wave_stat(st);
    if ((tid & (kWave - 1)) == 0) sh[tid / kWave] = st;
    __syncthreads();
    st = sh[0];
#pragma unroll
    for (int w = 1; w < NT / kWave; ++w) stat_join(st, sh[w]);
    __syncthreads();
    return st;
}

// Statistics of a unit, in every thread. `sh` is scratch of kWaves entries; ends with a barrier.
template <typename T, int NT>
__device__ __forceinline__ Stat unit_stat(const T *student, const UnitRange &ur, float s, Stat *sh,
                                          int tid) {
    constexpr int EV = Elem<T>::kPerVec;
    Stat st{-INFINITY, kNoRef, 0.f};
    stream<NT>(
        reinterpret_cast<const u32x4 *>(student) + ur.c0, ur.nv, tid,
        [&](const u32x4 *v, int) {
            float x[kU * EV];
#pragma unroll
            for (int u = 0; u < kU; ++u) Elem<T>::unpack(v[u], x + u * EV);
            stat_add<kU * EV>(st, x, s);
        },
        [&](const u32x4 &v, int) {
            float x[EV];
            Elem<T>::unpack(v, x);
            stat_add<EV>(st, x, s);
        });
    const int64_t e = ragged_element(ur, tid);
    if (e >= 0) {
        const float x = Elem<T>::load(student, e);
        stat_add<1>(st, &x, s);
    }
    return group_stat<NT>(st, sh, tid);
}

// Sigma of a whole row without a usable reference, by one wave: the sum of exp2((z - m) s).
template <typename T>
__device__ __noinline__ double far_row_sum(const T *student, int64_t row, int V, float m, float s,
                                           int lane) {
    double sum = 0.0;
    constexpr int kAhead = 16;  // loads in flight per lane
    for (int v0 = lane; v0 < V; v0 += kAhead * kWave) {
        float x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            x[u] = Elem<T>::load(student, row * V + min(v0 + u * kWave, V - 1));
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (v0 + u * kWave < V) sum += (double)__builtin_amdgcn_exp2f((x[u] - m) * s);
    }
    return wave_sum64(sum);
}

// Sigma of a row from its joined statistics (one wave); NaN where the row holds a NaN or +inf, 0
// where it holds nothing above -inf.
template <typename T>
__device__ __forceinline__ double row_sigma(const Stat &st, const T *student, int64_t row, int V,
                                            float s, int lane) {
    // nothing moved the reference, so the sum is a NaN only if an element is
    if (st.m == -INFINITY) return st.sum != st.sum ? (double)st.sum : 0.0;
    if (!(fabsf(st.m * s) < kMaxRef)) return far_row_sum<T>(student, row, V, st.m, s, lane);
    return (double)st.sum * exp2((double)st.ref - (double)st.m * (double)s);
}

struct Args {
    const int32_t *ids;
    const float *teacher;
    int R, V, K;
    double tau, inv_tau;
    float s;  // log2(e) / tau
};

// Forward: a unit (row, slice) per workgroup. One slice: the row's statistics and loss at once;
// more: the slice's statistics go to `part` [R][S], joined by distill_join_kernel.
template <typename T>
__global__ __launch_bounds__(kThreads) void distill_forward_kernel(const T *__restrict__ student,
                                                                   Args a, int S,
                                                                   float *__restrict__ loss,
                                                                   float *__restrict__ row_stats,
                                                                   Stat *__restrict__ part) {
    __shared__ Stat sh[kWaves];
    const int tid = threadIdx.x;
    const UnitRange ur = unit_range(blockIdx.x, a.V, S, Elem<T>::kPerVec);
    const Stat st = unit_stat<T, kThreads>(student, ur, a.s, sh, tid);
    if (S > 1) {
        if (tid == 0) part[blockIdx.x] = st;
        return;
    }
    if (tid >= kWave) return;
    const int64_t row = blockIdx.x;
    const double sigma = row_sigma<T>(st, student, row, a.V, a.s, tid);
    const Teacher t = teacher_row(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, tid);
    const double l = row_loss<T>(t, student, row, a.V, (double)st.m, sigma, a.tau);
    if (tid == 0) {
        loss[row] = (float)l;
        row_stats[2 * row] = st.m;
        row_stats[2 * row + 1] = (float)sigma;
    }
}

// Joins the slices of a row and computes its loss: one wave per row.
template <typename T>
__global__ __launch_bounds__(kWave) void distill_join_kernel(const T *__restrict__ student, Args a,
                                                             int S, const Stat *__restrict__ part,
                                                             float *__restrict__ loss,
                                                             float *__restrict__ row_stats) {
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    const Teacher t = teacher_row(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, lane);
    Stat st{-INFINITY, kNoRef, 0.f};
    for (int i = lane; i < S; i += kWave) stat_join(st, part[row * S + i]);
    st = wave_stat(st);
    const double sigma = row_sigma<T>(st, student, row, a.V, a.s, lane);
    const double l = row_loss<T>(t, student, row, a.V, (double)st.m, sigma, a.tau);
    if (lane == 0) {
        loss[row] = (float)l;
        row_stats[2 * row] = st.m;
        row_stats[2 * row + 1] = (float)sigma;
    }
}

// ---- gradient ------------------------------------------------------------------------------

// The gradient at the teacher's ids of one row, a value per lane; lanes whose id a lower lane
// holds too, and lanes without an entry, get id -1. Computed in fp64 from the stored logit.
struct Patch {
    int id;
    float value;
};

template <typename T>
__device__ __forceinline__ Patch teacher_patch(const Teacher &t, const T *student, int64_t row,
                                               int V, int K, double m, double sigma, double g,
                                               double tau, int lane) {
    Patch out{-1, 0.f};
    double p = 0.0;
    bool first = true;
    for (int i = 0; i < K; ++i) {
        const int id = __builtin_amdgcn_readlane(t.id, i);
        const double pi = __shfl(t.p, i);
        if (id == t.id) {
            p += pi;
            if (i < lane) first = false;
        }
    }
    if (t.id >= 0 && first && t.any) {
        const double z = (double)Elem<T>::load(student, row * V + t.id);
        const double q = sigma == 0.0 ? 0.0 : exp((z - m) / tau) / sigma;
        out.id = t.id;
        out.value = sigma == 0.0 ? 0.f : (float)(g * tau * (q - p));
    }
    return out;
}

// dz over a unit's elements as if no teacher entry were there: coef 2^((z - m) s), coef = g tau /
// Sigma; zeros where `live` is false. The difference to the maximum comes first: it is exact where
// q is large.
template <typename T, int NT>
__device__ __forceinline__ void unit_gradient(const T *student, const UnitRange &ur, float m,
                                              float s, float coef, bool live, T *grad, int tid) {
    constexpr int EV = Elem<T>::kPerVec;
    u32x4 *out = reinterpret_cast<u32x4 *>(grad) + ur.c0;
    if (!live) {
        for (int i = tid; i < ur.nv; i += NT) out[i] = u32x4{0u, 0u, 0u, 0u};
        const int64_t e = ragged_element(ur, tid);
        if (e >= 0) Pack<T>::one(grad + e, 0.f);
        return;
    }
    auto one = [&](const u32x4 &v, int i) {
        float x[EV];
        Elem<T>::unpack(v, x);
#pragma unroll
        for (int k = 0; k < EV; ++k) x[k] = coef * __builtin_amdgcn_exp2f((x[k] - m) * s);
        out[i] = Pack<T>::vec(x);
    };
    stream<NT>(
        reinterpret_cast<const u32x4 *>(student) + ur.c0, ur.nv, tid,
        [&](const u32x4 *v, int i) {
#pragma unroll
            for (int u = 0; u < kU; ++u) one(v[u], i + u * NT);
        },
        one);
    const int64_t e = ragged_element(ur, tid);
    if (e >= 0)
        Pack<T>::one(grad + e,
                     coef * __builtin_amdgcn_exp2f((Elem<T>::load(student, e) - m) * s));
}

// The element range of a unit, ragged ends included.
__device__ __forceinline__ bool unit_holds(const UnitRange &u, int64_t e, int EV) {
    const int64_t v0 = u.c0 * EV;
    return (e >= v0 && e < v0 + (int64_t)u.nv * EV) || (e >= u.h0 && e < u.h1) ||
           (e >= u.t0 && e < u.t1);
}

// Backward: a unit (row, slice) per workgroup. Wave 0 prepares the values at the teacher's ids
// while the others start to stream; after the barrier they overwrite what the stream put there.
template <typename T>
__global__ __launch_bounds__(kThreads) void distill_backward_kernel(
    const T *__restrict__ student, Args a, int S, const float *__restrict__ row_stats,
    const float *__restrict__ grad_loss, T *__restrict__ grad) {
    const int tid = threadIdx.x;
    const UnitRange ur = unit_range(blockIdx.x, a.V, S, Elem<T>::kPerVec);
    const int64_t row = (uint32_t)blockIdx.x / (uint32_t)S;
    const float m = row_stats[2 * row], sigma = row_stats[2 * row + 1], g = grad_loss[row];
    Patch patch{-1, 0.f};
    const int lane = tid & (kWave - 1);
    const bool live =
        teacher_any(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, lane) && sigma != 0.f;
    if (tid < kWave) {
        const Teacher t = teacher_row(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, lane);
        patch = teacher_patch<T>(t, student, row, a.V, a.K, (double)m, (double)sigma, (double)g,
                                 a.tau, lane);
    }
    const float coef = (float)((double)g * a.tau / (double)sigma);
    unit_gradient<T, kThreads>(student, ur, m, a.s, coef, live, grad, tid);
    __syncthreads();
    if (patch.id >= 0 && unit_holds(ur, row * a.V + patch.id, Elem<T>::kPerVec))
        Pack<T>::one(grad + row * a.V + patch.id, patch.value);
}

// Loss and gradient: a row per workgroup, read twice (the second time mostly from cache).
template <typename T>
__global__ __launch_bounds__(kThreads) void distill_step_kernel(
    const T *__restrict__ student, Args a, const float *__restrict__ grad_loss,
    float *__restrict__ loss, T *__restrict__ grad) {
    __shared__ Stat sh[kWaves];
    __shared__ double sh_sigma;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const UnitRange ur = unit_range(row, a.V, 1, Elem<T>::kPerVec);
    const Stat st = unit_stat<T, kThreads>(student, ur, a.s, sh, tid);
    const int lane = tid & (kWave - 1);
    const bool any = teacher_any(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, lane);
    const float g = grad_loss[row];
    Patch patch{-1, 0.f};
    if (tid < kWave) {
        const Teacher t = teacher_row(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, lane);
        const double sigma = row_sigma<T>(st, student, row, a.V, a.s, lane);
        const double l = row_loss<T>(t, student, row, a.V, (double)st.m, sigma, a.tau);
        if (lane == 0) {
            loss[row] = (float)l;
            sh_sigma = sigma;
        }
        patch = teacher_patch<T>(t, student, row, a.V, a.K, (double)st.m, sigma, (double)g, a.tau,
                                 lane);
    }
    __syncthreads();
    const double sigma = sh_sigma;
    const bool live = any && sigma != 0.0;
    const float coef = (float)((double)g * a.tau / sigma);
    unit_gradient<T, kThreads>(student, ur, st.m, a.s, coef, live, grad, tid);
    __syncthreads();
    if (patch.id >= 0) Pack<T>::one(grad + row * a.V + patch.id, patch.value);
}

// Statistics and gradient of long rows: a row per workgroup of NT threads, NV vectors of it per thread
// held in registers between the two passes, so that they come from memory once. What does not fit
// (`rest`: the row's first vectors) is streamed and read again. All fp32, and without the teacher's
// entries: the fp64 work for those (distill_finish_kernel) would cost the registers that hold the row.
// Against distill_step_kernel's two reads (us, bf16): 4096 rows x 10000 50 / 69, 1024 x 50021 49 / 52,
// 1024 x 70000 66 / 80, 1024 x 100001 115 / 115, 1024 x 151936 151 / 180, 4096 x 151936 512 / 734,
// 1024 x 262144 280 / 298, 1024 x 400000 446 / 486; float32: 1024 x 17000 27 / 37, 1024 x 50021
// 97 / 122, 1024 x 151936 302 / 374.
template <typename T, int NT, int NV>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(4))) void
distill_held_kernel(const T *__restrict__ student, Args a, const float *__restrict__ grad_loss,
                    Stat *__restrict__ stats, T *__restrict__ grad) {
    constexpr int EV = Elem<T>::kPerVec;
    __shared__ Stat sh[NT / kWave];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const UnitRange ur = unit_range(row, a.V, 1, EV);
    const int rest = max(ur.nv - NV * NT, 0), held = ur.nv - rest;
    const u32x4 *p = reinterpret_cast<const u32x4 *>(student) + ur.c0 + rest;
    u32x4 *out = reinterpret_cast<u32x4 *>(grad) + ur.c0 + rest;
    // (Buffer accesses: 32-bit offsets, and what lies past the row's end is neither read nor stored.
    // A vector's place is all in the vector offset, because a scalar offset is not part of the check.)
    const __amdgpu_buffer_rsrc_t src = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<u32x4 *>(p), 0, held * 16, kBufferWord3);
    const __amdgpu_buffer_rsrc_t dst =
        __builtin_amdgcn_make_buffer_rsrc(out, 0, held * 16, kBufferWord3);
    u32x4 v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        v[j] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(src, (tid + j * NT) * 16, 0, 0));
    const int64_t e = ragged_element(ur, tid);
    const float end = e >= 0 ? Elem<T>::load(student, e) : -INFINITY;
    const float g = grad_loss[row];
    const bool any = teacher_any(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, tid & (kWave - 1));
    Stat st{-INFINITY, kNoRef, 0.f};
    // f(elements of vectors j, j + 1; how many of the two the row has) over the held vectors
    auto pairs = [&](auto &&f) {
#pragma unroll
        for (int j = 0; j < NV; j += 2) {
            // (a new value to the compiler: it would keep the widened logits from pass to pass, twice
            // the registers, to save widening them again; and unpacked ahead of their turn they
            // would not fit either)
            asm("" : "+v"(v[j]), "+v"(v[j + 1]));
            float x[2 * EV];
            Elem<T>::unpack(v[j], x);
            Elem<T>::unpack(v[j + 1], x + EV);
            f(j, x, tid + (j + 1) * NT < held ? 2 : tid + j * NT < held ? 1 : 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    pairs([&](int, const float *x, int n) {
        if (n == 2)
            stat_add<2 * EV>(st, x, a.s);
        else if (n == 1)
            stat_add<EV>(st, x, a.s);
    });
    for (int i = tid - rest; i < 0; i += NT) {
        float x[EV];
        Elem<T>::unpack(p[i], x);
        stat_add<EV>(st, x, a.s);
    }
    if (e >= 0) stat_add<1>(st, &end, a.s);
    st = group_stat<NT>(st, sh, tid);
    if (tid == 0) stats[row] = st;
    const float m = st.m;
    float sigma = st.sum * __builtin_amdgcn_exp2f(__builtin_fmaf(-m, a.s, st.ref));
    if (m > -INFINITY && !(fabsf(m * a.s) < kMaxRef)) {  // no reference: from the differences
        Stat far{m, 0.f, 0.f};
        auto add = [&](float x) { far.sum += __builtin_amdgcn_exp2f((x - m) * a.s); };
        pairs([&](int, const float *x, int n) {
#pragma unroll
            for (int k = 0; k < 2 * EV; ++k)
                if (k < n * EV) add(x[k]);
        });
        for (int i = tid - rest; i < 0; i += NT) {
            float x[EV];
            Elem<T>::unpack(p[i], x);
#pragma unroll
            for (int k = 0; k < EV; ++k) add(x[k]);
        }
        if (e >= 0) add(end);
        sigma = group_stat<NT>(far, sh, tid).sum;
    }
    // (nothing above -inf: the sum is 0, or NaN if the row holds one)
    const bool live = any && (m > -INFINITY || st.sum != st.sum);
    // (g tau / sigma from mantissas and exponents: g tau alone may pass the largest number)
    const float tau = (float)a.tau;
    const float coef =
        live ? __builtin_amdgcn_ldexpf(__builtin_amdgcn_frexp_mantf(g) *
                                           __builtin_amdgcn_frexp_mantf(tau) / sigma,
                                       __builtin_amdgcn_frexp_expf(g) + __builtin_amdgcn_frexp_expf(tau))
             : 0.f;
    auto gradient = [&](float *x) {
#pragma unroll
        for (int k = 0; k < EV; ++k)
            x[k] = live ? coef * __builtin_amdgcn_exp2f((x[k] - m) * a.s) : 0.f;
        return Pack<T>::vec(x);
    };
    int at = tid * 16;
    asm("" : "+v"(at));  // (the loads' offsets would be kept for the stores otherwise)
    pairs([&](int j, float *x, int) {
        // (With a scalar offset, moreover, the compiler lets the instruction after a 16-byte store
        // overwrite the first stored register, and stores with a logit difference in that word have
        // been seen.)
        __builtin_amdgcn_raw_buffer_store_b128(gradient(x), dst, at + j * NT * 16, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(gradient(x + EV), dst, at + (j + 1) * NT * 16, 0, 0);
    });
    for (int i = tid - rest; i < 0; i += NT) {
        float x[EV];
        Elem<T>::unpack(p[i], x);
        out[i] = gradient(x);
    }
    if (e >= 0)
        Pack<T>::one(grad + e, live ? coef * __builtin_amdgcn_exp2f((end - m) * a.s) : 0.f);
}

// The loss of a row, and its gradient at the teacher's ids: one wave per row, after
// distill_held_kernel.
template <typename T>
__global__ __launch_bounds__(kWave) void distill_finish_kernel(const T *__restrict__ student,
                                                               Args a,
                                                               const float *__restrict__ grad_loss,
                                                               const Stat *__restrict__ stats,
                                                               float *__restrict__ loss,
                                                               T *__restrict__ grad) {
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    const Stat st = stats[row];
    const Teacher t = teacher_row(a.ids, a.teacher, row, a.K, a.V, a.inv_tau, lane);
    const double sigma = row_sigma<T>(st, student, row, a.V, a.s, lane);
    const double l = row_loss<T>(t, student, row, a.V, (double)st.m, sigma, a.tau);
    if (lane == 0) loss[row] = (float)l;
    const Patch patch = teacher_patch<T>(t, student, row, a.V, a.K, (double)st.m, sigma,
                                         (double)grad_loss[row], a.tau, lane);
    if (patch.id >= 0) Pack<T>::one(grad + row * a.V + patch.id, patch.value);
}

template <typename T, int NT, int NV>
hipError_t held(const T *x, const Args &a, const float *grad_loss, float *loss, T *grad, void *ws,
                hipStream_t stream) {
    Stat *stats = static_cast<Stat *>(ws);
    hipLaunchKernelGGL((distill_held_kernel<T, NT, NV>), dim3((unsigned)a.R), dim3(NT), 0, stream, x,
                       a, grad_loss, stats, grad);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((distill_finish_kernel<T>), dim3((unsigned)a.R), dim3(kWave), 0, stream, x, a,
                       grad_loss, stats, loss, grad);
    return hipGetLastError();
}

Args make_args(const int32_t *ids, const float *teacher, int R, int V, int K, float tau) {
    Args a;
    a.ids = ids;
    a.teacher = teacher;
    a.R = R;
    a.V = V;
    a.K = K;
    a.tau = (double)tau;
    a.inv_tau = 1.0 / (double)tau;
    a.s = (float)(1.4426950408889634 / (double)tau);
    return a;
}

// Slices per row where rows are cut: enough units to fill the chip (1024 workgroups) when rows are
// few, each of at least kUnitVectors vectors.
int plan_slices(int R, int V, int elem_bytes) {
    const int64_t nvec = (int64_t)V * elem_bytes / 16;
    int64_t s = (1024 + R - 1) / R;
    const int64_t most = nvec / kUnitVectors;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

// Slices per row of the forward pass: 1 where the row is short for the number of rows, as a second
// kernel has to join slices. Measured in a graph, one workgroup per row against slices (us, bf16):
// V = 32000: 1 row 6.4 / 7.4, 128 rows 7.2 / 9.6; V = 100001: 16 rows 9.4 / 8.1, 48 rows 9.7 / 10.9;
// V = 200003: 48 rows 13.9 / 13.7, 128 rows 15.0 / 17.1; V = 500000: 48 rows 26.3 / 17.9, 128 rows
// 32.3 / 31.6; V = 151936: 256 rows 17.3 / 21.1, 512 rows 29.0 / 32.6 (float32: the same borders).
// By itself the second launch also costs the host 2.6 us, more than slices save up to V = 160000:
// 16 rows x 151936 take 12.5 us in one launch, 15.1 in two (11.3 and 9.0 in a graph).
int forward_slices(int R, int V, int elem_bytes, bool alone) {
    int64_t most = 50000 + 2500 * (int64_t)R;
    if (alone && most < 160000) most = 160000;
    return V <= most ? 1 : plan_slices(R, V, elem_bytes);
}

// Whether a step holds its rows in registers (distill_held_kernel, a workgroup per row) or runs forward
// and backward pass one after the other (rows cut into slices, at least by the latter). Held against
// the two passes (us, in a graph, bf16): V = 32000: 16 rows 12.2 / 11.9, 100 rows 13.4 / 14.9;
// V = 65536: 16 rows 15.5 / 13.2, 100 rows 18.1 / 20.4; V = 151936: 100 rows 29.7 / 27.8, 128 rows
// 31.6 / 29, 200 rows 33.8 / 41, 512 rows 82 / 103; V = 262144: 512 rows 149 / 164. float32: V = 10000:
// 1 row 8.8 / 10.3; V = 32000: 64 rows 13.4 / 15.1; V = 151936: 127 rows 46.9 / 48.4.
bool held_step(int R, int V, int elem_bytes) {
    return R >= kHeldRows || V <= 40000 + 300 * R || plan_slices(R, V, elem_bytes) == 1;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <typename T>
hipError_t forward(const void *student, const Args &a, bool alone, float *loss, float *row_stats,
                   void *ws, hipStream_t stream) {
    const int S = forward_slices(a.R, a.V, (int)sizeof(T), alone);
    const T *x = static_cast<const T *>(student);
    Stat *part = static_cast<Stat *>(ws);
    hipLaunchKernelGGL((distill_forward_kernel<T>), dim3((unsigned)(a.R * (int64_t)S)),
                       dim3(kThreads), 0, stream, x, a, S, loss, row_stats, part);
    if (S > 1)
        hipLaunchKernelGGL((distill_join_kernel<T>), dim3((unsigned)a.R), dim3(kWave), 0, stream, x,
                           a, S, part, loss, row_stats);
    return hipGetLastError();
}

template <typename T>
hipError_t backward(const void *student, const Args &a, const float *row_stats,
                    const float *grad_loss, void *grad, hipStream_t stream) {
    const int S = plan_slices(a.R, a.V, (int)sizeof(T));
    hipLaunchKernelGGL((distill_backward_kernel<T>), dim3((unsigned)(a.R * (int64_t)S)),
                       dim3(kThreads), 0, stream, static_cast<const T *>(student), a, S, row_stats,
                       grad_loss, static_cast<T *>(grad));
    return hipGetLastError();
}

template <typename T>
hipError_t step(const void *student, const Args &a, const float *grad_loss, float *loss, void *grad,
                void *ws, hipStream_t stream) {
    if (held_step(a.R, a.V, (int)sizeof(T))) {
        const T *x = static_cast<const T *>(student);
        T *out = static_cast<T *>(grad);
        // The smallest shape that holds the row (at most 128 registers a thread: 1024 threads a CU),
        // so that short rows share a CU; the largest one also takes what none holds.
        const int n = (int)((int64_t)a.V * (int)sizeof(T) / 16);  // vectors of a row
        if (n > 16 * 1024) return held<T, 1024, 20>(x, a, grad_loss, loss, out, ws, stream);
        if (n > 12 * 1024) return held<T, 1024, 16>(x, a, grad_loss, loss, out, ws, stream);
        if (n > 20 * 512) return held<T, 1024, 12>(x, a, grad_loss, loss, out, ws, stream);
        if (n > 16 * 512) return held<T, 512, 20>(x, a, grad_loss, loss, out, ws, stream);
        if (n > 12 * 512) return held<T, 512, 16>(x, a, grad_loss, loss, out, ws, stream);
        if (n > 20 * 256) return held<T, 512, 12>(x, a, grad_loss, loss, out, ws, stream);
        if (n > 16 * 256) return held<T, 256, 20>(x, a, grad_loss, loss, out, ws, stream);
        if (n > 12 * 256) return held<T, 256, 16>(x, a, grad_loss, loss, out, ws, stream);
        if (n > kShortRow) return held<T, 256, 12>(x, a, grad_loss, loss, out, ws, stream);
        hipLaunchKernelGGL((distill_step_kernel<T>), dim3((unsigned)a.R), dim3(kThreads), 0, stream,
                           x, a, grad_loss, loss, out);
        return hipGetLastError();
    }
    float *row_stats = static_cast<float *>(ws);
    char *part = static_cast<char *>(ws) + align256((size_t)a.R * 2 * sizeof(float));
    const hipError_t e = forward<T>(student, a, false, loss, row_stats, part, stream);
    if (e != hipSuccess) return e;
    return backward<T>(student, a, row_stats, grad_loss, grad, stream);
}

}  // namespace

size_t distill_workspace_bytes(int R, int V, int elem_bytes) {
    const int S = plan_slices(R, V, elem_bytes);
    if (S == 1) return align256((size_t)R * sizeof(Stat));  // of distill_held_kernel
    // row_stats of a step's two passes and the slices' statistics (more than the held kernel needs)
    return align256((size_t)R * 2 * sizeof(float)) + align256((size_t)R * S * sizeof(Stat));
}

hipError_t launch_distill(const void *student, int dtype, const int32_t *ids, const float *teacher,
                          int R, int V, int K, float tau, float *loss, float *row_stats, void *ws,
                          hipStream_t stream) {
    const Args a = make_args(ids, teacher, R, V, K, tau);
    return dtype == 0 ? forward<float>(student, a, true, loss, row_stats, ws, stream)
                      : forward<uint16_t>(student, a, true, loss, row_stats, ws, stream);
}

hipError_t launch_distill_backward(const void *student, int dtype, const int32_t *ids,
                                   const float *teacher, const float *row_stats,
                                   const float *grad_loss, int R, int V, int K, float tau,
                                   void *grad, hipStream_t stream) {
    const Args a = make_args(ids, teacher, R, V, K, tau);
    return dtype == 0 ? backward<float>(student, a, row_stats, grad_loss, grad, stream)
                      : backward<uint16_t>(student, a, row_stats, grad_loss, grad, stream);
}

hipError_t launch_distill_step(const void *student, int dtype, const int32_t *ids,
                               const float *teacher, const float *grad_loss, int R, int V, int K,
                               float tau, float *loss, void *grad, void *ws, hipStream_t stream) {
    const Args a = make_args(ids, teacher, R, V, K, tau);
    return dtype == 0 ? step<float>(student, a, grad_loss, loss, grad, ws, stream)
                      : step<uint16_t>(student, a, grad_loss, loss, grad, ws, stream);
}

}  // namespace dflash2
