// The global norm over many gradients, and the gradients clipped by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g min(1, max_norm / norm)
//
// Design (gfx950):
//   * The tensors' addresses and sizes travel as kernel arguments, kNormTensors a launch: nothing is
//     copied to the device, and a captured launch holds them. A tensor is cut into chunks of one
//     length; workgroups take chunks in turn and find a chunk's tensor by a binary search over the
//     tensors' first chunks.
//   * Squares are added in 64 bits (no square of a finite float leaves them, and the sum of a
//     billion keeps its digits): one partial sum per workgroup, joined in a fixed order.
//   * Clipping is one more launch: every workgroup adds up the partial sums itself (at most
//     kNormPartials, from L2) rather than wait for a kernel that would. It takes the chunks in the
//     opposite order, so that what the norm's pass read last comes from a cache. Where nothing is to
//     be scaled and the output is the gradient itself, it ends there.
//   * Tensors may start at any element: 16-byte accesses need no alignment here.
//   * Both passes are bound by the bytes: 68 bf16 and f32 tensors of 1.11 billion elements (2.2 GB), the norm
//     409 us (5.4 TB/s), clipping 841 us (5.3 TB/s read and written). 400 tensors of 58 million: 46 and
//     82 us in four launches each, less than the host needs to hand 800 tensors over; 20 of 8192: 4.1
//     and 4.7 us, latency. From about 1000 tensors on a launch has fewer workgroups than it could use
//     (kNormPartials).
#include <float.h>
#include <math.h>

#include <type_traits>

#include "device_common.h"
#include "kernels.h"

namespace dflash2 {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormTensors = 128;    // per launch
// Partial sums, all launches together, which share them evenly: a launch's workgroups in either pass. Norm, and
// norm with clipping, with 1024, 2048 and 8192: 68 tensors of 16 million 367, 383, 375 us and 1219, 1228, 1194; 400
// of 145 000, 48, 44, 41 and 102, 98, 95; 1000 of 100 000, 124, 82, 67 and 316, 229, 216; 2000 of 100 000, 510,
// 296, 150 and 1132, 706, 517 (on the GPU; the host takes about 0.6 us a tensor beside it).
constexpr int kNormPartials = 2048;
constexpr int kNormUnit = 2048;      // elements: a workgroup's step
// A chunk. Norm, and norm with clipping, with 8192, 32768 and 131072: 68 tensors of 16 million 385, 383, 380 us
// and 1237, 1228, 1253; 1000 of 100 000, 106, 82, 88 and 272, 229, 276.
constexpr int kNormLongest = 32768;

struct NormBatch {
    const void *grad[kNormTensors];
    int64_t size[kNormTensors];
    int32_t first[kNormTensors];  // the tensor's first chunk
    uint32_t wide[kNormTensors / 32];  // a bit per tensor: float
    int count, chunks, length;         // tensors; chunks; elements of a chunk
};
struct NormOut {
    void *out[kNormTensors];
};
static_assert(sizeof(NormBatch) + sizeof(NormOut) + 64 < 4096, "kernel arguments");

// 16 bytes at any element's address
struct __attribute__((packed, aligned(2))) Bytes16 { u32x4 v; };

template <typename T> __device__ __forceinline__ u32x4 load16(const T *p) {
    return reinterpret_cast<const Bytes16 *>(p)->v;
}
template <typename T> __device__ __forceinline__ void store16(T *p, u32x4 v) {
    reinterpret_cast<Bytes16 *>(p)->v = v;
}

// The tensor of a chunk: the last one whose first chunk is not behind it.
__device__ __forceinline__ int tensor_of(const NormBatch &b, int chunk) {
    int lo = 0, hi = b.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (b.first[mid] <= chunk) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, kWave);
    return x;
}

// The sum over the workgroup, in every thread.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kNormThreads / kWave];
    x = wave_sum64(x);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = x;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kNormThreads / kWave; ++w) s += part[w];
    return s;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int n) {
    constexpr int kPer = 16 / (int)sizeof(T);
    constexpr int kAhead = 4;  // loads in flight per thread
    double s[2] = {0.0, 0.0};
    int i = threadIdx.x * kPer;
    for (; i + ((kAhead - 1) * kNormThreads + 1) * kPer <= n; i += kAhead * kNormThreads * kPer) {
        u32x4 v[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) v[a] = load16(p + i + a * kNormThreads * kPer);
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            float x[kPer];
            Elem<T>::unpack(v[a], x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) s[e & 1] = fma((double)x[e], (double)x[e], s[e & 1]);
        }
    }
    for (; i + kPer <= n; i += kNormThreads * kPer) {
        float x[kPer];
        Elem<T>::unpack(load16(p + i), x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) s[e & 1] = fma((double)x[e], (double)x[e], s[e & 1]);
    }
    for (int e = i; e < n && e < i + kPer; ++e) {
        const double x = Elem<T>::load(p, e);
        s[0] = fma(x, x, s[0]);
    }
    return s[0] + s[1];
}

__global__ __launch_bounds__(kNormThreads) void grad_norm_kernel(NormBatch b, double *partial) {
    double s = 0.0;
    for (int c = blockIdx.x; c < b.chunks; c += gridDim.x) {
        const int t = tensor_of(b, c);
        const int64_t at = (int64_t)(c - b.first[t]) * b.length, left = b.size[t] - at;
        const int n = (int)(left < b.length ? left : b.length);
        if ((b.wide[t / 32] >> (t % 32)) & 1u)
            s += chunk_squares(static_cast<const float *>(b.grad[t]) + at, n);
        else
            s += chunk_squares(static_cast<const uint16_t *>(b.grad[t]) + at, n);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the partial sums; the same in every workgroup.
__device__ __forceinline__ double norm_of(const double *partial, int n) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kNormThreads) s += partial[i];
    return sqrt(block_sum(s));
}

__global__ __launch_bounds__(kNormThreads) void grad_norm_out_kernel(const double *partial, int n,
                                                                     float *norm) {
    const double x = norm_of(partial, n);
    if (threadIdx.x == 0) *norm = (float)x;
}

// F: float, or double for factors below the normal floats (chunk_scale).
template <typename T, typename F>
__device__ __forceinline__ u32x4 scaled(u32x4 v, F f) {
    float x[Elem<T>::kPerVec];
    Elem<T>::unpack(v, x);
#pragma unroll
    for (int e = 0; e < Elem<T>::kPerVec; ++e) x[e] = (float)((F)x[e] * f);
    if constexpr (sizeof(T) == 4) {
        return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                     __float_as_uint(x[3])};
    } else {
        bf16x8 y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (__bf16)x[e];
        return __builtin_bit_cast(u32x4, y);
    }
}

// (The product is rounded to fp32 and then to bf16: 2^-24 on top of the 2^-8.)
template <typename T, typename F>
__device__ __forceinline__ void chunk_scale(const T *p, T *out, int n, F f) {
    constexpr int kPer = 16 / (int)sizeof(T);
    constexpr int kAhead = 4;
    int i = threadIdx.x * kPer;
    for (; i + ((kAhead - 1) * kNormThreads + 1) * kPer <= n; i += kAhead * kNormThreads * kPer) {
        u32x4 v[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) v[a] = load16(p + i + a * kNormThreads * kPer);
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            store16(out + i + a * kNormThreads * kPer, scaled<T>(v[a], f));
    }
    for (; i + kPer <= n; i += kNormThreads * kPer) store16(out + i, scaled<T>(load16(p + i), f));
    for (int e = i; e < n && e < i + kPer; ++e) {
        const float y = (float)((F)Elem<T>::load(p, e) * f);
        if constexpr (sizeof(T) == 4)
            out[e] = y;
        else
            *reinterpret_cast<__bf16 *>(out + e) = (__bf16)y;
    }
}

__global__ __launch_bounds__(kNormThreads) void clip_grads_kernel(NormBatch b, NormOut o,
                                                                  const double *partial,
                                                                  int partials, float max_norm,
                                                                  float *norm) {
    const double x = norm_of(partial, partials);
    const float xf = (float)x;
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = xf;
    // (a norm that is not finite scales nothing)
    const bool clips = xf > max_norm && xf < INFINITY;
    const double f = clips ? (double)max_norm / x : 1.0;
    for (int i = blockIdx.x; i < b.chunks; i += gridDim.x) {
        const int c = b.chunks - 1 - i, t = tensor_of(b, c);
        if (!clips && o.out[t] == b.grad[t]) continue;
        const int64_t at = (int64_t)(c - b.first[t]) * b.length, left = b.size[t] - at;
        const int n = (int)(left < b.length ? left : b.length);
        const auto scale = [&](auto *out) {
            const auto *p = static_cast<const std::remove_pointer_t<decltype(out)> *>(b.grad[t]) + at;
            // (a factor that is no normal float, as of a norm of 1e36 and a limit of 1e-9, would lose
            // its digits as one, and every result with it)
            if (f < (double)FLT_MIN)
                chunk_scale(p, out + at, n, f);
            else
                chunk_scale(p, out + at, n, (float)f);
        };
        if ((b.wide[t / 32] >> (t % 32)) & 1u)
            scale(static_cast<float *>(o.out[t]));
        else
            scale(static_cast<uint16_t *>(o.out[t]));
    }
}

}  // namespace

size_t grad_norm_workspace_bytes() { return kNormPartials * sizeof(double); }

hipError_t launch_clip_grads(const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                             int count, void *const *out, float max_norm, float *norm, void *ws,
                             hipStream_t stream) {
    double *partial = static_cast<double *>(ws);
    int64_t total = 0;
    int used = 0;
    for (int i = 0; i < count; ++i) {
        total += sizes[i];
        used += sizes[i] > 0;
    }
    const int launches = (used + kNormTensors - 1) / kNormTensors;
    // a chunk: long enough for full workgroups, short enough to fill the chip; (with a cap on the
    // workgroups of a launch, so that the partial sums of all of them fit)
    int64_t length = total / 1024 / kNormUnit * kNormUnit;
    length = length < kNormUnit ? kNormUnit : length > kNormLongest ? kNormLongest : length;
    const int most = launches > 0 ? kNormPartials / launches : 0;
    if (launches > kNormPartials) return hipErrorInvalidValue;  // (the caller refuses such a count)
    int partials = 0;
    for (int pass = 0; pass < (out ? 2 : 1); ++pass) {
        int next = 0;
        for (int l = 0; l < launches; ++l) {
            NormBatch b = {};
            NormOut o = {};
            int64_t chunks = 0;
            for (; next < count && b.count < kNormTensors; ++next) {
                if (sizes[next] == 0) continue;
                b.grad[b.count] = grads[next];
                if (out) o.out[b.count] = out[next];
                b.size[b.count] = sizes[next];
                b.first[b.count] = (int32_t)chunks;
                if (dtypes[next] == 0) b.wide[b.count / 32] |= 1u << (b.count % 32);
                chunks += (sizes[next] + length - 1) / length;
                ++b.count;
            }
            b.chunks = (int)chunks;
            b.length = (int)length;
            const int grid = (int)(chunks < most ? chunks : most);
            if (pass == 0) {
                grad_norm_kernel<<<grid, kNormThreads, 0, stream>>>(b, partial + partials);
                partials += grid;
            } else {
                clip_grads_kernel<<<grid, kNormThreads, 0, stream>>>(b, o, partial, partials, max_norm,
                                                                     l == 0 ? norm : nullptr);
            }
        }
    }
    if (!out || launches == 0)
        grad_norm_out_kernel<<<1, kNormThreads, 0, stream>>>(partial, partials, norm);
    return hipGetLastError();
}

}  // namespace dflash2
