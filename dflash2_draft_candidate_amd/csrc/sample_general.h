// Sampling a token from a row of vocabulary logits, by one workgroup of NT threads: the general path
// (any type, any values). sample.hip has the definitions and the faster path for bf16 rows.
//
// The token is a whole number that a rounding can change, and a flat row has more than 10^5 tokens
// whose shares a 32-bit sum cannot tell apart: weights and masses are held to 2^-40 of themselves, up to
// V = 2^23 - 1, and half as fine for each doubling from there, where the fixed point below moves.
// With z = 32 log2(e) (ref - x) / T + shift in fp64 and b the integer nearest to it, a weight is, but for
// a factor of the row, 2^(-b/32) 2^(-(z-b)/32); the second factor, within 1.1% of 1, is a polynomial
// of degree 4 (error 1.6e-13, 1 at 0). b (counted from the middle of the bins) is also the weight's
// bin: bins follow the candidate order, because z does. A bin's second factors are summed as 64-bit
// integers (41 bits behind the point up to V = 2^22 - 1, 62 - floor(log2 V) from there on, so that
// V of them fit) by LDS atomics: whole numbers have no order of summation, so results do not depend on
// which wave came first.
//
// One pass finds the maximum and fills the bins: ref is the largest of the first logits that the
// workgroup loads (2 vectors a thread), with 40 octaves of bins left above it and 88 below. Only if
// the row's maximum lies above the bins is the pass made again with the maximum itself. (For T = 0
// the pass is for the maximum alone, and where it first stands.) Then each cut is found among the
// bins' running masses and inside its bin. Where the tokens from the top to the lowest cut are few
// (<= NT) they are gathered once, sorted, and everything is settled in that list. Otherwise each cut
// gathers and sorts its own bin, which is split by value first if it holds more than NT tokens; when
// a single value remains, its tokens are equal and a division tells how many of them a cut takes.
//
// The first pass is bound by its arithmetic where a row has a CU to itself (about 20 instructions a
// logit, half of them fp64: 31 us for a row of 151936; 28 without the atomics) and by memory where
// all CUs read (256 rows: 35 us, 4.4 TB/s). The rest is latency: running sums over the bins 2 us, a
// cut's bin 2, bounds of bins 2, gathering 2 where few groups of 64 logits reach the range and up to
// 12 where most do, sorting and sums 2-5 (by the tokens), cuts in the list 3. Groups of 32 logits
// made the first pass 2 us longer and gained nothing; gathering with five vectors a thread in flight
// in place of three was slower (256 rows 90 us against 86).
#pragma once

#include <float.h>

#include "device_common.h"
#include "row_stream.h"

namespace dflash2 {

constexpr int kPerOctave = 32;          // bins to a factor of two
constexpr int kBins = 128 * kPerOctave;
constexpr int kHeadroom = 40 * kPerOctave;  // the bin of the first estimate of the maximum
constexpr int kFar = 64 * kPerOctave;  // counts of bf16 values: weights from here on count as 0
constexpr int kCountWords = 2 * 3652;
constexpr double kBinsPerE = kPerOctave * 1.4426950408889634;
constexpr double kTwo52 = 4503599627370496.0;
// added to z, this leaves the bin's number in the low bits
constexpr double kToBin = 1.5 * kTwo52 + kBins / 2;

enum Cut { kNumber, kReach, kPass };  // the n-th token; first S >= target; first S > target

// The settings of one row.
struct RowSettings {
    float temperature;
    int top_k;
    float top_p, min_p;
    double u;  // in [0, 1)
};

// The weights of a row.
struct Weights {
    float m;              // row maximum (finite): its weight is 1
    double c;             // kBinsPerE / T
    double one;           // fixed-point 1 (2^41, less for very long rows)
    const double *scale;  // 2^(-i/kPerOctave), i < kPerOctave
    // general path: a bin's weights are `unit` 2^(-b/kPerOctave) times their second factors
    float ref;
    double shift, unit;
};

__device__ __forceinline__ double weight_y(const Weights &w, float x) {
    return ((double)w.m - (double)x) * w.c;
}

// p f + c; c uniform, from a scalar register (the compiler copies it to a vector register first).
__device__ __forceinline__ double fma_const(double p, double f, double c) {
    double r;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(p), "v"(f), "s"(c));
    return r;
}

// 2^(-f/32) for |f| <= 1/2: 1 + f times the cubic that meets (2^(-f/32) - 1) / f at the four Chebyshev
// nodes of the interval; relative error 1.6e-13.
__device__ __forceinline__ double fraction(double f) {
    static_assert(kPerOctave == 32, "coefficients");
    double p = fma_const(f, 0x1.3b2b07bdf358dp-27, -0x1.c6b13c3465457p-20);
    p = fma_const(p, f, 0x1.ebfbdff82240ap-13);
    p = fma_const(p, f, -0x1.62e42fef8dc67p-6);
    return __builtin_fma(p, f, 1.0);
}

// round(one * fraction): adding 2^52 leaves the integer in the low mantissa bits.
__device__ __forceinline__ uint64_t fixed_fraction(const Weights &w, double f) {
    const double v = __builtin_fma(fraction(f), w.one, kTwo52);
    return (uint64_t)__double_as_longlong(v) & 0xFFFFFFFFFFFFFull;
}

__device__ __forceinline__ double bin_scale(const Weights &w, int b) {
    return ldexp(w.scale[b & (kPerOctave - 1)], -(b / kPerOctave));  // (b >= 0)
}

// 2^(-y/kPerOctave) for y >= 0.
__device__ __forceinline__ double weight_at(const Weights &w, double y) {
    y = fmin(y, 1e6);
    const double b = rint(y);
    return fraction(y - b) * bin_scale(w, (int)b);
}
__device__ __forceinline__ double weight_of(const Weights &w, float x) {
    return weight_at(w, weight_y(w, x));
}

__device__ __forceinline__ double bin_z(const Weights &w, float x) {
    return __builtin_fma((double)w.ref - (double)x, w.c, w.shift);
}
// Whether the integer nearest to z is a bin's, up to kBins / 2 - 1 (a tie goes to kBins / 2): the same
// integer decides which keys are a bin's (keys_of), so what is gathered of the last bin was counted. (With
// |z| below that integer itself, half of the last bin was gathered without having been counted:
// where a fill lay there, the list overflowed.) No NaN has a bin.
__device__ __forceinline__ bool has_bin(double z) { return fabs(z) < kBins / 2 - 0.5; }
__device__ __forceinline__ int bin_of(double z) {
    return (int)(uint32_t)__double_as_longlong(z + kToBin);
}
// z's distance from its bin's middle.
__device__ __forceinline__ double bin_fraction(double z) { return z - ((z + kToBin) - kToBin); }

// A place in the candidate order.
struct Place {
    double mass;  // running mass up to and including the token
    double w;     // its weight
    int32_t id;   // its id, or -1: number `nth` of the tokens of logit `value`
    float value;
    uint32_t nth;
};

// The cut among `size` tokens of one value.
__device__ __forceinline__ Place cut_equal(float value, double w, uint32_t size, Cut cut,
                                           double target, uint32_t nth, double below,
                                           uint32_t before) {
    uint32_t n;  // how many of them are taken
    if (cut == kNumber) {
        n = nth - before;
    } else {
        double q = floor((target - below) / w);
        q = fmin(fmax(q - 1.0, 0.0), (double)size);
        n = (uint32_t)q;
        if (n < 1) n = 1;
        while (n < size && !(cut == kReach ? below + n * w >= target : below + n * w > target)) ++n;
    }
    if (n > size) n = size;
    Place p;
    p.mass = below + (double)n * w;
    p.w = w;
    p.id = -1;
    p.value = value;
    p.nth = n - 1;
    return p;
}

template <typename T, int NT>
struct RowSampler {
static constexpr int EV = Elem<T>::kPerVec;
static constexpr int kThreads = NT;
static constexpr int kWaves = NT / kWave;
static constexpr int kPer = kBins / NT;  // bins per thread
static constexpr int kCap = NT;          // gathered tokens, one per thread
static constexpr int kTops = sizeof(T) == 4 ? 4096 : 1;  // (bf16 rows come here rarely)
static constexpr int kGroups = NT / 8;  // groups of an iteration of each: eight threads' vectors
static constexpr int kParts = 1024;      // parts that a bin is split into

struct alignas(16) Shared {  // (`words` is cleared and written by 16-byte vectors)
    union {
        struct {
            uint64_t mass[kBins];
            uint32_t count[kBins];
        };
        uint32_t words[sizeof(T) == 2 ? kCountWords : 1];  // sample.hip: counts of bf16 values
    };
    uint64_t part_mass[kParts];  // of a bin that is split
    uint32_t part_count[kParts];
    uint64_t list[kCap];
    float tops[kTops];    // the groups' maxima (see each)
    uint16_t hit[kTops];  // groups to look through
    uint32_t hits;
    double scale[kPerOctave];  // 2^(-i/kPerOctave)
    double wave_mass[kWaves];
    uint32_t wave_count[kWaves];
    int wave_first[kWaves];
    uint32_t first_key[4];
    float wave_max[kWaves];
    uint32_t listed;
    int32_t token;
    double spot_mass;
    uint32_t spot_count;
    int spot_bin;
    uint32_t spot_size;
};

static __device__ __forceinline__ void fill_scale(Shared &sh, int tid) {
    if (tid < kPerOctave) sh.scale[tid] = exp2((double)tid * (-1.0 / kPerOctave));
}

// ---- workgroup steps -------------------------------------------------------------------------

// Exclusive running sum over the threads; `total` is the sum. The result of thread t + 1 is at
// least that of thread t plus its v up to one rounding.
static __device__ __forceinline__ double scan_mass(Shared &sh, double v, int tid, double &total) {
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const double s = wave_running_sum(v);
    if (lane == kWave - 1) sh.wave_mass[wave] = s;
    __syncthreads();
    double base = 0.0, all = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i == wave) base = all;
        all += sh.wave_mass[i];
    }
    __syncthreads();
    total = all;
    const double before = __shfl_up(s, 1);
    return lane == 0 ? base : base + before;
}

static __device__ __forceinline__ uint32_t scan_count(Shared &sh, uint32_t v, int tid, uint32_t &total) {
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const uint32_t s = wave_running_sum(v);
    if (lane == kWave - 1) sh.wave_count[wave] = s;
    __syncthreads();
    uint32_t base = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i == wave) base = all;
        all += sh.wave_count[i];
    }
    __syncthreads();
    total = all;
    return base + s - v;
}

// The first thread for which `c` holds, kThreads if none.
static __device__ __forceinline__ int first_thread(Shared &sh, bool c, int tid) {
    const uint64_t b = __ballot(c);
    if ((tid & (kWave - 1)) == 0)
        sh.wave_first[tid / kWave] = b ? (tid + __builtin_ctzll(b)) : kThreads;
    __syncthreads();
    int first = kThreads;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) first = min(first, sh.wave_first[i]);
    __syncthreads();
    return first;
}

// The row: f(x, id) for each of its elements, in no particular order; the next two vectors are in
// flight while two are worked on (the passes that use this are bound by their arithmetic).
static __device__ __forceinline__ void first_vectors(const T *logits, const UnitRange &ur, int tid,
                                                     u32x4 &a, u32x4 &b) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(logits) + ur.c0;
    a = b = u32x4{};
    if (tid < ur.nv) a = p[tid];
    if (tid + NT < ur.nv) b = p[tid + NT];
}
// `group` is called after each pair of vectors, with the number of the pair.
template <typename F, typename G>
static __device__ __forceinline__ void each(const T *logits, const UnitRange &ur, int tid, u32x4 a,
                                            u32x4 b, F &&f, G &&group) {
    const int32_t id0 = (int32_t)(ur.c0 * EV - ur.g0);
    const u32x4 *p = reinterpret_cast<const u32x4 *>(logits) + ur.c0;
    auto one = [&](const u32x4 &v, int i) {
        float x[EV];
        Elem<T>::unpack(v, x);
#pragma unroll
        for (int k = 0; k < EV; ++k) f(x[k], id0 + i * EV + k);
    };
#pragma unroll 1
    for (int i0 = 0; i0 < ur.nv; i0 += 2 * NT) {
        // (past the end: the last vector once more, not looked at; the loads are not conditional)
        const int i = i0 + tid;
        const u32x4 c = p[min(i + 2 * NT, ur.nv - 1)], d = p[min(i + 3 * NT, ur.nv - 1)];
        if (i < ur.nv) one(a, i);
        if (i + NT < ur.nv) one(b, i + NT);
        group(i0 / (2 * NT));
        a = c;
        b = d;
    }
    const int64_t e = ragged_element(ur, tid);
    if (e >= 0) f(Elem<T>::load(logits, e), (int32_t)(e - ur.g0));
}
template <typename F>
static __device__ __forceinline__ void each(const T *logits, const UnitRange &ur, int tid, F &&f) {
    u32x4 a, b;
    first_vectors(logits, ur, tid, a, b);
    each(logits, ur, tid, a, b, f, [](int) {});
}

// The row's whole vectors, f(vector, index), with more in flight, for cheap f: those passes wait for
// memory. (One copy of the body: with stream()'s five the compiler keeps every copy's ids in
// registers.)
template <typename F>
static __device__ __forceinline__ void each_vector(const T *logits, const UnitRange &ur, int tid,
                                                   F &&f) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(logits) + ur.c0;
    constexpr int kDeep = 3;
    u32x4 v[kDeep], next[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
        v[u] = u32x4{};
        if (tid + u * NT < ur.nv) v[u] = p[tid + u * NT];
    }
#pragma unroll 1
    for (int i = tid; i < ur.nv; i += kDeep * NT) {
#pragma unroll
        for (int u = 0; u < kDeep; ++u) next[u] = p[min(i + (kDeep + u) * NT, ur.nv - 1)];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            if (i + u * NT < ur.nv) f(v[u], i + u * NT);
            v[u] = next[u];
        }
    }
}
// The largest of a value over the workgroup.
static __device__ __forceinline__ float group_top(Shared &sh, float m, int tid) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((tid & (kWave - 1)) == 0) sh.wave_max[tid / kWave] = m;
    __syncthreads();
    m = sh.wave_max[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sh.wave_max[w]);
    __syncthreads();
    return m;
}

// The lowest id of the row's largest logit (NaN aside), -1 if nothing lies above -inf.
static __device__ __forceinline__ int32_t first_of_top(const T *logits, const UnitRange &ur,
                                                       Shared &sh, int tid) {
    float mine = -INFINITY;
    int at = -1;  // the first vector of this thread that holds its largest
    each_vector(logits, ur, tid, [&](const u32x4 &v, int i) {
        float x[EV];
        Elem<T>::unpack(v, x);
        float c = x[0];
#pragma unroll
        for (int k = 1; k < EV; ++k) c = fmaxf(c, x[k]);
        if (c > mine) {
            mine = c;
            at = i;
        }
    });
    const int64_t e = ragged_element(ur, tid);
    const float end = e >= 0 ? Elem<T>::load(logits, e) : -INFINITY;
    if (tid == 0) sh.token = 0x7FFFFFFF;
    const float m = group_top(sh, fmaxf(mine, end), tid);
    if (m == -INFINITY) return -1;
    int32_t id = 0x7FFFFFFF;
    if (mine == m) {
        float x[EV];
        Elem<T>::unpack(reinterpret_cast<const u32x4 *>(logits)[ur.c0 + at], x);
#pragma unroll
        for (int k = EV - 1; k >= 0; --k)
            if (x[k] == m) id = (int32_t)((ur.c0 + at) * EV + k - ur.g0);
    }
    if (e >= 0 && end == m) id = min(id, (int32_t)(e - ur.g0));
    if (id != 0x7FFFFFFF) atomicMin(&sh.token, id);
    __syncthreads();
    id = sh.token;
    __syncthreads();
    return id;
}

// How many logits of a unit equal `value`, and the id of number `nth` (from 0, by id) among them,
// -1 if there are not so many. Wave w takes the w-th run of the unit's vectors, kSweep vectors a lane
// in flight. A comparison leaves a mask of lanes in a scalar register, and the scalar unit
// counts its bits: the vector units see two instructions an element (they are what bounds this
// otherwise: every wave of the workgroup runs here).
static constexpr int kSweep = sizeof(T) == 2 ? 8 : 4;
static __device__ __forceinline__ int32_t nth_equal(const T *logits, const UnitRange &ur, Shared &sh,
                                                    int tid, float value, uint32_t nth,
                                                    uint32_t &total) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(logits) + ur.c0;
    const int32_t id0 = (int32_t)(ur.c0 * EV - ur.g0);
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int v0 = (int)((int64_t)ur.nv * wave / kWaves);
    const int v1 = (int)((int64_t)ur.nv * (wave + 1) / kWaves);
    // matches among the 64 vectors at i (those below v1): of all lanes
    auto count = [&](const u32x4 &v, int i) {
        float x[EV];
        Elem<T>::unpack(v, x);
        const uint64_t on = v1 - i >= kWave ? ~0ull : (1ull << (v1 - i)) - 1ull;
        uint32_t n = 0;
#pragma unroll
        for (int k = 0; k < EV; ++k) n += __builtin_popcountll(__ballot(x[k] == value) & on);
        return n;
    };
    auto at = [&](int i) { return p[min(i + lane, v1 - 1)]; };
    uint32_t mine = 0;
    for (int i = v0; i < v1; i += kSweep * kWave) {
        u32x4 v[kSweep];
#pragma unroll
        for (int u = 0; u < kSweep; ++u)
            if (i + u * kWave < v1) v[u] = at(i + u * kWave);
#pragma unroll
        for (int u = 0; u < kSweep; ++u)
            if (i + u * kWave < v1) mine += count(v[u], i + u * kWave);
    }
    // the ragged ends: lanes of every wave look at one element each
    const int nh = (int)(ur.h1 - ur.h0);
    const int64_t e = ragged_element(ur, lane);
    const uint64_t ends = __ballot(e >= 0 && Elem<T>::load(logits, e >= 0 ? e : ur.g0) == value);
    const uint64_t head_mask = (1ull << nh) - 1ull;  // (fewer than 64 of them)
    if (lane == 0) sh.wave_count[wave] = mine;
    if (tid == 0) sh.token = -1;
    __syncthreads();
    const uint32_t head = __popcll(ends & head_mask), tail = __popcll(ends & ~head_mask);
    uint32_t before = head, base = head;
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) base = before;
        before += sh.wave_count[w];
    }
    total = before + tail;
    if (tid == 0 && (nth < head || (nth >= before && nth < total))) {
        uint64_t b = nth < head ? ends & head_mask : ends & ~head_mask;
        for (uint32_t left = nth < head ? nth : nth - before; left > 0; --left) b &= b - 1;
        sh.token = (int32_t)(ragged_element(ur, __builtin_ctzll(b)) - ur.g0);
    }
    if (nth >= base && nth < base + mine) {  // this wave's run holds it: once more, in order
        uint32_t left = nth - base;
        for (int i = v0; i < v1; i += kWave) {
            const u32x4 v = at(i);
            const uint32_t all = count(v, i);
            if (left >= all) {
                left -= all;
                continue;
            }
            float x[EV];
            Elem<T>::unpack(v, x);
            uint32_t bits = 0;
#pragma unroll
            for (int k = 0; k < EV; ++k) bits |= x[k] == value ? 1u << k : 0u;
            if (i + lane >= v1) bits = 0;
            const uint32_t own = __popc(bits);
            const uint32_t s = wave_running_sum(own);
            if (left >= s - own && left < s) {
                for (uint32_t k = left - (s - own); k > 0; --k) bits &= bits - 1;
                sh.token = id0 + (i + lane) * EV + (__ffs(bits) - 1);
            }
            break;
        }
    }
    __syncthreads();
    const int32_t id = sh.token;
    __syncthreads();
    return id;
}

// Appends the keys of a unit's matching logits to sh.list (sh.listed counts them; what does not fit
// in `cap` is dropped).
template <typename F>
static __device__ __forceinline__ void collect(const T *logits, const UnitRange &ur, Shared &sh,
                                               int tid, uint32_t cap, F &&match) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(logits) + ur.c0;
    const int32_t id0 = (int32_t)(ur.c0 * EV - ur.g0);
    auto append = [&](float x, int32_t id) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < cap) sh.list[at] = cand_key(x, id);
    };
    for (int i = tid; i < ur.nv; i += kSweep * NT) {
        u32x4 v[kSweep];
#pragma unroll
        for (int u = 0; u < kSweep; ++u)
            if (i + u * NT < ur.nv) v[u] = p[i + u * NT];
#pragma unroll
        for (int u = 0; u < kSweep; ++u) {
            if (i + u * NT >= ur.nv) continue;
            float x[EV];
            Elem<T>::unpack(v[u], x);
#pragma unroll
            for (int k = 0; k < EV; ++k)
                if (match(x[k])) append(x[k], id0 + (i + u * NT) * EV + k);
        }
    }
    const int64_t e = ragged_element(ur, tid);
    if (e >= 0 && match(Elem<T>::load(logits, e)))
        append(Elem<T>::load(logits, e), (int32_t)(e - ur.g0));
}

// ---- the gathered list --------------------------------------------------------------------------

// One gathered token per thread in candidate order (threads below n), with running masses.
struct Listed {
    uint64_t key;
    double w;      // 0 for threads from n on
    double below;  // masses of the tokens before it
    double total;
    int n;
};

// Sorts sh.list[0 .. n) in candidate order, a key per thread: waves sort 64 by lane exchanges,
// larger strides go through LDS. Keys are distinct, so the order is unique.
static __device__ __forceinline__ uint64_t sort_list(Shared &sh, int n, int tid) {
    const int lane = tid & (kWave - 1);
    uint64_t key = tid < n ? sh.list[tid] : 0ull;
    key = bitonic_merge_steps<1>(key, lane, (lane & 2) == 0);
    key = bitonic_merge_steps<2>(key, lane, (lane & 4) == 0);
    key = bitonic_merge_steps<4>(key, lane, (lane & 8) == 0);
    key = bitonic_merge_steps<8>(key, lane, (lane & 16) == 0);
    key = bitonic_merge_steps<16>(key, lane, (lane & 32) == 0);
    int size = kWave;
    while (size < n) size <<= 1;
    key = bitonic_merge_steps<32>(key, lane, size == kWave || (tid & kWave) == 0);
    for (int k = 2 * kWave; k <= size; k <<= 1) {
        const bool desc = k == size || (tid & k) == 0;
        for (int j = k >> 1; j >= kWave; j >>= 1) {
            __syncthreads();
            sh.list[tid] = key;
            __syncthreads();
            const uint64_t other = sh.list[tid ^ j];
            const bool keep_max = ((tid & j) == 0) == desc;
            key = ((key > other) == keep_max) ? key : other;
        }
        key = bitonic_merge_steps<32>(key, lane, desc);
    }
    __syncthreads();
    return key;
}

static __device__ __forceinline__ Listed make_list(Shared &sh, const Weights &w, int n, int tid) {
    Listed l;
    l.n = n;
    l.key = sort_list(sh, n, tid);
    l.w = tid < n ? weight_of(w, key_logit(l.key)) : 0.0;
    l.below = scan_mass(sh, l.w, tid, l.total);
    return l;
}

// The smallest value key in [key(-FLT_MAX), key(FLT_MAX)] for which `holds` is true, one past the range
// if there is none; holds(x) must not fall back to false as x grows. By one wave, 64 keys at a time.
template <typename F>
static __device__ __forceinline__ uint32_t first_key(int lane, F &&holds) {
    uint32_t a = value_key(-FLT_MAX), e = value_key(FLT_MAX) + 1u;  // a <= answer <= e
#pragma unroll 1
    while (a < e) {
        const uint32_t step = (e - a) / kWave + 1u;
        const uint64_t probe = (uint64_t)a + (uint64_t)lane * step;
        const bool yes = probe >= e || holds(key_value((uint32_t)probe));
        const uint64_t b = __ballot(yes);
        const uint32_t t = b ? (uint32_t)__builtin_ctzll(b) : (uint32_t)kWave;
        const uint32_t base = a;
        if (t > 0) a = base + (t - 1u) * step + 1u;
        const uint64_t top = (uint64_t)base + (uint64_t)t * step;
        if (t < kWave && top < e) e = (uint32_t)top;
    }
    return a;
}
// Value keys of the bins [b0, b1].
struct Keys {
    uint32_t lo, hi;  // lo <= key <= hi
};
static constexpr uint32_t kMinusZero = 0x7FFFFFFFu;  // key_value gives -0, value_key never this
// The keys of the bins [a0, a1] and of [b0, b1]: four searches, a wave each (side by side they take
// 2 us; by every wave, one after the other, 7).
static __device__ __forceinline__ void keys_of(Shared &sh, const Weights &w, int a0, int a1, int b0,
                                               int b1, int tid, Keys &a, Keys &b) {
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    if (wave < 4) {  // the first key in bin `bin` or above it in the order
        const int bin = wave == 0 ? a1 : wave == 1 ? a0 - 1 : wave == 2 ? b1 : b0 - 1;
        const double last = (double)(bin - kBins / 2);
        const uint32_t key = first_key(tid & (kWave - 1), [&](float x) {
            const double z = bin_z(w, x);
            return z - bin_fraction(z) <= last;
        });
        if ((tid & (kWave - 1)) == 0) sh.first_key[wave] = key;
    }
    __syncthreads();
    a = Keys{sh.first_key[0], sh.first_key[1] - 1u};
    b = Keys{sh.first_key[2], sh.first_key[3] - 1u};
    __syncthreads();
}

// Whether the pass keeps the maxima of this row's groups.
static __device__ __forceinline__ bool keeps_tops(const UnitRange &ur) {
    return kTops > 1 && (ur.nv + 2 * NT - 1) / (2 * NT) * kGroups <= kTops;
}

// Gathers the tokens whose keys lie in `one` or `two`: at most kCap, known from the histogram, which
// counted each logit by the bin or part that the keys were made from. Only groups whose maximum reaches
// the lowest of them can hold any; where those are few, the rest of the row is not read again.
static __device__ __forceinline__ Listed gather(const T *logits, const UnitRange &ur, Shared &sh,
                                         const Weights &w, const Keys &one, const Keys &two,
                                         int tid) {
    const float lo1 = key_value(one.lo), hi1 = key_value(one.hi);
    const float lo2 = key_value(two.lo), hi2 = key_value(two.hi);
    const float lo = fminf(lo1, lo2);  // (finite: keys of finite logits)
    const int groups = (ur.nv + 2 * NT - 1) / (2 * NT) * kGroups;
    const bool keep = keeps_tops(ur);
    if (tid == 0) sh.listed = sh.hits = 0;
    __syncthreads();
    if (keep) {
        for (int g = tid; g < groups; g += NT)
            if (sh.tops[g] >= lo) sh.hit[atomicAdd(&sh.hits, 1u)] = (uint16_t)g;
        __syncthreads();
    }
    const bool single = one.lo == two.lo && one.hi == two.hi;
    // (x lies in a range where the median of it and the range's ends is x itself; one branch a vector)
    auto in_one = [&](float x) { return __builtin_amdgcn_fmed3f(x, lo1, hi1) == x; };
    auto in = [&](float x) { return in_one(x) || __builtin_amdgcn_fmed3f(x, lo2, hi2) == x; };
    auto append = [&](float x, int32_t id) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kCap) sh.list[at] = cand_key(x, id);
    };
    const u32x4 *p = reinterpret_cast<const u32x4 *>(logits) + ur.c0;
    const int32_t id0 = (int32_t)(ur.c0 * EV - ur.g0);
    auto take = [&](const u32x4 &v, int i) {
        float x[EV];
        Elem<T>::unpack(v, x);
        bool any = false;
        if (single) {
#pragma unroll
            for (int k = 0; k < EV; ++k) any |= in_one(x[k]);
        } else {
#pragma unroll
            for (int k = 0; k < EV; ++k) any |= in(x[k]);
        }
        if (any) {
#pragma unroll
            for (int k = 0; k < EV; ++k)
                if (in(x[k])) append(x[k], id0 + i * EV + k);
        }
    };
    if (keep && (int)sh.hits * 2 < groups) {
#pragma unroll 1
        for (int h = tid / 8; h < (int)sh.hits; h += kGroups) {
            const int g = sh.hit[h];
            const int i = g / kGroups * 2 * NT + g % kGroups * 8 + (tid & 7);
            u32x4 v[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (i + u * NT < ur.nv) v[u] = p[i + u * NT];
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (i + u * NT < ur.nv) take(v[u], i + u * NT);
        }
    } else {
        each_vector(logits, ur, tid, take);
    }
    const int64_t e = ragged_element(ur, tid);
    if (e >= 0) {
        const float x = Elem<T>::load(logits, e);
        if (in(x)) append(x, (int32_t)(e - ur.g0));
    }
    __syncthreads();
    const int n = min((int)sh.listed, kCap);
    __syncthreads();
    return make_list(sh, w, n, tid);
}

// ---- cuts -------------------------------------------------------------------------------------

// A histogram in LDS: kPerThread bins per thread, of mass sum[b] `unit`, times 2^(-b/kPerOctave) where
// `by_bin` is set.
template <int kPerThread>
struct Level {
    const uint64_t *sum;
    const uint32_t *counts;
    double unit;
    bool by_bin;
    __device__ __forceinline__ double mass(const Weights &w, int b) const {
        return (double)sum[b] * (by_bin ? bin_scale(w, b) * unit : unit);
    }
};
// What lies before this thread's bins, and in all.
struct Bins {
    double below, total;
    uint32_t before, number;
};

template <int kPerThread>
static __device__ __forceinline__ Bins sum_bins(Shared &sh, const Level<kPerThread> &v,
                                                const Weights &w, double below, uint32_t before,
                                                int tid) {
    Bins h;
    double sum = 0.0;
    uint32_t number = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        const int b = tid * kPerThread + j;
        sum += v.mass(w, b);
        number += v.counts[b];
    }
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const double upto = wave_running_sum(sum);
    const uint32_t upto_n = wave_running_sum(number);
    if (lane == kWave - 1) {
        sh.wave_mass[wave] = upto;
        sh.wave_count[wave] = upto_n;
    }
    __syncthreads();
    h.below = h.total = 0.0;
    h.before = h.number = 0u;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i == wave) {
            h.below = h.total;
            h.before = h.number;
        }
        h.total += sh.wave_mass[i];
        h.number += sh.wave_count[i];
    }
    __syncthreads();
    const double prev = __shfl_up(upto, 1);
    h.below += below + (lane == 0 ? 0.0 : prev);
    h.before += before + upto_n - number;
    h.total += below;
    h.number += before;
    return h;
}

// The bin that holds a cut: the result is in sh.spot_*. Roundings may leave a mass cut behind the
// last bin: it is then the last that holds anything.
template <int kPerThread>
static __device__ __forceinline__ void find_bin(Shared &sh, const Level<kPerThread> &v,
                                                const Weights &w, const Bins &h, Cut cut,
                                                double target, uint32_t nth, int tid) {
    // the first bin of this thread that meets the cut, or (any) the last that holds a token
    auto look = [&](bool any, double &run, uint32_t &num, uint32_t &size) {
        int bin = -1;
        double mass = h.below;
        uint32_t number = h.before;
#pragma unroll 1
        for (int j = 0; j < kPerThread; ++j) {
            const int b = tid * kPerThread + j;
            const uint32_t n = v.counts[b];
            if (n == 0) continue;
            const double next = mass + v.mass(w, b);
            const bool in = cut == kNumber ? number + n >= nth
                            : cut == kReach ? next >= target
                                            : next > target;
            if (any || (in && bin < 0)) {
                bin = b;
                run = mass;
                num = number;
                size = n;
            }
            mass = next;
            number += n;
        }
        return bin;
    };
    double spot_mass = 0.0;
    uint32_t spot_count = 0, spot_size = 0;
    int bin = look(false, spot_mass, spot_count, spot_size);
    int first = first_thread(sh, bin >= 0, tid);
    if (first == kThreads) {
        bin = look(true, spot_mass, spot_count, spot_size);
        const uint64_t b = __ballot(bin >= 0);
        const int lane = tid & (kWave - 1), wave = tid / kWave;
        if (lane == 0) sh.wave_first[wave] = b ? wave * kWave + 63 - __builtin_clzll(b) : -1;
        __syncthreads();
        first = -1;
        for (int i = 0; i < kWaves; ++i) first = max(first, sh.wave_first[i]);
        __syncthreads();
    }
    if (tid == first) {
        sh.spot_bin = bin;
        sh.spot_mass = spot_mass;
        sh.spot_count = spot_count;
        sh.spot_size = spot_size;
    }
    __syncthreads();
}

// The cut inside a sorted list whose first token has `below` mass and `before` tokens before it.
static __device__ __forceinline__ Place cut_list(Shared &sh, const Listed &l, Cut cut, double target,
                                          uint32_t nth, double below, uint32_t before, int tid) {
    const double s = below + l.below + l.w;
    const bool in = tid < l.n && (cut == kNumber ? before + tid + 1 >= nth
                                  : cut == kReach ? s >= target
                                                  : s > target);
    int at = first_thread(sh, in, tid);
    if (at >= l.n) at = l.n - 1;
    if (tid == at) {
        sh.spot_mass = s;
        sh.list[0] = l.key;
    }
    __syncthreads();
    Place p;
    p.mass = sh.spot_mass;
    const uint64_t key = sh.list[0];
    __syncthreads();
    p.id = key_id(key);
    p.value = key_logit(key);
    p.nth = 0;
    p.w = 0.0;
    return p;
}

// The cut inside bin `bin` of the row (size tokens, `below` mass and `before` tokens before it).
static __device__ __forceinline__ Place cut_bin(const T *logits, const UnitRange &ur, Shared &sh,
                                      const Weights &w, int bin, uint32_t size, Cut cut,
                                      double target, uint32_t nth, double below, uint32_t before,
                                      int tid) {
    Keys keys, same;
    keys_of(sh, w, bin, bin, bin, bin, tid, keys, same);
    // Split by value until a part is small or a single value; every step narrows the range to a
    // kParts-th of it or to one value.
#pragma unroll 1
    while (size > kCap && keys.lo != keys.hi) {
        const int bits = 32 - __clz(keys.hi - keys.lo);
        const int shift = bits > 10 ? bits - 10 : 0;
        for (int b = tid; b < kParts; b += kThreads) {
            sh.part_mass[b] = 0ull;
            sh.part_count[b] = 0u;
        }
        __syncthreads();
        const float lo = key_value(keys.lo), hi = key_value(keys.hi);
        each(logits, ur, tid, [&](float x, int32_t) {
            if (x >= lo && x <= hi) {
                const uint32_t part = (keys.hi - value_key(x)) >> shift;
                atomicAdd((unsigned long long *)&sh.part_mass[part],
                          (unsigned long long)fixed_fraction(w, bin_fraction(bin_z(w, x))));
                atomicAdd(&sh.part_count[part], 1u);
            }
        });
        __syncthreads();
        const Level<kParts / NT> v{sh.part_mass, sh.part_count,
                                   bin_scale(w, bin) * w.unit / w.one, false};
        const Bins h = sum_bins(sh, v, w, below, before, tid);
        find_bin(sh, v, w, h, cut, target, nth, tid);
        const uint32_t part = (uint32_t)sh.spot_bin;
        below = sh.spot_mass;
        before = sh.spot_count;
        size = sh.spot_size;
        __syncthreads();
        keys.hi -= part << shift;
        const uint32_t width = (1u << shift) - 1u;
        if (keys.hi - keys.lo > width) keys.lo = keys.hi - width;
        // (The key of -0 is no logit's, as zeros of both signs have that of +0. Logits are compared by
        // value, so as an upper end it would let the zeros in, whose key lies above the range.)
        if (keys.hi == kMinusZero) --keys.hi;
    }
    if (size > kCap) {
        const float value = key_value(keys.hi);
        return cut_equal(value, weight_of(w, value), size, cut, target, nth, below, before);
    }
    const Listed l = gather(logits, ur, sh, w, keys, keys, tid);
    Place p = cut_list(sh, l, cut, target, nth, below, before, tid);
    p.w = weight_of(w, p.value);
    return p;
}

// One row: its token and log-probability, written by thread 0.
static __device__ __forceinline__ void run(const T *logits, const UnitRange &ur, Shared &sh,
                                           const RowSettings &st, double one, int tid,
                                           int32_t *token, float *logprob) {
    const int top_k = st.top_k;
    const float top_p = st.top_p, min_p = st.min_p, temperature = st.temperature;
    const double u = st.u;
    auto answer = [&](int32_t id, double lp) {
        if (tid == 0) {
            *token = id;
            if (logprob) *logprob = (float)lp;
        }
    };
    if (!(temperature > 0.f)) {
        const int32_t id = first_of_top(logits, ur, sh, tid);
        answer(id, id < 0 ? -INFINITY : 0.0);
        return;
    }
    u32x4 a, b;
    first_vectors(logits, ur, tid, a, b);
    fill_scale(sh, tid);
    float m = -INFINITY;
    {
        float x[2 * EV];
        Elem<T>::unpack(a, x);
        Elem<T>::unpack(b, x + EV);
#pragma unroll
        for (int k = 0; k < 2 * EV; ++k)
            if (tid + (k < EV ? 0 : NT) < ur.nv) m = fmaxf(m, x[k]);
    }
    Weights w{0.f, kBinsPerE / (double)temperature, one, sh.scale, group_top(sh, m, tid),
              (double)(kHeadroom - kBins / 2), 1.0};
    const bool keep = keeps_tops(ur);
#pragma unroll 1
    for (;;) {
        for (int i = tid; i < kBins; i += kThreads) {
            sh.mass[i] = 0ull;
            sh.count[i] = 0u;
        }
        __syncthreads();
        float pair = -INFINITY;
        each(
            logits, ur, tid, a, b,
            [&](float x, int32_t) {
                pair = fmaxf(pair, x);
                const double z = bin_z(w, x);
                if (has_bin(z)) {  // (false for NaN and -inf)
                    const int i = bin_of(z);
                    atomicAdd((unsigned long long *)&sh.mass[i],
                              (unsigned long long)fixed_fraction(w, bin_fraction(z)));
                    atomicAdd(&sh.count[i], 1u);
                }
            },
            [&](int number) {
                m = fmaxf(m, pair);
                if (keep) {
                    pair = fmaxf(pair, lane_move<kDppQuadXor1>(pair));
                    pair = fmaxf(pair, lane_move<kDppQuadXor2>(pair));
                    pair = fmaxf(pair, lane_move<0x141>(pair));  // row_half_mirror
                    if ((tid & 7) == 0) sh.tops[number * kGroups + tid / 8] = pair;
                }
                pair = -INFINITY;
            });
        m = fmaxf(m, pair);  // (of the ragged ends)
        w.m = group_top(sh, m, tid);
        // (nothing to weigh, or the maximum has its bin; a second time it always has)
        if (!(fabsf(w.m) < INFINITY) || (w.ref > -INFINITY && has_bin(bin_z(w, w.m)))) break;
        w.ref = w.m;
        w.shift = kPerOctave - kBins / 2;  // an octave of bins above it stays empty
        first_vectors(logits, ur, tid, a, b);
    }
    if (w.m == -INFINITY) {  // nothing to draw
        answer(-1, -INFINITY);
        return;
    }
    if (w.m == INFINITY) {  // only the infinite logits have weight, all the same
        uint32_t n;
        nth_equal(logits, ur, sh, tid, INFINITY, 0u, n);
        if (top_k >= 1 && (uint32_t)top_k < n) n = (uint32_t)top_k;
        double whole = (double)n;
        if (top_p < 1.f)
            whole = cut_equal(INFINITY, 1.0, n, kReach, (double)top_p * whole, 0u, 0.0, 0u).mass;
        const Place p = cut_equal(INFINITY, 1.0, n, kPass, u * whole, 0u, 0.0, 0u);
        answer(nth_equal(logits, ur, sh, tid, INFINITY, p.nth, n), -log(whole));
        return;
    }
    // The maximum's weight is 1; where it is the reference itself, its bin is a whole number of octaves
    // down, so that equal tokens weigh 1 each exactly.
    const double top_z = bin_z(w, w.m) + kBins / 2;
    w.unit = w.ref == w.m ? ldexp(1.0, (int)top_z / kPerOctave) : exp2(top_z * (1.0 / kPerOctave));
    const Level<kPer> all{sh.mass, sh.count, w.unit / one, true};
    const Bins h = sum_bins(sh, all, w, 0.0, 0u, tid);

    // The lowest bin that the cuts can reach. (A top-k beyond the counted tokens cuts only among
    // weights below 2^-64.)
    const bool by_number = top_k >= 1 && (uint32_t)top_k < h.number;
    const bool by_mass = top_p < 1.f;
    const double least = min_p > 0.f ? fmin((double)min_p, 1.0) : 0.0;
    const bool by_weight = least > 0x1p-64;  // (lower weights need not count)
    const int weight_bin =
        by_weight ? min((int)(top_z - kPerOctave * log2(least)) + 2, kBins - 1) : kBins - 1;
    bool mass_inside = false;  // the nucleus ends in the bins up to `low`
    int low = by_weight ? weight_bin : kBins - 1;
    if (by_number) {
        find_bin(sh, all, w, h, kNumber, 0.0, (uint32_t)top_k, tid);
        // (top-p needs the whole mass of the top-k tokens, whatever min-p leaves of them)
        low = by_mass ? sh.spot_bin : min(low, sh.spot_bin);
    } else if (by_mass) {
        find_bin(sh, all, w, h, kReach, (double)top_p * h.total, 0u, tid);
        mass_inside = sh.spot_bin <= low;
        low = min(low, sh.spot_bin);
    }
    // tokens in the bins up to `low` (after a search: of which sh.spot_* still has the result)
    uint32_t upto = h.number;
    if ((by_number || by_mass) && low == sh.spot_bin) {
        upto = sh.spot_count + sh.spot_size;
    } else if (low < kBins - 1) {
        upto = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (tid * kPer + j <= low) upto += sh.count[tid * kPer + j];
        uint32_t total;
        scan_count(sh, upto, tid, total);
        upto = total;
    }
    if (upto <= kCap) {
        Keys keys, same;
        keys_of(sh, w, low, low, low, low, tid, keys, same);
        keys.hi = value_key(w.m);
        const Listed l = gather(logits, ur, sh, w, keys, keys, tid);
        // (the list's weights are exact where equal tokens tie; the bins give only what lies below it)
        double z = 0.0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (tid * kPer + j > low) z += all.mass(w, tid * kPer + j);
        double tail;
        scan_mass(sh, z, tid, tail);
        z = l.total + tail;
        if (by_number)
            z = cut_list(sh, l, kNumber, 0.0, (uint32_t)top_k, 0.0, 0u, tid).mass;
        double whole = z;
        if (by_mass) {
            const double target = (double)top_p * z;
            // (the list may end before the nucleus does, at a min-p cut)
            if (mass_inside || first_thread(sh, tid < l.n && l.below + l.w >= target, tid) < l.n)
                whole = fmin(whole, cut_list(sh, l, kReach, target, 0u, 0.0, 0u, tid).mass);
        }
        if (by_weight) {
            const int n = first_thread(sh, !(tid < l.n && l.w >= least), tid);
            whole = fmin(whole, cut_list(sh, l, kNumber, 0.0, (uint32_t)max(n, 1), 0.0, 0u, tid).mass);
        }
        const Place p = cut_list(sh, l, kPass, u * whole, 0u, 0.0, 0u, tid);
        answer(p.id, log(weight_of(w, p.value) / whole));
        return;
    }

    // Cut by cut, each in its own bin; the draw is the last.
    double z = h.total, whole = h.total;
    if (by_weight) {
        // the bins above the one that the border falls in, and of that one what reaches it
        const float border = key_value(
            first_key(tid & (kWave - 1), [&](float x) { return x >= w.m || weight_of(w, x) >= least; }));
        const int bin = bin_of(bin_z(w, border));
        double part = 0.0;
        each(logits, ur, tid, [&](float x, int32_t) {
            if (x >= border && x <= w.m && bin_of(bin_z(w, x)) == bin) part += weight_of(w, x);
        });
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (tid * kPer + j < bin) part += all.mass(w, tid * kPer + j);
        double sum;
        scan_mass(sh, part, tid, sum);
        whole = fmin(whole, sum);
    }
    if (by_mass && !by_number) {
        // The nucleus' end and the draw, gathered in one pass: the kept mass is known to within the
        // end's bin, and with it where the draw can fall.
        const double target = (double)top_p * z;
        const int end = sh.spot_bin;  // (found above)
        const double end_below = sh.spot_mass;
        const uint32_t end_before = sh.spot_count, end_size = sh.spot_size;
        __syncthreads();
        find_bin(sh, all, w, h, kPass, u * fmin(whole, end_below), 0u, tid);
        const int from = sh.spot_bin;
        const double from_below = sh.spot_mass;
        const uint32_t from_before = sh.spot_count;
        __syncthreads();
        find_bin(sh, all, w, h, kPass, u * fmin(whole, end_below + all.mass(w, end)), 0u, tid);
        const int to = sh.spot_bin;
        const uint32_t to_before = sh.spot_count + sh.spot_size;
        __syncthreads();
        const bool apart = to < end;  // otherwise one run of bins, from `from` to `end`
        const uint32_t drawn = apart ? to_before - from_before : 0u;  // tokens of the draw's bins
        const uint32_t in_all =
            apart ? drawn + end_size : end_before + end_size - min(from_before, end_before);
        if (in_all <= kCap) {
            Keys head, tail;
            const int last_run = apart ? end : min(from, end);
            keys_of(sh, w, apart ? from : last_run, apart ? to : end, last_run, end, tid, head, tail);
            const Listed l = gather(logits, ur, sh, w, head, tail, tid);
            // the running mass of this thread's token in the row
            if (tid == (int)drawn) sh.spot_mass = l.below;
            __syncthreads();
            const double split = sh.spot_mass;
            __syncthreads();
            const double s = apart && tid >= (int)drawn ? end_below + (l.below - split) + l.w
                                                        : fmin(from_below, end_below) + l.below + l.w;
            int at = min(first_thread(sh, tid >= (int)drawn && tid < l.n && s >= target, tid), l.n - 1);
            if (tid == at) sh.spot_mass = s;
            __syncthreads();
            whole = fmin(whole, sh.spot_mass);
            __syncthreads();
            const int last = apart ? (int)drawn : l.n;
            at = min(first_thread(sh, tid < last && s > u * whole, tid), last - 1);
            if (tid == at) {
                *token = key_id(l.key);
                if (logprob) *logprob = (float)log(l.w / whole);
            }
            return;
        }
    }
    Place p;
#pragma unroll 1
    for (int step = by_number ? 0 : by_mass ? 1 : 2; step < 3; ++step) {
        if (step == 1 && !by_mass) continue;
        const Cut cut = step == 0 ? kNumber : step == 1 ? kReach : kPass;
        const double target = step == 1 ? (double)top_p * z : u * whole;
        find_bin(sh, all, w, h, cut, target, (uint32_t)top_k, tid);
        const int bin = sh.spot_bin;
        const double below = sh.spot_mass;
        const uint32_t before = sh.spot_count, size = sh.spot_size;
        __syncthreads();
        p = cut_bin(logits, ur, sh, w, bin, size, cut, target, (uint32_t)top_k, below, before, tid);
        if (step == 0) z = p.mass;
        if (step < 2) whole = fmin(whole, p.mass);
    }
    int32_t id = p.id;
    if (id < 0) {
        uint32_t n;
        id = nth_equal(logits, ur, sh, tid, p.value, p.nth, n);
    }
    answer(id, log(p.w / whole));
}
};

}  // namespace dflash2
