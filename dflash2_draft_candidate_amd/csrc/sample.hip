// Sampling a token from each row of vocabulary logits with temperature, top-k, top-p and min-p, from
// given uniform numbers.
//
// For a row x with maximum m and temperature T the weights are w_v = exp((x_v - m) / T). In the
// candidate order (higher logit first, equal logits by lower id) with running sums S_j:
//   n_k = top_k if 1 <= top_k < N, else N;  Z = S_{n_k};  n_p = min{j: S_j >= top_p Z};
//   n_m = #{v: w_v >= min_p};  n = max(1, min(n_k, n_p, n_m));  W = S_n;
//   the token is number min{j: S_j > u W} of the order.
// Each cut keeps a prefix of the order and S grows along it, so W is the smallest of the cuts' masses
// and nothing else of a cut is needed.
//
// float32 rows take the general path (sample_general.h). bf16 rows have few distinct values, so it is
// enough to count how often each occurs: the masses of all cuts follow from the counts, a weight per
// value, and the draw gives a value and how many of its equals come before the token. The counts
// are whole numbers (LDS atomics in any order), there is one atomic and a handful of integer
// instructions per logit in place of an exponential, and the pass needs no maximum first.
//   * Counted values: 2^-20 <= |x| < 2^8, 28 binades of 128 values, a word each: positive values
//     in its low half, negative ones in its high half. A word below takes what is smaller, 64
//     above what is larger (from 382 on a lane has its own: the masked tokens of a row all count
//     there, and atomics on one word take turns: 1024 rows x 151936 of which 90% are masked took
//     570 us with one word for them, 71 with 64; of a finite mask nearer than that they still take
//     320 to 590). The row is counted in parts (words of their own), so that a
//     half-word is enough; a part's overflow shows as a wrong total.
//   * Smaller values are rare (one in 10^6 of a normal row): up to 64 of them are listed and take
//     their place between the positive and the negative values. Larger negative ones are masks,
//     or so far below the maximum that they have no weight. Anything else (large or infinite
//     logits, many tiny or zero ones, a row of masks) sends the row to the general path.
//   * The token is then the n-th logit of a value, and the parts' counts say in which part: only
//     that part is read a second time.
// Rows that are many (kRowGroups and more) or short have a workgroup each, with two parts; a few long
// rows are cut into slices, a part and a workgroup each, whose counts go through the workspace to a
// second kernel (plan_slices).
//
// What bounds it and what it takes (V = 151936, settings mixed; a row's bytes are read once, and the
// part that holds the token for the groups that can hold it):
//   1024 rows bf16: 82 us, 3.8 TB/s of logits; the reading and counting alone 55 us (5.6 TB/s, what a
//     plain read reaches), the rest is the settling of a row, a chain of 11-13 us that the other
//     workgroup of the CU hides in part;
//   64 rows bf16: 27 us: counting 9 us, settling 18 us; 1 row: 17 us, 4 + 13 us. Latency: barriers,
//     two dependent reads of the counts, fp64 exponentials, the second read of the part;
//   256 rows float32: 85 us; the first pass 35 us, at the rate of a read, 64 rows 32 us: there the
//     fp64 arithmetic of one CU per row is what it takes. Settling: 11 us a row whose cuts leave few
//     tokens, about 25 us where 1024 tokens are gathered from most of the row.
#include <stddef.h>

#include "kernels.h"
#include "sample_general.h"

namespace dflash2 {
namespace {

constexpr int kNT = 512;        // threads of the bf16 kernels: two workgroups share a CU, and two
                                // waves share a SIMD where all waves do the same (four workgroups
                                // of 256: 1024 rows x 151936 82 us, 81 with two of 512)
constexpr int kParts = 2;       // parts of a row that a workgroup counts by itself (with one, whose
                                // atomics meet more often and of which all is read again, 256 rows
                                // x 151936 took 40 us, 33 with two; 1024 rows 102, 87)
constexpr int kNT32 = 1024;     // threads of the float32 kernel
constexpr int kBase = 0x3580;  // bf16 pattern of 2^-20
constexpr int kValues = 3584;  // counted values of a sign: up to 2^8
constexpr int kAbove = 64;      // words for what is larger, one to a lane
constexpr int kStride = 3652;  // words of a part: below, kValues, kAbove, three unused
constexpr int kRows = 2 * kValues / kWave;  // places in rows of 64, one to a lane
constexpr int kRowGroups = 128;
constexpr int kMaxSlices = 16;  // (8: 1 row 18.2 us, 18.1 with 16; 64 rows 27.3, 27.8)
constexpr int kMaxTops = 1280;  // groups of a row whose maxima are kept
constexpr uint32_t kListed = 256;  // equal logits of a part that are listed
constexpr int kSmallCap = 64;  // gathered values below 2^-20
static_assert(kCountWords == 2 * kStride && kStride >= 1 + kValues + kAbove, "counts in LDS");
static_assert(kRows <= 2 * kWave && kValues % kWave == 0, "rows of places: two to a lane");
static_assert(kStride % 4 == 0, "a part's words are whole 16-byte vectors");

template <int NT> using S16 = RowSampler<uint16_t, NT>;
static_assert(alignof(S16<kNT>::Shared) == 16 && offsetof(S16<kNT>::Shared, words) % 16 == 0,
              "counts are accessed by 16-byte vectors");
using S32 = RowSampler<float, kNT32>;

struct Settings {
    const float *temperature;
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
    const float *uniforms;
    float all_temperature;
    int all_top_k;
    float all_top_p;
    float all_min_p;
};

__device__ __forceinline__ RowSettings row_settings(const Settings &st, int64_t row) {
    RowSettings r;
    r.temperature = st.temperature ? st.temperature[row] : st.all_temperature;
    r.top_k = st.top_k ? st.top_k[row] : st.all_top_k;
    r.top_p = st.top_p ? st.top_p[row] : st.all_top_p;
    r.min_p = st.min_p ? st.min_p[row] : st.all_min_p;
    const float u = st.uniforms[row];
    r.u = u > 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.0;
    return r;
}

__global__ __launch_bounds__(kNT32) void sample_f32_kernel(const float *__restrict__ logits, int V,
                                                           double one, Settings st,
                                                           int32_t *__restrict__ tokens,
                                                           float *__restrict__ logprob) {
    __shared__ S32::Shared sh;
    const int64_t row = blockIdx.x;
    const UnitRange ur = unit_range(row, V, 1, Elem<float>::kPerVec);
    S32::run(logits, ur, sh, row_settings(st, row), one, threadIdx.x, tokens + row,
             logprob ? logprob + row : nullptr);
}

// The general path of a bf16 row.
template <int NT>
__device__ __forceinline__ void general_row(const uint16_t *logits, int64_t row, int V,
                                            typename S16<NT>::Shared &sh, const RowSettings &st,
                                            double one, int32_t *token, float *logprob) {
    const UnitRange ur = unit_range(row, V, 1, Elem<uint16_t>::kPerVec);
    S16<NT>::run(logits, ur, sh, st, one, threadIdx.x, token, logprob);
}

// ---- counting ----------------------------------------------------------------------------------

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

// Counts two logits packed in a word: the words' indexes by packed 16-bit arithmetic (a saturating
// subtraction and a minimum), the increments 1 or 2^16 as sign mask + 1. Returns the pair as integers
// in the order of the logits (negative ones with their magnitude inverted); `lowest` becomes 0 in a
// half that met a small value. `high` has the last word that larger values may take, twice.
__device__ __forceinline__ i16x2 tally2(uint32_t *words, uint32_t pair, u16x2 high,
                                        u16x2 &lowest) {
    const u16x2 low = {(uint16_t)(kBase - 1), (uint16_t)(kBase - 1)};
    const u16x2 mag = __builtin_bit_cast(u16x2, pair & 0x7FFF7FFFu);
    const u16x2 at = __builtin_elementwise_min(__builtin_elementwise_sub_sat(mag, low), high);
    lowest = __builtin_elementwise_min(lowest, at);
    const uint32_t mask = __builtin_bit_cast(uint32_t, __builtin_bit_cast(i16x2, pair) >> 15);
    const u16x2 sign = __builtin_bit_cast(u16x2, mask);
    __hip_atomic_fetch_add(words + at.x, (uint32_t)sign.x + 1u, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_WORKGROUP);
    __hip_atomic_fetch_add(words + at.y, (uint32_t)sign.y + 1u, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_WORKGROUP);
    return __builtin_bit_cast(i16x2, pair ^ (mask & 0x7FFF7FFFu));
}
__device__ __forceinline__ int order_key(float value) {  // of a bf16 value, as tally2 returns it
    const int h = (int)(__float_as_uint(value)) >> 16;
    return h ^ ((h >> 15) & 0x7FFF);
}

// Counts one logit.
__device__ __forceinline__ void tally(uint32_t *words, uint32_t h) {
    const int at = min(max((int)(h & 0x7FFFu) - (kBase - 1), 0), kValues + 1);
    __hip_atomic_fetch_add(words + at, (h >> 15) * 65535u + 1u, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_WORKGROUP);
}

__device__ __forceinline__ i16x2 tally_vector(uint32_t *words, const u32x4 &v, u16x2 high,
                                              u16x2 &lowest) {
    const i16x2 a = __builtin_elementwise_max(tally2(words, v.x, high, lowest),
                                              tally2(words, v.y, high, lowest));
    const i16x2 b = __builtin_elementwise_max(tally2(words, v.z, high, lowest),
                                              tally2(words, v.w, high, lowest));
    return __builtin_elementwise_max(a, b);
}

// A group is what eight neighbouring threads load in one batch of the stream (256 logits); the rest
// of the part, less than a batch, makes a last row of groups. The largest logit of each group tells
// later where a value can be found. kGroupLanes lanes' maximum, in each of them:
constexpr int kGroupLanes = 8;
__device__ __forceinline__ int group_max(i16x2 m) {
    int v = max((int)m.x, (int)m.y);
    v = max(v, __builtin_amdgcn_mov_dpp(v, kDppQuadXor1, 0xF, 0xF, true));
    v = max(v, __builtin_amdgcn_mov_dpp(v, kDppQuadXor2, 0xF, 0xF, true));
    return max(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));  // row_half_mirror
}

// What a workgroup keeps of its stream beside the counts (null pointers: nothing).
struct Notes {
    int16_t *tops;         // maxima of the part's groups
    uint64_t *small_keys;  // the row's values below 2^-20: candidate keys, at most kSmallCap
    uint32_t *small_n;     // how many there were
};

__device__ __forceinline__ void note_small(const Notes &notes, uint32_t h, int64_t id) {
    if ((h & 0x7FFFu) >= kBase) return;
    const uint32_t at = atomicAdd(notes.small_n, 1u);
    if (at < kSmallCap) notes.small_keys[at] = cand_key(__uint_as_float(h << 16), (int32_t)id);
}
__device__ __forceinline__ void note_small(const Notes &notes, const u32x4 &v, int64_t id) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) note_small(notes, (w[k / 2] >> (16 * (k & 1))) & 0xFFFFu, id + k);
}

// Counts a part by NT threads.
template <int NT>
__device__ __forceinline__ void count_part(const uint16_t *logits, const UnitRange &ur,
                                           uint32_t *words, const Notes &notes, int tid) {
    constexpr int kStep = NT * kStreamVectors, kPerBatch = NT / kGroupLanes;
    const int slot = tid / kGroupLanes;
    const bool first = (tid & (kGroupLanes - 1)) == 0, keep = notes.tops != nullptr;
    const int64_t id0 = ur.c0 * 8 - ur.g0;
    const uint16_t top = (uint16_t)(kValues + 1 + (tid & (kAbove - 1)));
    const u16x2 high = {top, top};
    i16x2 rest = {-32768, -32768};
    stream<NT>(
        reinterpret_cast<const u32x4 *>(logits) + ur.c0, ur.nv, tid,
        [&](const u32x4 *v, int i) {
            u16x2 lowest = {0xFFFF, 0xFFFF};
            i16x2 m = tally_vector(words, v[0], high, lowest);
#pragma unroll
            for (int u = 1; u < kStreamVectors; ++u)
                m = __builtin_elementwise_max(m, tally_vector(words, v[u], high, lowest));
            if (keep) {
                const int top = group_max(m);
                if (first) notes.tops[i / kStep * kPerBatch + slot] = (int16_t)top;
                if (lowest.x == 0 || lowest.y == 0) {  // rare
                    for (int u = 0; u < kStreamVectors; ++u) {
                        // (one vector at a time, read again: the registers are not to be indexed)
                        const int j = i + u * NT;
                        note_small(notes, reinterpret_cast<const u32x4 *>(logits)[ur.c0 + j],
                                   id0 + (int64_t)j * 8);
                    }
                }
            }
        },
        [&](const u32x4 &v, int i) {
            u16x2 lowest = {0xFFFF, 0xFFFF};
            rest = __builtin_elementwise_max(rest, tally_vector(words, v, high, lowest));
            if (keep && (lowest.x == 0 || lowest.y == 0))
                note_small(notes, v, id0 + (int64_t)i * 8);
        });
    if (keep) {
        const int top = group_max(rest);
        if (first) notes.tops[ur.nv / kStep * kPerBatch + slot] = (int16_t)top;
    }
    const int64_t e = ragged_element(ur, tid);
    if (e >= 0) {
        tally(words, logits[e]);
        if (keep) note_small(notes, (uint32_t)logits[e], e - ur.g0);
    }
}

// The value at place q of the candidate order: positive values from the largest down, then the
// negative ones.
__device__ __forceinline__ uint32_t place_word(int q) {  // its word
    return (uint32_t)(q < kValues ? kValues - q : q - kValues + 1);
}
__device__ __forceinline__ float place_value(int q) {
    const uint32_t mag = place_word(q) + (kBase - 1);
    return __uint_as_float((q < kValues ? mag : mag | 0x8000u) << 16);
}
__device__ __forceinline__ uint32_t half(uint32_t word, bool negative) {
    return negative ? word >> 16 : word & 0xFFFFu;
}

// Where the counts of a row's parts are: in this workgroup's LDS, ...
template <int NT>
struct LocalCounts {
    static constexpr int kPartThreads = NT / kParts;
    const uint32_t *words;  // [kParts][kStride]
    const int16_t *maxima;  // of the parts' groups, `stride` apart; null: not kept
    int stride;
    __device__ __forceinline__ bool has_tops() const { return maxima != nullptr; }
    __device__ __forceinline__ bool small_listed() const { return maxima != nullptr; }
    __device__ __forceinline__ const int16_t *tops(int p) const { return maxima + p * stride; }
    __device__ __forceinline__ int parts() const { return kParts; }
    __device__ __forceinline__ uint32_t part(int p, uint32_t word, bool negative) const {
        return half(words[p * kStride + word], negative);
    }
    __device__ __forceinline__ uint32_t count(uint32_t word, bool negative) const {
        uint32_t n = 0;
#pragma unroll
        for (int p = 0; p < kParts; ++p) n += half(words[p * kStride + word], negative);
        return n;
    }
};

// ... or in the workspace, with their sums in LDS (positive, then negative).
struct SlicedCounts {
    static constexpr int kPartThreads = kNT;
    const uint32_t *words;  // [slices][kStride]
    const uint32_t *sums;   // [2][kStride]
    int slices;
    __device__ __forceinline__ bool has_tops() const { return false; }
    __device__ __forceinline__ bool small_listed() const { return false; }
    __device__ __forceinline__ const int16_t *tops(int) const { return nullptr; }
    __device__ __forceinline__ int parts() const { return slices; }
    __device__ __forceinline__ uint32_t part(int p, uint32_t word, bool negative) const {
        return half(words[(size_t)p * kStride + word], negative);
    }
    __device__ __forceinline__ uint32_t count(uint32_t word, bool negative) const {
        return sums[(negative ? kStride : 0) + word];
    }
};

// ---- a row from its counts -----------------------------------------------------------------------
//
// The 7168 places are kRows rows of 64, a place to a lane. The waves take the rows in turn for their
// counts and masses; after that one wave holds all rows' running sums (lane l: rows 2l and 2l + 1)
// and finds each cut by itself, first among the rows, then among the row's lanes: no barriers. (When
// all waves did the same, to save handing the result on, that cost the many-rows pass a third of its
// time: it is a long chain of fp64 instructions, and a SIMD issues one in four cycles.)

// Two rows per lane: masses and counts, and what lies before them.
struct Rows {
    double mass[2], below[2];
    uint32_t count[2], before[2];
};

// The gathered small values (|x| < 2^-20), in candidate order.
struct Small {
    int n;
    double mass, below;
    uint32_t before;
};

// The value a cut falls on.
struct Spot {
    float value;
    double w, below;
    uint32_t size, before;
    int small;  // index into the gathered small values, -1 if a counted value
    int q;
};

template <int NT, typename Counts>
__device__ __forceinline__ Spot find_spot(const typename S16<NT>::Shared &sh, const Counts &counts,
                                          const Weights &w, const Rows &rows, const Small &small,
                                          Cut cut, double target, uint32_t nth, int lane) {
    auto meets = [&](double mass, uint32_t number) {
        return cut == kNumber ? number >= nth : cut == kReach ? mass >= target : mass > target;
    };
    uint64_t in[2], any[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        any[i] = __ballot(rows.count[i] > 0);
        in[i] = any[i] & __ballot(meets(rows.below[i] + rows.mass[i], rows.before[i] + rows.count[i]));
    }
    int row;
    if (in[0] | in[1]) {
        const int l = __builtin_ctzll(in[0] | in[1]);
        row = 2 * l + ((in[0] >> l) & 1 ? 0 : 1);
    } else {
        row = 2 * kRows;
    }
    Spot s;
    s.small = -1;
    if (small.n > 0 && row >= kRows / 2 &&
        (meets(small.below + small.mass, small.before + (uint32_t)small.n) ||
         (any[0] | any[1]) == 0ull)) {
        s.q = -1;
        s.below = small.below;
        s.before = small.before;
        s.size = 1;
        for (int i = 0; i < small.n; ++i) {  // few
            s.value = key_logit(sh.list[i]);
            s.w = weight_of(w, s.value);
            s.small = i;
            if (i == small.n - 1 || meets(s.below + s.w, s.before + 1)) break;
            s.below += s.w;
            ++s.before;
        }
        return s;
    }
    if (row >= kRows) {  // roundings left a mass cut behind everything: the last counted value
        const int l = 63 - __builtin_clzll(any[0] | any[1]);
        row = 2 * l + ((any[1] >> l) & 1 ? 1 : 0);
    }
    const int owner = row >> 1;
    const double base = lane_value(row & 1 ? rows.below[1] : rows.below[0], owner);
    const uint32_t start = lane_value(row & 1 ? rows.before[1] : rows.before[0], owner);
    const int q = row * kWave + lane;
    const float value = place_value(q);
    const bool counted = value <= w.m && weight_y(w, value) < (double)kFar;
    const uint32_t n = counted ? counts.count(place_word(q), q >= kValues) : 0u;
    const double wt = n > 0 ? weight_of(w, value) : 0.0;
    const double mass = wave_running_sum(wt * (double)n);
    const uint32_t number = wave_running_sum(n);
    const uint64_t here = __ballot(n > 0);
    const uint64_t hit = here & __ballot(meets(base + mass, start + number));
    const int at = hit ? __builtin_ctzll(hit) : here ? 63 - __builtin_clzll(here) : 0;
    s.below = at > 0 ? base + lane_value(mass, at - 1) : base;
    s.before = at > 0 ? start + lane_value(number, at - 1) : start;
    s.value = __uint_as_float(lane_value(__float_as_uint(value), at));
    s.w = lane_value(wt, at);
    s.size = lane_value(n, at);
    s.q = row * kWave + at;
    return s;
}

// Scratch of settle.
template <int NT>
struct SettleShared {
    uint32_t weighed[2 * kWave];  // tokens with weight, by row
    double mass[2 * kWave];
    double heavy[S16<NT>::kWaves];
    uint32_t total[S16<NT>::kWaves];  // by wave: tokens counted, and the first row that holds any
    int first[S16<NT>::kWaves];
    // what is drawn: a value and how many of its equals come before, or a token
    float value;
    uint32_t nth;
    int q;
    int32_t id;
    double share;
    uint32_t hits;  // groups to look through for it
    uint16_t hit[kMaxTops];
};

// Settles a row from the counts of its parts. False (in every thread) if the row is one for the
// general path; nothing is written then.
template <int NT, typename Counts>
__device__ __forceinline__ bool settle(const uint16_t *logits, int64_t row, int V,
                                       const Counts &counts, typename S16<NT>::Shared &sh,
                                       SettleShared<NT> &ss, const RowSettings &st, int tid,
                                       int32_t *token, float *logprob) {
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    // A binade is four rows: two of its positive values, two of its negative ones. The waves take the
    // binades in turn.
    constexpr int kTurns = (kRows / 4 + S16<NT>::kWaves - 1) / S16<NT>::kWaves;
    auto row_of = [&](int binade, int i) {  // descending values: larger magnitudes first, then last
        return i < 2 ? kRows / 2 - 1 - 2 * binade - i : kRows / 2 + 2 * binade + (i - 2);
    };
    S16<NT>::fill_scale(sh, tid);
    uint32_t tokens = 0, held = 0;  // held: which of the wave's binades hold a token
    int first = kRows;
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int binade = wave + k * S16<NT>::kWaves;
        if (binade >= kRows / 4) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row_of(binade, i);
            const uint32_t n = counts.count(place_word(r * kWave + lane), i >= 2);
            tokens += n;
            if (__ballot(n > 0) != 0ull) {
                held |= 1u << k;
                first = min(first, r);
            }
        }
    }
    const uint32_t large_pos = counts.count(kValues + 1 + lane, false);
    const uint32_t large_neg = counts.count(kValues + 1 + lane, true);
    const bool any_large_neg = __ballot(large_neg > 0) != 0ull;
    if (wave == 0) tokens += large_pos + large_neg;
    tokens = wave_running_sum(tokens);
    if (lane == kWave - 1) {
        ss.total[wave] = tokens;
        ss.first[wave] = first;
    }
    if (tid < 2 * kWave) {
        ss.weighed[tid] = 0u;
        ss.mass[tid] = 0.0;
    }
    const uint32_t small_n = counts.count(0, false) + counts.count(0, true);
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int i = 0; i < S16<NT>::kWaves; ++i) {
        total += ss.total[i];
        first = min(first, ss.first[i]);
    }
    if (total + small_n != (uint32_t)V || __ballot(large_pos > 0) != 0ull ||
        small_n > kSmallCap || (first == kRows && small_n == 0))
        return false;
    // the small values, listed and sorted
    Small small{(int)small_n, 0.0, 0.0, 0u};
    if (small_n > 0) {
        if (!counts.small_listed()) {
            if (tid == 0) sh.listed = 0;
            __syncthreads();
            for (int part = 0; part < counts.parts(); ++part) {
                if (counts.part(part, 0, false) + counts.part(part, 0, true) == 0) continue;
                const UnitRange ur = unit_range(row * counts.parts() + part, V, counts.parts(),
                                                Elem<uint16_t>::kPerVec);
                S16<NT>::collect(logits, ur, sh, tid, kSmallCap,
                                 [](float x) { return fabsf(x) < 0x1p-20f; });
            }
            __syncthreads();
        }
        if (tid < kWave) {
            const uint64_t key = wave_sort_desc(lane < (int)small_n ? sh.list[lane] : 0ull, lane);
            sh.list[lane] = key;
        }
        __syncthreads();
    }
    // the maximum: the first place with a count, unless a small value comes before it
    int top_q = 2 * kValues;
    if (first < kRows) {
        const uint32_t n = counts.count(place_word(first * kWave + lane), first >= kRows / 2);
        top_q = first * kWave + __builtin_ctzll(__ballot(n > 0));
    }
    const bool top_small = small_n > 0 && top_q >= kValues;
    const float m = top_small ? key_logit(sh.list[0]) : place_value(top_q);

    if (st.temperature > 0.f) {
        const Weights w{m, kBinsPerE / (double)st.temperature, 1.0, sh.scale, m, 0.0, 1.0};
        if (any_large_neg && !(weight_y(w, -256.f) >= (double)kFar)) return false;
        const bool by_number = st.top_k >= 1, by_weight = st.min_p > 0.f;
        const double least = by_weight ? fmin((double)st.min_p, 1.0) : 0.0;
        double heavy = 0.0;  // mass of the weights that min_p keeps
        // A row's values are equidistant, so its weights are that of its first value times
        // exp(-lane distance / T), which the four rows of a binade share. Lane j has the first
        // weight of the wave's row j. The row of the maximum, which may begin above it, is weighed
        // value by value: the maximum's weight is 1 exactly.
        double base = 0.0;
        if (lane < 4 * kTurns) {
            const int binade = wave + lane / 4 * S16<NT>::kWaves;
            const int r = row_of(min(binade, kRows / 4 - 1), lane & 3);
            base = weight_at(w, fmax(weight_y(w, place_value(r * kWave)), 0.0));
        }
#pragma unroll 1
        for (int k = 0; k < kTurns; ++k) {
            if (!((held >> k) & 1u)) continue;
            const int binade = wave + k * S16<NT>::kWaves;
            const double distance = ldexp(1.0, binade - 27);  // (128 values from 2^(binade - 20) on)
            const double falloff = weight_at(w, distance * (double)lane * w.c);
            double mass[4];
            uint32_t n[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row_of(binade, i);
                n[i] = counts.count(place_word(r * kWave + lane), i >= 2);
                double wt = lane_value(base, 4 * k + i) * falloff;
                if (r == first) {
                    const float x = place_value(r * kWave + lane);
                    wt = x <= m ? weight_of(w, x) : 0.0;
                }
                if (!(wt >= 0x1p-64)) n[i] = 0;
                mass[i] = n[i] > 0 ? wt * (double)n[i] : 0.0;
                if (wt >= least) heavy += mass[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mass[i] = wave_running_sum(mass[i]);
                // (how many they are matters to top-k only; otherwise whether there are any)
                n[i] = by_number ? wave_running_sum(n[i]) : (uint32_t)(__ballot(n[i] > 0) != 0ull);
            }
            if (lane == kWave - 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ss.mass[row_of(binade, i)] = mass[i];
                    ss.weighed[row_of(binade, i)] = n[i];
                }
            }
        }
        for (int i = 0; i < small.n; ++i) {
            const float x = key_logit(sh.list[i]);
            if (!(weight_y(w, x) < (double)kFar)) {  // (they are in order: the rest has none either)
                small.n = i;
                break;
            }
            const double wt = weight_of(w, x);
            small.mass += wt;
            if (tid == 0 && wt >= least) heavy += wt;
        }
        if (by_weight) {
            heavy = wave_running_sum(heavy);
            if (lane == kWave - 1) ss.heavy[wave] = heavy;
        }
        __syncthreads();
        if (wave == 0) {
            Rows rows;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                rows.mass[i] = ss.mass[2 * lane + i];
                rows.count[i] = ss.weighed[2 * lane + i];
            }
            const double upto = wave_running_sum(rows.mass[0] + rows.mass[1]);
            const uint32_t upto_n = wave_running_sum(rows.count[0] + rows.count[1]);
            rows.below[0] = dpp_or_zero<0x138, 0xF>(upto);  // wave_shr:1
            rows.before[0] = upto_n - rows.count[0] - rows.count[1];
            double z = lane_value(upto, kWave - 1);
            uint32_t number = lane_value(upto_n, kWave - 1);
            if (small.n > 0) {  // between the positive and the negative values
                small.below = lane_value(upto, kRows / 4 - 1);
                small.before = lane_value(upto_n, kRows / 4 - 1);
                if (lane >= kRows / 4) {
                    rows.below[0] += small.mass;
                    rows.before[0] += (uint32_t)small.n;
                }
                z += small.mass;
                number += (uint32_t)small.n;
            }
            rows.below[1] = rows.below[0] + rows.mass[0];
            rows.before[1] = rows.before[0] + rows.count[0];
            // top-k, top-p and the draw, in one loop: one copy of the search
            double whole = z;
            Spot s;
            uint32_t taken = 0;
#pragma unroll 1
            for (int step = 0; step < 3; ++step) {
                Cut cut = kNumber;
                double target = 0.0;
                if (step == 0) {
                    if (!by_number || (uint32_t)st.top_k >= number) continue;
                } else if (step == 1) {
                    if (!(st.top_p < 1.f)) continue;
                    cut = kReach;
                    target = (double)st.top_p * z;
                } else {
                    if (by_weight) {
                        double sum = 0.0;
                        for (int i = 0; i < S16<NT>::kWaves; ++i) sum += ss.heavy[i];
                        whole = fmin(whole, sum);
                    }
                    cut = kPass;
                    target = st.u * whole;
                }
                s = find_spot<NT>(sh, counts, w, rows, small, cut, target, (uint32_t)st.top_k, lane);
                const Place p = cut_equal(s.value, s.w, s.size, cut, target, (uint32_t)st.top_k, s.below,
                                          s.before);
                if (step == 0) z = p.mass;
                if (step < 2) whole = fmin(whole, p.mass);
                taken = p.nth;
            }
            if (lane == 0) {
                ss.value = s.value;
                ss.nth = taken;
                ss.q = s.q;
                ss.id = s.small >= 0 ? key_id(sh.list[s.small]) : -1;
                ss.share = s.w / whole;
                ss.hits = 0;
                sh.listed = 0;
            }
        }
    } else if (tid == 0) {
        ss.value = m;
        ss.nth = 0;
        ss.q = top_q;
        ss.id = top_small ? key_id(sh.list[0]) : -1;
        ss.share = 1.0;
        ss.hits = 0;
        sh.listed = 0;
    }
    __syncthreads();
    if (tid == NT - 1 && logprob) *logprob = (float)log(ss.share);
    if (ss.id >= 0) {
        if (tid == 0) *token = ss.id;
        return true;
    }
    // number nth of its equals: the part that holds it, then the logit itself
    const float value = ss.value;
    const uint32_t nth = ss.nth;
    const int q = ss.q;
    const uint32_t n = lane < counts.parts() ? counts.part(lane, place_word(q), q >= kValues) : 0u;
    const uint32_t upto = wave_running_sum(n);
    const int part = __builtin_ctzll(__ballot(upto > nth));
    const uint32_t equal = lane_value(n, part);
    const uint32_t left = nth - (lane_value(upto, part) - equal);
    const UnitRange ur =
        unit_range(row * counts.parts() + part, V, counts.parts(), Elem<uint16_t>::kPerVec);
    if (!counts.has_tops() || equal > kListed) {
        uint32_t found;
        const int32_t id = S16<NT>::nth_equal(logits, ur, sh, tid, value, left, found);
        if (tid == 0) *token = id;
        return true;
    }
    // Only groups whose maximum reaches the value can hold it: near the top, few of them.
    constexpr int kPart = Counts::kPartThreads;
    constexpr int kStep = kPart * kStreamVectors, kPerBatch = kPart / kGroupLanes;
    const int key = order_key(value);
    const int16_t *tops = counts.tops(part);
    const int groups = (ur.nv / kStep + 1) * kPerBatch;
    for (int g = tid; g < groups; g += NT)
        if (tops[g] >= key) ss.hit[atomicAdd(&ss.hits, 1u)] = (uint16_t)g;
    const int32_t id0 = (int32_t)(ur.c0 * Elem<uint16_t>::kPerVec - ur.g0);
    const uint32_t pattern = __float_as_uint(value) >> 16;
    const int64_t e = ragged_element(ur, tid);
    if (e >= 0 && logits[e] == pattern) sh.list[atomicAdd(&sh.listed, 1u)] = (uint32_t)(e - ur.g0);
    __syncthreads();
    const u32x4 *p = reinterpret_cast<const u32x4 *>(logits) + ur.c0;
    for (int h = tid / kGroupLanes; h < (int)ss.hits; h += NT / kGroupLanes) {
        const int g = ss.hit[h];
        const int i = g / kPerBatch * kStep + g % kPerBatch * kGroupLanes + (tid & (kGroupLanes - 1));
        u32x4 v[kStreamVectors];
#pragma unroll
        for (int u = 0; u < kStreamVectors; ++u) {
            v[u] = u32x4{};  // (zeros match nothing: small values are not looked for here)
            if (i + u * kPart < ur.nv) v[u] = p[i + u * kPart];
        }
#pragma unroll
        for (int u = 0; u < kStreamVectors; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (((w[k / 2] >> (16 * (k & 1))) & 0xFFFFu) == pattern)
                    sh.list[atomicAdd(&sh.listed, 1u)] = (uint32_t)(id0 + (i + u * kPart) * 8 + k);
        }
    }
    __syncthreads();
    if (tid < (int)equal) {  // all `equal` of them are listed: number `left` by id
        const uint32_t id = (uint32_t)sh.list[tid];
        uint32_t before = 0;
        for (uint32_t i = 0; i < equal; ++i) before += (uint32_t)sh.list[i] < id ? 1u : 0u;
        if (before == left) *token = (int32_t)id;
    }
    return true;
}

// A row per workgroup.
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(4))) void
sample_bf16_kernel(const uint16_t *__restrict__ logits, int V, double one, Settings st,
                   int32_t *__restrict__ tokens, float *__restrict__ logprob) {
    __shared__ typename S16<kNT>::Shared sh;
    __shared__ SettleShared<kNT> ss;
    __shared__ int16_t maxima[kMaxTops];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    constexpr int kGroup = kNT / kParts;
    const int part = tid / kGroup;
    const UnitRange ur = unit_range(row * kParts + part, V, kParts, Elem<uint16_t>::kPerVec);
    const RowSettings rs = row_settings(st, row);
    u32x4 *clear = reinterpret_cast<u32x4 *>(sh.words);
    for (int i = tid; i < kParts * kStride / 4; i += kNT) clear[i] = u32x4{0u, 0u, 0u, 0u};
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    // (the longest part has at most V / 8 / kParts + 1 vectors)
    const int stride = (V / 8 / kParts / (kGroup * kStreamVectors) + 2) * (kGroup / kGroupLanes);
    const bool keep = kParts * stride <= kMaxTops;
    Notes notes{nullptr, sh.list, &sh.listed};
    if (keep) notes.tops = maxima + part * stride;
    count_part<kGroup>(logits, ur, sh.words + part * kStride, notes, tid & (kGroup - 1));
    __syncthreads();
    int32_t *token = tokens + row;
    float *lp = logprob ? logprob + row : nullptr;
    const LocalCounts<kNT> counts{sh.words, keep ? maxima : nullptr, stride};
    if (!settle<kNT>(logits, row, V, counts, sh, ss, rs, tid, token, lp)) {
        __syncthreads();
        general_row<kNT>(logits, row, V, sh, rs, one, token, lp);
    }
}

// A slice per workgroup: its counts go to the workspace, [R][slices][kStride].
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(4))) void
sample_count_kernel(const uint16_t *__restrict__ logits, int V, int slices,
                    uint32_t *__restrict__ words) {
    __shared__ __attribute__((aligned(16))) uint32_t sh[kStride];
    const int tid = threadIdx.x;
    const UnitRange ur = unit_range(blockIdx.x, V, slices, Elem<uint16_t>::kPerVec);
    u32x4 *clear = reinterpret_cast<u32x4 *>(sh);
    for (int i = tid; i < kStride / 4; i += kNT) clear[i] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    count_part<kNT>(logits, ur, sh, Notes{nullptr, nullptr, nullptr}, tid);
    __syncthreads();
    u32x4 *out = reinterpret_cast<u32x4 *>(words + (size_t)blockIdx.x * kStride);
    for (int i = tid; i < kStride / 4; i += kNT) out[i] = clear[i];
}

// Joins a row's slices and settles it.
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(4))) void
sample_settle_kernel(const uint16_t *__restrict__ logits, int V, int slices, double one,
                     Settings st, const uint32_t *__restrict__ words,
                     int32_t *__restrict__ tokens, float *__restrict__ logprob) {
    __shared__ S16<kNT>::Shared sh;
    __shared__ SettleShared<kNT> ss;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const uint32_t *mine = words + (size_t)row * slices * kStride;
    uint32_t *sums = sh.words;  // [2][kStride]
    for (int i = tid; i < kStride / 4; i += kNT) {
        u32x4 v[kMaxSlices];  // all in flight together
#pragma unroll
        for (int s = 0; s < kMaxSlices; ++s) {
            v[s] = u32x4{0u, 0u, 0u, 0u};
            if (s < slices) v[s] = reinterpret_cast<const u32x4 *>(mine + (size_t)s * kStride)[i];
        }
        u32x4 lo = u32x4{0u, 0u, 0u, 0u}, hi = lo;
#pragma unroll
        for (int s = 0; s < kMaxSlices; ++s) {
            lo += v[s] & 0xFFFFu;
            hi += v[s] >> 16;
        }
        reinterpret_cast<u32x4 *>(sums)[i] = lo;
        reinterpret_cast<u32x4 *>(sums + kStride)[i] = hi;
    }
    __syncthreads();
    const RowSettings rs = row_settings(st, row);
    int32_t *token = tokens + row;
    float *lp = logprob ? logprob + row : nullptr;
    if (!settle<kNT>(logits, row, V, SlicedCounts{mine, sums, slices}, sh, ss, rs, tid, token, lp)) {
        __syncthreads();
        general_row<kNT>(logits, row, V, sh, rs, one, token, lp);
    }
}

// Slices per bf16 row: 1 (sample_bf16_kernel) where rows are many or short, otherwise about 512
// workgroups in all, of two vectors and more per thread. Slices read a row faster, but their counts
// go through the workspace to a second kernel, which costs more the more rows there are. Measured,
// one workgroup per row against slices (us, N(0, 2.5) logits, top-p): V = 32000: 1 row 14.9 / 16.7,
// 64 rows 16.4 / 20.0; V = 65536: 1 row 19.0 / 18.0, 8 rows 19.3 / 18.2, 64 rows 20.2 / 24.5;
// V = 100001: 8 rows 23.7 / 19.0, 64 rows 24.3 / 24.8; V = 151936: 1 row 26.9 / 18.0, 64 rows
// 29.6 / 26.7, 100 rows 30.1 / 30.0, 127 rows 30.8 / 33.2, 192 rows 31.3 / 43.7; V = 262144: 64 rows
// 41.6 / 30.5, 127 rows 43.3 / 41.9. (256 or 1024 workgroups in place of 512: 64 rows x 151936
// 27.9 / 28.3 against 26.7.)
int plan_slices(int R, int V) {
    if (R >= kRowGroups || V <= 60000 + 1000 * R) return 1;
    int s = 512 / R;
    if (s > kMaxSlices) s = kMaxSlices;
    const int most = V / 8 / (2 * kNT);
    return s > most ? most : s;
}

}  // namespace

size_t sample_workspace_bytes(int R, int V, int dtype) {
    const int slices = dtype == 0 ? 1 : plan_slices(R, V);
    return slices == 1 ? 0 : (size_t)R * slices * kStride * sizeof(uint32_t);
}

hipError_t launch_sample(const void *logits, int dtype, int R, int V, const float *temperature,
                         float all_temperature, const int32_t *top_k, int all_top_k,
                         const float *top_p, float all_top_p, const float *min_p, float all_min_p,
                         const float *uniforms, int32_t *tokens, float *logprob, void *ws,
                         hipStream_t stream) {
    const Settings st{temperature, top_k, top_p, min_p, uniforms, all_temperature, all_top_k,
                      all_top_p, all_min_p};
    // A bin's sum of up to V factors, each at most 1.011, stays below 2^64. (A weight errs by half a step
    // of its factor: below 2^-40 of itself with 40 bits behind the point and more, below 2^-frac with
    // fewer.)
    int bits = 0;
    while ((1ll << bits) <= V) ++bits;
    const int frac = bits <= 22 ? 41 : 63 - bits;
    const double one = (double)(1ull << frac);
    const dim3 rows((unsigned)R);
    if (dtype == 0) {
        hipLaunchKernelGGL(sample_f32_kernel, rows, dim3(kNT32), 0, stream,
                           static_cast<const float *>(logits), V, one, st, tokens, logprob);
        return hipGetLastError();
    }
    const uint16_t *x = static_cast<const uint16_t *>(logits);
    const int slices = plan_slices(R, V);
    if (slices == 1) {
        hipLaunchKernelGGL(sample_bf16_kernel, rows, dim3(kNT), 0, stream, x, V, one,
                           st, tokens, logprob);
        return hipGetLastError();
    }
    uint32_t *words = static_cast<uint32_t *>(ws);
    hipLaunchKernelGGL(sample_count_kernel, dim3((unsigned)(R * slices)), dim3(kNT), 0, stream, x,
                       V, slices, words);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sample_settle_kernel, rows, dim3(kNT), 0, stream, x, V, slices, one, st,
                       words, tokens, logprob);
    return hipGetLastError();
}

}  // namespace dflash2
