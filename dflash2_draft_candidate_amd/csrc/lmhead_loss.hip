// The loss of the LM head's product without its logits: softmax cross entropy with a target token,
// or the distillation loss from a teacher's top entries, and the gradients of the hidden states
// and of the head's weight.
//
//   x[r][v] = sum_h hidden[r][h] W[v][h];  q = softmax(x[r] / tau);  p = the teacher's softmax
//   over the row's entries (one entry with p = 1 for a target token)
//   loss[r] = tau^2 sum_j p_j (ln p_j - ln q[id_j])
//   G[r][v] = g[r] tau (q[r][v] - sum_{j: id_j = v} p_j)
//   grad_hidden = G W;  grad_W = G^T hidden
//
// Design (gfx950):
//   * Rows without an entry (prompts, padding) are left out: a first kernel copies the other rows'
//     hidden states behind one another (what stands in the rows left out, NaN among it, is never
//     read), and the products run over those alone. Their number stays on the device; workgroups
//     whose tile lies behind it end at once. Up to 64 bf16 rows stay where they are: the product's
//     workgroups look the kept ones up.
//   * Forward: the product's tiles (W's rows x hidden rows) end in a maximum and a sum of
//     exponentials per hidden row, 8 bytes instead of a tile of logits; a second kernel joins
//     them. The logits of the entries come out of the product (up to 64 bf16 rows), or from the
//     first kernel, which repeats the product's instructions for them.
//   * Backward: for a piece of the vocabulary at a time, the product again (the same sums in the
//     same order) with G as its epilogue, in a buffer of at most kPieceBytes; then the entries of
//     the piece; then the two products that read the piece. grad_hidden is summed over the pieces
//     in fp32, split along the vocabulary where it has few tiles.
//   * Three ways through the products. bf16, more than 128 rows: streams of 256 x 256 tiles, bound
//     by the matrix cores (and by the card's power). Fewer rows, f32, and logits of few such tiles:
//     rings, which read W in tiles as narrow as the rows, or of 128 rows. At most 32 bf16 rows of
//     1024 < H <= 4096: W in whole rows (lmhead_rows.h), bound by its bytes.
//   * bf16: G is rounded to bf16 for the matrix cores (2^-8 of each value, as a bf16 gradient of logits
//     would be). Up to 64 rows it is kept in two parts; above, what rounding left of it at the entries, its
//     largest values, is added to both gradients. Everything else is fp32. f32 inputs take the f32 matrix
//     instructions throughout.
#include <type_traits>

#include "dflash2.h"
#include "gemm_tile.h"
#include "kernels.h"

namespace dflash2 {
namespace {

constexpr int kTile = 256;                       // rows of W (or columns of hidden) per tile
constexpr int64_t kPieceBytes = 256ll << 20;     // of G
constexpr int kPieceMost = 1 << 20;              // columns of a piece (32-bit offsets in it)
constexpr int kPlaceGroup = 8;                   // rows of tiles that share columns of tiles
constexpr int kCus = 256;
// Up to so many 256 x 256 tiles of logits, the rings' tiles of half that size give every CU one at most.
// Forward, H = 4096: 256 rows x 32000 (125 tiles) 90 us, as streams 111; 1024 rows x 8000 (128) 80 and 105;
// 384 rows x 32000 (250) 148 and 118.
constexpr int kRingTiles = kCus / 2;
constexpr int kBothGroups = kCus / 2;  // (launch_both)

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Few kept rows: ranges of the vocabulary (of `width` columns, 16 at least each) for nr tiles of kept
// rows: a workgroup per CU.
__host__ __device__ __forceinline__ int few_ranges(int width, int nr) {
    const int units = (width + 15) / 16, most = nr > kCus ? 1 : kCus / (nr > 0 ? nr : 1);
    return units < most ? units : most;
}

// What a row's kept statistics hold, [K + 2] floats: the maximum of its logits, the sum of
// exp((x - max) / tau) (kLeftOut: a row without an entry), the entries' logits.
constexpr float kLeftOut = -1.f;

struct Entries {
    const int32_t *ids;     // [R, K]
    const float *teacher;   // [R, K], or null: every entry has mass 1 (K = 1)
    int K;
    float tau;
};

__device__ __forceinline__ bool id_ok(int id, int V) { return id >= 0 && id < V; }

// Over the wave's lanes, in every lane, in the VALU.
template <typename F>
__device__ __forceinline__ float wave_fold(float x, int lane, F f) {
    x = f(x, __uint_as_float(xor_lane<1>(__float_as_uint(x), lane)));
    x = f(x, __uint_as_float(xor_lane<2>(__float_as_uint(x), lane)));
    x = f(x, __uint_as_float(xor_lane<4>(__float_as_uint(x), lane)));
    x = f(x, __uint_as_float(xor_lane<8>(__float_as_uint(x), lane)));
    x = f(x, __uint_as_float(xor_lane<16>(__float_as_uint(x), lane)));
    return f(x, __uint_as_float(xor_lane<32>(__float_as_uint(x), lane)));
}

__device__ __forceinline__ float wave_sum(float x, int lane) {
    return wave_fold(x, lane, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ float wave_max(float x, int lane) {
    return wave_fold(x, lane, [](float a, float b) { return fmaxf(a, b); });
}

template <int S>
__device__ __forceinline__ double add_lane(double x, int lane) {
    return x + __longlong_as_double((long long)xor_lane64<S>((uint64_t)__double_as_longlong(x), lane));
}

__device__ __forceinline__ double wave_sum(double x, int lane) {
    x = add_lane<2>(add_lane<1>(x, lane), lane);
    x = add_lane<8>(add_lane<4>(x, lane), lane);
    return add_lane<32>(add_lane<16>(x, lane), lane);
}

// g tau / sum, and g tau times a mass: g tau alone may pass the largest float.
__device__ __forceinline__ float grad_scale(float g, float tau, float sum) {
    return (float)((double)g * (double)tau / (double)sum);
}
__device__ __forceinline__ float grad_mass(float g, float tau, float mass) {
    return (float)((double)g * (double)tau * (double)mass);
}

// Between a wave's writes of LDS and its other lanes' reads (LDS keeps a wave's order): for the compiler.
__device__ __forceinline__ void wave_lds_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// ---- the entries by columns ------------------------------------------------------------------------
// G of more than 64 bf16 rows is in one bf16 part. Its largest values, and most of what their rounding costs the
// gradients, are the entries' (q - p against a q): what rounding left of those is added to both gradients'
// fp32 sums, to grad_hidden with the entry's row of W (lmloss_hidden_out_kernel), to grad_W with the
// row's hidden state (add_listed). Entries of less than a 32nd of the row's largest mass are left as they are: even
// 63 of them come to a quarter of that one's rounding (64 entries a row, as a teacher's top logits fall: a third of
// them remain). For grad_W the entries are listed by units of 64 columns, in the order of the rows.
// The gradients' error, relative and over all elements, with and without: 1024 rows x 4096 x 151936, 0.00167 and
// 0.0024; rounded output alone 0.00166. It costs 1 - 2 % of a call with one entry a row (1024 rows: 4.23 ms and 4.31),
// 5 % with 64 (4.29 and 4.51), more where the vocabulary is small (kMany).
struct Listed {
    uint32_t where;  // the row, the column in the unit << 16
    int entry;       // of all rows' entries
};
static_assert(DFLASH2_MAX_LMHEAD_LOSS_ROWS <= 1 << 16, "Listed::where");
constexpr int kUnit = 64, kListUnits = 16;  // columns; units a workgroup lists at most
// From a quarter of the rows' number on (K entries a row of V / kMany columns) a unit's listed entries, 16 at a
// time, take grad_W's tiles longer than a second part of G, all zeros but for the entries' rests. The backward call
// with lists and with two parts: 2476 rows x 2592, 42 of 2575, 531 us and 335; 2048 x 512, 64 of 8000, 271 and 196;
// 2476 x 2592, 42 of 10000, 654 and 631; 4096 x 1024, 8 of 2048, 296 and 277, 4 of 2048, 246 and 274; 1024 x 4096,
// 64 of 16000, 562 and 565, of 40000, 1114 and 1231 (none of it kept: 233, 131, 443, 190, 189, 406 and 915).
constexpr int kMany = 256;

struct ListedRest {
    const Listed *list;
    const int2 *units;       // a unit's first entry in the list, and behind its last
    const float *left;       // [R, K] what rounding left of G (entries that are none, rows left out: anything)
    const uint16_t *hidden;  // [R, H], all rows
};

constexpr float kLn32 = 3.4657359f;  // (a 32nd of the largest mass)

struct ListsJob {
    const int32_t *ids;
    const uint64_t *mask;  // null: all; a row's entries of a 32nd of its largest mass and more
    int n, K, V;           // entries of all rows
    uint32_t inverse;      // 2^32 / K rounded up; K = 1: 0
    int per, groups;       // units a workgroup lists, workgroups
    Listed *list;
    int2 *units;
};

// A workgroup lists the entries of `per` units: it counts them, and those before its units (where its part of the
// list starts), and puts them there. Each wave takes a contiguous part of the entries; what it has found waits
// in LDS (of more than kWaiting it goes through all entries again).
template <int THREADS> struct Lists {
    static constexpr int kWaves = THREADS / kWave, kAhead = 8, kWaiting = 256;
    struct Waiting {
        int entry, column;
    };
    struct Lds {
        Waiting waiting[kWaves][kWaiting];
        int count[kWaves][kListUnits], total[kListUnits], before[kWaves];
    };

    static __device__ __forceinline__ void run(const ListsJob &job, int block, Lds &lds, int wave, int lane) {
        const int first = block * job.per * kUnit, end = min(first + job.per * kUnit, job.V);
        const int e0 = (int)((int64_t)job.n * wave / kWaves), e1 = (int)((int64_t)job.n * (wave + 1) / kWaves);
        const uint64_t below = (1ull << lane) - 1;
        // (exact below 2^22, and there are not more)
        const auto row_of = [&](int e) { return job.inverse ? (int)__umulhi((uint32_t)e, job.inverse) : e; };
        // f(entry, column, whether it is listed here, whether before) for a wave's entries, 64 at a time
        const auto each = [&](auto f) {
            for (int base = e0; base < e1; base += kAhead * kWave) {
                int id[kAhead];
                uint64_t takes[kAhead];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int e = min(base + a * kWave + lane, e1 - 1), r = row_of(e);
                    id[a] = job.ids[e];
                    takes[a] = job.mask ? job.mask[r] >> (e - r * job.K) : 1ull;
                }
                __builtin_amdgcn_sched_barrier(0);  // (all loads at once)
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int e = base + a * kWave + lane;
                    if (e >= e1) id[a] = -1;
                    f(e, id[a] - first, id[a] >= first && id[a] < end && (takes[a] & 1ull) != 0ull,
                      id[a] >= 0 && id[a] < first);
                }
            }
        };
        // g(unit, the lanes whose entries are listed in it, in one of these) for each unit among them
        const auto each_unit = [&](int column, bool in, auto g) {
            const int unit = column / kUnit;
            for (uint64_t m = __ballot(in); m != 0ull;) {
                const int u = __builtin_amdgcn_readlane(unit, __builtin_ctzll(m));
                const uint64_t same = __ballot(in && unit == u);
                g(u, same, in && unit == u);
                m &= ~same;
            }
        };
        int mine = 0, earlier = 0, found = 0;  // mine: lane u: entries of unit u
        each([&](int e, int column, bool in, bool is_before) {
            earlier += __popcll(__ballot(is_before));
            const uint64_t m = __ballot(in);
            if (m == 0ull) return;
            const int at = found + __popcll(m & below);
            if (in && at < kWaiting) lds.waiting[wave][at] = Waiting{e, column};
            found += __popcll(m);
            each_unit(column, in, [&](int u, uint64_t same, bool) { mine += lane == u ? __popcll(same) : 0; });
        });
        if (lane < kListUnits) lds.count[wave][lane] = mine;
        if (lane == 0) lds.before[wave] = earlier;
        __syncthreads();
        if (threadIdx.x < kListUnits) {
            int n = 0;
            for (int w = 0; w < kWaves; ++w) n += lds.count[w][threadIdx.x];
            lds.total[threadIdx.x] = n;
        }
        __syncthreads();
        int at = 0;  // lane u: where the wave's next entry of unit u goes
        if (lane < kListUnits) {
            for (int w = 0; w < kWaves; ++w) at += lds.before[w];
            for (int u = 0; u < lane; ++u) at += lds.total[u];
            if (wave == 0 && lane < job.per) job.units[block * job.per + lane] = int2{at, at + lds.total[lane]};
            for (int w = 0; w < wave; ++w) at += lds.count[w][lane];
        }
        const auto put = [&](int e, int column, bool in) {
            each_unit(column, in, [&](int u, uint64_t same, bool here) {
                const int to = __shfl(at, u, kWave) + __popcll(same & below);
                if (here)
                    job.list[to] = Listed{(uint32_t)row_of(e) | (uint32_t)(column % kUnit) << 16, e};
                if (lane == u) at += __popcll(same);
            });
        };
        if (found <= kWaiting) {
            for (int i = 0; i < found; i += kWave) {
                const Waiting x = lds.waiting[wave][min(i + lane, found - 1)];
                put(x.entry, x.column, i + lane < found);
            }
        } else {
            each([&](int e, int column, bool in, bool) { put(e, column, in); });
        }
    }
};

// ---- rows with an entry ------------------------------------------------------------------------

// flags[r] = whether row r has an entry with mass (or NaN). One wave per row.
__global__ __launch_bounds__(256) void lmloss_flags_kernel(Entries e, int R, int V, int32_t *flags) {
    const int r = blockIdx.x * 4 + threadIdx.x / kWave, j = threadIdx.x % kWave;
    if (r >= R) return;
    bool has = false;
    if (j < e.K && id_ok(e.ids[(int64_t)r * e.K + j], V))
        has = !(e.teacher[(int64_t)r * e.K + j] == -INFINITY);
    if (__ballot(has) != 0ull) has = true;
    if (j == 0) flags[r] = has ? 1 : 0;
}

enum class Rows { kTargets, kEntries, kFlags };

struct GatherJob {
    const char *hidden;   // [R, H]
    const char *W;        // [V, H]
    const int32_t *flags; // kFlags
    float *stats;         // [R, K + 2]: entries' logits out
    Entries e;
    int R, H, V;
    char *rows;           // [R, H] the kept rows, behind one another
    int32_t *place;       // [R] where row r went, -1: left out
    int32_t *count;
};

constexpr int kGatherRows = 4;     // rows per workgroup, one a wave
constexpr int kGatherEntries = 8;  // entries per wave
// Rows of W read whole above this H, rings up to it. V = 152000, loss and gradients, whole rows and rings:
// H = 520, 16 rows 176 us and 178, 32 rows 220 and 192; H = 1032, 16 rows 278 and 343, 32 rows 346 and
// 355; H = 2048, 16 rows 448 and 586, 32 rows 576 and 597. (More than 32 rows: 64 of H = 1032, 428 and
// 432; H = 520, 269 and 229.)
constexpr int kRowsFrom = 1024;
// Up to so many the gather looks at the entries itself (a launch less; every workgroup looks at all of the rows
// before its own). Forward, H = 256, V = 2000, inline and by flags: 256 rows x 16, 31 us and 32; 512 x 16, 31 and
// 32.5; 1024 x 16, 32.5 and 33; 1024 x 64, 57 and 42.
constexpr int kInlineEntries = 4096;

template <Rows M>
__device__ __forceinline__ bool row_kept(const GatherJob &job, int r) {
    if constexpr (M == Rows::kTargets) return id_ok(job.e.ids[r], job.V);
    if constexpr (M == Rows::kEntries) {
        const int32_t *ids = job.e.ids + (int64_t)r * job.e.K;
        const float *t = job.e.teacher + (int64_t)r * job.e.K;
        int has = 0;  // (no entry's loads wait for another's)
#pragma unroll 8
        for (int j = 0; j < job.e.K; ++j)
            has |= (int)id_ok(ids[j], job.V) & (int)!(t[j] == -INFINITY);
        return has != 0;
    }
    if constexpr (M == Rows::kFlags) return job.flags[r] != 0;
}

// Forward. Workgroup (x, y): rows 4 x .. 4 x + 3; y = 0 copies them to their places, and each y
// takes the logits of ENTRIES of the entries. A row's place is the number of kept rows before it,
// which every workgroup of y = 0 counts for itself.
// An entry's logit is the same fp32 number as in the row's maximum and sum: the same matrix
// instructions on the same values of k, one after the other, as the rings and streams make them
// (another order of sums is 10^-4 off where logits are about 1000, which is all of a sure row's loss).
// A wave reads 1 KB of its hidden row and of each entry's row of W at a time, through LDS of its own. H = 4096:
// 64 entries of each of 1024 rows 76 - 93 us (537 MB, bound by these bytes), one of each 12 us. f32 waits for the chain
// of its instructions, 4 us for every 1024 of H (15 us of a call more at H = 4096 than a free order of sums).
template <typename T, Rows M, int ENTRIES>
__global__ __launch_bounds__(256) void lmloss_gather_kernel(GatherJob job) {
    constexpr int kBlock = 16 * kWave;               // bytes of a row
    constexpr int kAhead = ENTRIES == 1 ? 4 : 2;     // blocks asked for at once (8 and 4: up to 8 us more)
    __shared__ int part[4];
    __shared__ __align__(16) char stage[kGatherRows][(ENTRIES + 1) * kBlock];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int first = blockIdx.x * kGatherRows, r = first + wave;
    const bool copies = blockIdx.y == 0;
    int before = 0;
    if (copies) {
        int n = 0;
        for (int i = threadIdx.x; i < first; i += 256) n += row_kept<M>(job, i) ? 1 : 0;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d, kWave);
        if (lane == 0) part[wave] = n;
        __syncthreads();
        before = part[0] + part[1] + part[2] + part[3];
        for (int i = first; i < r; ++i) before += row_kept<M>(job, min(i, job.R - 1)) ? 1 : 0;
    }
    if (r >= job.R) return;
    const bool kept = row_kept<M>(job, r);
    if (copies && lane == 0) {
        job.place[r] = kept ? before : -1;
        if (r == job.R - 1) *job.count = before + (kept ? 1 : 0);
    }
    if (!kept) return;
    const int K = job.e.K;
    const int64_t row_bytes = (int64_t)job.H * sizeof(T);
    const char *src = job.hidden + r * row_bytes;
    char *dst = job.rows + before * row_bytes;
    // (past the last entry, and for ids that are none: row 0, whose product nothing reads)
    const int j0 = blockIdx.y * ENTRIES, n = min(ENTRIES, K - j0);
    const char *w[ENTRIES];
#pragma unroll
    for (int e = 0; e < ENTRIES; ++e) {
        const int id = e < n ? job.e.ids[(int64_t)r * K + j0 + e] : 0;
        w[e] = job.W + (id_ok(id, job.V) ? id : 0) * row_bytes;
    }
    // LDS: 16-byte chunk c of entry e's block at c ^ e, behind them the hidden row's. Lane (g, j) of a
    // step takes chunk g of its 64 bytes: of entry j (the rows of the instruction repeat them), of
    // the hidden row in every column.
    static_assert((ENTRIES & (ENTRIES - 1)) == 0 && ENTRIES <= 16, "rows of the instruction");
    constexpr int kSteps = 4;  // whose fragments are read together
    char *lds = stage[wave];
    const int g = lane >> 4, m = lane % ENTRIES;
    typedef typename GemmSide<T, kTile, false>::Frag Frag;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int64_t b0 = 0; b0 < row_bytes; b0 += kAhead * kBlock) {
        u32x4 h[kAhead], x[kAhead][ENTRIES];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {  // (zeros behind the row, as in the product)
            const int64_t b = b0 + a * kBlock + lane * 16;
            const bool in = b < row_bytes;
            h[a] = in ? *reinterpret_cast<const u32x4 *>(src + b) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < ENTRIES; ++e)
                x[a][e] = in ? *reinterpret_cast<const u32x4 *>(w[e] + b) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int64_t left = row_bytes - (b0 + a * kBlock);
            if (left <= 0) break;
            if (copies && lane * 16 < left)
                *reinterpret_cast<u32x4 *>(dst + b0 + a * kBlock + lane * 16) = h[a];
            wave_lds_order();  // (the last block is read)
            *reinterpret_cast<u32x4 *>(lds + ENTRIES * kBlock + lane * 16) = h[a];
#pragma unroll
            for (int e = 0; e < ENTRIES; ++e)
                *reinterpret_cast<u32x4 *>(lds + e * kBlock + ((lane ^ e) << 4)) = x[a][e];
            wave_lds_order();
            for (int s0 = 0; s0 < 16 && s0 * 64 < left; s0 += kSteps) {
                Frag fw[kSteps], fh[kSteps];
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const int c = 4 * (s0 + s) + g;
                    fw[s] = *reinterpret_cast<const Frag *>(lds + m * kBlock + ((c ^ m) << 4));
                    fh[s] = *reinterpret_cast<const Frag *>(lds + ENTRIES * kBlock + (c << 4));
                }
#pragma unroll
                for (int s = 0; s < kSteps; ++s) sum = gemm_mfma(fw[s], fh[s], sum);
            }
        }
    }
    // lane (g, j) holds entries 4 g .. 4 g + 3
    if (lane % 16 == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * g + i < n) job.stats[(int64_t)r * (K + 2) + 2 + j0 + 4 * g + i] = sum[i];
    }
}

struct KeepJob {
    const char *hidden;  // [R, H]
    const float *stats;  // [R, K + 2]
    const float *grad_loss;
    int R, H, K;
    float tau;
    char *rows;          // as GatherJob's
    int32_t *place, *count;
    float2 *scale;       // [kept rows] (max, g tau / sum)
    const int32_t *ids;  // with mask: [R, K]
    const float *teacher;
    int V;
    uint64_t *mask;      // null, or out: ListsJob's
};
constexpr int kKeepThreads = 1024, kKeepRows = kKeepThreads / kWave;

// Backward: the kept rows to their places, by the forward call's statistics, a wave per row.
template <typename T>
__global__ __launch_bounds__(kKeepThreads) void lmloss_keep_kernel(KeepJob job) {
    __shared__ int part[kKeepRows];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const auto kept = [&](int r) { return !(job.stats[(int64_t)r * (job.K + 2) + 1] < 0.f); };
    const int first = blockIdx.x * kKeepRows, r = first + wave;
    int n = 0;
    for (int i = threadIdx.x; i < first; i += kKeepThreads) n += kept(i) ? 1 : 0;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d, kWave);
    if (lane == 0) part[wave] = n;
    const uint64_t keeps = __ballot(lane < kKeepRows && first + lane < job.R && kept(min(first + lane, job.R - 1)));
    __syncthreads();
    if (r >= job.R) return;
    int before = __popcll(keeps & ((1ull << wave) - 1));
#pragma unroll
    for (int w = 0; w < kKeepRows; ++w) before += part[w];
    const bool is_kept = (keeps >> wave) & 1ull;
    if (lane == 0) {
        job.place[r] = is_kept ? before : -1;
        if (r == job.R - 1) *job.count = before + (is_kept ? 1 : 0);
    }
    if (job.mask) {
        const int64_t at = (int64_t)r * job.K + min(lane, job.K - 1);
        const bool ok = lane < job.K && id_ok(job.ids[at], job.V);
        const float t = ok ? job.teacher[at] : -INFINITY, least = wave_max(t, lane) - job.tau * kLn32;
        const uint64_t takes = __ballot(is_kept && ok && t >= least);
        if (lane == 0) job.mask[r] = takes;
    }
    if (!is_kept) return;
    const int64_t row_bytes = (int64_t)job.H * sizeof(T);
    const char *src = job.hidden + r * row_bytes;
    char *dst = job.rows + before * row_bytes;
#pragma unroll 4
    for (int64_t b = lane * 16; b < row_bytes; b += kWave * 16)
        *reinterpret_cast<u32x4 *>(dst + b) = *reinterpret_cast<const u32x4 *>(src + b);
    if (lane == 0) {
        const float *st = job.stats + (int64_t)r * (job.K + 2);
        job.scale[before] = float2{st[0], grad_scale(job.grad_loss[r], job.tau, st[1])};
    }
}

// ---- the product's epilogues ---------------------------------------------------------------------

// log2(e) / tau: rounded, and what that left.
struct Coef {
    float c, low;
};

// exp(d / tau), d <= 0. The rounded product d c errs by up to |d c| 2^-24 (and as much from c), which is
// the result's relative error: nothing to what is rounded to bf16; in f32 a correction of first order
// brings it back (EXACT).
template <bool EXACT> __device__ __forceinline__ float scaled_exp(float d, Coef k) {
    const float t = d * k.c, e = __builtin_amdgcn_exp2f(t);
    if constexpr (!EXACT) return e;
    const float left = fmaf(d, k.c, -t) + d * k.low;
    return t > -150.f ? fmaf(e, left * (float)kLn2, e) : e;  // (also where d is infinite, or NaN)
}

// (ref, sum) pairs in natural units: sum counts exp((x - ref) / tau). NaN in either stays.
template <bool EXACT>
__device__ __forceinline__ void join(float &m, float &s, float om, float os, Coef k) {
    const float top = fmaxf(m, om), ref = top == -INFINITY ? 0.f : top;
    s = s * scaled_exp<EXACT>(m - ref, k) + os * scaled_exp<EXACT>(om - ref, k);
    m = top;
}

// With lane ^ S's pair, in the lower lane's order on both sides (a fused sum of products is not
// symmetric): every lane ends with the same pair.
template <bool EXACT, int S>
__device__ __forceinline__ void join_lane(float &m, float &s, int lane, Coef k) {
    const float om = __uint_as_float(xor_lane<S>(__float_as_uint(m), lane));
    const float os = __uint_as_float(xor_lane<S>(__float_as_uint(s), lane));
    float lm = lane & S ? om : m, ls = lane & S ? os : s;
    join<EXACT>(lm, ls, lane & S ? m : om, lane & S ? s : os, k);
    m = lm;
    s = ls;
}

struct LogitsJob {
    const char *rows;     // [count, H]
    const char *W;        // [V, H]
    const int32_t *count;
    int H, V;
    int v0, v1;           // the piece of the vocabulary
    int nv, nr;           // tiles (of all R rows)
    Coef c;               // log2(e) / tau
    float2 *parts;        // forward: per 16 rows, [nparts][16] (max, sum)
    int64_t nparts;
    void *G;              // backward: [count][ldg]
    int64_t ldg;          // columns
    const float2 *scale;  // backward: [count]
    int low;              // few rows: the row of G where what rounding left of row 0 stands, or 0
    bool whole;           // bf16 rings: all rows of a tile of G are written, zeros behind the kept ones
    // few rows that the workgroups find themselves (`rows`: all R; count and scale are not read)
    int R;
    Entries e;
    float *stats;         // [R, K + 2]: forward: the entries' logits out; else in
    const float *grad_loss;
    int32_t *place, *from, *kept;  // out: FewRows
};

// A tile's end: for GRAD G's values, else maxima and sums. Its vocabulary rows start at v0, its
// kept rows at r0 (of R); `part`: the place of its (max, sum) pairs.
template <typename T> using GradStream = GemmStream<T, false, false, 16>;
template <typename T> using StatsStream = GemmStream<T, false, false, 0>;

template <typename T, bool GRAD, typename Tile>
__device__ __forceinline__ void logits_done(const LogitsJob &job, Tile &tile, int v0, int r0, int R,
                                            int64_t part, char *lds, int wave, int lane) {
    lane = anew(lane);
    const int g = lane >> 4, j = lane & 15;
    const int vw = v0 + Tile::wave_m(wave) + 4 * g;
    const Coef c = job.c;
    const int64_t ldg = job.ldg * (int64_t)sizeof(T);
    const __amdgpu_buffer_rsrc_t out = out_rows(
        static_cast<char *>(job.G) + r0 * ldg + (int64_t)(v0 - job.v0) * sizeof(T), ldg,
        min(R - r0, Tile::kCols), kTile * sizeof(T));
    const bool ragged = v0 + kTile > job.v1;
#pragma unroll
    for (int ni = 0; ni < Tile::NI; ++ni) {
        const int rn = Tile::wave_n(wave) + 16 * ni + j, r = r0 + rn;
        if constexpr (!GRAD) {
            if (ragged) {
#pragma unroll
                for (int mi = 0; mi < Tile::MI; ++mi)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (vw + 16 * mi + i >= job.v1) tile.acc[mi][ni][i] = -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int mi = 0; mi < Tile::MI; ++mi)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, tile.acc[mi][ni][i]);
            top = fmaxf(top, __uint_as_float(xor_lane<16>(__float_as_uint(top), lane)));
            top = fmaxf(top, __uint_as_float(xor_lane<32>(__float_as_uint(top), lane)));
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int mi = 0; mi < Tile::MI; ++mi)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += scaled_exp<false>(tile.acc[mi][ni][i] - ref, c);
            sum += __uint_as_float(xor_lane<16>(__float_as_uint(sum), lane));
            sum += __uint_as_float(xor_lane<32>(__float_as_uint(sum), lane));
            if (g == 0 && r < R)
                job.parts[((r >> 4) * job.nparts + part + wave / Tile::WN) * 16 + (r & 15)] =
                    float2{top, sum};
        }
    }
    if constexpr (GRAD) {
        float2 s[Tile::NI];
#pragma unroll
        for (int ni = 0; ni < Tile::NI; ++ni)
            s[ni] = job.scale[min(r0 + Tile::wave_n(wave) + 16 * ni + j, R - 1)];
        tile.store_rows(out, (int)ldg, 0, kTile * 2, lds, wave, lane, [&](int mi, int ni) {
            f32x4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = s[ni].y * scaled_exp<false>(tile.acc[mi][ni][i] - s[ni].x, c);
                if (ragged && vw + 16 * mi + i >= job.v1) y[i] = 0.f;
            }
            return y;
        });
    }
}

// Tiles of 256 vocabulary rows x 256 kept rows, bf16. Bound by the matrix cores at the clock that the
// card's power leaves: 4096 rows x 4096 x 151936, forward 4.02 ms (1267 TFLOP/s); 1024 rows, 1.01 - 1.09 ms
// (1170 - 1260: 2376 tiles are 9.3 rounds of the CUs).
template <typename T, bool GRAD>
__global__ __launch_bounds__(kGemmThreads) void lmloss_logits_stream_kernel(LogitsJob job) {
    typedef typename std::conditional<GRAD, GradStream<T>, StatsStream<T>>::type Stream;
    static_assert(!GRAD || Stream::kRowStores == 16, "the stores a tile's end makes");
    __shared__ __align__(1024) char lds[Stream::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count, nr = (R + kTile - 1) / kTile, tiles = job.nv * nr;
    const int64_t ld = (int64_t)job.H * sizeof(T);
    auto place = [&](int i, int &v0, int &r0) {
        const int id = blockIdx.x + i * gridDim.x;
        if (id >= tiles) return false;
        int tm, tn;
        gemm_place(id, job.nv, nr, kPlaceGroup, tm, tn);
        v0 = job.v0 + tm * kTile;
        r0 = tn * kTile;
        return true;
    };
    Stream stream;
    stream.run(
        ld, ld,
        [&](int i) -> GemmWork {
            int v0, r0;
            if (!place(i, v0, r0)) return {{job.W, ld, 0}, {job.rows, ld, 0}, 0};
            return {operand_kc<T>(job.W, ld, v0, job.v1, 0), operand_kc<T>(job.rows, ld, r0, R, 0),
                    job.H};
        },
        [&](int i) {
            int v0 = 0, r0 = 0;
            place(i, v0, r0);
            logits_done<T, GRAD>(job, stream, v0, r0, R,
                                 (int64_t)((v0 - job.v0) / kTile) * Stream::WM, lds, wave, lane);
        },
        lds, wave, lane);
}

// ---- few rows ---------------------------------------------------------------------------------------
// Up to BN <= 64 rows: every workgroup finds the kept ones and their entries in its range of the
// vocabulary by itself (a launch and a pass over the rows less: 8 - 12 us of a call); the first one leaves
// the rows' places for the kernels that follow. The entries' logits are taken, and their masses
// subtracted, where their columns come by. All eight waves take part: a wave looks at rows wave,
// wave + 8, .., a lane at an entry.
template <int BN, int LIST> struct FewRowsLds {
    float x[BN * LIST];     // backward: an entry's mass times g tau; forward: its column and which it is
    uint16_t v[BN * LIST];  // backward: its column. Columns count from the range's first on; a forward
                            // range has up to 2^20 of them, one of a piece 2^12
    int listed[BN];         // entries of a kept row in the range
    int from[BN], keeps[BN];  // the row that a kept one is; whether a row is kept

    static constexpr int kWhich = 64;  // x = column * kWhich + entry
    __device__ __forceinline__ int column(int at, bool forward) const {
        return forward ? (int)(__float_as_uint(x[at]) / kWhich) : v[at];
    }
    __device__ __forceinline__ int entry(int at) const { return (int)(__float_as_uint(x[at]) % kWhich); }
};
static_assert(DFLASH2_MAX_K <= 64 && DFLASH2_MAX_V / kCus <= 1 << 20, "FewRowsLds::x");

template <int BN, int LIST, bool FORWARD> struct FewRows {
    typedef FewRowsLds<BN, LIST> Lds;
    static constexpr int kRounds = BN / kGemmWaves;
    int ids[kRounds];
    float teacher[kRounds], sums[kRounds], grads[kRounds];
    uint64_t mask;  // the kept rows
    int R;          // their number

    __device__ __forceinline__ void find(const Entries &e, int rows, int V, const float *stats,
                                         const float *grad_loss, Lds &lds, int32_t *place,
                                         int32_t *from, int32_t *kept, int wave, int lane) {
        const int K = e.K;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {  // (all loads at once)
            const int r = min(wave + kGemmWaves * i, rows - 1);
            const int64_t at = (int64_t)r * K + min(lane, K - 1);
            ids[i] = e.ids[at];
            teacher[i] = e.teacher ? e.teacher[at] : 0.f;
            if constexpr (!FORWARD) {
                sums[i] = stats[(int64_t)r * (K + 2) + 1];
                grads[i] = grad_loss[r];
            }
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = wave + kGemmWaves * i;
            bool has;
            if constexpr (FORWARD)
                has = __ballot(lane < K && id_ok(ids[i], V) && !(teacher[i] == -INFINITY)) != 0ull;
            else
                has = !(sums[i] < 0.f);
            if (lane == 0) lds.keeps[r] = has && r < rows ? 1 : 0;
        }
        __syncthreads();
        mask = __ballot(lane < BN && lds.keeps[min(lane, BN - 1)] != 0);
        R = __popcll(mask);
        if (wave == 0) {
            const int mine = __popcll(mask & ((1ull << lane) - 1));
            const bool is_kept = (mask >> lane) & 1ull;
            if (is_kept) lds.from[mine] = lane;
            if (blockIdx.x == 0) {
                if (lane < rows) place[lane] = is_kept ? mine : -1;
                if (is_kept) from[mine] = lane;
                if (lane == 0) *kept = R;
            }
        }
        __syncthreads();
    }

    // The entries in columns [first, end), in their order.
    __device__ __forceinline__ void list(const Entries &e, int V, Coef c, int first, int end, Lds &lds,
                                         int wave, int lane) const {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = wave + kGemmWaves * i, p = __popcll(mask & ((1ull << r) - 1));
            if (!((mask >> r) & 1ull)) continue;
            const bool any = lane < e.K && id_ok(ids[i], V);
            float x;
            if constexpr (FORWARD) {
                x = __uint_as_float((uint32_t)(ids[i] - first) * Lds::kWhich + lane);
            } else {
                x = 1.f;
                if (e.teacher) {
                    const float t = any ? teacher[i] : -INFINITY;
                    float high = wave_max(t, lane);
                    if (__ballot(any && t != t) != 0ull) high = NAN;
                    const float w = any ? scaled_exp<false>(t - high, c) : 0.f;
                    x = w / wave_sum(w, lane);
                }
                x = grad_mass(grads[i], e.tau, x);
            }
            const uint64_t m = __ballot(any && ids[i] >= first && ids[i] < end);
            if ((m >> lane) & 1ull) {
                const int at = p * LIST + __popcll(m & ((1ull << lane) - 1));
                if constexpr (!FORWARD) lds.v[at] = (uint16_t)(ids[i] - first);
                lds.x[at] = x;
            }
            if (lane == 0) lds.listed[p] = __popcll(m);
        }
        __syncthreads();
    }
};

// Entries a row that a ring's workgroup has a list for.
template <int BN> constexpr int ring_list() { return BN <= 32 ? 32 : 16; }

// Few kept rows (BN <= 128 a tile), or f32: a workgroup takes a range of the vocabulary (a multiple of 16
// rows of W) and goes through it in tiles of 128 or 256. Forward: each lane keeps its columns' (max, sum)
// over the whole range. G of few bf16 rows is kept in two parts (rounded, and what that left): the
// products that read it are bound by W and the gradient, and two parts cost them nothing. FIND: the
// workgroups find the kept rows (one tile of them) and take care of their entries.
// bf16 is bound by W: 64 rows x 4096 x 152000, 237 us a forward call (5.3 TB/s), 128 rows 268 us. f32 by
// the matrix cores: 298 rows x 1016 x 32003 200 us, 97 TFLOP/s of 154 (the cores are busy 0.72 of the time;
// reading a stage's fragments before its products, starting loads behind half of them, or one half of the
// waves behind the other moved nothing).
template <typename T, int BN, bool GRAD, bool FIND>
__global__ __launch_bounds__(kGemmThreads) void lmloss_logits_few_kernel(LogitsJob job) {
    // bf16 of up to 64 rows: stages of two K steps, 256 bytes of each of 128 rows of W. f32: the matrix
    // cores are the bound, and shorter tiles leave less of a range's last one unused.
    constexpr int SUB = sizeof(T) == 2 && BN <= 64 ? 2 : 1, BM = sizeof(T) == 4 || SUB == 2 ? 128 : 256;
    constexpr bool kExact = sizeof(T) == 4;
    constexpr int kFind = FIND ? BN : 8, kList = ring_list<BN>();
    typedef FewRows<kFind, kList, !GRAD> Few;
    typedef GemmRing<T, BM, BN, SUB, false, false, FIND ? sizeof(typename Few::Lds) : 0> Ring;
    __shared__ __align__(1024) char lds[Ring::kLdsBytes];
    __shared__ typename std::conditional<FIND, typename Few::Lds, int>::type few_lds;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    Few few;
    const int *from = nullptr;
    int R;
    if constexpr (FIND) {
        few.find(job.e, job.R, job.V, job.stats, job.grad_loss, few_lds, job.place, job.from, job.kept,
                 wave, lane);
        R = few.R;
        from = few_lds.from;
    } else {
        R = *job.count;
    }
    const int nr = (R + BN - 1) / BN, ranges = few_ranges(job.v1 - job.v0, nr);
    if ((int)blockIdx.x >= ranges * nr) return;
    int range, tn;
    gemm_place(blockIdx.x, ranges, nr, 1, range, tn);
    const int units = (job.v1 - job.v0 + 15) / 16, r0 = tn * BN;
    const int lo = job.v0 + 16 * (int)((int64_t)units * range / ranges);
    const int hi = min(job.v0 + 16 * (int)((int64_t)units * (range + 1) / ranges), job.v1);
    if constexpr (FIND) few.list(job.e, job.V, job.c, lo, hi, few_lds, wave, lane);
    const int64_t ld = (int64_t)job.H * sizeof(T);
    const Coef c = job.c;
    const int rows = FIND ? job.R : R;  // of `rows`
    float top[Ring::NI], sum[Ring::NI];
    float2 scale[Ring::NI];  // (read here: a load in a tile's end would wait for all that are in flight)
#pragma unroll
    for (int ni = 0; ni < Ring::NI; ++ni) {
        top[ni] = -INFINITY;
        sum[ni] = 0.f;
        if constexpr (GRAD) {
            const int r = min(r0 + 16 * ni + (lane & 15), R - 1);
            if constexpr (FIND) {
                const float *st = job.stats + (int64_t)from[r] * (job.e.K + 2);
                scale[ni] = float2{st[0], grad_scale(job.grad_loss[from[r]], job.e.tau, st[1])};
            } else {
                scale[ni] = job.scale[r];
            }
        }
    }
    Ring ring;
    ring.run(
        ld, ld,
        [&](int i) -> GemmWork {
            const int v0 = lo + i * BM;
            if (v0 >= hi) return {{job.W, ld, 0}, {job.rows, ld, 0}, 0};
            return {operand_kc<T>(job.W, ld, v0, hi, 0), operand_kc<T>(job.rows, ld, r0, rows, 0), job.H};
        },
        [&](int i) {
            const int at = anew(lane), g = at >> 4, j = at & 15;
            const int v0 = lo + i * BM, vw = v0 + Ring::wave_m(wave) + 4 * g;
            const int64_t ldg = job.ldg * (int64_t)sizeof(T);
            const bool ragged = v0 + BM > hi;
            const __amdgpu_buffer_rsrc_t out = out_rows(
                static_cast<char *>(job.G) + r0 * ldg + (int64_t)(v0 - job.v0) * sizeof(T), ldg,
                job.low ? 2 * job.low : sizeof(T) == 2 && job.whole ? BN : min(R - r0, BN), BM * sizeof(T));
#pragma unroll
            for (int ni = 0; ni < Ring::NI; ++ni) {
                const int rn = 16 * ni + j, r = r0 + rn;
                int listed = 0;
                if constexpr (FIND) listed = r < R ? few_lds.listed[min(r, kFind - 1)] : 0;
                if constexpr (!GRAD) {
                    if constexpr (FIND) {
                        for (int n = 0; n < listed; ++n) {
                            const int dv = lo + few_lds.column(r * kList + n, true) - vw;
                            const int j = few_lds.entry(r * kList + n);
#pragma unroll
                            for (int mi = 0; mi < Ring::MI; ++mi)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (dv == 16 * mi + k)
                                        job.stats[(int64_t)from[r] * (job.e.K + 2) + 2 + j] =
                                            ring.acc[mi][ni][k];
                        }
                    }
                    float high = top[ni];
#pragma unroll
                    for (int mi = 0; mi < Ring::MI; ++mi)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (ragged && vw + 16 * mi + k >= hi) ring.acc[mi][ni][k] = -INFINITY;
                            high = fmaxf(high, ring.acc[mi][ni][k]);
                        }
                    const float ref = high == -INFINITY ? 0.f : high;
                    float s = sum[ni] * scaled_exp<kExact>(top[ni] - ref, c);
#pragma unroll
                    for (int mi = 0; mi < Ring::MI; ++mi)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            s += scaled_exp<kExact>(ring.acc[mi][ni][k] - ref, c);
                    top[ni] = high;
                    sum[ni] = s;
                } else {
                    f32x4 y[Ring::MI];
#pragma unroll
                    for (int mi = 0; mi < Ring::MI; ++mi)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[mi][k] = scale[ni].y * scaled_exp<kExact>(ring.acc[mi][ni][k] - scale[ni].x, c);
                    if constexpr (FIND) {
                        for (int n = 0; n < listed; ++n) {
                            const int dv = lo + few_lds.column(r * kList + n, false) - vw;
                            const float x = few_lds.x[r * kList + n];
#pragma unroll
                            for (int mi = 0; mi < Ring::MI; ++mi)
#pragma unroll
                                for (int k = 0; k < 4; ++k) y[mi][k] -= dv == 16 * mi + k ? x : 0.f;
                        }
                    }
#pragma unroll
                    for (int mi = 0; mi < Ring::MI; ++mi) {
                        const int v = vw + 16 * mi;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (r >= R || (ragged && v + k >= job.v1)) y[mi][k] = 0.f;
                        // (hi is a multiple of 16 behind v0, or the piece's end)
                        const int off = v - 4 * g < hi ? rn * (int)ldg + (v - v0) * (int)sizeof(T)
                                                       : kGemmOutside;
                        store4<T>(out, off, y[mi]);
                        if (sizeof(T) == 2 && job.low) {
                            f32x4 z;
#pragma unroll
                            for (int k = 0; k < 4; ++k) z[k] = y[mi][k] - (float)(__bf16)y[mi][k];
                            store4<T>(out, off + (off == kGemmOutside ? 0 : job.low * (int)ldg), z);
                        }
                    }
                }
            }
        },
        lds, wave, lane, from, R);
    if constexpr (!GRAD) {
        float2 *pair = reinterpret_cast<float2 *>(lds);  // [waves][BN]
        const int g = lane >> 4, j = lane & 15;
#pragma unroll
        for (int ni = 0; ni < Ring::NI; ++ni) {
            float m = top[ni], s = sum[ni];
            join_lane<kExact, 16>(m, s, lane, c);
            join_lane<kExact, 32>(m, s, lane, c);
            if (g == 0) pair[wave * BN + 16 * ni + j] = float2{m, s};
        }
        __syncthreads();
        const int n = threadIdx.x, r = r0 + n;
        if (n < BN && r < R) {
            float2 x = pair[n];
            for (int w = 1; w < kGemmWaves; ++w) {
                const float2 y = pair[w * BN + n];
                join<kExact>(x.x, x.y, y.x, y.y, c);
            }
            job.parts[((int64_t)(r >> 4) * ranges + range) * 16 + (r & 15)] = x;
        }
    }
}

// ---- forward's end -------------------------------------------------------------------------------

constexpr int kFinishRows = 16;
constexpr int kFinishThreads = 1024;

struct FinishJob {
    const float2 *parts;
    int64_t nparts;      // pairs of a row; or 0: few_ranges
    const int32_t *place, *count;
    int bn;
    Entries e;
    int R, V;
    Coef c;
    float *loss;
    float *stats;
};

// 16 rows: their tiles' pairs in a fixed order, then a wave per row over its entries. 5 - 7 us for 16
// rows (the latency of its loads), 12 us for 1024.
__global__ __launch_bounds__(kFinishThreads) void lmloss_finish_kernel(FinishJob job) {
    constexpr int kGroups = kFinishThreads / kFinishRows;
    static_assert(kGroups == kWave, "a wave joins a row's groups");
    __shared__ float2 pair[kGroups][kFinishRows];
    const int first = blockIdx.x * kFinishRows;
    const int64_t nparts = job.nparts ? job.nparts : few_ranges(job.V, (*job.count + job.bn - 1) / job.bn);
    {
        const int k = threadIdx.x % kFinishRows, grp = threadIdx.x / kFinishRows;
        const int r = first + k, p = r < job.R ? job.place[r] : -1;
        float m = -INFINITY, s = 0.f;
        if (p >= 0) {
            const float2 *src = job.parts + (p >> 4) * nparts * 16 + (p & 15);
#pragma unroll 4
            for (int64_t i = grp; i < nparts; i += kGroups) {
                const float2 x = src[i * 16];
                join<true>(m, s, x.x, x.y, job.c);
            }
        }
        pair[grp][k] = float2{m, s};
    }
    __syncthreads();
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    constexpr int kWaves = kFinishThreads / kWave;
    for (int k = wave; k < kFinishRows; k += kWaves) {
        const int r = first + k;
        if (r >= job.R) break;
        const int K = job.e.K;
        float *st = job.stats + (int64_t)r * (K + 2);
        if (job.place[r] < 0) {
            for (int i = lane; i < K + 2; i += kWave) st[i] = i == 1 ? kLeftOut : 0.f;
            if (lane == 0) job.loss[r] = 0.f;
            continue;
        }
        float m = -INFINITY, s = 0.f;
        m = pair[lane][k].x;
        s = pair[lane][k].y;
        join_lane<true, 1>(m, s, lane, job.c);
        join_lane<true, 2>(m, s, lane, job.c);
        join_lane<true, 4>(m, s, lane, job.c);
        join_lane<true, 8>(m, s, lane, job.c);
        join_lane<true, 16>(m, s, lane, job.c);
        join_lane<true, 32>(m, s, lane, job.c);
        const int id = lane < K ? job.e.ids[(int64_t)r * K + lane] : -1;
        const bool ok = id_ok(id, job.V);
        if (lane < K && !ok) st[2 + lane] = 0.f;
        double term = 0.0;
        const double tau = job.e.tau;
        double p = ok ? 1.0 : 0.0, ln_p = 0.0;
        if (job.e.teacher) {
            const float t = ok ? job.e.teacher[(int64_t)r * K + lane] : -INFINITY;
            float top = wave_max(t, lane);
            if (__ballot(ok && t != t) != 0ull) top = NAN;
            ln_p = ((double)t - top) / tau;
            const double w = ok ? exp(ln_p) : 0.0;
            const double all = wave_sum(w, lane);
            p = w / all;
            ln_p -= log(all);
        }
        if (ok && !(p == 0.0)) {
            // (at most 0: the entry's logit is the one in the maximum and the sum)
            const double ln_q = ((double)st[2 + lane] - m) / tau - log((double)s);
            term = p * (ln_p - ln_q);
        }
        term = wave_sum(term, lane);
        if (lane == 0) {
            job.loss[r] = (float)(tau * tau * term);
            st[0] = m;
            st[1] = s;
        }
    }
}

// ---- backward: the entries of a piece ------------------------------------------------------------

struct EntriesJob {
    Entries e;
    const float *stats;
    const float *grad_loss;
    const int32_t *place;
    int R, V, v0, v1;
    Coef c;
    void *G;
    int64_t ldg;
    int low;
    float *rest;           // [R, K] or null: ListedRest::left
    const uint64_t *mask;  // as ListsJob's
    int groups;            // workgroups of 16 rows; those behind them make the lists
    ListsJob lists;
};

__global__ __launch_bounds__(256) void lmloss_zero_kernel(u32x4 *p, int64_t n) {
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256)
        p[i] = u32x4{0u, 0u, 0u, 0u};
}

// One wave per row: G at the row's entries, the masses of equal ids added in their order. f32: taken from
// what the product has written; bf16: from the kept logit, rounded once. Either way the logit is the
// one in the row's sum, so q - 1 of a sure row keeps its digits. The first piece's launch makes the lists of the
// entries by columns too, in workgroups of their own. 1024 rows: 5 us of one entry, 10 of 64; with the lists 6 and 34.
template <typename T>
__global__ __launch_bounds__(kKeepThreads) void lmloss_entries_kernel(EntriesJob job) {
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if constexpr (sizeof(T) == 2) {
        typedef Lists<kKeepThreads> Listing;
        __shared__ typename Listing::Lds lds;
        if ((int)blockIdx.x >= job.groups) {
            Listing::run(job.lists, blockIdx.x - job.groups, lds, wave, lane);
            return;
        }
    }
    const int r = blockIdx.x * kKeepRows + wave;
    if (r >= job.R) return;
    const int p = job.place[r];
    const int K = job.e.K;
    const int id = lane < K ? job.e.ids[(int64_t)r * K + lane] : -1;
    const bool ok = id_ok(id, job.V), in_piece = ok && id >= job.v0 && id < job.v1;
    if (p < 0) return;
    float mass = 1.f;
    if (job.e.teacher) {
        const float t = ok ? job.e.teacher[(int64_t)r * K + lane] : -INFINITY;
        float top = wave_max(t, lane);
        if (__ballot(ok && t != t) != 0ull) top = NAN;
        const float w = ok ? scaled_exp<true>(t - top, job.c) : 0.f;
        mass = w / wave_sum(w, lane);
    }
    float total = 0.f;
    bool earlier = false;
    for (int j = 0; j < K; ++j) {
        const int oid = __shfl(id, j, kWave);
        const float om = __shfl(mass, j, kWave);
        if (oid == id) {
            total += om;
            earlier |= j < lane;
        }
    }
    if (!in_piece) return;
    if (earlier) {
        if (sizeof(T) == 2 && job.rest) job.rest[(int64_t)r * K + lane] = 0.f;
        return;
    }
    T *out = static_cast<T *>(job.G) + p * job.ldg + (id - job.v0);
    const float g = job.grad_loss[r];
    float y;
    if constexpr (sizeof(T) == 4) {
        y = *out - grad_mass(g, job.e.tau, total);
    } else {
        const float *st = job.stats + (int64_t)r * (K + 2);
        const float q = scaled_exp<true>(st[2 + lane] - st[0], job.c) / st[1];
        y = grad_mass(g, job.e.tau, q - total);
    }
    if constexpr (sizeof(T) == 2) {
        const float high = (float)(__bf16)y;
        *reinterpret_cast<__bf16 *>(out) = (__bf16)y;
        if (job.low) *reinterpret_cast<__bf16 *>(out + job.low * job.ldg) = (__bf16)(y - high);
        // (nothing is added to what is infinite or NaN already)
        if (job.rest) {
            const bool takes = !job.mask || ((job.mask[r] >> lane) & 1ull) != 0ull;
            job.rest[(int64_t)r * K + lane] = takes && fabsf(high) < INFINITY ? y - high : 0.f;
        }
    } else {
        *out = y;
    }
}

// ---- what rounding left of the entries ---------------------------------------------------------------

// Adds a unit's listed entries to a wave's part of grad_W: acc[mi][ni][i] is column h0 + 16 mi + 4 g + i of the
// unit's row c0 + 16 ni + j. 16 entries at a time as a product of their hidden states and what is left of G, with
// the next 16's loads and the places of those behind them on their way. scratch: 16 rows of 16 MI columns of
// hidden in LDS (16-byte chunk c of row k at c ^ k), the wave's own, which transposing reads take them from.
template <int MI, int NI>
__device__ __forceinline__ void add_listed(f32x4 (&acc)[MI][NI], const ListedRest &rest, int unit, int c0, int H,
                                           int h0, char *scratch, int lane) {
    constexpr int kChunks = 2 * MI, kRows = 16 / kChunks, kLoads = 4 / kRows;  // of a row; of lanes' 4 rows
    const int2 range = rest.units[__builtin_amdgcn_readfirstlane(unit)];
    if (range.x >= range.y) return;
    const int g = lane >> 4, j = lane & 15, chunk = j % kChunks, sub = j / kChunks;
    const int column = min(h0 + 8 * chunk, H - 8);
    const int k_put = 4 * g + sub, k_get = 4 * g + (j >> 2);
    Listed x[4];
    u32x4 h[kLoads];
    float left[4];
    int at[4];  // columns
    const auto places = [&](int e) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = rest.list[(uint32_t)min(e + 4 * g + i, range.y - 1)];
    };
    const auto load = [&](int e) {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const uint32_t where = sub == 0 ? x[q * kRows].where : x[q * kRows + kRows - 1].where;
            h[q] = *reinterpret_cast<const u32x4 *>(rest.hidden + (int64_t)(where & 0xFFFFu) * H + column);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            left[i] = rest.left[(uint32_t)x[i].entry];
            at[i] = e + 4 * g + i < range.y ? (int)(x[i].where >> 16) - c0 : -1;
        }
    };
    places(range.x);
    load(range.x);
    places(range.x + 16);
    for (int e = range.x; e < range.y; e += 16) {
        wave_lds_order();
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int k = k_put + q * kRows;
            *reinterpret_cast<u32x4 *>(scratch + k * (kChunks * 16) + ((chunk ^ (k % kChunks)) << 4)) = h[q];
        }
        s16x4 b[NI];
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[ni][i] = __builtin_bit_cast(short, (__bf16)(at[i] == 16 * ni + j ? left[i] : 0.f));
        wave_lds_order();
        __builtin_amdgcn_sched_barrier(0);
        if (e + 16 < range.y) {  // (on their way during the products)
            load(e + 16);
            places(e + 32);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m0 = 0; m0 < MI; m0 += 4) {
            s16x4 a[4];
#pragma unroll
            for (int mi = 0; mi < 4; ++mi) {
                const int c = 2 * (m0 + mi) + ((j & 3) >> 1);
                a[mi] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(
                    scratch + k_get * (kChunks * 16) + ((c ^ (k_get % kChunks)) << 4) + 8 * (j & 1)));
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int mi = 0; mi < 4; ++mi)
#pragma unroll
                for (int ni = 0; ni < NI; ++ni)
                    acc[m0 + mi][ni] =
                        __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a[mi], b[ni], acc[m0 + mi][ni], 0, 0, 0);
        }
    }
    wave_lds_order();
}

// ---- the gradients' products -----------------------------------------------------------------------

// Streams of tiles: splits of the vocabulary for grad_hidden, given how many tiles of kept rows there are
// (known on the device only) and the width of the first piece. A tile's end, with its sums read and
// written, takes as long as 17 K steps. Rounds of tiles over the CUs count as whole ones, but the card's
// power is the limit from about three quarters of the CUs on (192 tiles as 192, or in 4 splits as 768,
// take the same time; 160 tiles in 3 splits take 0.9 of the time of 160).
constexpr int kSplitTiles = 768;  // splits x tiles, at most, where there is more than one split

__host__ __device__ __forceinline__ int split_columns(int width, int splits) {
    return ((width + splits - 1) / splits + 63) / 64 * 64;
}

__host__ __device__ __forceinline__ int stream_splits(int tiles, int width) {
    int best = 1, least = 0x7FFFFFFF;
    for (int rounds = 1; rounds <= kSplitTiles / kCus; ++rounds) {  // as many as fit the rounds
        const int fit = rounds * kCus / tiles, most = width / 256;
        const int s = fit < most ? fit : most;
        if (s < 1) continue;
        const int steps = split_columns(width, s) / 64 + 17;
        const int all = (int)((int64_t)s * tiles * steps * 333 >> 16);  // 1.3 / 256: at 0.77 of the CUs
        const int cost = rounds * steps > all ? rounds * steps : all;
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    const int per = split_columns(width, best);
    return (width + per - 1) / per;
}

struct HiddenJob {
    const char *W;       // [V, H]
    const char *G;       // [count][ldg]
    const int32_t *count;
    int R, H, v0, v1;    // R: rows of G and of the sums
    int64_t ldg;
    int nh, nr, splits, per;  // tiles (of all R rows); splits of the piece, `per` columns each
    bool first;          // the first piece: nothing to add to
    float *sums;         // [splits][R][H]
    int low;             // as the logits' job's
    int width;           // streams: of the first piece (nr, splits, per and R come from the kept rows)
};

template <bool few, typename Tile>
__device__ __forceinline__ void hidden_done(const HiddenJob &job, Tile &tile, int split, int rows,
                                            int h0, int r0, int R, int wave, int lane) {
    lane = anew(lane);
    const int g = lane >> 4, j = lane & 15;
    const int ld = job.H * 4;
    const __amdgpu_buffer_rsrc_t out = out_rows(
        job.sums + ((int64_t)split * rows + r0) * job.H, ld, min(R - r0, Tile::kCols), ld);
#pragma unroll
    for (int ni = 0; ni < Tile::NI; ++ni) {
        const int n = Tile::wave_n(wave) + 16 * ni + j, row = n * ld;
        // (few rows: those that hold something)
        const bool some = !few || (n >= job.low && job.low ? n - job.low : n) < *job.count;
#pragma unroll
        for (int mi = 0; mi < Tile::MI; ++mi) {
            const int h = h0 + Tile::wave_m(wave) + 16 * mi + 4 * g;
            const int off = some && h < job.H ? row + 4 * h : kGemmOutside;
            f32x4 x = tile.acc[mi][ni];
            if (!job.first)
                x += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(out, off, 0, 0));
            store4<float>(out, off, x);
        }
    }
}

// Few kept rows, or f32: tiles of 256 columns of H x BN rows of G over a split of the piece, one a
// workgroup. bf16 is bound by the read of W (64 rows x 4096 x 152000, G and this: 472 us), f32 by the matrix
// cores (298 rows x 1016 x 32003: 182 us, 106 TFLOP/s, busy 0.76).
template <typename T, int BN> using HiddenRing = GemmRing<T, kTile, BN, 1, true, false>;

template <typename T, int BN>
__device__ __forceinline__ void hidden_few(const HiddenJob &job, int block, char *lds) {
    typedef HiddenRing<T, BN> Ring;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = sizeof(T) == 2 ? BN : *job.count, nr = (R + BN - 1) / BN;
    if (block >= job.nh * job.splits * nr) return;
    int tm, tn;
    gemm_place(block, job.nh * job.splits, nr, kPlaceGroup, tm, tn);
    const int split = tm / job.nh, h0 = tm % job.nh * kTile, r0 = tn * BN;
    const int k0 = split * job.per, k1 = min(k0 + job.per, job.v1 - job.v0);
    const int64_t ldw = (int64_t)job.H * sizeof(T), ldg = job.ldg * (int64_t)sizeof(T);
    Ring ring;
    ring.run(
        ldw, ldg,
        [&](int i) -> GemmWork {
            if (i > 0) return {{job.W, ldw, 0}, {job.G, ldg, 0}, 0};
            return {operand_ks<T>(job.W, ldw, h0, job.v0 + k0), operand_kc<T>(job.G, ldg, r0, R, k0),
                    k1 - k0};
        },
        [&](int) { hidden_done<sizeof(T) == 2>(job, ring, split, job.R, h0, r0, R, wave, lane); }, lds,
        wave, lane);
}

template <typename T, int BN>
__global__ __launch_bounds__(kGemmThreads) void lmloss_hidden_few_kernel(HiddenJob job) {
    __shared__ __align__(1024) char lds[HiddenRing<T, BN>::kLdsBytes];
    hidden_few<T, BN>(job, blockIdx.x, lds);
}

// Tiles of 256 columns of H x 256 kept rows over a split of the piece, bf16. 4096 rows x 4096 x 151936:
// 3.8 ms (1330 TFLOP/s); 1024 rows, 64 tiles in splits, 0.98 ms (1300).
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void lmloss_hidden_stream_kernel(HiddenJob job) {
    typedef GemmStream<T, true, false, 32> Stream;  // (hidden_done: 32 stores)
    __shared__ __align__(1024) char lds[Stream::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count, nr = (R + kTile - 1) / kTile;
    if (R == 0) return;
    const int width = job.v1 - job.v0;
    const int per = split_columns(width, stream_splits(job.nh * nr, job.width));
    const int splits = (width + per - 1) / per, tiles = job.nh * splits * nr;
    const int64_t ldw = (int64_t)job.H * sizeof(T), ldg = job.ldg * (int64_t)sizeof(T);
    auto place = [&](int i, int &split, int &h0, int &r0) {
        const int id = blockIdx.x + i * gridDim.x;
        if (id >= tiles) return false;
        int tm, tn;
        gemm_place(id, job.nh * splits, nr, kPlaceGroup, tm, tn);
        split = tm / job.nh;
        h0 = tm % job.nh * kTile;
        r0 = tn * kTile;
        return true;
    };
    Stream stream;
    stream.run(
        ldw, ldg,
        [&](int i) -> GemmWork {
            int split, h0, r0;
            if (!place(i, split, h0, r0)) return {{job.W, ldw, 0}, {job.G, ldg, 0}, 0};
            const int k0 = split * per, k1 = min(k0 + per, width);
            return {operand_ks<T>(job.W, ldw, h0, job.v0 + k0), operand_kc<T>(job.G, ldg, r0, R, k0),
                    k1 - k0};
        },
        [&](int i) {
            int split = 0, h0 = 0, r0 = 0;
            place(i, split, h0, r0);
            hidden_done<false>(job, stream, split, nr * kTile, h0, r0, R, wave, lane);
        },
        lds, wave, lane);
}

// grad_hidden from the splits' sums, added in a fixed order (and from the two parts of G, `low` rows
// apart, or the entries' rests); zeros for the rows left out. Workgroup (x, y): 256 columns of row x, a wave per
// WAVES-th split and entry. Bound by the latency of its loads: 1024 rows x 4096 in 4 splits, 37 us (75 MB, 2.0 TB/s),
// 44 with an entry's rest a row, 58 with those of 64. Few rows leave few workgroups, and many splits a chain of loads; the calls for grad_hidden with 16 waves and with 4: 7 rows x 72 in
// 256 splits, 29 us and 33; 40 x 256 x 50000, 38 and 41; 64 x 1024 x 50000 in 64, 62 and 63; 64 x 2048 in 32, 92
// and 91; below that 4 are as fast or faster (331 x 1016 x 32003, f32: 385 us, with 16 waves 388).
template <typename T, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void lmloss_hidden_out_kernel(
    const float *sums, int splits, int rows, int low, const int32_t *count, int width,
    const int32_t *place, int H, T *grad, Entries e, int V, const float *rest, const T *W) {
    __shared__ f32x4 part[WAVES][kWave];
    if (width > 0) {  // a stream's: as it has split them
        const int nr = (*count + kTile - 1) / kTile, nh = (H + kTile - 1) / kTile;
        splits = nr > 0 ? stream_splits(nh * nr, width) : 0;
        rows = nr * kTile;
    }
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = blockIdx.x, p = place[r], h = (blockIdx.y * kWave + lane) * 4;
    // the entries of which something is left, every WAVES-th to a wave
    int id = -1;
    float left = 0.f;
    uint64_t mine = 0ull;
    if (sizeof(T) == 2 && rest && p >= 0) {
        const int64_t at = (int64_t)r * e.K + min(lane, e.K - 1);
        id = lane < e.K ? e.ids[at] : -1;
        left = rest[at];
        const bool some = id_ok(id, V) && left != 0.f;
        mine = __ballot(some && __popcll(__ballot(some) & ((1ull << lane) - 1)) % WAVES == wave);
    }
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (p >= 0 && h < H) {
        const auto add = [&](int row) {
#pragma unroll 8
            for (int s = wave; s < splits; s += WAVES)
                x += *reinterpret_cast<const f32x4 *>(sums + ((int64_t)s * rows + row) * H + h);
        };
        add(p);
        if (low) add(p + low);
        while (sizeof(T) == 2 && mine != 0ull) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            constexpr int kAhead = 4;
            u32x2 w[kAhead];
            float of[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {  // (behind the last: the first row, for nothing)
                const int j = mine != 0ull ? __builtin_ctzll(mine) : 0;
                const int v = mine != 0ull ? __builtin_amdgcn_readlane(id, j) : 0;
                const uint32_t bits = __builtin_amdgcn_readlane(__float_as_uint(left), j);
                of[n] = mine != 0ull ? __uint_as_float(bits) : 0.f;
                w[n] = *reinterpret_cast<const u32x2 *>(W + (int64_t)v * H + h);
                if (mine == 0ull) w[n] = u32x2{0u, 0u};
                mine &= mine - 1ull;
            }
#pragma unroll
            for (int n = 0; n < kAhead; ++n)
                x += of[n] * f32x4{bf16_lo(w[n].x), bf16_hi(w[n].x), bf16_lo(w[n].y), bf16_hi(w[n].y)};
        }
    }
    if (wave > 0) part[wave][lane] = x;
    __syncthreads();
    if (wave > 0 || h >= H) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) x += part[w][lane];
    const auto y = packed4<T>(x);
    *reinterpret_cast<decltype(packed4<T>(x)) *>(grad + (int64_t)r * H + h) = y;
}

struct WeightJob {
    const char *rows;    // [count, H]
    const char *G;       // [count][ldg]
    const int32_t *count;
    const int32_t *from; // null, or where in `rows` each kept row is (lmloss_weight_few_kernel)
    int H, v0, v1;
    int64_t ldg;
    int nh, nv;
    void *grad;          // [V, H]
    ListedRest rest;     // bf16 in one part
    int low;             // bf16, many entries: the row of G where what rounding left of row 0 stands, or 0
};

template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_rows(const WeightJob &job, int v0,
                                                              int most) {
    const int ld = job.H * (int)sizeof(T);
    return out_rows(static_cast<char *>(job.grad) + (int64_t)(job.v0 + v0) * ld, ld,
                    min(job.v1 - job.v0 - v0, most), ld);
}

// f32: tiles of 256 columns of H x 128 vocabulary rows, over the kept rows; one a workgroup. 298 rows x 1016
// x 32003: 181 us, 107 TFLOP/s, busy 0.74 (10 K steps a tile, whose end no product covers).
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void lmloss_weight_kernel(WeightJob job) {
    typedef GemmTile<T, kTile, 128, true, true, 4> Tile;
    __shared__ __align__(1024) char lds[Tile::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count;
    int tm, tn;
    gemm_place(blockIdx.x, job.nh, job.nv, kPlaceGroup, tm, tn);
    const int h0 = tm * kTile, v0 = tn * Tile::kCols;
    Tile tile;
    tile.run(operand_ks<T>(job.rows, (int64_t)job.H * sizeof(T), h0, 0),
             operand_ks<T>(job.G, job.ldg * (int64_t)sizeof(T), v0, 0), R, lds, wave, lane);
    const int at = anew(lane), g = at >> 4, j = at & 15;
    const __amdgpu_buffer_rsrc_t out = weight_rows<T>(job, v0, Tile::kCols);
#pragma unroll
    for (int ni = 0; ni < Tile::NI; ++ni) {
        const int row = (Tile::wave_n(wave) + 16 * ni + j) * job.H * (int)sizeof(T);
#pragma unroll
        for (int mi = 0; mi < Tile::MI; ++mi) {
            const int h = h0 + Tile::wave_m(wave) + 16 * mi + 4 * g;
            store4<T>(out, h < job.H ? row + h * (int)sizeof(T) : kGemmOutside, tile.acc[mi][ni]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// bf16, more rows than that, or many entries: tiles of 256 columns of H x 256 vocabulary rows. 4096 rows x 4096 x
// 151936: 3.86 ms (1320 TFLOP/s); 1024 rows 1.15 ms (1100): of 16 K steps a tile, the end takes a sixth; with listed
// entries, one a row, 1.21, with 64, 1.31.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void lmloss_weight_stream_kernel(WeightJob job) {
    typedef GemmStream<T, true, true, 16, true> Stream;
    static_assert(Stream::kRowStores == 16, "the stores a tile's end makes");
    __shared__ __align__(1024) char lds[Stream::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    // (without a kept row the products are over a row of zeros)
    const int R = *job.count, K = max(R, 1), tiles = job.nh * job.nv, parts = job.low ? 2 : 1;
    const int64_t ldh = (int64_t)job.H * sizeof(T), ldg = job.ldg * (int64_t)sizeof(T);
    auto place = [&](int i, int &h0, int &v0) {
        const int id = blockIdx.x + i / parts * gridDim.x;
        if (id >= tiles) return false;
        int tm, tn;
        gemm_place(id, job.nh, job.nv, kPlaceGroup, tm, tn);
        h0 = tm * kTile;
        v0 = tn * kTile;
        return true;
    };
    Stream stream;
    stream.run(
        ldh, ldg,
        [&](int i) -> GemmWork {
            int h0, v0;
            if (!place(i, h0, v0)) return {{job.rows, ldh, 0}, {job.G, ldg, 0}, 0};
            const int low = i % parts;
            GemmWork w = {operand_ks<T>(job.rows, ldh, h0, 0), operand_ks<T>(job.G, ldg, v0, low * job.low), K};
            w.more = parts == 2 && low == 0;
            if (R == 0) w.a.valid = w.b.valid = 1 << 30;  // (past every row: nothing is read)
            return w;
        },
        [&](int i) {
            int h0 = 0, v0 = 0;
            place(i, h0, v0);
            static_assert(Stream::BN / Stream::WN == kUnit, "a wave's columns");
            if (!job.low) add_listed(stream.acc, job.rest, (job.v0 + v0 + Stream::wave_n(wave)) / kUnit, 0, job.H,
                       h0 + Stream::wave_m(wave), lds + Stream::kStageBytes + wave * Stream::kScratch,
                       anew(lane));
            stream.store_rows(weight_rows<T>(job, v0, kTile), (int)ldh, h0 * 2, (int)ldh, lds, wave, lane,
                              [&](int mi, int ni) { return stream.acc[mi][ni]; });
        },
        lds, wave, lane);
}

// bf16, few kept rows: 64 STEPS rows of G (with `low`, in two parts). The output is the bound. A wave
// keeps the kept rows' values at 64 columns of H as fragments, for a workgroup's 512, and goes through a
// range of the vocabulary, 64 rows at a time: G's columns come through LDS, two buffers, and the output
// goes through 4 KB of LDS, so that a store covers whole lines (128 bytes of each of 8 rows). 16 rows x
// 4096 x 151936 (1.245 GB written): 231 us, 5.4 TB/s (a plain fill reaches 6.9).
struct WeightFewJob {
    const uint16_t *rows;  // [count, H], or with `from` all rows
    const char *G;         // [grows][ldg], at most 64 STEPS rows
    const int32_t *count, *from;
    int H, v0, v1, low;
    int grows;             // rows of G, 0: the kept rows
    int64_t ldg;
    int slabs, ranges;     // of 512 columns of H; of the vocabulary, a multiple of 8
    uint16_t *grad;        // [V, H]
    ListedRest rest;       // more than one step and G in one part
};

// TWO: G in two parts of 32 STEPS rows, which meet the same rows of hidden.
template <int STEPS> constexpr int weight_few_lds() {
    return 2 * STEPS * GemmSide<uint16_t, 64, true>::kBytes + kGemmWaves * 4096;
}

template <int STEPS, bool TWO>
__device__ __forceinline__ void weight_few(const WeightFewJob &job, int block, char *lds) {
    typedef uint16_t T;
    typedef GemmSide<T, 64, true> Side;
    constexpr int kBuffer = STEPS * Side::kBytes;
    constexpr int kStores = 8;  // a wave's, for 64 rows
    const int lane = threadIdx.x % kWave, g = lane >> 4, j = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count, rows = job.grows ? job.grows : R;
    // (the slabs of a range run on one XCD, whose L2 gives them G)
    const int at = block / 8, slab = at % job.slabs;
    const int range = block % 8 + 8 * (at / job.slabs);
    const int units = (job.v1 - job.v0 + 63) / 64;
    const int u0 = (int)((int64_t)units * range / job.ranges);
    const int u1 = (int)((int64_t)units * (range + 1) / job.ranges);
    if (u0 >= u1) return;
    const int h0 = slab * 512 + wave * 64;

    Side side;
    const int64_t ldg = job.ldg * (int64_t)sizeof(T);
    side.init(ldg, wave, lane);
    const uint32_t base = lds_address(lds);
    auto issue = [&](int u, int buf) {
        const bool in = u < u1 && R > 0;  // (without a kept row nothing has written G: zeros)
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            side.issue(base + buf * kBuffer + s * Side::kBytes,
                       job.G + 64 * s * ldg + (int64_t)u * 128, (int)ldg, u * 128,
                       in ? rows - 64 * s : 0, wave);
    };
    issue(u0, 0);
    constexpr int kHeld = TWO ? STEPS : 2 * STEPS;
    bf16x8 fa[kHeld][4];
    // Where the rows are (`from` has 64 places, of which the kept rows' are used). Loads are of the first
    // kept row where there is none.
    typedef int __attribute__((ext_vector_type(4))) i32x4;
    i32x4 at_row[kHeld][2];
#pragma unroll
    for (int s = 0; s < kHeld; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = 32 * s + 8 * g + 4 * i, r = !TWO && job.low && k >= job.low ? k - job.low : k;
            at_row[s][i] = job.from ? *reinterpret_cast<const i32x4 *>(job.from + r)
                                    : i32x4{r, r + 1, r + 2, r + 3};
        }
    const int first = R > 0 && job.from ? job.from[0] : 0;
#pragma unroll
    for (int s = 0; s < kHeld; ++s) {
        uint32_t src[8];  // (bytes: at most 256 rows of 128 KiB)
        bool in[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = 32 * s + 8 * g + e, r = !TWO && job.low && k >= job.low ? k - job.low : k;
            in[e] = r < R;
            src[e] = (uint32_t)(in[e] ? at_row[s][e / 4][e % 4] : first) * (uint32_t)job.H * 2u;
        }
#pragma unroll
        for (int mi = 0; mi < 4; ++mi) {
            const int h = h0 + 16 * mi + j;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint16_t x = *reinterpret_cast<const uint16_t *>(
                    reinterpret_cast<const char *>(job.rows) + src[e] + 2u * (uint32_t)min(h, job.H - 1));
                fa[s][mi][e] = __builtin_bit_cast(__bf16, in[e] && h < job.H ? x : (uint16_t)0);
            }
        }
    }
    Side::template Reader<4> rb;
    rb.init(0, lane);
    char *scratch = lds + 2 * kBuffer + wave * 4096;
    const int ld = job.H * (int)sizeof(T);
    const int row_in = lane >> 3, chunk = lane & 7;  // of the stores
    const int h_out = h0 + 8 * chunk;
    for (int u = u0; u < u1; ++u) {
        const int buf = (u - u0) & 1;
        // the loads of this buffer are older than the last 64 rows' stores
        if (u == u0) gemm_barrier<0>(); else gemm_barrier<kStores>();
        issue(u + 1, buf ^ 1);
        const int v = job.v0 + u * 64;
        const __amdgpu_buffer_rsrc_t out =
            out_rows(reinterpret_cast<char *>(job.grad) + (int64_t)v * ld, ld, min(job.v1 - v, 64), ld);
        // (of two steps in one part: all four 16 columns at once, so that listed entries are added once)
        constexpr bool kListed = STEPS > 1 && !TWO;
        constexpr int kOnce = STEPS == 2 && !TWO ? 4 : 2;
#pragma unroll
        for (int n0 = 0; n0 < 4; n0 += kOnce) {
            f32x4 acc[4][kOnce];
#pragma unroll
            for (int mi = 0; mi < 4; ++mi)
#pragma unroll
                for (int ni = 0; ni < kOnce; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 2 * STEPS; ++s)
#pragma unroll
                for (int ni = 0; ni < kOnce; ++ni) {
                    const bf16x8 fb = rb.read(lds + buf * kBuffer + (s / 2) * Side::kBytes, n0 + ni, s % 2);
#pragma unroll
                    for (int mi = 0; mi < 4; ++mi)
                        acc[mi][ni] = gemm_mfma(fa[s % kHeld][mi], fb, acc[mi][ni]);
                }
            if constexpr (kListed)
                add_listed(acc, job.rest, job.v0 / kUnit + u, 16 * n0, job.H, h0, scratch, anew(lane));
#pragma unroll
            for (int half = 0; half < kOnce / 2; ++half) {
#pragma unroll
                for (int ni = 0; ni < 2; ++ni)
#pragma unroll
                    for (int mi = 0; mi < 4; ++mi) {
                        const auto x = packed4<T>(acc[mi][2 * half + ni]);
                        const int row = 16 * ni + j;
                        *reinterpret_cast<decltype(packed4<T>(f32x4{})) *>(
                            scratch + row * 128 + (((2 * mi + (g >> 1)) ^ (row & 7)) << 4) + (g & 1) * 8) = x;
                    }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int row = 8 * q + row_in;
                    const u32x4 x =
                        *reinterpret_cast<const u32x4 *>(scratch + row * 128 + ((chunk ^ (row & 7)) << 4));
                    __builtin_amdgcn_raw_buffer_store_b128(
                        x, out,
                        h_out < job.H ? (16 * n0 + 32 * half + row) * ld + h_out * (int)sizeof(T)
                                      : kGemmOutside,
                        0, 0);
                }
            }
        }
    }
    wait_for<0, 0>();  // no load is in flight when the workgroup ends
}

template <int STEPS, bool TWO>
__global__ __launch_bounds__(kGemmThreads) void lmloss_weight_few_kernel(WeightFewJob job) {
    __shared__ __align__(1024) char lds[weight_few_lds<STEPS>()];
    weight_few<STEPS, TWO>(job, blockIdx.x, lds);
}

// Both gradients of little work in one launch, whose two parts do not wait for each other: the first
// `groups` workgroups take grad_hidden's tiles. 40 rows x 256 x 1024: 9 us, 19 as two launches.
template <int BN, int STEPS, bool TWO>
__global__ __launch_bounds__(kGemmThreads) void lmloss_both_few_kernel(HiddenJob hidden,
                                                                       WeightFewJob weight, int groups) {
    constexpr int kHidden = HiddenRing<uint16_t, BN>::kLdsBytes, kWeight = weight_few_lds<STEPS>();
    __shared__ __align__(1024) char lds[kHidden > kWeight ? kHidden : kWeight];
    if ((int)blockIdx.x < groups)
        hidden_few<uint16_t, BN>(hidden, blockIdx.x, lds);
    else
        weight_few<STEPS, TWO>(weight, blockIdx.x - groups, lds);
}

}  // namespace
}  // namespace dflash2

#include "lmhead_rows.h"

namespace dflash2 {
namespace {

// ---- plans and launches ------------------------------------------------------------------------

size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
    int bn, nr;              // kept rows of a tile, tiles
    bool few;                // tiles of at most 128 rows: rings (f32: always)
    int kc;                  // few bf16 rows, H <= 4096: columns of H a wave (lmhead_rows.h); or 0
    bool find;               // few bf16 rows: rings whose workgroups find the kept rows
    bool ring;               // logits by rings of 128 rows though not few (bf16, few tiles of 256 x 256)
    int low;                 // few bf16 rows: G in two parts, this many rows apart; or 0
    int grows;               // rows of G
    // forward
    int nv;                  // tiles of the vocabulary
    // backward
    int piece, pieces;       // columns (a multiple of 256), number
    int splits;              // of a piece, for grad_hidden: at most, all of them in the first one
    size_t rows, place, count, flags, parts, scale, from, G, sums, rest, mask, list, units, forward, backward;

    // what rounding left of G's entries is added to the gradients
    bool listed(int elem) const { return elem == 2 && !low; }
    // G has room for its second part
    bool pair;
    // a unit's entries are as many as a quarter of the rows (kMany)
    bool many(int K, int V) const { return pair && (int64_t)K * kMany > V; }

    // grad_hidden together with the logits
    bool fused() const { return kc && bn == 16; }
    // the logits' tiles of rows
    int logits_bn() const { return ring ? 128 : bn; }
    // workgroups of a rows kernel
    int rows_grid(int width) const {
        const int units = ceil_div(width, kRowsTile);
        return units < kCus ? units : kCus;
    }
    // columns of a split in a piece of `width`
    int per(int width) const { return split_columns(width, splits); }
};

// Rows of a tile for R rows. bf16: 256 from 129 rows on (two tiles of 128 read W twice); f32: 128 at
// most.
int row_tile(int R, int elem) {
    if (elem == 2) return R > 128 ? 256 : R > 64 ? 128 : R > 32 ? 64 : 32;
    // f32: the matrix cores are the bound, so tiles are as short as the rows allow (331 rows x 1016 x
    // 32003, loss and gradients: tiles of 112 758 us, of 128 818; 96 rows x 1024 x 100000: 861, of 128
    // 1012)
    const int even = ceil_div(R, ceil_div(R, 128));
    return even > 64 ? ceil_div(even, 16) * 16 : even > 32 ? 64 : 32;
}

Plan plan(int R, int H, int V, int K, int elem) {
    Plan p;
    p.bn = row_tile(R, elem);
    p.nr = ceil_div(R, p.bn);
    p.few = p.bn <= 128;
    // rows read whole: as many as a wave's registers hold of its columns
    p.kc = elem == 2 && R <= 32 && H <= 4096 && H > kRowsFrom ? H <= 2048 ? 256 : 512 : 0;
    if (p.kc && R <= 16) p.bn = 16;
    p.find = elem == 2 && !p.kc && p.bn <= 64 && K <= (p.bn <= 32 ? ring_list<32>() : ring_list<64>());
    p.low = elem == 2 && p.bn <= 64 ? p.bn : 0;
    p.grows = elem == 2 && p.few ? p.bn + p.low : R;
    p.pair = p.listed(elem) && V < DFLASH2_MAX_K * kMany;
    const int g_rows = p.pair ? 2 * p.grows : p.grows;
    p.nv = ceil_div(V, kTile);
    p.ring = !p.few && p.nv * (int64_t)p.nr <= kRingTiles;
    // a piece: whole rounds of tiles over the CUs, if as many fit
    int64_t most = kPieceBytes / ((int64_t)g_rows * elem) / kTile;
    most = most < 1 ? 1 : most > kPieceMost / kTile ? kPieceMost / kTile : most;
    int round = kCus;
    for (int n = p.nr; n % 2 == 0 && round > 1; n /= 2) round /= 2;
    if (most > round) most = most / round * round;
    p.piece = (int)(most < p.nv ? most : p.nv) * kTile;
    p.pieces = ceil_div(V, p.piece);
    // grad_hidden (rings): a workgroup for every CU, splits of 256 columns at least
    const int tiles = ceil_div(H, kTile) * p.nr, width = p.piece < V ? p.piece : V;
    const int longest = width / 256;
    p.splits = kCus / tiles < longest ? kCus / tiles : longest;
    p.splits = p.splits < 1 ? 1 : p.splits;
    p.splits = ceil_div(width, p.per(width));
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t a = at;
        at += up(n);
        return a;
    };
    p.rows = take((size_t)R * H * elem);
    p.place = take((size_t)R * 4);
    p.count = take(4);
    p.from = take(64 * 4);  // (of at most 64 rows)
    const size_t common = at;
    p.flags = take((size_t)R * 4);
    // (few_ranges of the kept rows' tiles: 256 bn pairs, or one for each of more rows than that)
    const size_t rows16 = (size_t)ceil_div(R, 16) * 16, few_most = (size_t)kCus * p.logits_bn();
    const size_t pairs = p.few || p.ring ? (rows16 > few_most ? rows16 : few_most) : rows16 * p.nv * 2;
    p.parts = take(pairs * sizeof(float2));
    p.forward = at;
    at = common;
    p.scale = take((size_t)R * sizeof(float2));
    p.G = take((size_t)g_rows * p.piece * elem);
    const size_t split_rows = (size_t)kSplitTiles / ceil_div(H, kTile) * kTile;
    const size_t stream_rows = (size_t)p.nr * kTile > split_rows ? (size_t)p.nr * kTile : split_rows;
    const size_t sum_rows = p.fused() ? (size_t)p.rows_grid(width) * 16
                            : p.few   ? (size_t)p.splits * p.grows
                                      : stream_rows;
    p.sums = take(sum_rows * H * 4);
    if (p.listed(elem)) {
        p.rest = take((size_t)R * DFLASH2_MAX_K * sizeof(float));
        p.mask = take((size_t)R * sizeof(uint64_t));
        p.list = take((size_t)R * DFLASH2_MAX_K * sizeof(Listed));
        p.units = take((size_t)((int64_t)p.nv * kTile / kUnit + kListUnits) * sizeof(int2));
    }
    p.backward = at;
    return p;
}

template <int KC>
void launch_rows_kc(const Plan &p, RowsDo what, const RowsJob &job, hipStream_t s) {
    const dim3 grid(p.rows_grid(job.v1 - job.v0)), block(kGemmThreads);
    if (p.bn == 32) {
        if (what == RowsDo::kStats)
            lmloss_rows_kernel<KC, 32, RowsDo::kStats><<<grid, block, 0, s>>>(job);
        else
            lmloss_rows_kernel<KC, 32, RowsDo::kGrad><<<grid, block, 0, s>>>(job);
        return;
    }
    switch (what) {
    case RowsDo::kStats: lmloss_rows_kernel<KC, 16, RowsDo::kStats><<<grid, block, 0, s>>>(job); break;
    case RowsDo::kGrad: lmloss_rows_kernel<KC, 16, RowsDo::kGrad><<<grid, block, 0, s>>>(job); break;
    default: lmloss_rows_kernel<KC, 16, RowsDo::kHidden><<<grid, block, 0, s>>>(job); break;
    }
}

void launch_rows(const Plan &p, RowsDo what, const RowsJob &job, hipStream_t s) {
    if (p.kc == 256)
        launch_rows_kc<256>(p, what, job, s);
    else
        launch_rows_kc<512>(p, what, job, s);
}

template <typename T, int BN, bool GRAD>
void launch_logits_f32(dim3 grid, const LogitsJob &job, hipStream_t s) {
    if constexpr (sizeof(T) == 4)
        lmloss_logits_few_kernel<T, BN, GRAD, false><<<grid, kGemmThreads, 0, s>>>(job);
}

template <typename T, bool GRAD>
void launch_logits(const Plan &p, const LogitsJob &job, hipStream_t s) {
    const dim3 block(kGemmThreads);
    if constexpr (sizeof(T) == 2) {
        if (!p.few && !p.ring) {
            const int tiles = job.nv * job.nr;
            lmloss_logits_stream_kernel<T, GRAD><<<tiles < kCus ? tiles : kCus, block, 0, s>>>(job);
            return;
        }
    }
    // (at least what few_ranges gives for the kept rows, whose tiles are job.nr at most)
    const int64_t all = (int64_t)ceil_div(job.v1 - job.v0, 16) * job.nr;
    const dim3 grid(job.nr > kCus ? job.nr : all < kCus ? (int)all : kCus);
    if constexpr (sizeof(T) == 2) {
        if (p.find) {
            if (p.bn == 64)
                lmloss_logits_few_kernel<T, 64, GRAD, true><<<grid, block, 0, s>>>(job);
            else
                lmloss_logits_few_kernel<T, 32, GRAD, true><<<grid, block, 0, s>>>(job);
            return;
        }
    }
    switch (p.logits_bn()) {
    case 128: lmloss_logits_few_kernel<T, 128, GRAD, false><<<grid, block, 0, s>>>(job); break;
    case 64: lmloss_logits_few_kernel<T, 64, GRAD, false><<<grid, block, 0, s>>>(job); break;
    case 80: launch_logits_f32<T, 80, GRAD>(grid, job, s); break;
    case 96: launch_logits_f32<T, 96, GRAD>(grid, job, s); break;
    case 112: launch_logits_f32<T, 112, GRAD>(grid, job, s); break;
    default: lmloss_logits_few_kernel<T, 32, GRAD, false><<<grid, block, 0, s>>>(job); break;
    }
}

template <typename T, int BN>
void launch_hidden_f32(dim3 grid, const HiddenJob &job, hipStream_t s) {
    if constexpr (sizeof(T) == 4) lmloss_hidden_few_kernel<T, BN><<<grid, kGemmThreads, 0, s>>>(job);
}

template <typename T>
void launch_hidden(const Plan &p, const HiddenJob &job, hipStream_t s) {
    const int tiles = job.nh * job.nr * job.splits;
    const dim3 grid(tiles), block(kGemmThreads);
    if constexpr (sizeof(T) == 2) {
        if (!p.few) {
            lmloss_hidden_stream_kernel<T><<<kCus, block, 0, s>>>(job);
            return;
        }
    }
    switch (p.bn + p.low) {
    case 128: lmloss_hidden_few_kernel<T, 128><<<grid, block, 0, s>>>(job); break;
    case 64: lmloss_hidden_few_kernel<T, 64><<<grid, block, 0, s>>>(job); break;
    case 112: launch_hidden_f32<T, 112>(grid, job, s); break;
    case 96: launch_hidden_f32<T, 96>(grid, job, s); break;
    case 80: launch_hidden_f32<T, 80>(grid, job, s); break;
    default: launch_hidden_f32<T, 32>(grid, job, s); break;
    }
}

WeightFewJob weight_few_job(const Plan &p, const WeightJob &job, int groups) {
    WeightFewJob w = {reinterpret_cast<const uint16_t *>(job.rows), job.G, job.count, job.from, job.H,
                      job.v0, job.v1, p.low, p.few ? p.grows : 0, job.ldg, ceil_div(job.H, 512), 0,
                      static_cast<uint16_t *>(job.grad), job.rest};
    const int most = ceil_div(job.v1 - job.v0, 64);  // (a range has 64 columns at least)
    w.ranges = 8 * ceil_div(groups < (int64_t)most * w.slabs ? groups : most * w.slabs, 8 * w.slabs);
    return w;
}

template <typename T>
void launch_weight(const Plan &p, const WeightJob &job, hipStream_t s) {
    if constexpr (sizeof(T) == 4) {
        lmloss_weight_kernel<T><<<job.nh * job.nv, kGemmThreads, 0, s>>>(job);
    } else if (p.grows <= kTile && !job.low) {
        const WeightFewJob w = weight_few_job(p, job, kCus);
        const int grid = w.slabs * w.ranges;
        switch (p.low) {
        case 64: lmloss_weight_few_kernel<2, true><<<grid, kGemmThreads, 0, s>>>(w); break;
        case 32: lmloss_weight_few_kernel<1, true><<<grid, kGemmThreads, 0, s>>>(w); break;
        case 16: lmloss_weight_few_kernel<1, false><<<grid, kGemmThreads, 0, s>>>(w); break;
        default:
            if (p.grows > 128)
                lmloss_weight_few_kernel<4, false><<<grid, kGemmThreads, 0, s>>>(w);
            else
                lmloss_weight_few_kernel<2, false><<<grid, kGemmThreads, 0, s>>>(w);
        }
    } else {
        const int tiles = job.nh * job.nv;
        lmloss_weight_stream_kernel<T><<<tiles < kCus ? tiles : kCus, kGemmThreads, 0, s>>>(job);
    }
}

// Both gradients of up to 128 bf16 rows in one launch, where grad_hidden's tiles leave the weight half of
// the CUs and more. The backward call in one launch and in two: 40 rows x 256 x 8000 28 us and 37, x 32000
// (125 tiles) 49 and 49; 100 rows x 1000 x 8000 63 and 70. Whether they were launched.
bool launch_both(const Plan &p, const HiddenJob &hj, const WeightJob &wj, hipStream_t s) {
    const int groups = hj.nh * hj.nr * hj.splits;
    if (!p.few || groups > kBothGroups || wj.low) return false;
    const WeightFewJob w = weight_few_job(p, wj, kCus - groups);
    const dim3 grid(groups + w.slabs * w.ranges), block(kGemmThreads);
    switch (p.low) {
    case 64: lmloss_both_few_kernel<128, 2, true><<<grid, block, 0, s>>>(hj, w, groups); break;
    case 32: lmloss_both_few_kernel<64, 1, true><<<grid, block, 0, s>>>(hj, w, groups); break;
    default: lmloss_both_few_kernel<128, 2, false><<<grid, block, 0, s>>>(hj, w, groups); break;
    }
    return true;
}

Coef coef(float tau) {
    const double exact = 1.4426950408889634 / (double)tau;
    const float c = (float)exact;
    return {c, (float)(exact - (double)c)};
}

RowsJob rows_job(const Plan &p, const void *hidden, const void *W, const Entries &e, int R, int H, int V,
                 float *stats, char *ws) {
    RowsJob job = {};
    job.hidden = static_cast<const uint16_t *>(hidden);
    job.W = static_cast<const uint16_t *>(W);
    job.R = R;
    job.H = H;
    job.V = V;
    job.c = coef(e.tau);
    job.e = e;
    job.stats = stats;
    job.place = reinterpret_cast<int32_t *>(ws + p.place);
    job.from = reinterpret_cast<int32_t *>(ws + p.from);
    job.count = reinterpret_cast<int32_t *>(ws + p.count);
    return job;
}

void few_rows(const Plan &p, const Entries &e, int R, float *stats, const float *grad_loss, char *ws,
              LogitsJob &job) {
    job.R = R;
    job.e = e;
    job.stats = stats;
    job.grad_loss = grad_loss;
    job.place = reinterpret_cast<int32_t *>(ws + p.place);
    job.from = reinterpret_cast<int32_t *>(ws + p.from);
    job.kept = reinterpret_cast<int32_t *>(ws + p.count);
}

template <typename T>
hipError_t forward(const Plan &p, const void *hidden, const void *W, Entries e, int R, int H, int V,
                   float *loss, float *stats, char *ws, hipStream_t s) {
    const Coef c = coef(e.tau);
    int32_t *place = reinterpret_cast<int32_t *>(ws + p.place);
    int32_t *count = reinterpret_cast<int32_t *>(ws + p.count);
    float2 *parts = reinterpret_cast<float2 *>(ws + p.parts);
    const auto finish = [&](int64_t nparts) {
        FinishJob fj = {parts, nparts, place, count, p.logits_bn(), e, R, V, c, loss, stats};
        lmloss_finish_kernel<<<ceil_div(R, kFinishRows), kFinishThreads, 0, s>>>(fj);
        return hipGetLastError();
    };
    if (p.kc) {
        RowsJob rj = rows_job(p, hidden, W, e, R, H, V, stats, ws);
        rj.v1 = V;
        rj.parts = parts;
        launch_rows(p, RowsDo::kStats, rj, s);
        return finish(p.rows_grid(V));
    }
    if (!p.find) {
        GatherJob gj = {};
        gj.hidden = static_cast<const char *>(hidden);
        gj.W = static_cast<const char *>(W);
        gj.flags = reinterpret_cast<int32_t *>(ws + p.flags);
        gj.stats = stats;
        gj.e = e;
        gj.R = R;
        gj.H = H;
        gj.V = V;
        gj.rows = ws + p.rows;
        gj.place = place;
        gj.count = count;
        const dim3 grid(ceil_div(R, kGatherRows), e.teacher ? ceil_div(e.K, kGatherEntries) : 1);
        if (e.teacher && (int64_t)R * e.K <= kInlineEntries) {
            lmloss_gather_kernel<T, Rows::kEntries, kGatherEntries><<<grid, 256, 0, s>>>(gj);
        } else if (e.teacher) {
            lmloss_flags_kernel<<<ceil_div(R, 4), 256, 0, s>>>(e, R, V, const_cast<int32_t *>(gj.flags));
            lmloss_gather_kernel<T, Rows::kFlags, kGatherEntries><<<grid, 256, 0, s>>>(gj);
        } else {
            lmloss_gather_kernel<T, Rows::kTargets, 1><<<grid, 256, 0, s>>>(gj);
        }
    }
    LogitsJob lj = {};
    lj.rows = p.find ? static_cast<const char *>(hidden) : ws + p.rows;
    lj.W = static_cast<const char *>(W);
    lj.count = count;
    few_rows(p, e, R, stats, nullptr, ws, lj);
    lj.H = H;
    lj.V = V;
    lj.v0 = 0;
    lj.v1 = V;
    lj.nv = p.nv;
    lj.nr = ceil_div(R, p.logits_bn());
    lj.c = c;
    lj.parts = parts;
    lj.nparts = p.few || p.ring ? 0 : p.nv * 2;
    launch_logits<T, false>(p, lj, s);
    return finish(lj.nparts);
}

template <typename T>
hipError_t backward(const Plan &p, const void *hidden, const void *W, Entries e,
                    const float *stats, const float *grad_loss, int R, int H, int V,
                    void *grad_hidden, void *grad_W, char *ws, hipStream_t s) {
    const Coef c = coef(e.tau);
    int32_t *place = reinterpret_cast<int32_t *>(ws + p.place);
    int32_t *count = reinterpret_cast<int32_t *>(ws + p.count);
    int32_t *from = reinterpret_cast<int32_t *>(ws + p.from);
    float2 *scale = reinterpret_cast<float2 *>(ws + p.scale);
    const bool listed = p.listed(sizeof(T)), many = listed && grad_W && p.many(e.K, V);
    float *rest = listed ? reinterpret_cast<float *>(ws + p.rest) : nullptr;
    uint64_t *mask = listed && e.teacher ? reinterpret_cast<uint64_t *>(ws + p.mask) : nullptr;
    if (!p.kc && !p.find) {
        KeepJob kj = {};
        kj.hidden = static_cast<const char *>(hidden);
        kj.stats = stats;
        kj.grad_loss = grad_loss;
        kj.R = R;
        kj.H = H;
        kj.K = e.K;
        kj.tau = e.tau;
        kj.rows = ws + p.rows;
        kj.place = place;
        kj.count = count;
        kj.scale = scale;
        if (listed && e.teacher) {
            kj.ids = e.ids;
            kj.teacher = e.teacher;
            kj.V = V;
            kj.mask = mask;
        }
        lmloss_keep_kernel<T><<<ceil_div(R, kKeepRows), kKeepThreads, 0, s>>>(kj);
    }
    ListsJob lists = {};
    if (listed && grad_W && !many) {
        const int units = p.nv * (kTile / kUnit), per = ceil_div(units, kCus / 2);
        lists.ids = e.ids;
        lists.mask = mask;
        lists.n = R * e.K;
        lists.K = e.K;
        lists.V = V;
        lists.inverse = e.K == 1 ? 0u : (uint32_t)(((1ull << 32) + e.K - 1) / e.K);
        lists.per = per < kListUnits ? per : kListUnits;
        lists.groups = ceil_div(units, lists.per);
        lists.list = reinterpret_cast<Listed *>(ws + p.list);
        lists.units = reinterpret_cast<int2 *>(ws + p.units);
    }
    const ListedRest left = {lists.list, lists.units, rest, static_cast<const uint16_t *>(hidden)};
    const bool fused = p.fused() && grad_hidden;
    const int nh = ceil_div(H, kTile);
    for (int i = 0; i < p.pieces; ++i) {
        const int v0 = i * p.piece, v1 = v0 + p.piece < V ? v0 + p.piece : V;
        const char *Wb = static_cast<const char *>(W);
        const int nv = ceil_div(v1 - v0, kTile);
        if (p.kc) {
            RowsJob rj = rows_job(p, hidden, W, e, R, H, V, const_cast<float *>(stats), ws);
            rj.v0 = v0;
            rj.v1 = v1;
            rj.grad_loss = grad_loss;
            rj.G = fused && !grad_W ? nullptr : reinterpret_cast<uint16_t *>(ws + p.G);
            rj.ldg = p.piece;
            rj.low = p.low;
            rj.sums = reinterpret_cast<float *>(ws + p.sums);
            rj.first = i == 0;
            launch_rows(p, fused ? RowsDo::kHidden : RowsDo::kGrad, rj, s);
        } else {
            LogitsJob lj = {};
            lj.rows = p.find ? static_cast<const char *>(hidden) : ws + p.rows;
            lj.W = Wb;
            lj.count = count;
            few_rows(p, e, R, const_cast<float *>(stats), grad_loss, ws, lj);
            lj.H = H;
            lj.V = V;
            lj.v0 = v0;
            lj.v1 = v1;
            lj.nv = nv;
            lj.nr = ceil_div(R, p.logits_bn());
            lj.c = c;
            lj.G = ws + p.G;
            lj.ldg = p.piece;
            lj.scale = scale;
            lj.low = p.low;
            lj.whole = p.few;
            launch_logits<T, true>(p, lj, s);
            if (!p.find) {
                const int low = many ? p.grows : p.low;
                if (many) {
                    const int64_t n = (int64_t)p.grows * p.piece / 8;  // (of bf16 rows of whole vectors)
                    lmloss_zero_kernel<<<(int)(n / 1024 < 8 * kCus ? n / 1024 + 1 : 8 * kCus), 256, 0, s>>>(
                        reinterpret_cast<u32x4 *>(ws + p.G) + n, n);
                }
                EntriesJob ej = {e, stats, grad_loss, place, R, V, v0, v1, c, lj.G, p.piece, low, rest, mask,
                                 ceil_div(R, kKeepRows), lists};
                lmloss_entries_kernel<T>
                    <<<ej.groups + (i == 0 ? lists.groups : 0), kKeepThreads, 0, s>>>(ej);
            }
        }
        const int per = p.per(v1 - v0);
        const HiddenJob hj = {Wb, ws + p.G, count, p.grows, H, v0, v1, p.piece, nh, p.nr,
                              ceil_div(v1 - v0, per), per, i == 0, reinterpret_cast<float *>(ws + p.sums),
                              p.low, p.piece < V ? p.piece : V};
        const bool found = p.kc || p.find;  // (the kept rows are where they were)
        const WeightJob wj = {found ? static_cast<const char *>(hidden) : ws + p.rows, ws + p.G, count,
                              found ? from : nullptr, H, v0, v1, p.piece, nh,
                              sizeof(T) == 4 ? ceil_div(v1 - v0, 128) : nv, grad_W, left, many ? p.grows : 0};
        if constexpr (sizeof(T) == 2)
            if (grad_hidden && !fused && grad_W && launch_both(p, hj, wj, s)) continue;
        if (grad_hidden && !fused) launch_hidden<T>(p, hj, s);
        if (grad_W) launch_weight<T>(p, wj, s);
    }
    if (grad_hidden) {
        const dim3 grid(R, ceil_div(H, 256));
        const float *sums = reinterpret_cast<const float *>(ws + p.sums);
        const int width = p.piece < V ? p.piece : V;
        const int splits = p.fused() ? p.rows_grid(width) : p.splits, rows = p.fused() ? 16 : p.grows;
        const int low = p.fused() ? 0 : p.low, stream = p.few ? 0 : width;
        T *out = static_cast<T *>(grad_hidden);
        if (p.few && splits >= 32)
            lmloss_hidden_out_kernel<T, 16>
                <<<grid, 16 * kWave, 0, s>>>(sums, splits, rows, low, count, stream, place, H, out, e, V, rest,
                                             static_cast<const T *>(W));
        else
            lmloss_hidden_out_kernel<T, 4>
                <<<grid, 4 * kWave, 0, s>>>(sums, splits, rows, low, count, stream, place, H, out, e, V, rest,
                                            static_cast<const T *>(W));
    }
    return hipGetLastError();
}

}  // namespace

size_t lmloss_workspace_bytes(int R, int H, int V, int elem_bytes) {
    const Plan p = plan(R, H, V, 1, elem_bytes);  // (K decides nothing that takes space)
    return p.forward;
}

size_t lmloss_backward_workspace_bytes(int R, int H, int V, int elem_bytes) {
    const Plan p = plan(R, H, V, 1, elem_bytes);  // (K decides nothing that takes space)
    return p.backward;
}

hipError_t launch_lmloss(const void *hidden, const void *W, int elem_bytes, const int32_t *ids,
                         const float *teacher, int R, int H, int V, int K, float tau, float *loss,
                         float *row_stats, void *ws, hipStream_t stream) {
    const Plan p = plan(R, H, V, K, elem_bytes);
    const Entries e = {ids, teacher, K, tau};
    char *w = static_cast<char *>(ws);
    return elem_bytes == 2
               ? forward<uint16_t>(p, hidden, W, e, R, H, V, loss, row_stats, w, stream)
               : forward<float>(p, hidden, W, e, R, H, V, loss, row_stats, w, stream);
}

hipError_t launch_lmloss_backward(const void *hidden, const void *W, int elem_bytes,
                                  const int32_t *ids, const float *teacher, const float *row_stats,
                                  const float *grad_loss, int R, int H, int V, int K, float tau,
                                  void *grad_hidden, void *grad_W, void *ws, hipStream_t stream) {
    const Plan p = plan(R, H, V, K, elem_bytes);
    const Entries e = {ids, teacher, K, tau};
    char *w = static_cast<char *>(ws);
    return elem_bytes == 2 ? backward<uint16_t>(p, hidden, W, e, row_stats, grad_loss, R, H, V,
                                                grad_hidden, grad_W, w, stream)
                           : backward<float>(p, hidden, W, e, row_stats, grad_loss, R, H, V,
                                             grad_hidden, grad_W, w, stream);
}

}  // namespace dflash2
