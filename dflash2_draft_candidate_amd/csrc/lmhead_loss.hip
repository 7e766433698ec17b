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
//     whose tile lies behind it end at once.
//   * Forward: the product's tiles (W's rows x hidden rows) end in a maximum and a sum of
//     exponentials per hidden row, 8 bytes instead of a tile of logits; a second kernel joins
//     them. The logits of the entries come from dot products of their own, in the first kernel.
//   * Backward: for a piece of the vocabulary at a time, the product again (the same sums in the
//     same order) with G as its epilogue, in a buffer of at most kPieceBytes that stays in the
//     last-level cache; then the entries of the piece, whose value is formed from the kept logit
//     and rounded once; then the two products that read the piece. grad_hidden is summed over the
//     pieces in fp32, split along the vocabulary where it has few tiles.
//   * bf16: G is rounded to bf16 for the matrix cores (2^-9 of each entry, as a bf16 gradient of
//     logits would be); everything else is fp32. f32 inputs take the f32 matrix instructions
//     throughout.
#include <type_traits>

#include "gemm_tile.h"
#include "kernels.h"

namespace dflash2 {
namespace {

constexpr int kTile = 256;                       // rows of W (or columns of hidden) per tile
constexpr int64_t kPieceBytes = 128ll << 20;     // of G
constexpr int kPieceMost = 1 << 20;              // columns of a piece (32-bit offsets in it)
constexpr int kPlaceGroup = 8;                   // rows of tiles that share columns of tiles
constexpr int kCus = 256;

// Rows of a tile's hidden side for R rows.
int row_tile(int R) { return R > 128 ? 256 : R > 64 ? 128 : R > 32 ? 64 : 32; }

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

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

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, kWave);
    return x;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, kWave);
    return x;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, kWave));
    return x;
}

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

enum class Rows { kTargets, kFlags, kStats };

struct GatherJob {
    const char *hidden;   // [R, H]
    const char *W;        // [V, H] (forward: the entries' logits)
    const int32_t *flags; // kFlags
    float *stats;         // [R, K + 2]: forward: entries' logits out; kStats: in
    const float *grad_loss;
    Entries e;
    int R, H, V;
    char *rows;           // [R, H] the kept rows, behind one another
    int32_t *place;       // [R] where row r went, -1: left out
    int32_t *count;
    float2 *scale;        // kStats: [kept rows] (max, g tau / sum)
};

constexpr int kGatherRows = 4;     // rows per workgroup, one a wave
constexpr int kGatherEntries = 8;  // entries per wave

template <Rows M>
__device__ __forceinline__ bool row_kept(const GatherJob &job, int r) {
    if constexpr (M == Rows::kTargets) return id_ok(job.e.ids[r], job.V);
    if constexpr (M == Rows::kFlags) return job.flags[r] != 0;
    if constexpr (M == Rows::kStats) return !(job.stats[(int64_t)r * (job.e.K + 2) + 1] < 0.f);
}

// Workgroup (x, y): rows 4 x .. 4 x + 3; y = 0 copies them to their places, and (forward) each y
// takes the dot products of 8 of the entries. A row's place is the number of kept rows before it,
// which every workgroup of y = 0 counts for itself.
template <typename T, Rows M>
__global__ __launch_bounds__(256) void lmloss_gather_kernel(GatherJob job) {
    constexpr bool kForward = M != Rows::kStats;
    constexpr int kPer = 16 / (int)sizeof(T);
    __shared__ int part[4];
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
    if constexpr (!kForward) {
        char *dst = job.rows + before * row_bytes;
        for (int64_t b = lane * 16; b < row_bytes; b += kWave * 16)
            *reinterpret_cast<u32x4 *>(dst + b) = *reinterpret_cast<const u32x4 *>(src + b);
        if (lane == 0) {
            const float *st = job.stats + (int64_t)r * (K + 2);
            job.scale[before] = float2{st[0], job.grad_loss[r] * job.e.tau / st[1]};
        }
        return;
    } else {
        char *dst = job.rows + before * row_bytes;
        const int j0 = blockIdx.y * kGatherEntries, n = min(kGatherEntries, K - j0);
        const char *w[kGatherEntries];
        float sum[kGatherEntries];
#pragma unroll
        for (int j = 0; j < kGatherEntries; ++j) {
            const int id = j < n ? job.e.ids[(int64_t)r * K + j0 + j] : 0;
            w[j] = job.W + (id_ok(id, job.V) ? id : 0) * row_bytes;
            sum[j] = 0.f;
        }
        for (int64_t b = lane * 16; b < row_bytes; b += kWave * 16) {
            const u32x4 h = *reinterpret_cast<const u32x4 *>(src + b);
            if (copies) *reinterpret_cast<u32x4 *>(dst + b) = h;
            float x[kPer];
            Elem<T>::unpack(h, x);
#pragma unroll
            for (int j = 0; j < kGatherEntries; ++j) {
                if (j >= n) break;
                float y[kPer];
                Elem<T>::unpack(*reinterpret_cast<const u32x4 *>(w[j] + b), y);
#pragma unroll
                for (int i = 0; i < kPer; ++i) sum[j] = fmaf(x[i], y[i], sum[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kGatherEntries; ++j) {
            if (j >= n) break;
            const float s = wave_sum(sum[j]);
            if (lane == 0) job.stats[(int64_t)r * (K + 2) + 2 + j0 + j] = s;
        }
    }
}

// ---- the product's epilogues ---------------------------------------------------------------------

struct LogitsJob {
    const char *rows;     // [count, H]
    const char *W;        // [V, H]
    const int32_t *count;
    int H, V;
    int v0, v1;           // the piece of the vocabulary
    int nv, nr;           // tiles (of all R rows)
    float c;              // log2(e) / tau
    float2 *parts;        // forward: per 16 rows, [nparts][16] (max, sum)
    int64_t nparts;
    void *G;              // backward: [count][ldg]
    int64_t ldg;          // columns
    const float2 *scale;  // backward: [count]
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
    const float c = job.c;
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
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int mi = 0; mi < Tile::MI; ++mi)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += __builtin_amdgcn_exp2f((tile.acc[mi][ni][i] - ref) * c);
            sum += __shfl_xor(sum, 16, kWave);
            sum += __shfl_xor(sum, 32, kWave);
            if (g == 0 && r < R)
                job.parts[((r >> 4) * job.nparts + part + wave / Tile::WN) * 16 + (r & 15)] =
                    float2{top, sum};
        } else if constexpr (std::is_same<Tile, GradStream<T>>::value) {
            break;  // (stored below)
        } else {
            const float2 s = job.scale[min(r, R - 1)];
            const int off = rn * (int)ldg + (vw - v0) * (int)sizeof(T);
#pragma unroll
            for (int mi = 0; mi < Tile::MI; ++mi) {
                f32x4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[i] = s.y * __builtin_amdgcn_exp2f((tile.acc[mi][ni][i] - s.x) * c);
                    if (ragged && vw + 16 * mi + i >= job.v1) y[i] = 0.f;
                }
                store4<T>(out, off + 16 * mi * (int)sizeof(T), y);
                __builtin_amdgcn_sched_barrier(0);  // (all at once would not fit the registers)
            }
        }
    }
    if constexpr (GRAD && std::is_same<Tile, GradStream<T>>::value) {
        float2 s[Tile::NI];
#pragma unroll
        for (int ni = 0; ni < Tile::NI; ++ni)
            s[ni] = job.scale[min(r0 + Tile::wave_n(wave) + 16 * ni + j, R - 1)];
        tile.store_rows(out, (int)ldg, 0, kTile * 2, lds, wave, lane, [&](int mi, int ni) {
            f32x4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = s[ni].y * __builtin_amdgcn_exp2f((tile.acc[mi][ni][i] - s[ni].x) * c);
                if (ragged && vw + 16 * mi + i >= job.v1) y[i] = 0.f;
            }
            return y;
        });
    }
}

// Tiles of 256 vocabulary rows x BN kept rows, one a workgroup.
template <typename T, int BN, int WM_, bool GRAD>
__global__ __launch_bounds__(kGemmThreads) void lmloss_logits_kernel(LogitsJob job) {
    typedef GemmTile<T, kTile, BN, false, false, WM_> Tile;
    __shared__ __align__(1024) char lds[Tile::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count, nr = (R + BN - 1) / BN;
    if ((int)blockIdx.x >= job.nv * nr) return;
    int tm, tn;
    gemm_place(blockIdx.x, job.nv, nr, kPlaceGroup, tm, tn);
    const int v0 = job.v0 + tm * kTile, r0 = tn * BN;
    const int64_t ld = (int64_t)job.H * sizeof(T);
    Tile tile;
    tile.run(operand_kc<T>(job.W, ld, v0, job.v1, 0), operand_kc<T>(job.rows, ld, r0, R, 0), job.H,
             lds, wave, lane);
    logits_done<T, GRAD>(job, tile, v0, r0, R, (int64_t)tm * WM_, lds, wave, lane);
}

// The same with 256 kept rows a tile, as a stream.
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

// ---- forward's end -------------------------------------------------------------------------------

// (ref, sum) pairs in natural units: sum counts exp((x - ref) / tau). NaN in either stays.
__device__ __forceinline__ void join(float &m, float &s, float om, float os, float c) {
    const float top = fmaxf(m, om), ref = top == -INFINITY ? 0.f : top;
    s = s * __builtin_amdgcn_exp2f((m - ref) * c) + os * __builtin_amdgcn_exp2f((om - ref) * c);
    m = top;
}

constexpr int kFinishRows = 16;
constexpr int kFinishThreads = 512;

struct FinishJob {
    const float2 *parts;
    int64_t nparts;
    const int32_t *place;
    Entries e;
    int R, V;
    float c;
    float *loss;
    float *stats;
};

// 16 rows: their tiles' pairs in a fixed order, then a wave per row over its entries.
__global__ __launch_bounds__(kFinishThreads) void lmloss_finish_kernel(FinishJob job) {
    constexpr int kGroups = kFinishThreads / kFinishRows;
    __shared__ float2 pair[kGroups][kFinishRows];
    const int first = blockIdx.x * kFinishRows;
    {
        const int k = threadIdx.x % kFinishRows, grp = threadIdx.x / kFinishRows;
        const int r = first + k, p = r < job.R ? job.place[r] : -1;
        float m = -INFINITY, s = 0.f;
        if (p >= 0) {
            const float2 *src = job.parts + (p >> 4) * job.nparts * 16 + (p & 15);
            for (int64_t i = grp; i < job.nparts; i += kGroups) {
                const float2 x = src[i * 16];
                join(m, s, x.x, x.y, job.c);
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
        if (lane < kGroups) {
            m = pair[lane][k].x;
            s = pair[lane][k].y;
        }
#pragma unroll
        for (int d = 1; d < kGroups; d *= 2) {
            const float om = __shfl_down(m, d, kWave), os = __shfl_down(s, d, kWave);
            if (lane % (2 * d) == 0) join(m, s, om, os, job.c);
        }
        m = __shfl(m, 0, kWave);
        s = __shfl(s, 0, kWave);
        const int id = lane < K ? job.e.ids[(int64_t)r * K + lane] : -1;
        const bool ok = id_ok(id, job.V);
        double term = 0.0;
        const double tau = job.e.tau;
        double p = ok ? 1.0 : 0.0, ln_p = 0.0;
        if (job.e.teacher) {
            const float t = ok ? job.e.teacher[(int64_t)r * K + lane] : -INFINITY;
            float top = wave_max(t);
            if (__ballot(ok && t != t) != 0ull) top = NAN;
            ln_p = ((double)t - top) / tau;
            const double w = ok ? exp(ln_p) : 0.0;
            const double all = wave_sum(w);
            p = w / all;
            ln_p -= log(all);
        }
        if (ok && !(p == 0.0)) {
            // (the entry's logit comes from another order of sums than the row's: at most 0)
            double ln_q = ((double)st[2 + lane] - m) / tau - log((double)s);
            ln_q = ln_q > 0.0 ? 0.0 : ln_q;
            term = p * (ln_p - ln_q);
        }
        term = wave_sum(term);
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
    float c;
    void *G;
    int64_t ldg;
};

// One wave per row: G at the row's entries, the masses of equal ids added in their order.
template <typename T>
__global__ __launch_bounds__(256) void lmloss_entries_kernel(EntriesJob job) {
    const int r = blockIdx.x * 4 + threadIdx.x / kWave, lane = threadIdx.x % kWave;
    if (r >= job.R) return;
    const int p = job.place[r];
    if (p < 0) return;
    const int K = job.e.K;
    const int id = lane < K ? job.e.ids[(int64_t)r * K + lane] : -1;
    const bool ok = id_ok(id, job.V);
    float mass = 1.f;
    if (job.e.teacher) {
        const float t = ok ? job.e.teacher[(int64_t)r * K + lane] : -INFINITY;
        float top = wave_max(t);
        if (__ballot(ok && t != t) != 0ull) top = NAN;
        const float w = ok ? __builtin_amdgcn_exp2f((t - top) * job.c) : 0.f;
        mass = w / wave_sum(w);
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
    if (!ok || earlier || id < job.v0 || id >= job.v1) return;
    const float *st = job.stats + (int64_t)r * (K + 2);
    const float q = fminf(__builtin_amdgcn_exp2f((st[2 + lane] - st[0]) * job.c) / st[1], 1.f);
    // (fminf drops a NaN: a row whose sum is NaN keeps it)
    const float y = job.grad_loss[r] * job.e.tau * ((st[1] != st[1] ? st[1] : q) - total);
    T *out = static_cast<T *>(job.G) + p * job.ldg + (id - job.v0);
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<__bf16 *>(out) = (__bf16)y;
    else
        *out = y;
}

// ---- the gradients' products -----------------------------------------------------------------------

struct HiddenJob {
    const char *W;       // [V, H]
    const char *G;       // [count][ldg]
    const int32_t *count;
    int R, H, v0, v1;
    int64_t ldg;
    int nh, nr, splits, per;  // tiles (of all R rows); splits of the piece, `per` columns each
    bool first;          // the first piece: nothing to add to
    float *sums;         // [splits][R][H]
};

template <typename Tile>
__device__ __forceinline__ void hidden_done(const HiddenJob &job, Tile &tile, int split, int h0,
                                            int r0, int R, int wave, int lane) {
    lane = anew(lane);
    const int g = lane >> 4, j = lane & 15;
    const int ld = job.H * 4;
    const __amdgpu_buffer_rsrc_t out = out_rows(
        job.sums + ((int64_t)split * job.R + r0) * job.H, ld, min(R - r0, Tile::kCols), ld);
#pragma unroll
    for (int ni = 0; ni < Tile::NI; ++ni) {
        const int row = (Tile::wave_n(wave) + 16 * ni + j) * ld;
#pragma unroll
        for (int mi = 0; mi < Tile::MI; ++mi) {
            const int h = h0 + Tile::wave_m(wave) + 16 * mi + 4 * g;
            const int off = h < job.H ? row + 4 * h : kGemmOutside;
            f32x4 x = tile.acc[mi][ni];
            if (!job.first)
                x += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(out, off, 0, 0));
            store4<float>(out, off, x);
        }
    }
}

// Tiles of 256 columns of H x BN kept rows over a split of the piece, one a workgroup.
template <typename T, int BN, int WM>
__global__ __launch_bounds__(kGemmThreads) void lmloss_hidden_kernel(HiddenJob job) {
    typedef GemmTile<T, kTile, BN, true, false, WM> Tile;
    __shared__ __align__(1024) char lds[Tile::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count, nr = (R + BN - 1) / BN;
    if ((int)blockIdx.x >= job.nh * job.splits * nr) return;
    int tm, tn;
    gemm_place(blockIdx.x, job.nh * job.splits, nr, kPlaceGroup, tm, tn);
    const int split = tm / job.nh, h0 = tm % job.nh * kTile, r0 = tn * BN;
    const int k0 = split * job.per, k1 = min(k0 + job.per, job.v1 - job.v0);
    Tile tile;
    tile.run(operand_ks<T>(job.W, (int64_t)job.H * sizeof(T), h0, job.v0 + k0),
             operand_kc<T>(job.G, job.ldg * (int64_t)sizeof(T), r0, R, k0), k1 - k0, lds, wave, lane);
    hidden_done(job, tile, split, h0, r0, R, wave, lane);
}

// The same with 256 kept rows a tile, as a stream.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void lmloss_hidden_stream_kernel(HiddenJob job) {
    typedef GemmStream<T, true, false, 32> Stream;  // (hidden_done: 32 stores)
    __shared__ __align__(1024) char lds[Stream::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count, nr = (R + kTile - 1) / kTile, tiles = job.nh * job.splits * nr;
    const int64_t ldw = (int64_t)job.H * sizeof(T), ldg = job.ldg * (int64_t)sizeof(T);
    auto place = [&](int i, int &split, int &h0, int &r0) {
        const int id = blockIdx.x + i * gridDim.x;
        if (id >= tiles) return false;
        int tm, tn;
        gemm_place(id, job.nh * job.splits, nr, kPlaceGroup, tm, tn);
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
            const int k0 = split * job.per, k1 = min(k0 + job.per, job.v1 - job.v0);
            return {operand_ks<T>(job.W, ldw, h0, job.v0 + k0), operand_kc<T>(job.G, ldg, r0, R, k0),
                    k1 - k0};
        },
        [&](int i) {
            int split = 0, h0 = 0, r0 = 0;
            place(i, split, h0, r0);
            hidden_done(job, stream, split, h0, r0, R, wave, lane);
        },
        lds, wave, lane);
}

// grad_hidden from the splits' sums, in split order; zeros for the rows left out. One workgroup per
// row.
template <typename T>
__global__ __launch_bounds__(256) void lmloss_hidden_out_kernel(const float *sums, int splits,
                                                                const int32_t *place, int R, int H,
                                                                T *grad) {
    const int r = blockIdx.x, p = place[r];
    for (int h = threadIdx.x * 4; h < H; h += 1024) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        if (p >= 0)
            for (int s = 0; s < splits; ++s)
                x += *reinterpret_cast<const f32x4 *>(sums + ((int64_t)s * R + p) * H + h);
        const auto y = packed4<T>(x);
        *reinterpret_cast<decltype(packed4<T>(x)) *>(grad + (int64_t)r * H + h) = y;
    }
}

struct WeightJob {
    const char *rows;    // [count, H]
    const char *G;       // [count][ldg]
    const int32_t *count;
    int H, v0, v1;
    int64_t ldg;
    int nh, nv;
    void *grad;          // [V, H]
};

template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_rows(const WeightJob &job, int v0) {
    const int ld = job.H * (int)sizeof(T);
    return out_rows(static_cast<char *>(job.grad) + (int64_t)(job.v0 + v0) * ld, ld,
                    min(job.v1 - job.v0 - v0, kTile), ld);
}

// Tiles of 256 columns of H x 256 vocabulary rows, over the kept rows; one a workgroup.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void lmloss_weight_kernel(WeightJob job) {
    typedef GemmTile<T, kTile, kTile, true, true, 2> Tile;
    __shared__ __align__(1024) char lds[Tile::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int R = *job.count;
    int tm, tn;
    gemm_place(blockIdx.x, job.nh, job.nv, kPlaceGroup, tm, tn);
    const int h0 = tm * kTile, v0 = tn * kTile;
    Tile tile;
    tile.run(operand_ks<T>(job.rows, (int64_t)job.H * sizeof(T), h0, 0),
             operand_ks<T>(job.G, job.ldg * (int64_t)sizeof(T), v0, 0), R, lds, wave, lane);
    const int g = lane >> 4, j = lane & 15;
    const __amdgpu_buffer_rsrc_t out = weight_rows<T>(job, v0);
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

// The same as a stream.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void lmloss_weight_stream_kernel(WeightJob job) {
    typedef GemmStream<T, true, true, 16> Stream;
    static_assert(Stream::kRowStores == 16, "the stores a tile's end makes");
    __shared__ __align__(1024) char lds[Stream::kLdsBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    // (without a kept row the products are over a row of zeros)
    const int R = *job.count, K = max(R, 1), tiles = job.nh * job.nv;
    const int64_t ldh = (int64_t)job.H * sizeof(T), ldg = job.ldg * (int64_t)sizeof(T);
    auto place = [&](int i, int &h0, int &v0) {
        const int id = blockIdx.x + i * gridDim.x;
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
            GemmWork w = {operand_ks<T>(job.rows, ldh, h0, 0), operand_ks<T>(job.G, ldg, v0, 0), K};
            if (R == 0) w.a.valid = w.b.valid = 1 << 30;  // (past every row: nothing is read)
            return w;
        },
        [&](int i) {
            int h0 = 0, v0 = 0;
            place(i, h0, v0);
            stream.store_rows(weight_rows<T>(job, v0), (int)ldh, h0 * 2, (int)ldh, lds, wave, lane,
                              [&](int mi, int ni) { return stream.acc[mi][ni]; });
        },
        lds, wave, lane);
}

// ---- plans and launches ------------------------------------------------------------------------

size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
    int elem;
    int bn;                  // row_tile
    int nr;                  // tiles of rows
    int wm;                  // waves along the vocabulary in a logits tile
    // forward
    int nv;
    // backward
    int piece, pieces;       // columns (a multiple of 256), number
    int splits;              // of a piece, for grad_hidden: at most, all of them in the first one
    size_t rows, place, count, flags, parts, scale, G, sums, forward, backward;

    // columns of a split in a piece of `width`
    int per(int width) const { return ceil_div(ceil_div(width, splits), 64) * 64; }
};

int waves_m(int bn) { return bn == 256 ? 2 : bn == 128 ? 4 : 8; }

Plan plan(int R, int H, int V, int elem) {
    Plan p;
    p.elem = elem;
    p.bn = row_tile(R);
    p.nr = ceil_div(R, p.bn);
    p.wm = waves_m(p.bn);
    p.nv = ceil_div(V, kTile);
    // a piece: whole rounds of tiles over the CUs, if as many fit
    int64_t most = kPieceBytes / ((int64_t)R * elem) / kTile;
    most = most < 1 ? 1 : most > kPieceMost / kTile ? kPieceMost / kTile : most;
    int round = kCus;
    for (int n = p.nr; n % 2 == 0 && round > 1; n /= 2) round /= 2;
    if (most > round) most = most / round * round;
    p.piece = (int)(most < p.nv ? most : p.nv) * kTile;
    p.pieces = ceil_div(V, p.piece);
    // grad_hidden: a workgroup for every CU, splits of 1024 columns at least
    const int tiles = ceil_div(H, kTile) * p.nr, width = p.piece < V ? p.piece : V;
    const int longest = width / 1024;
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
    const size_t common = at;
    p.flags = take((size_t)R * 4);
    p.parts = take((size_t)ceil_div(R, 16) * 16 * p.nv * p.wm * sizeof(float2));
    p.forward = at;
    at = common;
    p.scale = take((size_t)R * sizeof(float2));
    p.G = take((size_t)R * p.piece * elem);
    p.sums = take((size_t)p.splits * R * H * 4);
    p.backward = at;
    return p;
}

// (bf16 tiles of 256 rows go through a stream, one workgroup per CU.)
template <typename T, bool GRAD>
void launch_logits(int bn, const LogitsJob &job, hipStream_t s) {
    const int tiles = job.nv * job.nr;
    const dim3 grid(tiles), block(kGemmThreads);
    if constexpr (sizeof(T) == 2) {
        if (bn == kTile) {
            lmloss_logits_stream_kernel<T, GRAD><<<tiles < kCus ? tiles : kCus, block, 0, s>>>(job);
            return;
        }
    } else if (bn == kTile) {
        lmloss_logits_kernel<T, 256, 2, GRAD><<<grid, block, 0, s>>>(job);
        return;
    }
    switch (bn) {
    case 128: lmloss_logits_kernel<T, 128, 4, GRAD><<<grid, block, 0, s>>>(job); break;
    case 64: lmloss_logits_kernel<T, 64, 8, GRAD><<<grid, block, 0, s>>>(job); break;
    default: lmloss_logits_kernel<T, 32, 8, GRAD><<<grid, block, 0, s>>>(job); break;
    }
}

template <typename T>
void launch_hidden(int bn, const HiddenJob &job, hipStream_t s) {
    const int tiles = job.nh * job.nr * job.splits;
    const dim3 grid(tiles), block(kGemmThreads);
    if constexpr (sizeof(T) == 2) {
        if (bn == kTile) {
            lmloss_hidden_stream_kernel<T><<<tiles < kCus ? tiles : kCus, block, 0, s>>>(job);
            return;
        }
    } else if (bn == kTile) {
        lmloss_hidden_kernel<T, 256, 2><<<grid, block, 0, s>>>(job);
        return;
    }
    switch (bn) {
    case 128: lmloss_hidden_kernel<T, 128, 4><<<grid, block, 0, s>>>(job); break;
    case 64: lmloss_hidden_kernel<T, 64, 8><<<grid, block, 0, s>>>(job); break;
    default: lmloss_hidden_kernel<T, 32, 8><<<grid, block, 0, s>>>(job); break;
    }
}

template <typename T>
void launch_weight(const WeightJob &job, hipStream_t s) {
    const int tiles = job.nh * job.nv;
    if constexpr (sizeof(T) == 2)
        lmloss_weight_stream_kernel<T>
            <<<tiles < kCus ? tiles : kCus, kGemmThreads, 0, s>>>(job);
    else
        lmloss_weight_kernel<T><<<tiles, kGemmThreads, 0, s>>>(job);
}

template <typename T>
hipError_t forward(const Plan &p, const void *hidden, const void *W, Entries e, int R, int H, int V,
                   float *loss, float *stats, char *ws, hipStream_t s) {
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
    gj.place = reinterpret_cast<int32_t *>(ws + p.place);
    gj.count = reinterpret_cast<int32_t *>(ws + p.count);
    const dim3 grid(ceil_div(R, kGatherRows), ceil_div(e.K, kGatherEntries));
    if (e.teacher) {
        lmloss_flags_kernel<<<ceil_div(R, 4), 256, 0, s>>>(e, R, V, const_cast<int32_t *>(gj.flags));
        lmloss_gather_kernel<T, Rows::kFlags><<<grid, 256, 0, s>>>(gj);
    } else {
        lmloss_gather_kernel<T, Rows::kTargets><<<grid, 256, 0, s>>>(gj);
    }
    const float c = kLog2e / e.tau;
    LogitsJob lj = {};
    lj.rows = gj.rows;
    lj.W = gj.W;
    lj.count = gj.count;
    lj.H = H;
    lj.V = V;
    lj.v0 = 0;
    lj.v1 = V;
    lj.nv = p.nv;
    lj.nr = p.nr;
    lj.c = c;
    lj.parts = reinterpret_cast<float2 *>(ws + p.parts);
    lj.nparts = (int64_t)p.nv * p.wm;
    launch_logits<T, false>(p.bn, lj, s);
    FinishJob fj = {lj.parts, lj.nparts, gj.place, e, R, V, c, loss, stats};
    lmloss_finish_kernel<<<ceil_div(R, kFinishRows), kFinishThreads, 0, s>>>(fj);
    return hipGetLastError();
}

template <typename T>
hipError_t backward(const Plan &p, const void *hidden, const void *W, Entries e,
                    const float *stats, const float *grad_loss, int R, int H, int V,
                    void *grad_hidden, void *grad_W, char *ws, hipStream_t s) {
    GatherJob gj = {};
    gj.hidden = static_cast<const char *>(hidden);
    gj.stats = const_cast<float *>(stats);
    gj.grad_loss = grad_loss;
    gj.e = e;
    gj.R = R;
    gj.H = H;
    gj.V = V;
    gj.rows = ws + p.rows;
    gj.place = reinterpret_cast<int32_t *>(ws + p.place);
    gj.count = reinterpret_cast<int32_t *>(ws + p.count);
    gj.scale = reinterpret_cast<float2 *>(ws + p.scale);
    lmloss_gather_kernel<T, Rows::kStats><<<ceil_div(R, kGatherRows), 256, 0, s>>>(gj);
    const float c = kLog2e / e.tau;
    const int nh = ceil_div(H, kTile);
    for (int i = 0; i < p.pieces; ++i) {
        const int v0 = i * p.piece, v1 = v0 + p.piece < V ? v0 + p.piece : V;
        LogitsJob lj = {};
        lj.rows = gj.rows;
        lj.W = static_cast<const char *>(W);
        lj.count = gj.count;
        lj.H = H;
        lj.V = V;
        lj.v0 = v0;
        lj.v1 = v1;
        lj.nv = ceil_div(v1 - v0, kTile);
        lj.nr = p.nr;
        lj.c = c;
        lj.G = ws + p.G;
        lj.ldg = p.piece;
        lj.scale = gj.scale;
        launch_logits<T, true>(p.bn, lj, s);
        EntriesJob ej = {e, stats, grad_loss, gj.place, R, V, v0, v1, c, lj.G, p.piece};
        lmloss_entries_kernel<T><<<ceil_div(R, 4), 256, 0, s>>>(ej);
        if (grad_hidden) {
            const int per = p.per(v1 - v0);
            HiddenJob hj = {lj.W, ws + p.G, gj.count, R, H, v0, v1, p.piece, nh, p.nr,
                            ceil_div(v1 - v0, per), per, i == 0,
                            reinterpret_cast<float *>(ws + p.sums)};
            launch_hidden<T>(p.bn, hj, s);
        }
        if (grad_W) {
            WeightJob wj = {gj.rows, ws + p.G, gj.count, H, v0, v1, p.piece, nh, lj.nv, grad_W};
            launch_weight<T>(wj, s);
        }
    }
    if (grad_hidden)
        lmloss_hidden_out_kernel<T><<<R, 256, 0, s>>>(reinterpret_cast<float *>(ws + p.sums),
                                                      p.splits, gj.place, R, H,
                                                      static_cast<T *>(grad_hidden));
    return hipGetLastError();
}

}  // namespace

size_t lmloss_workspace_bytes(int R, int H, int V, int elem_bytes) {
    const Plan p = plan(R, H, V, elem_bytes);
    return p.forward;
}

size_t lmloss_backward_workspace_bytes(int R, int H, int V, int elem_bytes) {
    const Plan p = plan(R, H, V, elem_bytes);
    return p.backward;
}

hipError_t launch_lmloss(const void *hidden, const void *W, int elem_bytes, const int32_t *ids,
                         const float *teacher, int R, int H, int V, int K, float tau, float *loss,
                         float *row_stats, void *ws, hipStream_t stream) {
    const Plan p = plan(R, H, V, elem_bytes);
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
    const Plan p = plan(R, H, V, elem_bytes);
    const Entries e = {ids, teacher, K, tau};
    char *w = static_cast<char *>(ws);
    return elem_bytes == 2 ? backward<uint16_t>(p, hidden, W, e, row_stats, grad_loss, R, H, V,
                                                grad_hidden, grad_W, w, stream)
                           : backward<float>(p, hidden, W, e, row_stats, grad_loss, R, H, V,
                                             grad_hidden, grad_W, w, stream);
}

}  // namespace dflash2
