// The LM head's losses for at most 32 rows (bf16, kRowsFrom < H <= 4096): one read of W a pass, at the
// rate of its stream. 16 rows x 4096 x 151936: loss 203 us in the kernel (6.1 TB/s), logits again and
// grad_hidden 270 us (W, and 67 MB of sums). Included by lmhead_loss.hip.
//
// Design:
//   * A wave owns KC columns of H (an eighth, rounded up to 256 or 512) for the whole pass: the kept
//     rows' values there are matrix fragments in its registers. A workgroup takes a contiguous range of the
//     vocabulary, 8 rows of W a tile: the waves together read whole rows (8 KB at H = 4096). Tiles of 256
//     rows x 256 bytes, which the ring of stages reads, touch every row of the range over and over and
//     ran at 5.0 - 5.4 TB/s; rows read whole, at 6.0.
//   * A wave's part of a tile goes straight from memory into LDS that only it reads, two tiles deep, so
//     the stream needs no barrier: it waits for its own loads.
//   * The waves' partial logits (8 x 16 or 8 x 32) are added through LDS in a fixed order, one barrier a
//     tile, by groups of threads that own an element (row, v) each and keep its running maximum and sum,
//     or form G there.
//   * The workgroups find the kept rows and their entries (FewRows) while their first tiles are on their
//     way.
//   * With at most 16 rows the backward pass multiplies G, in two bf16 parts, with the tile of W while it
//     is still in LDS (v_mfma_f32_16x16x16_bf16: 8 rows, two parts): 16 x KC sums a wave in registers.
//     W is read once for the logits and grad_hidden (G and its product in passes of their own: 450 us for
//     16 x 4096 x 151936).
#pragma once

#include "dflash2.h"

namespace dflash2 {
namespace {

constexpr int kRowsTile = 8;

enum class RowsDo { kStats, kGrad, kHidden };

struct RowsJob {
    const uint16_t *hidden;  // [R, H]
    const uint16_t *W;       // [V, H]
    int R, H, V, v0, v1;     // the piece
    Coef c;                  // log2(e) / tau
    Entries e;
    float *stats;            // [R, K + 2]: kStats: the entries' logits out; else in
    const float *grad_loss;  // kGrad, kHidden
    int32_t *place;          // out: [R] a row's place among the kept ones, -1: left out
    int32_t *from, *count;   // out: [kept rows] the row, their number
    float2 *parts;           // kStats: per 16 rows, [workgroups][16] (max, sum)
    uint16_t *G;             // [2 low][ldg], null: not kept
    int64_t ldg;
    int low;
    float *sums;             // kHidden: [workgroups][16][H]
    bool first;
};

template <int KC, int BN, RowsDo DO>
__global__ __launch_bounds__(kGemmThreads) void lmloss_rows_kernel(RowsJob job) {
    static_assert(DO != RowsDo::kHidden || BN == 16, "the sums are a wave's registers");
    constexpr int NI = BN / 16, kSlices = KC / 32, kRowBytes = KC * 2;
    constexpr int kLoads = kRowsTile * kRowBytes / 1024;     // a wave's, per tile
    constexpr int kPartRow = BN * kRowsTile + 8;             // floats of a wave's partial tile
    constexpr int kOwners = kGemmThreads / (BN * kRowsTile); // threads per element
    // per tile, younger than what it waits for (at least): its stores, two loads that run further ahead
    constexpr bool kAhead = DO != RowsDo::kHidden;
    constexpr int kYounger = (DO == RowsDo::kStats ? 0 : 2) + (kAhead ? 2 : 0);
    constexpr int kList = DFLASH2_MAX_K;
    typedef FewRows<BN, kList, DO == RowsDo::kStats> Few;
    __shared__ __align__(1024) char stage[kGemmWaves][2][kRowsTile * kRowBytes];
    __shared__ __align__(16) uint32_t dump[kAhead ? kGemmWaves : 1][kWave];
    __shared__ __align__(16) float part[2][kGemmWaves][kPartRow];
    __shared__ __align__(16) uint16_t gt[DO == RowsDo::kHidden ? 16 * 16 : 8];  // [row][8 hi, 8 lo]
    __shared__ typename Few::Lds few_lds;

    const int lane = threadIdx.x % kWave, g = lane >> 4, j = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int H = job.H, h0 = wave * KC, K = job.e.K;
    const int units = (job.v1 - job.v0 + kRowsTile - 1) / kRowsTile;
    const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x);
    const int u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
    const int64_t ld = (int64_t)H * 2;

    // Loads: lane `at` of a tile's KC / 8 chunks a row takes chunk p ^ (row & 7) for place p.
    int voff[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = i * kWave + lane, row = at / (KC / 8), c = (at % (KC / 8)) ^ (row & 7);
        voff[i] = h0 + 8 * c < H ? row * (int)ld + 16 * c : kGemmOutside;
    }
    // this wave's columns of tile u (of nothing behind the last)
    auto buffer = [&](int u) {
        const int v = job.v0 + u * kRowsTile, n = u < u1 ? min(kRowsTile, job.v1 - v) : 0;
        return scalar_buffer(job.W + (int64_t)v * H + h0,
                             n > 0 && h0 < H ? (n - 1) * (int)ld + (H - h0) * 2 : 0);
    };
    auto issue = [&](int u) {
        const u32x4 rs = buffer(u);
        const uint32_t to = lds_address(stage[wave][(u - u0) & 1]);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load_lds16(to + i * 1024, voff[i], rs);
    };
    // One load that touches every 128-byte line of this wave's part of a tile: the tile comes to the L2
    // while the two in LDS are still in use (16 x 4096 x 151936: 209 us without, 202 with). What it
    // brings lands in `dump`. Not for kHidden (276 us without, 298 with).
    constexpr int kLines = kRowBytes / 128;  // per row
    const int touch = lane < kRowsTile * kLines && h0 + (lane % kLines) * 64 < H
                          ? (lane / kLines) * (int)ld + (lane % kLines) * 128 : kGemmOutside;
    auto ahead = [&](int u) { load_lds4(lds_address(dump[wave]), touch, buffer(u)); };
    issue(u0);
    issue(u0 + 1);
    if constexpr (kAhead) ahead(u0 + 2);

    Few few;
    few.find(job.e, job.R, job.V, job.stats, job.grad_loss, few_lds, job.place, job.from, job.count, wave,
             lane);
    const int R = few.R;
    const int *from = few_lds.from;
    if (R == 0) {  // (the loads in flight end before the workgroup does)
        wait_for<0, 0>();
        return;
    }

    // The kept rows as fragments: lane (j, g) of slice s holds row 16 ni + j at h0 + 32 s + 8 g .. + 7.
    bf16x8 hid[NI][kSlices];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
        const int p = 16 * ni + j;
        const uint16_t *row = job.hidden + (int64_t)from[min(p, R - 1)] * H;
#pragma unroll
        for (int s = 0; s < kSlices; ++s) {
            const int h = h0 + 32 * s + 8 * g;
            u32x4 x = {0u, 0u, 0u, 0u};
            if (p < R && h < H) x = *reinterpret_cast<const u32x4 *>(row + h);
            hid[ni][s] = __builtin_bit_cast(bf16x8, x);
        }
    }
    // This thread's element of a tile: kept row er, vocabulary row ev; `owner` of kOwners threads.
    constexpr int kMine = kWave / kOwners;  // elements of a wave
    const int el = wave * kMine + lane % kMine, owner = lane / kMine, er = el / kRowsTile;
    const int ev = el % kRowsTile, r_mine = from[min(er, R - 1)];
    float top = -INFINITY, sum = 0.f;
    float2 sc = {0.f, 0.f};
    float *stats = job.stats + (int64_t)r_mine * (K + 2);
    if constexpr (DO != RowsDo::kStats)
        sc = float2{stats[0], grad_scale(job.grad_loss[r_mine], job.e.tau, stats[1])};
    few.list(job.e, job.V, job.c, job.v0 + u0 * kRowsTile, job.v0 + u1 * kRowsTile, few_lds, wave, lane);
    const int nlist = er < R ? few_lds.listed[er] : 0;

    // Fragment addresses within a tile. Logits: row j & 7 (rows 8 .. 15 of the instruction repeat them),
    // chunk 4 s + g. grad_hidden: the 4 rows 4 (g & 1) .. of 16 columns, transposed.
    int xa[2], ta[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) xa[i] = (j & 7) * kRowBytes + (((4 * i + g) ^ (j & 7)) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * (g & 1) + (j >> 2), c = 2 * i + ((j & 3) >> 1);
        ta[i] = row * kRowBytes + ((c ^ row) << 4) + 8 * (j & 1);
    }
    constexpr int kSums = DO == RowsDo::kHidden ? KC / 16 : 1;
    f32x4 acc[kSums];
#pragma unroll
    for (int t = 0; t < kSums; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
        job.G, (short)0, job.G ? (int)(2 * job.low * job.ldg) * 2 : 0, kGemmWord3);

    wait_for<0, 15>();  // the first two tiles, and what was read above
    for (int u = u0; u < u1; ++u) {
        const int buf = (u - u0) & 1;
        const char *tile = stage[wave][buf];
        // this tile's loads: all but the next one's, and the stores behind those
        wait_for<kLoads + kYounger, 15>();
        // (two chains of sums; reads in batches, which the compiler would make and wait for one by one)
        constexpr int kBatch = DO == RowsDo::kHidden ? 4 : 8;
        static_assert(kSlices % kBatch == 0, "whole batches");
        f32x4 x[NI][2];
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) x[ni][0] = x[ni][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < kSlices; b += kBatch) {
            bf16x8 w[kBatch];
#pragma unroll
            for (int s = 0; s < kBatch; ++s)
                w[s] = *reinterpret_cast<const bf16x8 *>(tile + xa[s & 1] + ((b + s) >> 1) * 128);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < kBatch; ++s)
#pragma unroll
                for (int ni = 0; ni < NI; ++ni)
                    x[ni][s & 1] = gemm_mfma(w[s], hid[ni][b + s], x[ni][s & 1]);
        }
        // lane (j, g < 2) holds v = 4 g .. 4 g + 3 of row 16 ni + j
        if (g < 2) {
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
                *reinterpret_cast<f32x4 *>(&part[buf][wave][(16 * ni + j) * kRowsTile + 4 * g]) =
                    x[ni][0] + x[ni][1];
        }
        if constexpr (DO != RowsDo::kHidden) {
            wait_for<63, 0>();  // the tile is read
            issue(u + 2);
            ahead(u + 3);
        }
        wait_for<63, 0>();
        bare_barrier();
        // (the other buffer's partial tiles are written before the next barrier, this one's after it)
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kGemmWaves / kOwners; ++w)
            y += part[buf][owner * (kGemmWaves / kOwners) + w][el];
        if constexpr (kOwners >= 4) y += __uint_as_float(xor_lane<16>(__float_as_uint(y), lane));
        if constexpr (kOwners >= 2) y += __uint_as_float(xor_lane<32>(__float_as_uint(y), lane));
        const int v = job.v0 + u * kRowsTile + ev, in_range = (u - u0) * kRowsTile + ev;
        if constexpr (DO == RowsDo::kStats) {
            for (int i = 0; i < nlist; ++i)
                if (few_lds.column(er * kList + i, true) == in_range && owner == 0)
                    stats[2 + few_lds.entry(er * kList + i)] = y;
            if (v < job.v1) {
                const float high = fmaxf(top, y), ref = high == -INFINITY ? 0.f : high;
                sum = sum * scaled_exp<false>(top - ref, job.c) + scaled_exp<false>(y - ref, job.c);
                top = high;
            }
        } else {
            float z = sc.y * scaled_exp<false>(y - sc.x, job.c);
            for (int i = 0; i < nlist; ++i)
                if (few_lds.v[er * kList + i] == in_range) z -= few_lds.x[er * kList + i];
            if (er >= R || v >= job.v1) z = 0.f;
            const __bf16 hi = (__bf16)z, lo = (__bf16)(z - (float)hi);
            const uint16_t hb = __builtin_bit_cast(uint16_t, hi), lb = __builtin_bit_cast(uint16_t, lo);
            // (every wave makes both, whatever they write: the waits count them)
            const int off = owner == 0 ? (int)(er * job.ldg + u * kRowsTile + ev) * 2 : kGemmOutside;
            __builtin_amdgcn_raw_buffer_store_b16(hb, out, off, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b16(
                lb, out, owner == 0 ? off + (int)(job.low * job.ldg) * 2 : off, 0, 0);
            if constexpr (DO == RowsDo::kHidden) {
                if (owner == 0) {
                    gt[er * 16 + ev] = hb;
                    gt[er * 16 + 8 + ev] = lb;
                }
                wait_for<63, 0>();
                bare_barrier();
                // lane (j, g): row j, k = 4 g ..: hi of v 0 .. 7, then lo
                const s16x4 ga = *reinterpret_cast<const s16x4 *>(&gt[j * 16 + 4 * g]);
                constexpr int kGroup = 4;
                s16x4 w[2][kGroup];
                auto read = [&](int t0, s16x4(&f)[kGroup]) {
#pragma unroll
                    for (int t = t0; t < t0 + kGroup; ++t)
                        f[t - t0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (lds_s16x4 *)(tile + ta[t & 3] + (t >> 2) * 128));
                    __builtin_amdgcn_sched_barrier(0);
                };
                read(0, w[0]);
#pragma unroll
                for (int t0 = 0; t0 < kSums; t0 += kGroup) {
                    const int b = t0 / kGroup & 1;
                    if (t0 + kGroup < kSums) read(t0 + kGroup, w[b ^ 1]);
#pragma unroll
                    for (int t = t0; t < t0 + kGroup; ++t)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(ga, w[b][t - t0], acc[t], 0,
                                                                          0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                // the tile is read; (gt is written again behind the next tile's first barrier)
                wait_for<63, 0>();
                issue(u + 2);
            }
        }
    }
    wait_for<0, 0>();  // no load is in flight when the workgroup ends

    if constexpr (DO == RowsDo::kStats) {
        join_lane<false, 1>(top, sum, lane, job.c);
        join_lane<false, 2>(top, sum, lane, job.c);
        join_lane<false, 4>(top, sum, lane, job.c);
        if (ev == 0 && owner == 0 && er < R)
            job.parts[((int64_t)(er >> 4) * gridDim.x + blockIdx.x) * 16 + (er & 15)] = float2{top, sum};
    }
    if constexpr (DO == RowsDo::kHidden) {
#pragma unroll
        for (int t = 0; t < kSums; ++t) {
            const int h = h0 + 16 * t + j;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * g + i;
                if (r < R && h < H) {
                    float *at = job.sums + ((int64_t)blockIdx.x * 16 + r) * H + h;
                    *at = job.first ? acc[t][i] : *at + acc[t][i];
                }
            }
        }
    }
}

}  // namespace
}  // namespace dflash2
