// One workgroup's tile of a matrix product on the matrix cores: C[m][n] = sum_k A(m, k) B(n, k).
//
// An operand lies in memory in one of two ways: its rows hold k (KC: element (m, k) at
// base + m ld + k), or its rows hold m (KS: element (m, k) at base + k ld + m). The LM head's
// logits take two KC operands, the hidden states' gradient KS x KC, the weight's KS x KS; no
// operand is transposed in memory first.
//
// Design (gfx950, eight waves):
//   * A K step is 128 bytes of k per row (64 bf16, 32 f32), so a stage holds 128 B bytes of an
//     operand of B rows in either layout. Two stages per operand: the loads of step t + 1 go from
//     memory straight into LDS (16 bytes a lane) while step t is multiplied.
//   * The loads write LDS linearly, so the swizzle that keeps the fragment reads free of bank
//     conflicts is in the addresses they read: KC stages keep chunk c (16 bytes) of row m at slot
//     c ^ (m & 7); KS stages of bf16 keep the 32-byte piece s of row k at s ^ f(k), where f takes
//     16 values over the 16 rows that one transposing read touches; KS stages of f32 keep the
//     64-byte piece s at s ^ ((k >> 2) & 3).
//   * bf16: v_mfma_f32_16x16x32_bf16. Lane (g = lane / 16, j = lane % 16) takes row j and
//     k = 8 g .. 8 g + 7: one 16-byte LDS read from a KC stage, two transposing 8-byte reads
//     (rows k = 8 g .. + 3 and + 4 .. + 7) from a KS stage. f32: v_mfma_f32_16x16x4_f32, a lane's
//     16 bytes (k = 4 g .. 4 g + 3) feeding four of them; both operands agree on which k an
//     instruction multiplies. Sums are fp32 and their order depends on k alone, not on the tile.
//   * Out of range: a descriptor ends at the operand's last valid byte, so rows past the end read
//     zeros; a KC operand whose k ends inside a step masks the chunks behind it. What lies behind
//     the last column m of a KS row only reaches outputs that no caller stores.
#pragma once

#include "device_common.h"

namespace dflash2 {

constexpr int kGemmWaves = 8;
constexpr int kGemmThreads = kGemmWaves * kWave;
constexpr int kStepBytes = 128;
constexpr int kGemmOutside = 0x7FFFFFF0;  // an offset that no descriptor covers
constexpr int kGemmWord3 = 0x00020000;    // gfx9-family buffer descriptor word 3 (raw data)

constexpr int kWaitAll = 0x0070;          // s_waitcnt vmcnt(0) lgkmcnt(0)

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// An operand from the tile's first row (KC) or column (KS) and first k on.
struct GemmOperand {
    const char *base;
    int64_t ld;     // bytes from one row to the next
    int64_t bytes;  // valid bytes from base on
};

// The operand of rows [row0, rows) of a KC matrix, k in [k0, k1). (A row is a whole number of
// 16-byte chunks in memory; what k1 leaves of the last one holds zeros.)
template <typename T>
__device__ __forceinline__ GemmOperand operand_kc(const void *p, int64_t ld, int row0, int rows,
                                                  int most, int k0, int k1) {
    const int n = min(rows - row0, most);
    return {static_cast<const char *>(p) + row0 * ld + (int64_t)k0 * sizeof(T), ld,
            n > 0 ? (int64_t)(n - 1) * ld + ((int64_t)(k1 - k0) * (int)sizeof(T) + 15) / 16 * 16 : 0};
}

// The operand of columns from col0 on of a KS matrix, k in [k0, k1).
template <typename T>
__device__ __forceinline__ GemmOperand operand_ks(const void *p, int64_t ld, int col0, int k0,
                                                  int k1) {
    return {static_cast<const char *>(p) + (int64_t)k0 * ld + (int64_t)col0 * sizeof(T), ld,
            (int64_t)(k1 - k0) * ld - (int64_t)col0 * (int)sizeof(T)};
}

// One operand's stages: B rows (m) of a K step.
template <typename T, int B, bool KS> struct GemmSide {
    static constexpr int kBytes = B * kStepBytes;
    static constexpr int kStepK = kStepBytes / (int)sizeof(T);
    static constexpr int kLoads = kBytes / 1024;  // of 1 KB, one wave's
    static constexpr int kPerWave = (kLoads + kGemmWaves - 1) / kGemmWaves;
    static constexpr int kRowChunks = B * (int)sizeof(T) / 16;  // KS: 16-byte chunks per stage row

    int voff[kPerWave];  // the lane's bytes within the operand's step
    int kbyte;           // KC: the first byte of k that the lane reads

    __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
        kbyte = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
        for (int q = 0; q < kPerWave; ++q) {
            const int load = wave + kGemmWaves * q;
            if constexpr (!KS) {
                voff[q] = (8 * load + (lane >> 3)) * (int)ld + kbyte;
            } else {
                const int at = load * kWave + lane, k = at / kRowChunks, p = at % kRowChunks;
                int c;
                if constexpr (sizeof(T) == 2)
                    c = (((p >> 1) ^ swizzle(k)) << 1) | (p & 1);
                else
                    c = (((p >> 2) ^ ((k >> 2) & 3)) << 2) | (p & 3);
                voff[q] = k * (int)ld + c * 16;
            }
        }
    }

    // KS, bf16: f(k) for the 32-byte pieces of row k
    static __device__ __forceinline__ int swizzle(int k) {
        return ((((k >> 3) & 3) << 2) | (k & 3)) & (kRowChunks / 2 - 1);
    }

    // Bytes from one step to the next.
    static __device__ __forceinline__ int64_t stride(int64_t ld) {
        return KS ? ld * kStepK : (int64_t)kStepBytes;
    }

    // Starts the loads of a step whose first element is at `p`, with `bytes` valid bytes from there
    // and (KC) `kleft` bytes of k left.
    __device__ __forceinline__ void issue(char *stage, const char *p, int64_t bytes, int kleft,
                                          int wave) const {
        const int n = (int)(bytes < 0 ? 0 : bytes > kGemmOutside ? kGemmOutside : bytes);
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), (short)0, n, kGemmWord3);
#pragma unroll
        for (int q = 0; q < kPerWave; ++q) {
            const int load = wave + kGemmWaves * q;
            if (kLoads % kGemmWaves != 0 && load >= kLoads) break;
            int off = voff[q];
            if constexpr (!KS) off = kbyte < kleft ? off : kGemmOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(stage + load * 1024), 16, off,
                                                     0, 0, 0);
        }
    }

    typedef typename std::conditional<sizeof(T) == 2, bf16x8, f32x4>::type Frag;

    // Lane addresses (bytes within a stage) of the fragments of rows m0 + 16 i + j, i < N.
    template <int N> struct Reader {
        int at[KS ? N : 2];
        __device__ __forceinline__ void init(int m0, int lane) {
            const int g = lane >> 4, j = lane & 15;
            if constexpr (!KS) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    at[h] = (m0 + j) * kStepBytes + (((4 * h + g) ^ (j & 7)) << 4);
            } else if constexpr (sizeof(T) == 2) {
                const int k = 8 * g + (j >> 2);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    at[i] = k * (B * 2) + (((m0 / 16 + i) ^ swizzle(k)) << 5) + 8 * (j & 3);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    at[i] = 4 * g * (B * 4) + (((m0 / 16 + i) ^ g) << 6) + 4 * j;
            }
        }
        // half h of the step: bf16 k = 32 h .. 32 h + 31, f32 k = 16 h .. 16 h + 15
        __device__ __forceinline__ Frag read(const char *stage, int i, int h) const {
            if constexpr (!KS) {
                return *reinterpret_cast<const Frag *>(stage + at[h] + i * 16 * kStepBytes);
            } else if constexpr (sizeof(T) == 2) {
                const char *p = stage + at[i] + 32 * h * (B * 2);
                struct { s16x4 lo, hi; } v;
                v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
                v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * (B * 2)));
                return __builtin_bit_cast(Frag, v);
            } else {
                const char *p = stage + at[i] + 16 * h * (B * 4);
                Frag v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float *>(p + e * (B * 4));
                return v;
            }
        }
    };
};

__device__ __forceinline__ f32x4 gemm_mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 gemm_mfma(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// A tile of BM x BN over WM x (8 / WM) waves. Wave (wm, wn) holds rows m = wm BM / WM + 16 mi +
// 4 g + i and columns n = wn BN / WN + 16 ni + j in acc[mi][ni][i].
template <typename T, int BM, int BN, bool AS, bool BS, int WM> struct GemmTile {
    static constexpr int WN = kGemmWaves / WM;
    static constexpr int MI = BM / (16 * WM), NI = BN / (16 * WN);
    static_assert(MI * 16 * WM == BM && NI * 16 * WN == BN, "whole fragments");
    typedef GemmSide<T, BM, AS> SideA;
    typedef GemmSide<T, BN, BS> SideB;
    static constexpr int kStepK = SideA::kStepK;

    f32x4 acc[MI][NI];

    static __device__ __forceinline__ int wave_m(int wave) { return (wave / WN) * (BM / WM); }
    static __device__ __forceinline__ int wave_n(int wave) { return (wave % WN) * (BN / WN); }

    // The product over K values of k. a0/a1, b0/b1: the stages, objects of their own in LDS.
    __device__ __forceinline__ void run(const GemmOperand &A, const GemmOperand &B, int K, char *a0,
                                        char *a1, char *b0, char *b1, int wave, int lane) {
        SideA sa;
        SideB sb;
        sa.init(A.ld, wave, lane);
        sb.init(B.ld, wave, lane);
        typename SideA::template Reader<MI> ra;
        typename SideB::template Reader<NI> rb;
        ra.init(wave_m(wave), lane);
        rb.init(wave_n(wave), lane);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};

        const int steps = (K + kStepK - 1) / kStepK;
        const char *pa = A.base, *pb = B.base;
        int64_t na = A.bytes, nb = B.bytes;
        int kleft = K * (int)sizeof(T);
        auto issue = [&](char *sta, char *stb) {
            sa.issue(sta, pa, na, kleft, wave);
            sb.issue(stb, pb, nb, kleft, wave);
            const int64_t da = SideA::stride(A.ld), db = SideB::stride(B.ld);
            pa += da;
            na -= da;
            pb += db;
            nb -= db;
            kleft -= kStepBytes;
            __builtin_amdgcn_sched_barrier(0);  // (the compiler would start them after the products)
        };
        auto compute = [&](const char *sta, const char *stb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                typename SideA::Frag fa[MI];
                typename SideB::Frag fb[NI];
#pragma unroll
                for (int ni = 0; ni < NI; ++ni) fb[ni] = rb.read(stb, ni, h);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) fa[mi] = ra.read(sta, mi, h);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                    for (int ni = 0; ni < NI; ++ni)
                        acc[mi][ni] = gemm_mfma(fa[mi], fb[ni], acc[mi][ni]);
            }
        };
        // The barrier at a step's start: this wave's loads have landed (vmcnt), so after it all
        // waves' have, and every wave has read the other stage, which the next loads overwrite.
        auto ready = [&]() {
            __builtin_amdgcn_s_waitcnt(kWaitAll);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        };
        // (Loads past the last step read nothing and write zeros: the loop stays free of branches.)
        issue(a0, b0);
        for (int t = 0; t + 1 < steps; t += 2) {
            ready();
            issue(a1, b1);
            compute(a0, b0);
            ready();
            issue(a0, b0);
            compute(a1, b1);
        }
        ready();
        if (steps & 1) compute(a0, b0);
    }
};

// The tile of workgroup `id` of nm x nn tiles. Consecutive workgroups run on different XCDs, each
// with an L2 of its own: XCD x takes a contiguous eighth of the tiles, in groups of `group` rows
// of tiles, rows first, so that what it works on at a time shares operands.
__device__ __forceinline__ void gemm_place(int id, int nm, int nn, int group, int &tm, int &tn) {
    constexpr int kXcds = 8;
    const int total = nm * nn, x = id % kXcds, q = total / kXcds, r = total % kXcds;
    const int at = x * q + min(x, r) + id / kXcds;
    const int per = group * nn, g = at / per, first = g * group;
    const int rows = min(group, nm - first), in = at - g * per;
    tm = first + in % rows;
    tn = in / rows;
}

}  // namespace dflash2
