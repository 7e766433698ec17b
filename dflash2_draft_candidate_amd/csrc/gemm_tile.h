// Matrix products on the matrix cores: tiles of C[m][n] = sum_k A(m, k) B(n, k).
//
// An operand lies in memory in one of two ways: its rows hold k (KC: element (m, k) at
// base + m ld + k), or its rows hold m (KS: element (m, k) at base + k ld + m). The LM head's
// logits take two KC operands, the hidden states' gradient KS x KC, the weight's KS x KS; no
// operand is transposed in memory first.
//
// What both kernels below share (gfx950, eight waves):
//   * A K step is 128 bytes of k per row (64 bf16, 32 f32), so a stage holds 128 B bytes of an
//     operand of B rows in either layout. Loads go from memory straight into LDS, 16 bytes a lane.
//   * The loads write LDS linearly, so the swizzle that keeps the fragment reads free of bank
//     conflicts is in the addresses they read: KC stages keep chunk c (16 bytes) of row m at slot
//     c ^ (m & 7); KS stages of bf16 keep the 32-byte piece s of row k at s ^ f(k), where f takes
//     16 values (as many as fit the row) over the 16 rows that one transposing read touches; KS
//     stages of f32 keep the 64-byte piece s at s ^ ((k >> 2) & 3).
//   * bf16: v_mfma_f32_16x16x32_bf16. Lane (g = lane / 16, j = lane % 16) takes row j and
//     k = 8 g .. 8 g + 7: one 16-byte LDS read from a KC stage, two transposing 8-byte reads
//     (rows k = 8 g .. + 3 and + 4 .. + 7) from a KS stage. f32: v_mfma_f32_16x16x4_f32, a lane's
//     16 bytes (k = 4 g .. 4 g + 3) feeding four of them; both operands agree on which k an
//     instruction multiplies. Sums are fp32 and their order depends on k alone, not on the tile.
//   * Out of range: a load's descriptor ends at the operand's last valid byte, so rows past the end
//     read zeros; a KC operand whose k ends inside a step masks the chunks behind it. What lies
//     behind the last column m of a KS row only reaches outputs that no caller stores.
//   * The loads into LDS are inline assembly (they have no output registers): the compiler, which
//     cannot tell the stages apart, would wait for all of them before each read of LDS. Every wait
//     for them is written out below.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace dflash2 {

constexpr int kGemmWaves = 8;
constexpr int kGemmThreads = kGemmWaves * kWave;
constexpr int kStepBytes = 128;
constexpr int kGemmOutside = 0x7FFFFFF0;  // an offset that no descriptor covers
constexpr int kGemmWord3 = 0x00020000;    // gfx9-family buffer descriptor word 3 (raw data)

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A tile's operand: from its first row (KC) or column (KS) and first k on.
struct GemmOperand {
    const char *base;
    int64_t ld;  // bytes from one row to the next
    int valid;   // KC: rows in range, counted from the tile's first; KS: bytes of a row before base
};

// Rows from row0 on of a KC matrix of `rows` rows, k from k0 on. (A row is a whole number of 16-byte
// chunks in memory; what the last k leaves of its chunk holds zeros.)
template <typename T>
__device__ __forceinline__ GemmOperand operand_kc(const void *p, int64_t ld, int row0, int rows,
                                                  int k0) {
    return {static_cast<const char *>(p) + row0 * ld + (int64_t)k0 * sizeof(T), ld, rows - row0};
}

// Columns from col0 on of a KS matrix, k from k0 on.
template <typename T>
__device__ __forceinline__ GemmOperand operand_ks(const void *p, int64_t ld, int col0, int k0) {
    return {static_cast<const char *>(p) + (int64_t)k0 * ld + (int64_t)col0 * sizeof(T), ld,
            col0 * (int)sizeof(T)};
}

// A descriptor of `bytes` bytes from p on, in scalar registers.
__device__ __forceinline__ u32x4 scalar_buffer(const void *p, int bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    u32x4 rs;
    rs.x = __builtin_amdgcn_readfirstlane((uint32_t)a);
    rs.y = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);
    rs.z = __builtin_amdgcn_readfirstlane((uint32_t)(bytes < 0 ? 0 : bytes));
    rs.w = kGemmWord3;
    return rs;
}

// Starts a load of 16 (4) bytes a lane, from `off` bytes into the buffer, into LDS at `to` + 16 (4) lane.
// (A memory instruction may read a scalar register that a vector instruction wrote 5 states later; the
// compiler sees to that, but not inside assembly. M0 needs one state.)
__device__ __forceinline__ void load_lds16(uint32_t to, int off, u32x4 rs) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to),
                 "v"(off), "s"(rs)
                 : "memory");
}
__device__ __forceinline__ void load_lds4(uint32_t to, int off, u32x4 rs) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to),
                 "v"(off), "s"(rs)
                 : "memory");
}

// One stage of an operand: B rows (KC) or columns (KS) of a K step. Where G is not 0 they are every
// other run of G of the tile's: row i of the stage is row (i / G) 2 G + i % G.
template <typename T, int B, bool KS, int G = 0> struct GemmSide {
    static constexpr int kBytes = B * kStepBytes;
    static constexpr int kStepK = kStepBytes / (int)sizeof(T);
    static constexpr int kLoads = kBytes / 1024;  // of 1 KB, one wave's
    static constexpr int kPerWave = (kLoads + kGemmWaves - 1) / kGemmWaves;
    static_assert(kLoads % kGemmWaves == 0 || kGemmWaves % kLoads == 0 || !KS, "the waves share the loads");
    static constexpr int kRowBytes = B * (int)sizeof(T);  // KS
    static constexpr int kRowChunks = kRowBytes / 16;

    int voff[kPerWave];  // the lane's bytes within the operand's step
    int kbyte;           // KC: the first byte of k that the lane reads

    // Where the loads are no multiple of 8, some waves make the same one: every wave counts the same.
    static __device__ __forceinline__ int load_of(int wave, int q) {
        const int i = wave + kGemmWaves * q;
        return kLoads < kGemmWaves ? wave % kLoads : i < kLoads ? i : i - kGemmWaves;
    }

    static __device__ __forceinline__ int tile_row(int i) {
        return G == 0 ? i : (i / (G ? G : 1)) * 2 * G + i % (G ? G : 1);
    }

    __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
        kbyte = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
        for (int q = 0; q < kPerWave; ++q) {
            const int load = load_of(wave, q);
            if constexpr (!KS) {
                voff[q] = tile_row(8 * load + (lane >> 3)) * (int)ld + kbyte;
            } else {
                const int at = load * kWave + lane, k = at / kRowChunks, p = at % kRowChunks;
                int c;
                if constexpr (sizeof(T) == 2)
                    c = (((p >> 1) ^ swizzle(k)) << 1) | (p & 1);
                else
                    c = (((p >> 2) ^ ((k >> 2) & 3)) << 2) | (p & 3);
                voff[q] = k * (int)ld + tile_row(c * (16 / (int)sizeof(T))) * (int)sizeof(T);
            }
        }
    }

    // KC: the stage's row i is row rows[i] of the operand, for i < n.
    __device__ __forceinline__ void take_rows(const int *rows, int n, int ld, int wave, int lane) {
        static_assert(!KS, "rows that hold k");
#pragma unroll
        for (int q = 0; q < kPerWave; ++q) {
            const int i = tile_row(8 * load_of(wave, q) + (lane >> 3));
            voff[q] = i < n ? rows[i] * ld + kbyte : kGemmOutside;
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

    // Starts this wave's loads of a step into the stage at `to`. p: the step's first byte of the
    // operand; `valid` as the operand's, counted from p; kleft: values of k left.
    __device__ __forceinline__ void issue(uint32_t to, const char *p, int ld, int valid, int kleft,
                                          int wave) const {
        const int ks = kleft < 0 ? 0 : kleft < kStepK ? kleft : kStepK;
        int n;
        if constexpr (KS)
            n = ks * ld - valid;
        else
            n = ks == 0 ? 0 : (min(valid, 2 * B) - 1) * ld + (ks * (int)sizeof(T) + 15) / 16 * 16;
        const u32x4 rs = scalar_buffer(p, n);
#pragma unroll
        for (int q = 0; q < kPerWave; ++q) {
            int off = voff[q];
            if constexpr (!KS) off = kbyte < kleft * (int)sizeof(T) ? off : kGemmOutside;
            load_lds16(to + load_of(wave, q) * 1024, off, rs);
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
                    at[i] = k * kRowBytes + (((m0 / 16 + i) ^ swizzle(k)) << 5) + 8 * (j & 3);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    at[i] = 4 * g * kRowBytes + (((m0 / 16 + i) ^ g) << 6) + 4 * j;
            }
        }
        // half h of the step: bf16 k = 32 h .. 32 h + 31, f32 k = 16 h .. 16 h + 15
        __device__ __forceinline__ Frag read(const char *stage, int i, int h) const {
            if constexpr (!KS) {
                return *reinterpret_cast<const Frag *>(stage + at[h] + i * 16 * kStepBytes);
            } else if constexpr (sizeof(T) == 2) {
                const char *p = stage + at[i] + 32 * h * kRowBytes;
                struct { s16x4 lo, hi; } v;
                v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
                v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * kRowBytes));
                return __builtin_bit_cast(Frag, v);
            } else {
                const char *p = stage + at[i] + 16 * h * kRowBytes;
                Frag v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float *>(p + e * kRowBytes);
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

__device__ __forceinline__ uint32_t lds_address(void *p) {
    return (uint32_t)(uintptr_t)(lds_void *)p;
}

// ---- output --------------------------------------------------------------------------------------

// Four values of type T, rounded to nearest even.
template <typename T>
__device__ __forceinline__ auto packed4(f32x4 x) {
    if constexpr (sizeof(T) == 2) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(u32x2, bf16x4{(__bf16)x[0], (__bf16)x[1], (__bf16)x[2],
                                                (__bf16)x[3]});
    } else {
        return __builtin_bit_cast(u32x4, x);
    }
}

// Output rows as a descriptor and 32-bit offsets: `rows` rows of `ld` bytes from p on, the last
// one `width` bytes long. A store at kGemmOutside, or behind the last row, is dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t out_rows(void *p, int64_t ld, int rows,
                                                           int64_t width) {
    const int64_t n = rows > 0 ? (rows - 1) * ld + width : 0;
    return __builtin_amdgcn_make_buffer_rsrc(p, (short)0, (int)n, kGemmWord3);
}

template <typename T>
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t rs, int off, f32x4 x) {
    if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b64(packed4<T>(x), rs, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b128(packed4<T>(x), rs, off, 0, 0);
}

// The barrier with what it stands for: nothing moves across, for the compiler's passes over memory
// (which take the barrier itself for an instruction that has none) and for its scheduler.
__device__ __forceinline__ void bare_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// vmcnt(VM) lgkmcnt(LGKM). 63 and 15: no wait.
template <int VM, int LGKM> __device__ __forceinline__ void wait_for() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | 0x70 | (LGKM << 8));
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

template <int VM> __device__ __forceinline__ void gemm_barrier() {
    wait_for<VM, 0>();
    bare_barrier();
}

// `x` as a value of its own: what an epilogue computes from it is computed there, not kept in registers
// through the products.
__device__ __forceinline__ int anew(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// ---- one tile at a time ------------------------------------------------------------------------
// A tile of BM x BN over WM x (8 / WM) waves. Wave (wm, wn) holds rows m = wm BM / WM + 16 mi +
// 4 g + i and columns n = wn BN / WN + 16 ni + j in acc[mi][ni][i]. Two stages per operand: the loads
// of step t + 1 are in flight while step t is multiplied. For tiles below 256 x 256, and for f32,
// where the matrix cores are the bound whatever feeds them (4096 x 4096 x 2048: 142 TFLOP/s; the
// phases below: 132).
template <typename T, int BM, int BN, bool AS, bool BS, int WM> struct GemmTile {
    static constexpr int WN = kGemmWaves / WM;
    static constexpr int MI = BM / (16 * WM), NI = BN / (16 * WN);
    static constexpr int kCols = BN;
    static_assert(MI * 16 * WM == BM && NI * 16 * WN == BN, "whole fragments");
    typedef GemmSide<T, BM, AS> SideA;
    typedef GemmSide<T, BN, BS> SideB;
    static constexpr int kStepK = SideA::kStepK;
    static constexpr int kLdsBytes = 2 * (SideA::kBytes + SideB::kBytes);

    f32x4 acc[MI][NI];

    static __device__ __forceinline__ int wave_m(int wave) { return (wave / WN) * (BM / WM); }
    static __device__ __forceinline__ int wave_n(int wave) { return (wave % WN) * (BN / WN); }

    // The product over K values of k. lds: kLdsBytes.
    __device__ __forceinline__ void run(const GemmOperand &A, const GemmOperand &B, int K, char *lds,
                                        int wave, int lane) {
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

        constexpr int kStage = SideA::kBytes + SideB::kBytes;
        const uint32_t base = lds_address(lds);
        const int steps = (K + kStepK - 1) / kStepK;
        const char *pa = A.base, *pb = B.base;
        int kleft = K;
        auto issue = [&](int buf) {
            sa.issue(base + buf * kStage, pa, (int)A.ld, A.valid, kleft, wave);
            sb.issue(base + buf * kStage + SideA::kBytes, pb, (int)B.ld, B.valid, kleft, wave);
            pa += SideA::stride(A.ld);
            pb += SideB::stride(B.ld);
            kleft -= kStepK;
        };
        auto compute = [&](int buf) {
            const char *sta = lds + buf * kStage, *stb = sta + SideA::kBytes;
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
        // At a step's barrier this wave's loads have landed, so after it all waves' have, and every
        // wave has read the other stage, which the next loads overwrite. (Loads past the last step
        // read nothing and write zeros: the loop stays free of branches.)
        issue(0);
        for (int t = 0; t + 1 < steps; t += 2) {
            gemm_barrier<0>();
            issue(1);
            compute(0);
            gemm_barrier<0>();
            issue(0);
            compute(1);
        }
        gemm_barrier<0>();
        if (steps & 1) compute(0);
    }
};

// ---- few columns: a ring of stages ---------------------------------------------------------------
// Tiles of BM x BN where the read of A is the bound (BN <= 128): each wave takes BM / 8 rows and all
// columns. A stage is SUB consecutive K steps; the ring holds as many as LDS does, and all but the one
// that is read are on their way. The loads run ahead from one tile of the workgroup into the next.
struct GemmWork {
    GemmOperand a, b;
    int K;  // <= 0: no tile
    bool more = false;  // a stream of PARTS: the next work's products are this tile's too
};

// RESERVE: bytes of LDS that are not the ring's.
template <typename T, int BM_, int BN, int SUB, bool AS, bool BS, int RESERVE = 0> struct GemmRing {
    static constexpr int BM = BM_, WM = 8, WN = 1, MI = BM / 128, NI = BN / 16, kCols = BN;
    typedef GemmSide<T, BM, AS> SideA;
    typedef GemmSide<T, BN, BS> SideB;
    static constexpr int kStepK = SideA::kStepK;
    static constexpr int kStep = SideA::kBytes + SideB::kBytes, kStage = SUB * kStep;
    static constexpr int kStages = (163840 - RESERVE) / kStage;
    static constexpr int kLdsBytes = kStages * kStage;
    static constexpr int kLoads = SUB * (SideA::kPerWave + SideB::kPerWave);  // a wave's, per stage
    static_assert(kStages >= 3 && (kStages - 2) * kLoads < 64, "stages");

    f32x4 acc[MI][NI];

    static __device__ __forceinline__ int wave_m(int wave) { return wave * (BM / WM); }
    static __device__ __forceinline__ int wave_n(int) { return 0; }

    // work(i): the workgroup's tile i, K = 0 behind the last; done(i): its epilogue, on acc. All tiles
    // share the operands' ld. Behind the last tile LDS is free. b_rows: null, or (in LDS) the rows of B's
    // matrix that the tile's columns are, nb of them.
    template <typename Work, typename Done>
    __device__ __forceinline__ void run(int64_t lda, int64_t ldb, Work work, Done done, char *lds,
                                        int wave, int lane, const int *b_rows = nullptr, int nb = 0) {
        SideA sa;
        SideB sb;
        sa.init(lda, wave, lane);
        sb.init(ldb, wave, lane);
        if (b_rows) sb.take_rows(b_rows, nb, (int)ldb, wave, lane);
        typename SideA::template Reader<MI> ra;
        typename SideB::template Reader<NI> rb;
        ra.init(wave_m(wave), lane);
        rb.init(0, lane);
        const uint32_t base = lds_address(lds);
        const int64_t da = SideA::stride(lda), db = SideB::stride(ldb);
        GemmWork at = work(0);
        int next = 1, kleft = at.K;
        auto issue = [&](int slot) {
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                const uint32_t to = base + slot * kStage + u * kStep;
                sa.issue(to, at.a.base, (int)lda, at.a.valid, kleft, wave);
                sb.issue(to + SideA::kBytes, at.b.base, (int)ldb, at.b.valid, kleft, wave);
                at.a.base += da;
                at.b.base += db;
                kleft -= kStepK;
            }
            if (kleft <= 0 && at.K > 0) {  // (behind the last tile: loads of nothing)
                at = work(next++);
                kleft = at.K;
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        int slot = 0;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(i);
        for (int i = 0;; ++i) {
            const int K = work(i).K;
            if (K <= 0) break;
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < K; k += SUB * kStepK) {
                // this stage has landed in every wave, and every wave has read the one before it
                gemm_barrier<(kStages - 2) * kLoads>();
                issue(slot == 0 ? kStages - 1 : slot - 1);
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    const char *sta = lds + slot * kStage + u * kStep, *stb = sta + SideA::kBytes;
                    // (all reads first: the products wait for theirs only, and cover the others)
                    typename SideA::Frag fa[2][MI];
                    typename SideB::Frag fb[2][NI];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int mi = 0; mi < MI; ++mi) fa[h][mi] = ra.read(sta, mi, h);
#pragma unroll
                        for (int ni = 0; ni < NI; ++ni) fb[h][ni] = rb.read(stb, ni, h);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
                            for (int mi = 0; mi < MI; ++mi)
                                acc[mi][ni] = gemm_mfma(fa[h][mi], fb[h][ni], acc[mi][ni]);
                }
                slot = slot == kStages - 1 ? 0 : slot + 1;
            }
            done(i);
        }
        gemm_barrier<0>();
    }
};

// ---- a stream of 256 x 256 tiles ---------------------------------------------------------------
// The waves form two groups of four, one wave of each on every SIMD. A K step is four phases, each a
// quarter of the wave's 128 x 64 (64 x 32: 16 matrix instructions); in a phase a wave first reads the
// fragments of the quarter from LDS and starts two loads, then multiplies. The second group runs one
// barrier behind the first, so on every SIMD one wave multiplies while the other one reads.
//   * A and B are staged in halves of 128 rows (the rows of every wave's first and second half), each
//     in a place of its own: 8 x 16 KB, two steps. Phases read A0 | B1 | A1 | B0 of the next step, and
//     each starts the load of the half that the phase before has read, for two steps later: seven
//     phases pass before it is read, so the waits leave six halves (12 loads a wave) in flight.
//   * A wave's reads of a half are done (lgkmcnt) before the barrier that ends its reading; no wave
//     starts a load into that half before that barrier, whichever group it is in.
//   * The loads run ahead over the end of a tile into the next one of the workgroup, so a tile's
//     epilogue, which uses no LDS, finds the next tile's first two steps on their way.
//   * An epilogue's stores count in vmcnt like loads. kStores is how many a wave surely makes in one;
//     the first six phases behind it, whose halves were asked for before them, do not wait for them.
// 4096 x 4096 x 16384 bf16: 1314 TFLOP/s (KC x KC), 1319 (KS x KC), 1366 (KS x KS); one stage of
// 64 KB ahead and a barrier per step (GemmTile): 1123, 1201, 1217.
template <typename T, bool AS, bool BS, int kStores, bool PARTS = false> struct GemmStream {
    static constexpr int WM = 2, WN = 4, MI = 8, NI = 4, BM = 256, BN = 256, kCols = BN;
    typedef GemmSide<T, 128, AS, 64> SideA;
    typedef GemmSide<T, 128, BS, 32> SideB;
    static constexpr int kStepK = SideA::kStepK;
    static constexpr int kHalf = SideA::kBytes;
    static constexpr int kStageBytes = 8 * kHalf;  // per buffer: A0 A1 B0 B1
    static constexpr int kScratch = 4096;          // a wave's, for its stores
    static constexpr int kLdsBytes = kStageBytes + kGemmWaves * kScratch;
    static_assert(12 + kStores < 64, "vmcnt");

    f32x4 acc[MI][NI];

    static __device__ __forceinline__ int wave_m(int wave) { return (wave / WN) * (BM / WM); }
    static __device__ __forceinline__ int wave_n(int wave) { return (wave % WN) * (BN / WN); }

    // steps of a tile: an even number, so that every tile starts in buffer 0
    static __device__ __forceinline__ int steps_of(int K) {
        return ((K + kStepK - 1) / kStepK + 1) & ~1;
    }

    // work(i): the workgroup's tile i (PARTS: or a part of its k), K = 0 behind the last; done(i): its epilogue,
    // on acc. All tiles share the operands' ld.
    template <typename Work, typename Done>
    __device__ __forceinline__ void run(int64_t lda, int64_t ldb, Work work, Done done, char *lds,
                                        int wave, int lane) {
        SideA sa;
        SideB sb;
        sa.init(lda, wave, lane);
        sb.init(ldb, wave, lane);
        typename SideA::template Reader<4> ra;
        typename SideB::template Reader<2> rb;
        ra.init((wave / WN) * 64, lane);
        rb.init((wave % WN) * 32, lane);

        // what the loads are at: two steps ahead of the products
        const uint32_t base = lds_address(lds);
        const int64_t da = SideA::stride(lda), db = SideB::stride(ldb);
        const int64_t half_a = AS ? 64 * (int)sizeof(T) : 64 * lda;
        const int64_t half_b = BS ? 32 * (int)sizeof(T) : 32 * ldb;
        constexpr int kPartA = AS ? 64 * (int)sizeof(T) : -64;  // on `valid`, for the second half
        constexpr int kPartB = BS ? 32 * (int)sizeof(T) : -32;
        GemmWork at = work(0);
        if (at.K <= 0) return;
        int next = 1, load_left = steps_of(at.K), kleft = at.K;
        auto load_a = [&](int half, int buf) {
            sa.issue(base + (buf * 4 + half) * kHalf, at.a.base + half * half_a, (int)lda,
                     at.a.valid + half * kPartA, kleft, wave);
        };
        auto load_b = [&](int half, int buf) {
            sb.issue(base + (buf * 4 + 2 + half) * kHalf, at.b.base + half * half_b, (int)ldb,
                     at.b.valid + half * kPartB, kleft, wave);
        };
        auto advance = [&]() {
            at.a.base += da;
            at.b.base += db;
            kleft -= kStepK;
            if (--load_left == 0) {
                at = work(next++);
                kleft = at.K;
                load_left = at.K > 0 ? steps_of(at.K) : -1;  // (behind the last tile: loads of nothing)
            }
        };
        typename SideA::Frag fa[4][2];
        typename SideB::Frag fb0[2][2], fb1[2][2], fbn[2][2];
        auto read_a = [&](int buf, int half) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) fa[i][h] = ra.read(lds + (buf * 4 + half) * kHalf, i, h);
        };
        auto read_b = [&](int buf, int half, typename SideB::Frag(&f)[2][2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) f[i][h] = rb.read(lds + (buf * 4 + 2 + half) * kHalf, i, h);
        };
        auto multiply = [&](int ah, int bh, typename SideB::Frag(&f)[2][2]) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[4 * ah + i][2 * bh + j] =
                            gemm_mfma(fa[i][h], f[j][h], acc[4 * ah + i][2 * bh + j]);
            __builtin_amdgcn_s_setprio(0);
        };
#pragma unroll
        for (int buf = 0; buf < 2; ++buf) {
            load_b(0, buf);
            load_a(0, buf);
            load_b(1, buf);
            load_a(1, buf);
            advance();
        }
        gemm_barrier<14>();  // the first of the 8 halves has landed
        read_b(0, 0, fb0);
        gemm_barrier<12>();  // the second
        if (wave >= kGemmWaves / 2) bare_barrier();  // from here on this group runs one barrier behind
        bool stored = false;  // an epilogue's stores are younger than what is waited for
        auto landed = [&](bool may_be_young) {
            if (kStores > 0 && may_be_young && stored)
                gemm_barrier<12 + kStores>();
            else
                gemm_barrier<12>();
        };
        auto step = [&](int buf, typename SideB::Frag(&b0)[2][2], typename SideB::Frag(&bn)[2][2]) {
            read_a(buf, 0);
            load_b(0, buf);
            landed(true);
            multiply(0, 0, b0);
            bare_barrier();
            read_b(buf, 1, fb1);
            load_a(0, buf);
            landed(true);
            multiply(0, 1, fb1);
            bare_barrier();
            read_a(buf, 1);
            load_b(1, buf);
            landed(buf == 0);
            multiply(1, 1, fb1);
            bare_barrier();
            read_b(buf ^ 1, 0, bn);
            load_a(1, buf);
            advance();
            landed(buf == 0);
            multiply(1, 0, b0);
            bare_barrier();
        };
        bool more = false;
        for (int i = 0;; ++i) {
            const int K = work(i).K;
            if (K <= 0) break;
            if (!PARTS || !more) {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            for (int t = steps_of(K); t > 0; t -= 2) {
                step(0, fb0, fbn);
                step(1, fbn, fb0);
                stored = false;
            }
            if constexpr (PARTS) {
                more = work(i).more;
                if (more) continue;
            }
            done(i);
            stored = true;
        }
        if (wave < kGemmWaves / 2) bare_barrier();  // (the other group's last barrier)
        wait_for<0, 0>();  // no load is in flight when the workgroup ends
    }

    // The tile as bf16 rows of output: row n of it at `out` + n ld, its columns m from byte `first` on,
    // those from byte `end` of a row on left out. value(mi, ni): the wave's four values. A wave's
    // accumulators hold 8 bytes of each of 16 rows; 16 rows of its 128 columns go through 4 KB of LDS
    // (16-byte chunk c of row j at c ^ j), so that a store covers 256 bytes of each of 4 rows: a store
    // takes its time by the lines it touches (4096 x 65536 x 1024: 630 us with 8-byte stores from the
    // accumulators).
    template <typename Value>
    __device__ __forceinline__ void store_rows(__amdgpu_buffer_rsrc_t out, int ld, int first, int end,
                                               char *lds, int wave, int lane, Value value) {
        char *scratch = lds + kStageBytes + wave * kScratch;
        lane = anew(lane);
        const int g = lane >> 4, j = lane & 15;
        const int put = j * 256 + (g & 1) * 8;
        const int column = first + wave_m(wave) * 2 + j * 16;  // (in the second half lane j takes chunk j)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
#pragma unroll
            for (int mi = 0; mi < MI; ++mi) {
                const auto x = packed4<uint16_t>(value(mi, ni));
                *reinterpret_cast<decltype(packed4<uint16_t>(f32x4{}))  *>(
                    scratch + put + (((2 * mi + (g >> 1)) ^ j) << 4)) = x;
                __builtin_amdgcn_sched_barrier(0);  // (all at once would not fit the registers)
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = 4 * q + g;
                const u32x4 x = *reinterpret_cast<const u32x4 *>(scratch + row * 256 + ((j ^ row) << 4));
                __builtin_amdgcn_raw_buffer_store_b128(
                    x, out, column < end ? (wave_n(wave) + 16 * ni + row) * ld + column : kGemmOutside,
                    0, 0);
            }
        }
    }
    static constexpr int kRowStores = 4 * NI;  // store_rows' stores
};

// The tile of place `id` of nm x nn tiles. Consecutive workgroups run on different XCDs, each with
// an L2 of its own: XCD x takes a contiguous eighth of the tiles, in groups of `group` rows of tiles,
// rows first, so that what it works on at a time shares operands.
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
