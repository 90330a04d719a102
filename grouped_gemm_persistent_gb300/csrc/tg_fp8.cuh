// tg_fp8.cuh - the 8-bit GEMM with a scale for each block of 128 along K.
//
//   C[m, n] = epilogue( sum_kb sa[m, kb] * sb[kb, n] * ( sum_{k in block kb} A[m, k] B[k, n] ) )
//
// The inner sum runs on the tensor cores (tcgen05.mma kind::f8f6f4, fp32 accumulator);
// the scales are fp32 of any value, so the outer sum cannot stay in tensor memory: each
// k-block's partial product is read back, scaled and added to fp32 registers.  One ring
// stage is one scale block (128 bytes of K per row, four MMAs of K = 32).
//
//   warp 0       TMA producer: A and B k-blocks into a STAGES-deep ring.
//   warps 1, 2   MMA issuers, one for each of two TMEM buffers (even and odd k-blocks): four
//                MMAs, then a commit that frees the ring stage and one that hands the
//                buffer over.  Warp 1 also allocates and frees tensor memory.
//   warp 3       scale loader: the scales of the k-blocks ahead, by cp.async into a ring of
//                their own.  (Loaded by the accumulating warps into registers, four k-blocks
//                ahead, they made every tcgen05.wait::ld wait for global loads: 8192^3 took
//                1340 us.)
//   warps 4-11   accumulation and epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 and
//                half the tile's columns: acc += scale * partial while the MMAs of the next
//                k-block run; after the last k-block bias, GELU, rounding and the store.
//
// 256 x 256 tiles of a CTA pair: per k-block and SM the tensor cores need 512 cycles
// (128 x 256 x 128 at 8192 MAC/cycle) and the additions 256 issue slots a quarter of the SM, but
// a k-block takes ~700: with two buffers, its MMAs wait for the read-back of the k-block two
// before it, and that is a chain of four tensor-memory loads (~80 cycles each, 130 before the
// first) and a barrier on either side.  8192^3, bf16 out: 390 to 400 us, 2750 TFLOP/s, in a few launches
// at a time, 430 to 447 us, 2490 TFLOP/s, back to back at the power limit; the MMAs and barriers
// without the read-back 296 us.  128 accumulator registers a thread for eight warps
// need the registers of the first four (setmaxnreg).
//
// Spills: none with block scales; 28 bytes of stores and 116 of loads a thread in the pair form with a
// scale per column.  Waits, aborts and draining are those of tg_kernel.cuh.
#pragma once

#include "tg_kernel.cuh"

namespace tg {

constexpr int F8_BK = 128;                 // K per stage: one scale block
constexpr int F8_THREADS = 384;
constexpr int F8_EPI_WARP0 = 4;
constexpr int F8_EPI_WARPS = 8;
constexpr int F8_GROUP = 4;                // k-blocks whose scales share a slot
constexpr int F8_C_STAGE = 32 * 64;        // per-warp store staging: 32 rows of 64 bytes

// What the 8-bit form needs besides Params (whose `dense` problem holds the maps, sizes,
// bias and epilogue; tma_c is unused).
struct Fp8Params {
    const float* sa;           // sa[(m >> sa_shift) * sa_mn + kb * sa_k]
    const float* sb;           // sb[expert * sb_g + (n >> sb_shift) * sb_mn + kb * sb_k]
    int64_t sa_mn, sa_k;
    int64_t sb_mn, sb_k, sb_g;
    int32_t sa_shift;          // 0: a scale per row, 7: per 128 rows
    uint32_t a_mn, b_mn;       // A stored M-contiguous, B stored N-contiguous
    uint32_t vec_c;            // rows of C are 16-byte aligned
    uint32_t a_bytes;          // of A's box: all 128 rows, or as many as a short A has
    uint32_t halves;           // pairs: the last wave's tiles may run as half tiles
    int32_t splits;            // SPLIT: CTAs that share a tile (the cluster's size)
    void* c;
    int64_t ldc;
};

// SPLIT (single CTAs, dense): the CTAs of a cluster share one tile, each summing its own range of
// k-blocks, and join their sums through distributed shared memory.
template <int CTA_GROUP_, bool SB_COL_, bool MOE_, bool SPLIT_ = false>
struct Fp8Config {
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int CTA_GROUP = CTA_GROUP_;
    static constexpr bool SB_COL = SB_COL_;          // B has a scale per column (else per 128 columns)
    static constexpr bool GROUPED = false;
    static constexpr bool MOE = MOE_;
    static constexpr int BN = 128 * CTA_GROUP;
    static constexpr int BN_CTA = 128;
    static constexpr int TILE_M = BM * CTA_GROUP;
    static constexpr int COLS = BN / 2;              // columns one epilogue warp accumulates
    static constexpr int A_BYTES = BM * F8_BK;
    static constexpr int B_BYTES = BN_CTA * F8_BK;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int C_BYTES = F8_EPI_WARPS * F8_C_STAGE;
    static constexpr int SB_COUNT = SB_COL ? BN : BN / 128;      // B scales of a tile and k-block
    static constexpr int SLOTS = 4;                            // groups of scales in flight
    static constexpr int SLOT_BYTES = (BM + SB_COUNT) * F8_GROUP * 4;
    static constexpr int SCALE_BYTES = SLOTS * SLOT_BYTES;
    static constexpr int TABLE_BYTES = MOE ? 8 * (MOE_MAX_G + 1) : 0;
    static constexpr int FIXED = C_BYTES + SCALE_BYTES + TABLE_BYTES + 512 + 1024;
    static constexpr int STAGES = (SMEM_LIMIT - FIXED) / (A_BYTES + B_BYTES);
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_C = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_SCALE = OFF_C + C_BYTES;
    static constexpr int OFF_TABLE = OFF_SCALE + SCALE_BYTES;
    static constexpr int OFF_BAR = OFF_TABLE + TABLE_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 6 + 2 * SLOTS;
    static constexpr int OFF_TMEM_SLOT = OFF_BAR + 8 * NUM_BARS;
    static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
    static constexpr int OFF_MOE_TOTAL = OFF_ABORT + 4;
    static constexpr int OFF_DRAIN_FLAG = OFF_MOE_TOTAL + 4;
    static constexpr int OFF_DRAIN_POS = OFF_DRAIN_FLAG + 4;
    static constexpr int OFF_DRAIN_LAST = OFF_DRAIN_POS + 4;
    static constexpr int OFF_DRAIN_BYTES = OFF_DRAIN_LAST + 4 * MAX_STAGES;
    static constexpr int SMEM_BYTES = OFF_DRAIN_BYTES + 4 * MAX_STAGES + 1024;
    static_assert(!SPLIT || (CTA_GROUP == 1 && !MOE), "split tiles are dense single-CTA ones");
    static_assert(!SPLIT || F8_EPI_WARPS * 32 * COLS * 4 <= STAGES * (A_BYTES + B_BYTES), "partial sums fit the ring");
    static_assert(STAGES >= 2 && STAGES <= MAX_STAGES, "ring depth");
    static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory budget");
    static_assert(OFF_BAR % 8 == 0, "barrier alignment");
};

namespace f8 {

// Prefix tables of a device-counts launch (one warp): rows and tiles before each expert, and the
// number of tiles; 0 tiles and an error record when the counts are negative or exceed the rows.
__device__ __forceinline__ int32_t build_moe_table(const Params& p, int tile_m, int64_t tiles_n, int32_t* tile_pref,
                                                   int32_t* row_off, int lane) {
    long long rows = 0, tiles = 0;
    bool bad = false;
    if (lane == 0) { tile_pref[0] = 0; row_off[0] = 0; }
    for (int g0 = 0; g0 < p.moe_groups; g0 += 32) {
        const int i = g0 + lane;
        long long c = i < p.moe_groups ? static_cast<long long>(__ldg(p.moe_counts + i)) : 0ll;
        bad |= c < 0;
        c = c < 0 ? 0 : c;
        long long t = (c + tile_m - 1) / tile_m * tiles_n;
        for (int d = 1; d < 32; d <<= 1) {
            const long long xc = __shfl_up_sync(0xffffffffu, c, d);
            const long long xt = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) { c += xc; t += xt; }
        }
        if (i < p.moe_groups) {
            row_off[i + 1] = static_cast<int32_t>(min(rows + c, 0x7fffffffll));
            tile_pref[i + 1] = static_cast<int32_t>(min(tiles + t, 0x7fffffffll));
        }
        rows += __shfl_sync(0xffffffffu, c, 31);
        tiles += __shfl_sync(0xffffffffu, t, 31);
    }
    bad = __any_sync(0xffffffffu, bad) || rows > p.moe_rows || tiles > 0x7fffffffll;
    if (bad && lane == 0 && blockIdx.x == 0 && atomicCAS(&p.err->code, ERR_NONE, ERR_COUNTS) == ERR_NONE) {
        p.err->role = 0;
        p.err->block = 0;
        p.err->stage = 0;
        p.err->tile = rows;
        p.err->waited_ns = 0;
    }
    return bad ? 0 : static_cast<int32_t>(tiles);
}

// Wait for all tcgen05.ld of this thread; the registers they fill are operands, so no use of
// them can be scheduled before the wait.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :: "memory");
}

// One k-block: four MMAs of K = 32 that start a new accumulator, the commit that frees the ring
// stage (`empty`) and the one that hands the accumulator over (`tfull`).  Executed by a
// converged warp; one elected lane issues.
template <int CTA_GROUP>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint64_t b, uint64_t a_step, uint64_t b_step,
                                          uint32_t idesc, uint32_t empty, uint32_t tfull) {
    if constexpr (CTA_GROUP == 2)
        asm volatile(
            "{\n\t.reg .pred g, f, t;\n\t"
            "elect.sync _|g, 0xffffffff;\n\t"
            "setp.ne.u32 f, 0, 0;\n\t"
            "setp.eq.u32 t, 0, 0;\n\t"
            "@g tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %5, %9, f;\n\t"
            "@g tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %2, %6, %9, t;\n\t"
            "@g tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %3, %7, %9, t;\n\t"
            "@g tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %4, %8, %9, t;\n\t"
            "@g tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%10], %12;\n\t"
            "@g tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%11], %12;\n\t"
            "}"
            :: "r"(d), "l"(a), "l"(a + a_step), "l"(a + 2 * a_step), "l"(a + 3 * a_step), "l"(b), "l"(b + b_step),
               "l"(b + 2 * b_step), "l"(b + 3 * b_step), "r"(idesc), "r"(empty), "r"(tfull),
               "h"(static_cast<uint16_t>(0x3)) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred g, f, t;\n\t"
            "elect.sync _|g, 0xffffffff;\n\t"
            "setp.ne.u32 f, 0, 0;\n\t"
            "setp.eq.u32 t, 0, 0;\n\t"
            "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %5, %9, f;\n\t"
            "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %6, %9, t;\n\t"
            "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %7, %9, t;\n\t"
            "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %8, %9, t;\n\t"
            "@g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t"
            "@g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11];\n\t"
            "}"
            :: "r"(d), "l"(a), "l"(a + a_step), "l"(a + 2 * a_step), "l"(a + 3 * a_step), "l"(b), "l"(b + b_step),
               "l"(b + 2 * b_step), "l"(b + 3 * b_step), "r"(idesc), "r"(empty), "r"(tfull) : "memory");
}

// Eight bf16 values from column `col` of a bias of N values (zeros past its end) as fp32.
__device__ __forceinline__ void load_bias8(const uint16_t* bias, int col, int N, float (&b)[8]) {
    const uint16_t* p = bias + col;
    if (col + 8 <= N && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[2 * i] = __uint_as_float(ws[i] << 16);
            b[2 * i + 1] = __uint_as_float(ws[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            b[i] = col + i < N ? __uint_as_float(static_cast<uint32_t>(__ldg(p + i)) << 16) : 0.0f;
    }
}

// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_each(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        for_each<N, I + 1>(f);
    }
}

template <int REGS>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REGS)); }

// A 4-byte asynchronous copy global -> shared, zero-filled when !ok (src is then not read), and
// an arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) { return __uint_as_float(ld_shared_u32(addr)); }

// Lane 0 arrives on a barrier of the cluster (address from mapa), predicated rather than
// branched to.  The release is of CTA scope: what it orders are the warp's tensor-memory loads,
// complete by tcgen05.wait::ld; with cluster scope every arrival waited for the warp's
// outstanding global and local accesses.
__device__ __forceinline__ void arrive_lane0(uint32_t cluster_bar, int lane) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" :: "r"(cluster_bar), "r"(lane) : "memory");
}

// GELU(tanh) of two values for fp32 output: z / (1 + e^-2u), which equals z/2 (1 + tanh u) and loses nothing where
// 1 + tanh u cancels; -2u log2(e) is one polynomial, e^-2u and the reciprocal are the hardware's, good to 22 bits and
// more.  (gelu_tanh_f32x2 takes the hardware's tanh, off by up to 2^-11.  4096^3 with fp32 output and GELU: 78 us with
// that tanh, 82 with this, 105 with expf and an IEEE division.)
__device__ __forceinline__ void gelu_full_f32x2(float& a, float& b) {
    constexpr float K0 = -2.302208198144325f, K1 = -0.10294323958f;      // -2 log2(e) sqrt(2/pi), and that times 0.044715
    const uint64_t z = ptx::f32x2_pack(a, b);
    const uint64_t poly = ptx::f32x2_fma(ptx::f32x2_pack(K1, K1), ptx::f32x2_mul(z, z), ptx::f32x2_pack(K0, K0));
    float ta, tb;
    ptx::f32x2_unpack(ptx::f32x2_mul(z, poly), ta, tb);
    a *= ptx::rcp_approx(1.0f + ptx::ex2_approx(ta));
    b *= ptx::rcp_approx(1.0f + ptx::ex2_approx(tb));
}

// GELU of two values that are stored as fp32 (F32) or rounded to 16 bits
template <bool F32>
__device__ __forceinline__ void gelu2(float& a, float& b) {
    if constexpr (F32) gelu_full_f32x2(a, b);
    else gelu_tanh_f32x2(a, b);
}

// Where a lane of an epilogue warp stores: four lanes to a row, four columns a lane, rows
// lane / 4, + 8, + 16, + 24 of the warp's 32.
struct StorePlan {
    uint8_t* at;            // this lane's first row, the warp's first column + 4 (lane % 4)
    int64_t row_step;       // bytes to eight rows down
    int rows;               // of its four rows, those inside C
    int cols;               // columns of C from `at` on (may exceed the warp's)
    const uint16_t* bias;   // of the column at `at`, or null
};

__device__ __forceinline__ void st_global_if(bool p, void* at, uint32_t a, uint32_t b) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.global.cs.v2.b32 [%1], {%2, %3};\n\t}"
                 :: "r"(static_cast<uint32_t>(p)), "l"(at), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_global_if(bool p, void* at, const float4& w) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.global.cs.v4.f32 [%1], {%2, %3, %4, %5};\n\t}"
                 :: "r"(static_cast<uint32_t>(p)), "l"(at), "f"(w.x), "f"(w.y), "f"(w.z), "f"(w.w) : "memory");
}

// 16 columns of 32 rows.  v holds one row a lane; the rows go through 2 KiB of shared memory
// (16-byte chunks swizzled by the row, so that neither side has bank conflicts) and come back
// four lanes to a row, where bias, GELU and rounding take place.  For what store_whole does not
// take: ragged columns, unaligned rows, fp16.
__device__ __forceinline__ void store16(const float* v, uint32_t stage, const StorePlan& sp, int chunk, int epi, uint32_t flags,
                                        bool whole, int lane) {
    __syncwarp();                         // the previous chunk has been read back
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                     :: "r"(stage + lane * 64 + ((static_cast<uint32_t>(j) ^ (lane >> 1 & 3u)) << 4)), "f"(v[4 * j]),
                        "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3]) : "memory");
    __syncwarp();
    const int cols = sp.cols - chunk * 16;
    // row i * 8 + lane / 4, chunk lane % 4; eight rows on, the swizzle is the same
    const uint32_t from = stage + (lane / 4) * 64 + ((static_cast<uint32_t>(lane % 4) ^ (lane >> 3 & 3u)) << 4);
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ptx::ld_shared_f4(from + i * 512);
    if (epi != EPI_NONE) {
        float b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b[i] = i < cols ? __uint_as_float(static_cast<uint32_t>(__ldg(sp.bias + chunk * 16 + i)) << 16) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) { w[i].x += b[0]; w[i].y += b[1]; w[i].z += b[2]; w[i].w += b[3]; }
        if (epi == EPI_BIAS_GELU) {
            if (flags & FLAG_C_F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) { gelu2<true>(w[i].x, w[i].y); gelu2<true>(w[i].z, w[i].w); }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) { gelu2<false>(w[i].x, w[i].y); gelu2<false>(w[i].z, w[i].w); }
            }
        }
    }
    uint8_t* at = sp.at + chunk * (flags & FLAG_C_F32 ? 64 : 32);
    if (flags & FLAG_C_F32) {
        if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global_if(i < sp.rows, at + i * sp.row_step, w[i]);
        } else {
#pragma unroll 1
            for (int i = 0; i < 4 && i < sp.rows; ++i) {
                float* c = reinterpret_cast<float*>(at + i * sp.row_step);
                const float4 y = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
                if (cols > 0) c[0] = y.x;
                if (cols > 1) c[1] = y.y;
                if (cols > 2) c[2] = y.z;
                if (cols > 3) c[3] = y.w;
            }
        }
        return;
    }
    uint32_t lo[4], hi[4];
    if (flags & FLAG_C_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) { lo[i] = pack_f16x2(w[i].x, w[i].y); hi[i] = pack_f16x2(w[i].z, w[i].w); }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) { lo[i] = pack_bf16x2(w[i].x, w[i].y); hi[i] = pack_bf16x2(w[i].z, w[i].w); }
    }
    if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) st_global_if(i < sp.rows, at + i * sp.row_step, lo[i], hi[i]);
    } else {
#pragma unroll 1
        for (int i = 0; i < 4 && i < sp.rows; ++i) {
            uint16_t* c = reinterpret_cast<uint16_t*>(at + i * sp.row_step);
            const uint32_t l = i == 0 ? lo[0] : i == 1 ? lo[1] : i == 2 ? lo[2] : lo[3];
            const uint32_t u = i == 0 ? hi[0] : i == 1 ? hi[1] : i == 2 ? hi[2] : hi[3];
            if (cols > 0) c[0] = static_cast<uint16_t>(l);
            if (cols > 1) c[1] = static_cast<uint16_t>(l >> 16);
            if (cols > 2) c[2] = static_cast<uint16_t>(u);
            if (cols > 3) c[3] = static_cast<uint16_t>(u >> 16);
        }
    }
}

// Scales first .. first + COUNT of `blocks` k-blocks into lines of COUNT floats; those past `limit` are zero.
// wide: four of a line are one aligned 16-byte word, a quarter of the copies (the weight gradient of 1536 x
// 4096 over 5000 rows 56.0 us with them, 57.0 without).
__device__ __forceinline__ bool lines_are_wide(const float* s, int64_t mn, int64_t k) {
    return mn == 1 && k % 4 == 0 && reinterpret_cast<uintptr_t>(s) % 16 == 0;
}
template <int COUNT>
__device__ __forceinline__ void scale_lines(uint32_t dst, const float* s, int first, int limit, int shift, int64_t mn,
                                            int64_t k, int kb, int blocks, bool wide, int lane) {
    if (wide) {
#pragma unroll
        for (int j = 0; j < COUNT; j += 128) {
            const int at = first + j + lane * 4, left = min(max(limit - at, 0), 4);
            const float* src = left > 0 ? s + at + kb * k : s;
            for (int i = 0; i < blocks; ++i)
                ptx::cp_async_16_part(dst + (i * COUNT + j + lane * 4) * 4, left > 0 ? src + i * k : s, left * 4);
        }
    } else {
#pragma unroll
        for (int j = 0; j < COUNT; j += 32) {
            const int64_t at = first + j + lane;
            const bool in = at < limit;
            const float* src = in ? s + (at >> shift) * mn + kb * k : s;
            for (int i = 0; i < blocks; ++i) cp_async_4(dst + (i * COUNT + j + lane) * 4, in ? src + i * k : s, in);
        }
    }
}

// From the lanes' rows and columns of tmem_ld_16x256b to a row a lane, 16 columns at a time through this
// warp's staging rows of 64 bytes: v[16 c + 8 (rows / 16) + 4 (columns / 8 % 2) + e] holds row
// lane / 4 + 8 (e / 2) of its 16 and column 2 (lane % 4) + e % 2 of its 8; v[n] is column n after.
template <int COLS>
__device__ __forceinline__ void turn(float* v, uint32_t stage, int lane) {
    // a row's four 16-byte units are swapped by its bits 1 and 2, crossed, so that neither the eight
    // bytes a lane writes (rows lane / 4) nor the sixteen it reads (row lane) meet in a bank
    const uint32_t w_swz = static_cast<uint32_t>(lane >> 3 & 1) * 2 + static_cast<uint32_t>(lane >> 4 & 1);
    const uint32_t r_swz = static_cast<uint32_t>(lane >> 1 & 1) * 2 + static_cast<uint32_t>(lane >> 2 & 1);
#pragma unroll
    for (int c = 0; c < COLS; c += 16) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t row = static_cast<uint32_t>(lane / 4 + i % 2 * 8 + i / 4 * 16);
            const uint32_t unit = static_cast<uint32_t>(i / 2 % 2 * 2 + lane % 4 / 2) ^ w_swz;
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};"
                         :: "r"(stage + row * 64 + (unit << 4) + (lane & 1) * 8),
                            "f"(v[c + i / 4 * 8 + i / 2 % 2 * 4 + i % 2 * 2]),
                            "f"(v[c + i / 4 * 8 + i / 2 % 2 * 4 + i % 2 * 2 + 1]) : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float4 w = ptx::ld_shared_f4(stage + lane * 64 + ((static_cast<uint32_t>(u) ^ r_swz) << 4));
            v[c + 4 * u] = w.x; v[c + 4 * u + 1] = w.y; v[c + 4 * u + 2] = w.z; v[c + 4 * u + 3] = w.w;
        }
    }
    __syncwarp();
}

// COLS columns of 32 rows, all inside C, 16-byte aligned, fp32 or bf16: straight code without a branch
// (rows past the end are predicated off).  Code runs once a tile here and every taken branch costs
// an instruction fetch: with branches around the types and epilogues of each store, a 128 x 256
// part of a tile took 5500 to 8000 cycles to store.
template <bool F32, int EPI, int COLS>
__device__ __forceinline__ void store_whole(const float* v, uint32_t stage, const StorePlan& sp, int lane) {
    const uint32_t to = stage + lane * 64, sw = lane >> 1 & 3u;
    const uint32_t from = stage + (lane / 4) * 64 + ((static_cast<uint32_t>(lane % 4) ^ (lane >> 3 & 3u)) << 4);
    if constexpr (!F32 && EPI == EPI_NONE) {
        // rounded first: 32 columns a pass, eight of a row in a lane afterwards (sp counts columns in
        // fours: this lane's eight start another 4 (lane % 4) columns on)
        uint8_t* at = sp.at + (lane % 4) * 8;
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                             :: "r"(to + ((static_cast<uint32_t>(j) ^ sw) << 4)), "r"(pack_bf16x2(v[c + 8 * j], v[c + 8 * j + 1])),
                                "r"(pack_bf16x2(v[c + 8 * j + 2], v[c + 8 * j + 3])),
                                "r"(pack_bf16x2(v[c + 8 * j + 4], v[c + 8 * j + 5])),
                                "r"(pack_bf16x2(v[c + 8 * j + 6], v[c + 8 * j + 7])) : "memory");
            __syncwarp();
            float4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ptx::ld_shared_f4(from + i * 512);
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global_if(i < sp.rows, at + i * sp.row_step + c * 2, w[i]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < COLS; c += 16) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                             :: "r"(to + ((static_cast<uint32_t>(j) ^ sw) << 4)), "f"(v[c + 4 * j]), "f"(v[c + 4 * j + 1]),
                                "f"(v[c + 4 * j + 2]), "f"(v[c + 4 * j + 3]) : "memory");
            __syncwarp();
            float4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ptx::ld_shared_f4(from + i * 512);
            if constexpr (EPI != EPI_NONE) {
                float b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = __uint_as_float(static_cast<uint32_t>(__ldg(sp.bias + c + i)) << 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i].x += b[0]; w[i].y += b[1]; w[i].z += b[2]; w[i].w += b[3];
                    if constexpr (EPI == EPI_BIAS_GELU) { gelu2<F32>(w[i].x, w[i].y); gelu2<F32>(w[i].z, w[i].w); }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint8_t* at = sp.at + i * sp.row_step + c * (F32 ? 4 : 2);
                if constexpr (F32) st_global_if(i < sp.rows, at, w[i]);
                else st_global_if(i < sp.rows, at, pack_bf16x2(w[i].x, w[i].y), pack_bf16x2(w[i].z, w[i].w));
            }
        }
    }
}

// Bias, GELU, rounding and the store of eight neighbouring columns of one row.
__device__ __forceinline__ void finish_and_store8(float (&v)[8], const Problem& pr, const Fp8Params& x, int row, int n) {
    if (row >= pr.M || n >= pr.N) return;
    if (pr.epi != EPI_NONE) {
        float b[8];
        load_bias8(static_cast<const uint16_t*>(pr.bias), n, pr.N, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += b[i];
        if (pr.epi == EPI_BIAS_GELU) {
            if (pr.flags & FLAG_C_F32) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) gelu2<true>(v[i], v[i + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) gelu2<false>(v[i], v[i + 1]);
            }
        }
    }
    const int64_t at = static_cast<int64_t>(row) * x.ldc + n;
    const bool whole = x.vec_c && n + 8 <= pr.N;
    if (pr.flags & FLAG_C_F32) {
        float* c = static_cast<float*>(x.c) + at;
        if (whole) {
            reinterpret_cast<float4*>(c)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(c)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n + i < pr.N) c[i] = v[i];
        }
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (pr.flags & FLAG_C_F16) ? pack_f16x2(v[2 * i], v[2 * i + 1]) : pack_bf16x2(v[2 * i], v[2 * i + 1]);
    uint16_t* c = static_cast<uint16_t*>(x.c) + at;
    if (whole) {
        *reinterpret_cast<uint4*>(c) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < pr.N) c[i] = static_cast<uint16_t>(w[i / 2] >> ((i & 1) * 16));
    }
}

}  // namespace f8

// ----------------------------------------------------------------------------------------

template <class Cfg>
__global__ void __launch_bounds__(F8_THREADS, 1) fp8_kernel(const __grid_constant__ Params p,
                                                            const __grid_constant__ Fp8Params x) {
    constexpr int STAGES = Cfg::STAGES;
    constexpr int CG = Cfg::CTA_GROUP;
    constexpr int BN = Cfg::BN;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t sA = base + Cfg::OFF_A, sB = base + Cfg::OFF_B, sC = base + Cfg::OFF_C;
    const uint32_t bar0 = base + Cfg::OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
    auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 6 + s); };
    auto sempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 6 + Cfg::SLOTS + s); };
    const uint32_t sS = base + Cfg::OFF_SCALE;
    const uint32_t abort_addr = base + Cfg::OFF_ABORT;

    // broadcast, so that the compiler knows the warp's index and what follows from it as uniform
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const uint32_t cta = ptx::cluster_ctarank();              // in the cluster: of a pair, or of a split tile
    const int splits = Cfg::SPLIT ? x.splits : 1;
    const int unit = blockIdx.x / (CG * splits), num_units = gridDim.x / (CG * splits);
    // this CTA's k-blocks of every tile
    const int kb_begin = Cfg::SPLIT ? static_cast<int>(static_cast<int64_t>(p.dense.k_blocks) * cta / splits) : 0;
    const int kb_end = Cfg::SPLIT ? static_cast<int>(static_cast<int64_t>(p.dense.k_blocks) * (cta + 1) / splits)
                                  : p.dense.k_blocks;

    // ---- set-up
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(tfull_bar(b), 1);
            ptx::mbar_init(tempty_bar(b), F8_EPI_WARPS * CG);
        }
        for (int s = 0; s < Cfg::SLOTS; ++s) {
            ptx::mbar_init(sfull_bar(s), 32);                 // every lane of the loader
            ptx::mbar_init(sempty_bar(s), F8_EPI_WARPS);
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::mbar_init(drain_bar + 8u, 1);
        st_shared_u32(abort_addr, 0u);
        st_shared_u32(base + Cfg::OFF_DRAIN_FLAG, 0u);
        st_shared_u32(base + Cfg::OFF_DRAIN_POS, 0u);
        for (int s = 0; s < MAX_STAGES; ++s) {
            st_shared_u32(base + Cfg::OFF_DRAIN_LAST + 4 * s, 0xffffffffu);
            st_shared_u32(base + Cfg::OFF_DRAIN_BYTES + 4 * s, 0u);
        }
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&p.dense.tma_a);
        ptx::prefetch_tensormap(&p.dense.tma_b);
    }
    if (warp == 1) {
        ptx::tmem_alloc<CG>(base + Cfg::OFF_TMEM_SLOT, Cfg::TMEM_COLS);
        ptx::tmem_relinquish<CG>();
    }
    MoeTable mt{};
    if constexpr (Cfg::MOE) {
        int32_t* tile_pref = reinterpret_cast<int32_t*>(smem + Cfg::OFF_TABLE);
        int32_t* row_off = tile_pref + (MOE_MAX_G + 1);
        if (warp == 2) {
            const int32_t n = f8::build_moe_table(p, Cfg::TILE_M, p.dense.tiles_n, tile_pref, row_off, lane);
            if (lane == 0) *reinterpret_cast<volatile int32_t*>(smem + Cfg::OFF_MOE_TOTAL) = n;
        }
        mt.tile_pref = tile_pref;
        mt.row_off = row_off;
    }
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2) ptx::cluster_sync(); else __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_TMEM_SLOT);
    int total_tiles = static_cast<int>(p.total_tiles);
    if constexpr (Cfg::MOE) total_tiles = *reinterpret_cast<volatile int32_t*>(smem + Cfg::OFF_MOE_TOTAL);

    // The last, partial wave of a pair launch: its R = tiles mod units tiles, when two of them fit a
    // unit each, run as 2R half tiles (128 rows of a pair, 64 a CTA), items whole, whole + 1, ..
    constexpr bool MAY_HALVE = CG == 2;
    const int last_wave = MAY_HALVE && x.halves ? total_tiles % num_units : 0;
    const int halved = 2 * last_wave <= num_units ? last_wave : 0;
    const int whole = total_tiles - halved, items = total_tiles + halved;
    auto tile_of = [&](int t) { return MAY_HALVE && t >= whole ? whole + (t - whole) % halved : t; };
    // tile_coord in 32 bits (the host refuses more than 2^30 tiles): with 64-bit divisions it took the
    // accumulating warps 1300 to 1900 cycles a tile, so ~800.
    auto coord_of_item = [&](int t, int g) {
        int local = tile_of(t), tiles_m = p.dense.tiles_m, rows_left = p.dense.M;
        TileCoord c;
        c.g = g;
        c.m0 = 0;
        c.row_end = INT32_MAX;
        if constexpr (Cfg::MOE) {
            local -= mt.tile_pref[g];
            c.m0 = mt.row_off[g];
            c.row_end = mt.row_off[g + 1];
            rows_left = c.row_end - c.m0;
            tiles_m = (rows_left + Cfg::TILE_M - 1) / Cfg::TILE_M;
        }
        // bands of p.band N-tiles, as raster()
        const int per_band = tiles_m * p.band, bi = local / per_band, r = local - bi * per_band;
        const int left = p.dense.tiles_n - bi * p.band, width = left < p.band ? left : p.band;
        const int row = r / width, mb = (bi & 1) ? tiles_m - 1 - row : row;
        c.n0 = (bi * p.band + r - row * width) * BN;
        c.half = MAY_HALVE && Cfg::MOE && rows_left - mb * Cfg::TILE_M <= BM;
        c.m0 += mb * Cfg::TILE_M + static_cast<int>(rank) * (c.half ? BM / 2 : BM);
        if (MAY_HALVE && t >= whole) {
            // (an expert's tile of at most 128 rows is a half tile already: its second half is empty)
            if (!c.half) c.m0 -= static_cast<int>(rank) * (BM / 2);
            c.m0 += (t - whole) / halved * BM;
            c.half = true;
        }
        return c;
    };
    const Problem& pr = p.dense;
    // Warp-uniform bounded wait: every lane polls once; if the phase is not yet complete, lane 0
    // runs the bounded wait and tells the others how it ended.  (Polling more than once before
    // that, or by lane 0 alone, was slower: 730 and 795 us at 8192^3 when this form took 470.)
    auto warp_wait = [&](uint32_t bar, uint32_t par, uint32_t role, int tile, uint32_t st) -> bool {
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, par))) return true;
        uint32_t ok = 1;
        if (lane == 0) ok = wait_bounded<CG, false>(bar, par, p, abort_addr, role, tile, st) ? 1u : 0u;
        return __shfl_sync(0xffffffffu, ok, 0) != 0;
    };
    // Registers: 384 x 168 at launch = 64512 = 128 x 72 + 256 x 216.  Each split stands at the head of
    // its own branch: after a common one the compiler kept to the smaller count.
    if (warp < F8_EPI_WARP0) {
    f8::regs_dec<72>();
    if (warp == 0) {
        // ================================ TMA producer ================================
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, pos = 0;
            int g = 0;
            bool aborted = false;
            bool withhold = p.withhold_kb >= 0 && blockIdx.x == static_cast<uint32_t>(p.withhold_block);
            const uint32_t tx = x.a_bytes + Cfg::B_BYTES;
            for (int t = unit; t < items && !aborted; t += num_units) {
                g = find_problem<Cfg>(p, tile_of(t), g, mt);
                const TileCoord tc = coord_of_item(t, g);
                const int nb0 = tc.n0 + static_cast<int>(rank) * Cfg::BN_CTA;
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    if (!ptx::mbar_test_wait(empty_bar(stage), phase ^ 1u) &&
                        !wait_bounded<CG>(empty_bar(stage), phase ^ 1u, p, abort_addr, ROLE_PRODUCER, t, stage)) {
                        aborted = true;
                        break;
                    }
                    if (!(withhold && kb == p.withhold_kb)) {
                        const uint32_t fb = CG == 2 ? ptx::mapa(full_bar(stage), 0) : full_bar(stage);
                        if (leader) ptx::mbar_arrive_expect_tx(full_bar(stage), tx * CG);
                        const int k0 = kb * F8_BK;
                        const uint32_t a_dst = sA + stage * Cfg::A_BYTES, b_dst = sB + stage * Cfg::B_BYTES;
                        const int ax = x.a_mn ? tc.m0 : k0, ay = x.a_mn ? k0 : tc.m0;
                        const int bx = x.b_mn ? nb0 : k0, by = x.b_mn ? k0 : nb0;
                        if constexpr (CG == 2) ptx::tma_load_2d_pair(a_dst, &pr.tma_a, ax, ay, fb);
                        else ptx::tma_load_2d(a_dst, &pr.tma_a, ax, ay, fb);
                        if constexpr (Cfg::MOE) {
                            if constexpr (CG == 2) ptx::tma_load_3d_pair(b_dst, &pr.tma_b, bx, by, g, fb);
                            else ptx::tma_load_3d(b_dst, &pr.tma_b, bx, by, g, fb);
                        } else {
                            if constexpr (CG == 2) ptx::tma_load_2d_pair(b_dst, &pr.tma_b, bx, by, fb);
                            else ptx::tma_load_2d(b_dst, &pr.tma_b, bx, by, fb);
                        }
                        st_shared_u32(base + Cfg::OFF_DRAIN_LAST + 4 * stage, pos);
                        st_shared_u32(base + Cfg::OFF_DRAIN_BYTES + 4 * stage, tx);
                    }
                    ++pos;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                withhold = false;
            }
            if (!aborted) {
                // Tail: every slot released, so no commit arrives here after this CTA leaves.
                for (int i = 0; i < STAGES; ++i) {
                    if (!wait_bounded<CG>(empty_bar(stage), phase ^ 1u, p, abort_addr, ROLE_PRODUCER, -1, stage)) {
                        aborted = true;
                        break;
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            st_shared_u32(base + Cfg::OFF_DRAIN_POS, pos);
            ptx::st_release_cluster_u32(base + Cfg::OFF_DRAIN_FLAG, 1u);
            if (aborted && leader) drain_issued_loads<Cfg>(p, base);
        }
    } else if (warp == 1 || warp == 2) {
        // ================================ MMA issuers ================================
        // Warp 1 issues the even k-blocks (into TMEM buffer 0), warp 2 the odd ones (buffer 1): the
        // waits, four MMAs and two commits of a k-block take one warp about 520 cycles, as long as
        // the MMAs of a 256 x 256 tile and twice as long as those of a 128 x 128 one.
        if (leader) {
            const int mine = warp - 1;
            int stage = mine, g = 0, before = 0;       // k-blocks of the tiles before this one
            uint32_t phase = 0, acc_phase = 0;
            bool aborted = false, any_mma = false;
            // 8-row (K-major) or 8-k (MN-major) groups are 1024 bytes apart; the next 32 k of a
            // stage are 32 bytes along the row, or 32 rows of 128 bytes down
            const uint64_t a_desc0 = ptx::smem_desc_sw128(sA, 16, 1024), b_desc0 = ptx::smem_desc_sw128(sB, 16, 1024);
            const uint64_t a_step = x.a_mn ? 4096u >> 4 : 32u >> 4, b_step = x.b_mn ? 4096u >> 4 : 32u >> 4;
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(mine * BN);
            const uint32_t tfull = tfull_bar(mine), tempty = tempty_bar(mine);
            for (int t = unit; t < items && !aborted; t += num_units) {
                g = find_problem<Cfg>(p, tile_of(t), g, mt);
                uint32_t idesc = pr.idesc;
                if (coord_of_item(t, g).half) idesc = (idesc & ~(0x1Fu << 24)) | ((128u >> 4) << 24);
                for (int i = (mine ^ before) & 1; i < kb_end - kb_begin; i += 2) {
                    // both barriers are asked before either answer is needed
                    const bool filled = ptx::mbar_test_wait(full_bar(stage), phase);
                    const bool drained = ptx::mbar_test_wait(tempty, acc_phase ^ 1u);
                    if (!__all_sync(0xffffffffu, filled && drained) &&
                        (!warp_wait(full_bar(stage), phase, ROLE_MMA, t, stage) ||
                         !warp_wait(tempty, acc_phase ^ 1u, ROLE_MMA, t, 16 + mine))) {
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    f8::mma_block<CG>(d_tmem, a_desc0 + static_cast<uint64_t>((stage * Cfg::A_BYTES) >> 4),
                                      b_desc0 + static_cast<uint64_t>((stage * Cfg::B_BYTES) >> 4), a_step, b_step, idesc,
                                      empty_bar(stage), tfull);
                    any_mma = true;
                    stage += 2;
                    if (stage >= STAGES) { stage -= STAGES; phase ^= 1u; }
                    acc_phase ^= 1u;
                }
                before += kb_end - kb_begin;
            }
            if (aborted && any_mma && lane == 0) {
                const uint32_t bar = drain_bar + 8u * mine;
                if constexpr (CG == 2) ptx::mma_commit_pair(bar, 0x1);
                else ptx::mma_commit(bar);
                if (!wait_quiet(bar, 0, p.wait_budget_ns)) report_timeout(p, ROLE_DRAIN, -1, 0, p.wait_budget_ns);
            }
            __syncwarp();
        }
    } else {
        // ================================ scale loader ================================
        // A slot: the scales of F8_GROUP k-blocks: [128 rows][k-block] of A, then [block of 128
        // columns][k-block] of B; with column scales [k-block][rows], then [k-block][columns].
        [[maybe_unused]] const bool wide_a = x.sa_shift == 0 && f8::lines_are_wide(x.sa, x.sa_mn, x.sa_k);
        [[maybe_unused]] const bool wide_b = f8::lines_are_wide(x.sb, x.sb_mn, x.sb_k);
        int slot = 0, g = 0;
        uint32_t phase = 0;
        bool aborted = false;
        for (int t = unit; t < items && !aborted; t += num_units) {
            g = find_problem<Cfg>(p, tile_of(t), g, mt);
            const TileCoord tc = coord_of_item(t, g);
            for (int kb = kb_begin; kb < kb_end; kb += F8_GROUP) {
                if (!warp_wait(sempty_bar(slot), phase ^ 1u, ROLE_PRODUCER, t, 32 + slot)) {
                    aborted = true;
                    break;
                }
                const uint32_t dst = sS + slot * Cfg::SLOT_BYTES, dst_b = dst + BM * F8_GROUP * 4;
                if constexpr (Cfg::SB_COL) {
                    const int blocks = min(F8_GROUP, kb_end - kb);
                    f8::scale_lines<BM>(dst, x.sa, tc.m0, pr.M, x.sa_shift, x.sa_mn, x.sa_k, kb, blocks, wide_a, lane);
                    f8::scale_lines<BN>(dst_b, x.sb, tc.n0, pr.N, 0, x.sb_mn, x.sb_k, kb, blocks, wide_b, lane);
                } else {
#pragma unroll
                    for (int j = 0; j < BM / 32; ++j) {
                        const int64_t row = tc.m0 + j * 32 + lane;
                        const bool in = row < pr.M;
                        const float* src = in ? x.sa + (row >> x.sa_shift) * x.sa_mn + kb * x.sa_k : x.sa;
#pragma unroll
                        for (int i = 0; i < F8_GROUP; ++i)
                            if (kb + i < kb_end)
                                f8::cp_async_4(dst + ((j * 32 + lane) * F8_GROUP + i) * 4, in ? src + i * x.sa_k : src, in);
                    }
                    if (lane < Cfg::SB_COUNT * F8_GROUP) {
                        const int64_t n = tc.n0 + lane / F8_GROUP * 128;
                        const int i = lane % F8_GROUP;
                        const bool in = n < pr.N && kb + i < kb_end;
                        f8::cp_async_4(dst_b + lane * 4,
                                       in ? x.sb + (n >> 7) * x.sb_mn + (kb + i) * x.sb_k + (Cfg::MOE ? g * x.sb_g : 0) : x.sb, in);
                    }
                }
                f8::cp_async_arrive(sfull_bar(slot));
                if (++slot == Cfg::SLOTS) { slot = 0; phase ^= 1u; }
            }
        }
        ptx::cp_async_commit();
        ptx::cp_async_wait<0>();              // nothing lands after this warp has left
    }
    } else {
        f8::regs_inc<216>();
        // ================================ accumulation and epilogue ================================
        constexpr int COLS = Cfg::COLS;
        const int q = warp % 4, h = (warp - F8_EPI_WARP0) / 4;
        const uint32_t stage_c = sC + (warp - F8_EPI_WARP0) * F8_C_STAGE;
        int buf = 0, slot = 0, g = 0;
        uint32_t buf_phase = 0, slot_phase = 0;
        const uint32_t lead_tempty = ptx::mapa(tempty_bar(0), CG == 2 ? 0 : cta), own_sempty = ptx::mapa(sempty_bar(0), cta);
        for (int t = unit; t < items; t += num_units) {
            g = find_problem<Cfg>(p, tile_of(t), g, mt);
            const TileCoord tc = coord_of_item(t, g);
            // a half tile keeps 64 rows in lanes 0-63 (columns [0, BN/2)) and again in lanes 64-127
            // (columns [BN/2, BN)), in BN/2 TMEM columns: the two warps of a quarter split those
            const int local_row = tc.half ? (q % 2) * 32 : q * 32;
            const int local_col = tc.half ? (q / 2) * (BN / 2) + h * (BN / 4) : h * COLS;
            const int row0 = tc.m0 + local_row, n0 = tc.n0 + local_col;
            const uint32_t t_col = static_cast<uint32_t>(tc.half ? h * (BN / 4) : h * COLS);
            const int n_cols = tc.half ? COLS / 2 : COLS;
            int row_limit = pr.M;
            if constexpr (Cfg::MOE) row_limit = static_cast<int>(min(static_cast<int64_t>(tc.row_end), p.moe_rows));
            const bool active = row0 < row_limit && n0 < pr.N;
            const uint32_t tm0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + t_col;
            const uint32_t sa_at = sS + (Cfg::SB_COL ? local_row + lane / 4 : (local_row + lane) * F8_GROUP) * 4;
            const uint32_t sb_at = sS + BM * F8_GROUP * 4 +
                                   (Cfg::SB_COL ? local_col + lane % 4 * 2 : (local_col >> 7) * F8_GROUP) * 4;

            float acc[COLS];
#pragma unroll
            for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;
            // Block scales: a lane has one row, acc[32 C ..] += scale * partial columns [32 C, 32 C + 32).
            // Column scales: chunk C holds 64 columns of 16 rows, of which a lane has two rows and two
            // columns of every eight, so that it needs 16 of the columns' scales (fc), which serve the
            // next 16 rows too.  (With a row a lane every lane read all of them: 16 KB a warp and k-block
            // out of shared memory, 1024 cycles at 128 bytes a cycle for the eight warps; 8192^3 took
            // 744 us and takes 620, or up to 690 at the power limit.)  acc keeps 16 columns together, in the order turn() takes.
            // Scalar: a warp's fused multiply-add measured 1.03 issue cycles, a packed pair of them 2.34.
            auto add = [&](auto chunk_index, const uint32_t (&r)[32], const float* s, const float* fc) {
                constexpr int C = decltype(chunk_index)::value;
                if constexpr (Cfg::SB_COL) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float& sum = acc[(C / 2 * 4 + j / 2) * 16 + C % 2 * 8 + j % 2 * 4 + e];
                            sum = fmaf(__uint_as_float(r[4 * j + e]) * fc[2 * j + e % 2], s[C % 2 * 2 + e / 2], sum);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[C * 32 + i] = fmaf(__uint_as_float(r[i]), s[0], acc[C * 32 + i]);
                }
            };
            // Chunk C of the buffer at tm, into r
            auto load = [&](auto chunk_index, uint32_t tm, uint32_t (&r)[32]) {
                constexpr int C = decltype(chunk_index)::value;
                if constexpr (Cfg::SB_COL) ptx::tmem_ld_16x256b_x8(tm + C / 2 * 64 + (static_cast<uint32_t>(C % 2 * 16) << 16), r);
                else ptx::tmem_ld_32x32b_x32(tm + C * 32, r);
            };
            // Waits for the next slot.  Block scales: this lane's scales of four k-blocks (times B's, one
            // for all the warp's columns).  Read once per group, a k-block ahead: shared memory answers
            // slowly while the tensor cores and TMA use it.
            auto read_scales = [&](float (&f)[F8_GROUP]) -> bool {
                if (!warp_wait(sfull_bar(slot), slot_phase, ROLE_EPILOGUE, t, 32 + slot)) return false;
                if constexpr (!Cfg::SB_COL) {
                    const uint32_t off = slot * Cfg::SLOT_BYTES;
                    const float4 a = ptx::ld_shared_f4(sa_at + off);
                    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
                    const float4 b = ptx::ld_shared_f4(sb_at + off);
                    f[0] *= b.x; f[1] *= b.y; f[2] *= b.z; f[3] *= b.w;
                    __syncwarp();
                    f8::arrive_lane0(own_sempty + 8u * slot, lane);
                    if (++slot == Cfg::SLOTS) { slot = 0; slot_phase ^= 1u; }
                }
                return true;
            };
            // All k-blocks over the first 32 * CHUNKS columns of this warp (none: it only keeps the
            // barriers going).
            auto accumulate = [&](auto chunk_count) -> bool {
                constexpr int CHUNKS = decltype(chunk_count)::value;
                static_assert(F8_GROUP == 4, "a lane's scales of a group are one 16-byte word");
                float f[F8_GROUP];
                if (kb_begin == kb_end) return true;
                if (!read_scales(f)) return false;
                // (Asking for the next buffer's first chunk ahead of the last additions cost spills in both
                // forms: 623 us instead of 418 at 8192^3, with column scales 810 instead of 644.)
                uint32_t r[2][32];
                bool ready = ptx::mbar_test_wait(tfull_bar(buf), buf_phase);
                auto open = [&]() -> bool {
                    if (!__all_sync(0xffffffffu, ready) &&
                        !warp_wait(tfull_bar(buf), buf_phase, ROLE_EPILOGUE, t, 16 + buf)) return false;
                    ptx::tc_fence_after_sync();
                    if constexpr (CHUNKS > 0) load(std::integral_constant<int, 0>{}, tm0 + static_cast<uint32_t>(buf * BN), r[0]);
                    return true;
                };
                // One k-block, the u-th of its group
                auto block = [&](int u, bool more) -> bool {
                    const uint32_t tm = tm0 + static_cast<uint32_t>(buf * BN);
                    float s[Cfg::SB_COL ? 4 : 1];
                    [[maybe_unused]] float fc[16];
                    [[maybe_unused]] const uint32_t sb = sb_at + slot * Cfg::SLOT_BYTES + u * (BN * 4);   // SB_COL
                    if constexpr (Cfg::SB_COL) {
#pragma unroll
                        for (int i = 0; i < (CHUNKS > 0 ? 4 : 0); ++i)
                            s[i] = f8::ld_shared_f32(sa_at + slot * Cfg::SLOT_BYTES + u * (BM * 4) + i * 32);
                    } else {
                        s[0] = f[0];
                        f[0] = f[1]; f[1] = f[2]; f[2] = f[3];
                        if (u == F8_GROUP - 1 && more && !read_scales(f)) return false;
                    }
                    f8::for_each<(CHUNKS > 0 ? CHUNKS : 1)>([&](auto ci) {
                        constexpr int C = decltype(ci)::value;
                        if constexpr (CHUNKS > 0) f8::tmem_ld_wait32(r[C & 1]);
                        if constexpr (C + 1 < CHUNKS) {
                            load(std::integral_constant<int, C + 1>{}, tm, r[(C + 1) & 1]);
                        } else {
                            // everything is in registers: the buffer goes back to the MMA issuer; the next
                            // one's barrier is asked early, so that the answer is there after the additions
                            ptx::tc_fence_before_sync();
                            f8::arrive_lane0(lead_tempty + 8u * buf, lane);
                            if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                            ready = ptx::mbar_test_wait(tfull_bar(buf), buf_phase);
                        }
                        if constexpr (Cfg::SB_COL && CHUNKS > 0 && C % 2 == 0) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 v = ptx::ld_shared_f2(sb + (C * 32 + j * 8) * 4);
                                fc[2 * j] = v.x;
                                fc[2 * j + 1] = v.y;
                            }
                        }
                        if constexpr (CHUNKS > 0) add(ci, r[C & 1], s, fc);
                    });
                    if constexpr (Cfg::SB_COL) {
                        if (u == F8_GROUP - 1 || !more) {
                            // the columns' scales have been read: on to the next group's slot
                            __syncwarp();
                            f8::arrive_lane0(own_sempty + 8u * slot, lane);
                            if (++slot == Cfg::SLOTS) { slot = 0; slot_phase ^= 1u; }
                            if (more && !read_scales(f)) return false;
                        }
                    }
                    return true;
                };
#pragma unroll 1
                for (int kb = kb_begin; kb < kb_end; ++kb)
                    if (!open() || !block((kb - kb_begin) % F8_GROUP, kb + 1 < kb_end)) return false;
                return true;
            };
            bool ok;
            if (!active) {
                ok = accumulate(std::integral_constant<int, 0>{});
            } else if (MAY_HALVE && tc.half) {
                if constexpr (MAY_HALVE) ok = accumulate(std::integral_constant<int, COLS / 64>{});
            } else {
                ok = accumulate(std::integral_constant<int, COLS / 32>{});
            }
            if (!ok) break;
            if (!active) continue;
            if constexpr (Cfg::SB_COL) f8::turn<COLS>(acc, stage_c, lane);
            if constexpr (Cfg::SPLIT) {
                // the operand ring is idle (the last buffer's commit followed every MMA): leave this
                // warp's sums there, [column][row], for the cluster
                const uint32_t mine = sA + static_cast<uint32_t>(warp - F8_EPI_WARP0) * (COLS * 128);
#pragma unroll
                for (int j = 0; j < COLS; ++j) st_shared_u32(mine + (j * 32 + lane) * 4, __float_as_uint(acc[j]));
                continue;
            }

            // epilogue, 16 columns at a time
            const int esize = pr.flags & FLAG_C_F32 ? 4 : 2;
            const int first = n0 + (lane % 4) * 4, my_row = row0 + lane / 4;
            f8::StorePlan sp;
            sp.at = static_cast<uint8_t*>(x.c) + (static_cast<int64_t>(my_row) * x.ldc + first) * esize;
            sp.row_step = x.ldc * esize * 8;
            sp.rows = (row_limit - my_row + 7) / 8;            // (at most 0 when this lane has none)
            sp.cols = pr.N - first;
            sp.bias = static_cast<const uint16_t*>(pr.bias) + first + (Cfg::MOE ? static_cast<int64_t>(g) * pr.N : 0);
            if (x.vec_c && n0 + n_cols <= pr.N && !(pr.flags & FLAG_C_F16)) {
                auto whole = [&](auto f32_tag, auto epi_tag) {
                    constexpr bool F32 = decltype(f32_tag)::value;
                    constexpr int EPI = decltype(epi_tag)::value;
                    f8::store_whole<F32, EPI, 64>(acc, stage_c, sp, lane);
                    if constexpr (COLS > 64) {
                        if (n_cols > 64) {
                            sp.at += 64 * esize;
                            sp.bias += 64;
                            f8::store_whole<F32, EPI, 64>(acc + 64, stage_c, sp, lane);
                        }
                    }
                };
                auto with_epi = [&](auto f32_tag) {
                    if (pr.epi == EPI_NONE) whole(f32_tag, std::integral_constant<int, EPI_NONE>{});
                    else if (pr.epi == EPI_BIAS) whole(f32_tag, std::integral_constant<int, EPI_BIAS>{});
                    else whole(f32_tag, std::integral_constant<int, EPI_BIAS_GELU>{});
                };
                if (pr.flags & FLAG_C_F32) with_epi(std::true_type{});
                else with_epi(std::false_type{});
            } else {
                f8::for_each<COLS / 16>([&](auto i) {
                    constexpr int C = decltype(i)::value;
                    if (C * 16 < n_cols && n0 + C * 16 < pr.N)
                        f8::store16(acc + C * 16, stage_c, sp, C, pr.epi, pr.flags, x.vec_c && n0 + C * 16 + 16 <= pr.N, lane);
                });
            }
            __syncwarp();
        }
    }

    if constexpr (Cfg::SPLIT) {
        // ================================ joining a split tile ================================
        // CTA r of the cluster adds columns [r COLS / splits, ..) of every warp's part, in the order
        // of the k ranges, and finishes them.
        __syncwarp();
        ptx::cluster_sync();
        const TileCoord tc = coord_of_item(unit, 0);
        const int ew = warp - F8_EPI_WARP0;
        const int row = tc.m0 + (warp % 4) * 32 + lane, per = Cfg::COLS / splits;
        const int c_first = static_cast<int>(cta) * per;
        const int n_first = tc.n0 + (ew / 4) * Cfg::COLS + c_first;
        if (ew >= 0 && row - lane < pr.M && n_first < pr.N) {
            const uint32_t from = sA + static_cast<uint32_t>(ew) * (Cfg::COLS * 128) + lane * 4;
            for (int c = 0; c < per; c += 8) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.0f;
                for (int r = 0; r < splits; ++r) {
                    const uint32_t at = ptx::mapa(from + static_cast<uint32_t>(c_first + c) * 128, static_cast<uint32_t>(r));
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(ptx::ld_cluster_u32(at + i * 128));
                }
                f8::finish_and_store8(v, pr, x, row, n_first + c);
            }
        }
    }

    // ---- teardown
    __syncwarp();
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2 || Cfg::SPLIT) ptx::cluster_sync(); else __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == 1) ptx::tmem_dealloc<CG>(tmem_base, Cfg::TMEM_COLS);
}

}  // namespace tg
