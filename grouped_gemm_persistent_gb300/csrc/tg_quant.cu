// tg_quant.cu - 8-bit floating point with one scale for each block of 128 values:
// the operands of the 8-bit products (tg_quantize_blocks in include/tg.h).
//
// For a block B (128 values along a row, along a column, or a 128 x 128 square) with
// largest magnitude a and a type whose largest finite value is 1.75 * 2^E (e4m3: E = 8,
// e5m2: E = 15), the scale is the smallest power of two s >= 2^-126 with
// a <= 1.75 * 2^E * s, and q = round(x / s).  With a = m * 2^e, 1 <= m < 2, that is
// s = 2^(e - E) when m <= 1.75 and 2^(e - E + 1) otherwise: read off the bits of a, no
// division.  Scaling by a power of two is exact, so a value is rounded once, to nearest
// even, and dequantising is exact in fp32; the factor of two that a power of two can
// waste costs range (the type has 2^15 of it and more below its top), not precision.
//
// One block of 256 threads reads a tile once into registers (8 rows of 8 columns a thread,
// 16-byte loads), reduces the magnitudes in the wanted direction as integers (the bits of
// non-negative floats order like the values), and writes bytes.  Tiles are 128 x 128, and
// 32 x 512 for blocks along a row, which need no more than a row: 1 KiB of a bf16 row at a
// time instead of 256 bytes.  65536 x 4096 bf16 to e4m3: 115 us,
// 7.1 TB/s (128 x 128 tiles, three blocks an SM: 170 us; 32 x 512: 151; five blocks an SM: 135;
// straight code for inner tiles and a thread a scale instead of a warp a row of them: 115).
// (Five blocks an SM leave 48 registers a thread and cost 20 bytes of spills.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"

namespace tg {

namespace {

enum : int { BLOCK_ROW = 0, BLOCK_COLUMN = 1, BLOCK_SQUARE = 2 };

constexpr int QT = 128;          // values of a scale block
constexpr int QTHREADS = 256;
constexpr int QROWS = 8;         // rows a thread holds (ty, ty + TY, ...)

// Tile of a mode: TX threads of 8 columns by TY of QROWS rows
template <int MODE>
struct QTile {
    static constexpr int TX = MODE == BLOCK_ROW ? 64 : 16;
    static constexpr int TY = QTHREADS / TX;
    static constexpr int COLS = 8 * TX, ROWS = QROWS * TY;
};

// Eight values of one row as they lie in memory, and what is needed of them.
// 16-bit types: magnitudes compare as 15-bit integers.
template <bool F16>
struct Half8 {
    uint32_t w[4];
    static constexpr int BYTES = 2;
    static constexpr uint32_t INF = F16 ? 0x7c00u : 0x7f80u;      // magnitudes from here on are not finite

    __device__ __forceinline__ void load(const void* p) {
        const uint4 t = __ldg(static_cast<const uint4*>(p));
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void set(int i, const void* p) {
        w[i >> 1] |= static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p))) << ((i & 1) * 16);
    }
    __device__ __forceinline__ uint32_t bits(int i) const { return (w[i >> 1] >> ((i & 1) * 16)) & 0xffffu; }
    __device__ __forceinline__ uint32_t mag(int i) const { return bits(i) & 0x7fffu; }
    static __device__ __forceinline__ float widen_value(uint32_t h) {
        if constexpr (F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
        else return __uint_as_float(h << 16);
    }
    __device__ __forceinline__ float value(int i) const { return widen_value(bits(i)); }
    // largest magnitude of the eight
    __device__ __forceinline__ uint32_t max_mag() const {
        const uint32_t a = __vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), b = __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu);
        const uint32_t m = __vmaxu2(a, b);
        return max(m & 0xffffu, m >> 16);
    }
    // fp32 bits of a magnitude (any pattern from infinity's on when it is not finite)
    static __device__ __forceinline__ uint32_t widen(uint32_t m) {
        return m >= INF ? 0x7f800000u : __float_as_uint(widen_value(m));
    }
};

struct Float8 {
    uint32_t w[8];
    static constexpr int BYTES = 4;

    __device__ __forceinline__ void load(const void* p) {
        const uint4 a = __ldg(static_cast<const uint4*>(p));
        const uint4 b = __ldg(static_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void set(int i, const void* p) { w[i] = __ldg(static_cast<const uint32_t*>(p)); }
    __device__ __forceinline__ uint32_t mag(int i) const { return w[i] & 0x7fffffffu; }
    __device__ __forceinline__ float value(int i) const { return __uint_as_float(w[i]); }
    __device__ __forceinline__ uint32_t max_mag() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, mag(i));
        return m;
    }
    static __device__ __forceinline__ uint32_t widen(uint32_t m) { return m; }
};

// The scale of a block whose largest magnitude has fp32 bits `a`, and its reciprocal.  A
// block with a value that is not finite gets s = NaN and q = 0: the product of such a
// block is NaN, so the fault stays visible.
__device__ __forceinline__ void block_scale(uint32_t a, int top_exp, float& s, float& inv) {
    if (a >= 0x7f800000u) {
        s = __uint_as_float(0x7fc00000u);
        inv = 0.0f;
        return;
    }
    int j = static_cast<int>(a >> 23) - 127 - top_exp + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (j < -126) j = -126;
    if (a == 0u) j = 0;
    s = __uint_as_float(static_cast<uint32_t>(127 + j) << 23);
    inv = __uint_as_float(static_cast<uint32_t>(127 - j) << 23);
}

// Four values, scaled and rounded to 8 bits
template <bool E5M2>
__device__ __forceinline__ uint32_t pack8(float a, float b, float c, float d) {
    uint16_t lo, hi;
    if constexpr (E5M2) {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    return lo | static_cast<uint32_t>(hi) << 16;
}

struct QuantArgs {
    const uint8_t* x;
    int64_t ldx_bytes;
    int64_t M, K;
    uint8_t* q;
    int64_t ldq;
    float* scale;
    int64_t scale_ld;
    int tiles_k;
    int vec_in;       // 16-byte loads allowed
    int vec_out;      // 8-byte stores allowed
};

template <class E, int MODE, bool E5M2>
__global__ void __launch_bounds__(QTHREADS, E::BYTES == 4 ? 2 : MODE == BLOCK_COLUMN ? 4 : 5)
    quantize_kernel(const QuantArgs p) {
    constexpr int TOP_EXP = E5M2 ? 15 : 8;
    using Tile = QTile<MODE>;
    constexpr int TX = Tile::TX, TY = Tile::TY;
    __shared__ uint32_t s_mag[QTHREADS / 32][QT];      // column mode: per warp; square: a word of each; row: the first
    __shared__ float s_inv[QT];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t tile = blockIdx.x;
    const int64_t mb = tile / p.tiles_k;
    const int64_t kb = tile - mb * p.tiles_k;
    const int64_t row0 = mb * Tile::ROWS, col0 = kb * Tile::COLS + tx * 8;
    const int cols = static_cast<int>(p.K - col0 < 8 ? (p.K > col0 ? p.K - col0 : 0) : 8);

    // a tile inside X (and aligned) takes straight code: this kernel is as near to the issue limit as
    // to the memory's
    const bool inside = row0 + Tile::ROWS <= p.M && (kb + 1) * Tile::COLS <= p.K;
    E v[QROWS];
    const uint8_t* src = p.x + (row0 + ty) * p.ldx_bytes + col0 * E::BYTES;
    const int64_t src_step = p.ldx_bytes * TY;
    if (inside && p.vec_in) {
#pragma unroll
        for (int i = 0; i < QROWS; ++i) v[i].load(src + i * src_step);
    } else {
#pragma unroll
        for (int i = 0; i < QROWS; ++i) {
            v[i].zero();
            if (row0 + ty + TY * i < p.M) {
                if (cols == 8 && p.vec_in) {
                    v[i].load(src + i * src_step);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < cols) v[i].set(c, src + i * src_step + c * E::BYTES);
                }
            }
        }
    }

    if constexpr (MODE == BLOCK_ROW) {
        // 16 lanes hold a scale block; s_mag and s_inv are [block of the tile][row]
        constexpr int ROWS = Tile::ROWS, BLOCKS = Tile::COLS / QT;
        static_assert(ROWS * BLOCKS == QT, "a scale a thread of the first 128");
#pragma unroll
        for (int i = 0; i < QROWS; ++i) {
            uint32_t m = v[i].max_mag();
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            if (tx % 16 == 0) s_mag[0][tx / 16 * ROWS + ty + TY * i] = m;
        }
        __syncthreads();
        // scales lie block column after block column, a tile's rows side by side
        if (threadIdx.x < QT) {
            float s, f;
            block_scale(E::widen(s_mag[0][threadIdx.x]), TOP_EXP, s, f);
            s_inv[threadIdx.x] = f;
            const int64_t b = kb * BLOCKS + threadIdx.x / ROWS, row = row0 + threadIdx.x % ROWS;
            if (b * QT < p.K && row < p.M) p.scale[b * p.scale_ld + row] = s;
        }
        __syncthreads();
    } else if constexpr (MODE == BLOCK_COLUMN) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < QROWS; ++i) m = max(m, v[i].mag(c));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
            if (lane < 16) s_mag[warp][tx * 8 + c] = m;
        }
        __syncthreads();
        if (threadIdx.x < QT) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < QTHREADS / 32; ++w) m = max(m, s_mag[w][threadIdx.x]);
            float s, inv;
            block_scale(E::widen(m), TOP_EXP, s, inv);
            s_inv[threadIdx.x] = inv;
            const int64_t col = kb * QT + threadIdx.x;
            if (col < p.K) p.scale[mb * p.scale_ld + col] = s;
        }
        __syncthreads();
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < QROWS; ++i) m = max(m, v[i].max_mag());
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) s_mag[warp][0] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < QTHREADS / 32; ++w) m = max(m, s_mag[w][0]);
            float s, f;
            block_scale(E::widen(m), TOP_EXP, s, f);
            s_inv[0] = f;
            p.scale[mb * p.scale_ld + kb] = s;
        }
        __syncthreads();
    }

    float inv[8];
    if constexpr (MODE == BLOCK_COLUMN) {
#pragma unroll
        for (int c = 0; c < 8; ++c) inv[c] = s_inv[tx * 8 + c];
    }
    // the eight bytes of row i
    auto bytes = [&](int i) {
        uint32_t w[2];
        if constexpr (MODE != BLOCK_COLUMN) {
            const float f = s_inv[MODE == BLOCK_ROW ? tx / 16 * Tile::ROWS + ty + TY * i : 0];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[h] = pack8<E5M2>(v[i].value(4 * h) * f, v[i].value(4 * h + 1) * f, v[i].value(4 * h + 2) * f,
                                   v[i].value(4 * h + 3) * f);
                if (f == 0.0f) w[h] = 0u;          // a block that is not finite: zeros
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[h] = pack8<E5M2>(v[i].value(4 * h) * inv[4 * h], v[i].value(4 * h + 1) * inv[4 * h + 1],
                                   v[i].value(4 * h + 2) * inv[4 * h + 2], v[i].value(4 * h + 3) * inv[4 * h + 3]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (inv[4 * h + c] == 0.0f) w[h] &= ~(0xffu << (8 * c));
            }
        }
        return make_uint2(w[0], w[1]);
    };
    uint8_t* dst = p.q + (row0 + ty) * p.ldq + col0;
    const int64_t dst_step = p.ldq * TY;
    if (inside && p.vec_out) {
#pragma unroll
        for (int i = 0; i < QROWS; ++i) *reinterpret_cast<uint2*>(dst + i * dst_step) = bytes(i);
    } else {
#pragma unroll
        for (int i = 0; i < QROWS; ++i) {
            const uint2 w = bytes(i);
            if (row0 + ty + TY * i >= p.M) continue;
            if (cols == 8 && p.vec_out) {
                *reinterpret_cast<uint2*>(dst + i * dst_step) = w;
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < cols) dst[i * dst_step + c] = static_cast<uint8_t>((c < 4 ? w.x : w.y) >> ((c & 3) * 8));
            }
        }
    }
}

using QuantKernel = void (*)(const QuantArgs);

template <class E, bool E5M2>
QuantKernel pick_mode(int mode) {
    return mode == BLOCK_ROW ? &quantize_kernel<E, BLOCK_ROW, E5M2>
         : mode == BLOCK_COLUMN ? &quantize_kernel<E, BLOCK_COLUMN, E5M2> : &quantize_kernel<E, BLOCK_SQUARE, E5M2>;
}

template <bool E5M2>
QuantKernel pick_kernel(tg_dtype x, int mode) {
    return x == TG_BF16 ? pick_mode<Half8<false>, E5M2>(mode)
         : x == TG_F16 ? pick_mode<Half8<true>, E5M2>(mode) : pick_mode<Float8, E5M2>(mode);
}

}  // namespace

}  // namespace tg

extern "C" tg_status tg_quantize_blocks(const void* X, tg_dtype x_dtype, int64_t ldx, int64_t M, int64_t K,
                                     int block_rows, int block_cols, void* Q, tg_dtype q_dtype, int64_t ldq,
                                     float* scale, int64_t scale_ld, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    if (x_dtype != TG_BF16 && x_dtype != TG_F16 && x_dtype != TG_F32)
        return fail(TG_ERR_INVALID_ARG, "bad x_dtype %d (bf16, fp16 or fp32)", int(x_dtype));
    if (q_dtype != TG_E4M3 && q_dtype != TG_E5M2)
        return fail(TG_ERR_INVALID_ARG, "bad q_dtype %d (e4m3 or e5m2)", int(q_dtype));
    int mode;
    if (block_rows == 1 && block_cols == 128) mode = BLOCK_ROW;
    else if (block_rows == 128 && block_cols == 1) mode = BLOCK_COLUMN;
    else if (block_rows == 128 && block_cols == 128) mode = BLOCK_SQUARE;
    else return fail(TG_ERR_INVALID_ARG, "bad block %d x %d (1 x 128, 128 x 1 or 128 x 128)", block_rows, block_cols);
    if (M < 0 || K < 0) return fail(TG_ERR_INVALID_ARG, "negative size M=%lld K=%lld", (long long)M, (long long)K);
    if (M > host::MAX_DIM || K > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "sizes must be below 2^31");
    if (M == 0 || K == 0) return TG_OK;
    if (!X || !Q || !scale) return fail(TG_ERR_INVALID_ARG, "%s is NULL", !X ? "X" : !Q ? "Q" : "scale");
    const int64_t esize = x_dtype == TG_F32 ? 4 : 2;
    if (ldx < K) return fail(TG_ERR_INVALID_ARG, "ldx=%lld < K=%lld", (long long)ldx, (long long)K);
    if (ldq < K) return fail(TG_ERR_INVALID_ARG, "ldq=%lld < K=%lld", (long long)ldq, (long long)K);
    if (ldx > host::MAX_DIM || ldq > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "leading dimensions must be below 2^31");
    if (!host::aligned(X, esize)) return fail(TG_ERR_INVALID_ARG, "X is not aligned to its element size");
    if (!host::aligned(scale, 4)) return fail(TG_ERR_INVALID_ARG, "scale is not 4-byte aligned");
    const int64_t tile_rows = mode == BLOCK_ROW ? QTile<BLOCK_ROW>::ROWS : QT;
    const int64_t tile_cols = mode == BLOCK_ROW ? QTile<BLOCK_ROW>::COLS : QT;
    const int64_t tiles_m = (M + tile_rows - 1) / tile_rows, tiles_k = (K + tile_cols - 1) / tile_cols;
    const int64_t need = mode == BLOCK_ROW ? M : mode == BLOCK_COLUMN ? K : tiles_k;
    if (scale_ld < need) return fail(TG_ERR_INVALID_ARG, "scale_ld=%lld < %lld", (long long)scale_ld, (long long)need);
    if (tiles_m * tiles_k > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "X is too large (2^31 - 1 tiles of 2^14 values)");
    host::Device d;
    const tg_status s = host::device(&d);
    if (s != TG_OK) return s;
    QuantArgs a;
    a.x = static_cast<const uint8_t*>(X);
    a.ldx_bytes = ldx * esize;
    a.M = M;
    a.K = K;
    a.q = static_cast<uint8_t*>(Q);
    a.ldq = ldq;
    a.scale = scale;
    a.scale_ld = scale_ld;
    a.tiles_k = static_cast<int>(tiles_k);
    a.vec_in = host::aligned(X, 16) && a.ldx_bytes % 16 == 0;
    a.vec_out = host::aligned(Q, 8) && ldq % 8 == 0;
    const QuantKernel k = q_dtype == TG_E5M2 ? pick_kernel<true>(x_dtype, mode) : pick_kernel<false>(x_dtype, mode);
    k<<<static_cast<unsigned>(tiles_m * tiles_k), QTHREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host::cuda_fail(e, "quantiser launch");
    host::count_launches(1);
    return TG_OK;
}
