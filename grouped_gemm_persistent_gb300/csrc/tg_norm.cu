// tg_norm.cu - RMS norm of a residual stream, with the addition of a block's output in front of it and an 8-bit copy
// behind it, and its gradients (tg_rmsnorm and tg_rmsnorm_backward in include/tg.h).
//
//   h = round(x + residual)                      the stream, in its own type (h = x without a residual)
//   r = 1 / sqrt(mean_k h^2 + eps)               rounded to fp32 once
//   y = (h r) gain                               two fp32 products
//   q, scale                                     y in 8 bits, a power-of-two scale for each 128 values of a row
// and with d = dy gain, n = h r, S = sum_k d n:
//   dx = r d - n S r / K + d_hidden              d_hidden: what reaches h past the norm
//   d_gain = sum_t dy n
//
// Bound by memory: a row is read once, held in registers between the sum and the scaling, and written once.
//
// The row factor.  An 8-bit value next to a rounding border, and a scale next to a power of two, fall on one side or
// the other with the last bit of r, so r is worked out to well below fp32's half step and rounded once: every
// implementation of the definition then gives the same bytes (up to one row in some thousands whose r lies that near a
// border itself).  Eight neighbours' squares are added in fp32; their sums, independent and many, go into a pair of
// fp32 numbers (value and what its rounding lost) through the lanes and warps; 1 / sqrt is the hardware's
// approximation and one Newton step whose residual is worked out in such pairs.  Double precision would take 15
// cycles a warp instruction on this GPU, about 700 a row, against 1200 that a 4096-wide row's bytes take.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_block_scale.cuh"
#include "tg_host.cuh"
#include "tg_ptx.cuh"

namespace tg {

namespace {

constexpr uint32_t FULL = 0xffffffffu;
constexpr int N_MAX_K = TG_RMSNORM_MAX_COLUMNS;
constexpr int N_NONE = -1;          // no residual

constexpr int item_bytes(int dt) { return dt == TG_F32 ? 4 : 2; }

template <int DT>
__device__ __forceinline__ float widen16(uint32_t b) {
    if constexpr (DT == TG_F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
    else return __uint_as_float(b << 16);
}

// Eight neighbouring values of a row, as they lie in memory
template <int DT>
struct Oct {
    static constexpr int WORDS = DT == TG_F32 ? 8 : 4;
    uint32_t w[WORDS];

    // n of the eight are inside the row (the others are zero); vec: 16-byte loads allowed.  Plain loads: the memory may
    // be an output of the same call.
    __device__ __forceinline__ void load(const uint8_t* p, int n, bool vec) {
        if (n == 8 && vec) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const uint4 t = *(reinterpret_cast<const uint4*>(p) + i / 4);
                w[i] = t.x; w[i + 1] = t.y; w[i + 2] = t.z; w[i + 3] = t.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) continue;
            if constexpr (DT == TG_F32) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
            else w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (i % 2 * 16);
        }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (DT == TG_F32) return __uint_as_float(w[i]);
        else return widen16<DT>(w[i / 2] >> (i % 2 * 16) & 0xffffu);
    }
    // values 2 i and 2 i + 1, rounded to the type
    __device__ __forceinline__ void set2(int i, float a, float b) {
        if constexpr (DT == TG_F32) {
            w[2 * i] = __float_as_uint(a);
            w[2 * i + 1] = __float_as_uint(b);
        } else if constexpr (DT == TG_F16) {
            const __half2 h = __floats2half2_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    __device__ __forceinline__ void store(uint8_t* p, int n, bool vec) const {
        if (n == 8 && vec) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4)
                reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) continue;
            if constexpr (DT == TG_F32) reinterpret_cast<uint32_t*>(p)[i] = w[i];
            else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
        }
    }
};

template <int DT>
__device__ __forceinline__ void store8(uint8_t* p, const float (&f)[8], int n, bool vec) {
    Oct<DT> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.set2(i, f[2 * i], f[2 * i + 1]);
    o.store(p, n, vec);
}

// Eight values of the gain, or ones
__device__ __forceinline__ void load_gain(float (&g)[8], const uint8_t* gain, int dt, int64_t col, int n, bool vec) {
    if (!gain) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = 1.0f;
    } else if (dt == TG_F32) {
        Oct<TG_F32> o;
        o.load(gain + col * 4, n, vec);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = o.value(i);
    } else if (dt == TG_F16) {
        Oct<TG_F16> o;
        o.load(gain + col * 2, n, vec);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = o.value(i);
    } else {
        Oct<TG_BF16> o;
        o.load(gain + col * 2, n, vec);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = o.value(i);
    }
}

// A number as the sum of two fp32 ones, the second what rounding the first lost
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
    return {s, __fadd_rn(e, __fadd_rn(a.lo, b.lo))};
}

__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const Pair o{__shfl_xor_sync(FULL, v.hi, d), __shfl_xor_sync(FULL, v.lo, d)};
        v = pair_add(v, o);
    }
    return v;
}

// 1 / sqrt(sum / K + eps), 1 / K given as a pair.  A sum that is not finite, or zero with eps zero, takes the plain
// function of its value (0, infinity or NaN).
__device__ __forceinline__ float row_factor(Pair sum, float inv_hi, float inv_lo, float eps) {
    if (!(sum.hi < __int_as_float(0x7f800000))) return rsqrtf(sum.hi);
    const float p = __fmul_rn(sum.hi, inv_hi);
    const float pe = __fmaf_rn(sum.hi, inv_hi, -p) + (sum.hi * inv_lo + sum.lo * inv_hi);
    const Pair m0 = pair_add({p, pe}, {eps, 0.0f});
    const float m = __fadd_rn(m0.hi, m0.lo), ml = __fsub_rn(m0.lo, __fsub_rn(m, m0.hi));
    const float r = rsqrtf(m);
    if (!(m >= 1.17549435e-38f)) return r;            // below fp32's normal numbers r^2 would overflow
    const float t = __fmul_rn(r, r), tl = __fmaf_rn(r, r, -t);
    const float q = __fmul_rn(m, t), ql = __fmaf_rn(m, t, -q) + (m * tl + ml * t);
    const float e = __fsub_rn(1.0f, q) - ql;          // 1 - m r^2
    return __fmaf_rn(0.5f * r, e, r);
}

// The sum of eight values' squares, the values times f (1, or 2^-70)
template <int DT>
__device__ __forceinline__ float squares(const Oct<DT>& o, float f) {
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float u = o.value(2 * i) * f, v = o.value(2 * i + 1) * f;
        s[i] = fmaf(u, u, v * v);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

struct NormArgs {
    const uint8_t* x;
    int64_t ldx;                 // strides in bytes
    const uint8_t* residual;
    int64_t ldr;
    const uint8_t* gain;
    uint8_t* hidden;
    int64_t ldh;
    uint8_t* y;                  // null: not wanted
    int64_t ldy;
    uint8_t* q;                  // null: not wanted
    int64_t ldq;
    float* scale;
    int64_t scale_ld;
    float* r;
    int64_t M;
    int K;
    int gain_dtype, y_dtype, e5m2;
    int vec_x, vec_r, vec_h, vec_g, vec_y, vec_q;
    float eps, inv_hi, inv_lo;
};

// Add the parts of a row's warps in a fixed order (every thread gets the sum)
__device__ __forceinline__ Pair block_sum(Pair v, Pair* part) {
    v = warp_sum(v);
    const int warps = blockDim.x / 32;
    if (warps == 1) return v;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    if (warps > 4) return warp_sum(threadIdx.x % 32 < warps ? part[threadIdx.x % 32] : Pair{0.0f, 0.0f});
    Pair s = part[0];
    for (int w = 1; w < warps; ++w) s = pair_add(s, part[w]);
    return s;
}

// One row by the block's threads, NV vectors of eight values each; ROWS: a row a warp instead, for short rows.
template <int XT, int RT, int NV, bool ROWS>
__global__ void __launch_bounds__(ROWS ? 256 : NV == 1 ? 1024 : 512) norm_kernel(const NormArgs a) {
    constexpr int HT = RT == N_NONE ? XT : RT;
    __shared__ Pair part[ROWS ? 1 : 32];
    const int tpr = ROWS ? 32 : blockDim.x;
    const int in = ROWS ? threadIdx.x % 32 : threadIdx.x;
    const int64_t row = ROWS ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    if (ROWS && row >= a.M) return;
    auto left = [&](int j) {
        const int c = a.K - (in + j * tpr) * 8;
        return c < 0 ? 0 : c < 8 ? c : 8;
    };
    Oct<XT> x[NV];
    Oct<HT> h[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t col = (in + j * tpr) * 8;
        x[j].load(a.x + row * a.ldx + col * item_bytes(XT), left(j), a.vec_x);
        if constexpr (RT != N_NONE) h[j].load(a.residual + row * a.ldr + col * item_bytes(HT), left(j), a.vec_r);
    }
    Pair sum{0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if constexpr (RT != N_NONE) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[j].set2(i, x[j].value(2 * i) + h[j].value(2 * i), x[j].value(2 * i + 1) + h[j].value(2 * i + 1));
            const int64_t col = (in + j * tpr) * 8;
            h[j].store(a.hidden + row * a.ldh + col * item_bytes(HT), left(j), a.vec_h);
        } else {
#pragma unroll
            for (int i = 0; i < Oct<HT>::WORDS; ++i) h[j].w[i] = x[j].w[i];
        }
        sum = pair_add(sum, {squares(h[j], 1.0f), 0.0f});
    }
    sum = ROWS ? warp_sum(sum) : block_sum(sum, part);
    float r = row_factor(sum, a.inv_hi, a.inv_lo, a.eps);
    if (!(sum.hi < __int_as_float(0x7f800000))) {
        // a row whose squares' sum is past fp32's range (or that has an infinity or a NaN, and keeps it): once more,
        // scaled down; eps is nothing beside it
        constexpr float DOWN = 8.470329473e-22f;          // 2^-70
        Pair low{0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) low = pair_add(low, {squares(h[j], DOWN), 0.0f});
        if (!ROWS) __syncthreads();                      // part is read above
        low = ROWS ? warp_sum(low) : block_sum(low, part);
        r = row_factor(low, a.inv_hi, a.inv_lo, 0.0f) * DOWN;
    }
    if (in == 0) a.r[row] = r;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = in + j * tpr, n = left(j);
        const int64_t col = v * 8;
        if ((v & ~31) * 8 >= a.K) continue;              // (a whole warp: the shuffles below stay together)
        float y[8], g[8];
        load_gain(g, a.gain, a.gain_dtype, col, n, a.vec_g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(__fmul_rn(h[j].value(i), r), g[i]);
        if (a.y) {
            if (a.y_dtype == TG_F32) store8<TG_F32>(a.y + row * a.ldy + col * 4, y, n, a.vec_y);
            else if (a.y_dtype == TG_F16) store8<TG_F16>(a.y + row * a.ldy + col * 2, y, n, a.vec_y);
            else store8<TG_BF16>(a.y + row * a.ldy + col * 2, y, n, a.vec_y);
        }
        if (a.q) {
            // 16 lanes hold a block; magnitudes compare as integers.  Values past the row's end count as zero.
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, i < n ? __float_as_uint(y[i]) & 0x7fffffffu : 0u);
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(FULL, m, d));
            float s, inv;
            block_scale(m, a.e5m2 ? 15 : 8, s, inv);
            if (v % 16 == 0 && n > 0) a.scale[static_cast<int64_t>(v / 16) * a.scale_ld + row] = s;
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float* f = y + 4 * i;
                w[i] = a.e5m2 ? pack8<true>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv)
                              : pack8<false>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
                if (inv == 0.0f) w[i] = 0u;              // a block that is not finite: zeros
            }
            uint8_t* dst = a.q + row * a.ldq + col;
            if (n == 8 && a.vec_q) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < n) dst[i] = static_cast<uint8_t>(w[i / 4] >> (i % 4 * 8));
            }
        }
    }
}

struct NormBackArgs {
    const uint8_t* dy;
    int64_t lddy;
    const uint8_t* h;
    int64_t ldh;
    const float* r;
    const uint8_t* gain;
    const uint8_t* d_hidden;     // null: zero
    int64_t lddh;
    uint8_t* dx;
    int64_t lddx;
    float* part;                 // [units, K] sums of the gain's gradient over a unit's rows; null: not wanted
    int64_t M;
    int K;
    int gain_dtype;
    int vec_dy, vec_h, vec_g, vec_dh, vec_dx;
    float inv_k;
};

// A unit (the block, or with ROWS a warp) takes rows unit, unit + units, ...
template <int DT, int HT, int NV, bool ROWS>
__global__ void __launch_bounds__(ROWS ? 256 : 512) norm_backward_kernel(const NormBackArgs a) {
    ptx::grid_launch_dependents();
    __shared__ float part[2][16];
    const int tpr = ROWS ? 32 : blockDim.x;
    const int in = ROWS ? threadIdx.x % 32 : threadIdx.x;
    const int64_t unit = ROWS ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    const int64_t units = ROWS ? static_cast<int64_t>(gridDim.x) * (blockDim.x / 32) : gridDim.x;
    auto left = [&](int j) {
        const int c = a.K - (in + j * tpr) * 8;
        return c < 0 ? 0 : c < 8 ? c : 8;
    };
    float acc[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
    int turn = 0;
    for (int64_t row = unit; row < a.M; row += units, turn ^= 1) {
        Oct<DT> dy[NV];
        Oct<HT> h[NV], dh[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (in + j * tpr) * 8;
            dy[j].load(a.dy + row * a.lddy + col * item_bytes(DT), left(j), a.vec_dy);
            h[j].load(a.h + row * a.ldh + col * item_bytes(HT), left(j), a.vec_h);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (in + j * tpr) * 8;
            dh[j].load(a.d_hidden + row * a.lddh + col * item_bytes(HT), a.d_hidden ? left(j) : 0, a.vec_dh);
        }
        const float r = a.r[row];
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float g[8];
            load_gain(g, a.gain, a.gain_dtype, (in + j * tpr) * 8, left(j), a.vec_g);
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = h[j].value(i) * r;
                t = fmaf(dy[j].value(i) * g[i], n, t);
                acc[j][i] = fmaf(dy[j].value(i), n, acc[j][i]);
            }
            s += t;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(FULL, s, d);
        if (!ROWS && blockDim.x > 32) {
            // (two rows' sums in turn: a warp is at most one row ahead of the others)
            if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = s;
            __syncthreads();
            s = part[turn][0];
            for (int w = 1; w < static_cast<int>(blockDim.x / 32); ++w) s += part[turn][w];
        }
        const float c = s * (r * a.inv_k);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (in + j * tpr) * 8;
            float g[8], o[8];
            load_gain(g, a.gain, a.gain_dtype, col, left(j), a.vec_g);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(dy[j].value(i) * g[i], r, fmaf(-(h[j].value(i) * r), c, dh[j].value(i)));
            store8<HT>(a.dx + row * a.lddx + col * item_bytes(HT), o, left(j), a.vec_dx);
        }
    }
    if (a.part) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (in + j * tpr) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < a.K) a.part[unit * a.K + col + i] = acc[j][i];
        }
    }
}

// d_gain[k] = the units' sums added: 32 columns a block, the warps spread over the units, then a warp a column.
__global__ void __launch_bounds__(1024) norm_gain_kernel(const float* part, int64_t units, int K, float* d_gain) {
    __shared__ float s_part[32][33];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    ptx::grid_dependency_wait();
    const int col = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (col < K) {
#pragma unroll 8
        for (int64_t u = warp; u < units; u += 32) s += part[u * K + col];
    }
    s_part[warp][lane] = s;
    __syncthreads();
    s = s_part[lane][warp];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(FULL, s, d);
    if (lane == 0 && blockIdx.x * 32 + warp < K) d_gain[blockIdx.x * 32 + warp] = s;
}

using NormKernel = void (*)(const NormArgs);
using NormBackKernel = void (*)(const NormBackArgs);

// How a row of K values is spread: threads of a row and vectors a thread; `rows`: a row a warp, eight a block.
struct Spread {
    int threads, nv;
    bool rows;
};

// Few rows (`wide`): a vector a thread, as many warps as that takes, so that a row takes one round of loads.  Many rows:
// four a thread, a row a warp up to 1024 values; eight a thread above 16384 (a block has at most 512 threads then).
Spread spread_for(int64_t K, bool wide) {
    const int vectors = static_cast<int>((K + 7) / 8);
    if (wide && vectors > 32 && vectors <= 1024) return {(vectors + 31) / 32 * 32, 1, false};
    if (vectors <= 128) return {32, 4, true};
    const int nv = vectors <= 2048 ? 4 : 8;
    return {(vectors + 32 * nv - 1) / (32 * nv) * 32, nv, false};
}

template <int XT, int RT>
NormKernel norm_for(const Spread& s) {
    if (s.rows) return &norm_kernel<XT, RT, 4, true>;
    return s.nv == 1 ? &norm_kernel<XT, RT, 1, false> : s.nv == 4 ? &norm_kernel<XT, RT, 4, false> : &norm_kernel<XT, RT, 8, false>;
}

// (the residual has x's type or fp32)
NormKernel norm_for(tg_dtype x, bool residual, tg_dtype rt, const Spread& s) {
    switch (x) {
        case TG_F32: return residual ? norm_for<TG_F32, TG_F32>(s) : norm_for<TG_F32, N_NONE>(s);
        case TG_F16:
            return !residual ? norm_for<TG_F16, N_NONE>(s) : rt == TG_F32 ? norm_for<TG_F16, TG_F32>(s) : norm_for<TG_F16, TG_F16>(s);
        default:
            return !residual ? norm_for<TG_BF16, N_NONE>(s) : rt == TG_F32 ? norm_for<TG_BF16, TG_F32>(s) : norm_for<TG_BF16, TG_BF16>(s);
    }
}

template <int DT, int HT>
NormBackKernel back_for(const Spread& s) {
    if (s.rows) return &norm_backward_kernel<DT, HT, 4, true>;
    return s.nv == 4 ? &norm_backward_kernel<DT, HT, 4, false> : &norm_backward_kernel<DT, HT, 8, false>;
}

template <int DT>
NormBackKernel back_for(tg_dtype h, const Spread& s) {
    return h == TG_F32 ? back_for<DT, TG_F32>(s) : h == TG_F16 ? back_for<DT, TG_F16>(s) : back_for<DT, TG_BF16>(s);
}

bool value_type(tg_dtype t) { return t == TG_BF16 || t == TG_F16 || t == TG_F32; }

// A row-major matrix argument: its pointer, leading dimension and alignment
tg_status check_matrix(const char* name, const void* p, int64_t ld, int64_t K, int64_t esize) {
    using host::fail;
    if (!p) return fail(TG_ERR_INVALID_ARG, "%s is NULL", name);
    if (ld < K) return fail(TG_ERR_INVALID_ARG, "the leading dimension of %s, %lld, is below K=%lld", name, (long long)ld, (long long)K);
    if (ld > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "the leading dimension of %s must be below 2^31", name);
    if (!host::aligned(p, esize)) return fail(TG_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    return TG_OK;
}

tg_status check_sizes(int64_t M, int64_t K) {
    using host::fail;
    if (M < 0 || K < 0) return fail(TG_ERR_INVALID_ARG, "negative size M=%lld K=%lld", (long long)M, (long long)K);
    if (M > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "M must be below 2^31");
    if (K > N_MAX_K) return fail(TG_ERR_UNSUPPORTED, "K=%lld columns; the norm takes at most %d", (long long)K, N_MAX_K);
    return TG_OK;
}

bool vectors_of(const void* p, int64_t ld_bytes) { return host::aligned(p, 16) && ld_bytes % 16 == 0; }

}  // namespace

}  // namespace tg

extern "C" tg_status tg_rmsnorm(const tg_rmsnorm_args* args, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    if (!args) return fail(TG_ERR_INVALID_ARG, "args is NULL");
    const tg_rmsnorm_args& p = *args;
    if (!value_type(p.x_dtype)) return fail(TG_ERR_INVALID_ARG, "bad x_dtype %d (bf16, fp16 or fp32)", int(p.x_dtype));
    const bool residual = p.residual != nullptr;
    if (residual && p.residual_dtype != p.x_dtype && p.residual_dtype != TG_F32)
        return fail(TG_ERR_INVALID_ARG, "bad residual_dtype %d (x's or fp32)", int(p.residual_dtype));
    if (p.gain && !value_type(p.gain_dtype)) return fail(TG_ERR_INVALID_ARG, "bad gain_dtype %d (bf16, fp16 or fp32)", int(p.gain_dtype));
    if (p.y && !value_type(p.y_dtype)) return fail(TG_ERR_INVALID_ARG, "bad y_dtype %d (bf16, fp16 or fp32)", int(p.y_dtype));
    if (p.q && p.q_dtype != TG_E4M3 && p.q_dtype != TG_E5M2)
        return fail(TG_ERR_INVALID_ARG, "bad q_dtype %d (e4m3 or e5m2)", int(p.q_dtype));
    if (!(p.eps >= 0.0f) || p.eps > 3.0e38f) return fail(TG_ERR_INVALID_ARG, "eps must be finite and not negative");
    tg_status s = check_sizes(p.M, p.K);
    if (s != TG_OK || p.M == 0 || p.K == 0) return s;
    const tg_dtype ht = residual ? p.residual_dtype : p.x_dtype;
    const int64_t xs = item_bytes(p.x_dtype), hs = item_bytes(ht), ys = item_bytes(p.y_dtype);
    if ((s = check_matrix("x", p.x, p.ldx, p.K, xs)) != TG_OK) return s;
    if (residual) {
        if ((s = check_matrix("residual", p.residual, p.ldr, p.K, hs)) != TG_OK) return s;
        if ((s = check_matrix("hidden", p.hidden, p.ldh, p.K, hs)) != TG_OK) return s;
    }
    if (p.gain && !host::aligned(p.gain, item_bytes(p.gain_dtype)))
        return fail(TG_ERR_INVALID_ARG, "gain is not aligned to its element size");
    if (!p.y && !p.q) return fail(TG_ERR_INVALID_ARG, "neither y nor q is wanted");
    if (p.y && (s = check_matrix("y", p.y, p.ldy, p.K, ys)) != TG_OK) return s;
    if (p.q) {
        if ((s = check_matrix("q", p.q, p.ldq, p.K, 1)) != TG_OK) return s;
        if (!p.scale) return fail(TG_ERR_INVALID_ARG, "scale is NULL (needed with q)");
        if (!host::aligned(p.scale, 4)) return fail(TG_ERR_INVALID_ARG, "scale is not 4-byte aligned");
        if (p.scale_ld < p.M) return fail(TG_ERR_INVALID_ARG, "scale_ld=%lld < M=%lld", (long long)p.scale_ld, (long long)p.M);
    }
    if (!p.row_scale) return fail(TG_ERR_INVALID_ARG, "row_scale is NULL");
    if (!host::aligned(p.row_scale, 4)) return fail(TG_ERR_INVALID_ARG, "row_scale is not 4-byte aligned");
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    NormArgs a{};
    a.x = static_cast<const uint8_t*>(p.x);
    a.ldx = p.ldx * xs;
    a.gain = static_cast<const uint8_t*>(p.gain);
    a.gain_dtype = p.gain_dtype;
    a.vec_g = host::aligned(p.gain, 16);
    a.vec_x = vectors_of(p.x, a.ldx);
    if (residual) {
        a.residual = static_cast<const uint8_t*>(p.residual);
        a.ldr = p.ldr * hs;
        a.hidden = static_cast<uint8_t*>(p.hidden);
        a.ldh = p.ldh * hs;
        a.vec_r = vectors_of(p.residual, a.ldr);
        a.vec_h = vectors_of(p.hidden, a.ldh);
    }
    if (p.y) {
        a.y = static_cast<uint8_t*>(p.y);
        a.ldy = p.ldy * ys;
        a.y_dtype = p.y_dtype;
        a.vec_y = vectors_of(p.y, a.ldy);
    }
    if (p.q) {
        a.q = static_cast<uint8_t*>(p.q);
        a.ldq = p.ldq;
        a.scale = p.scale;
        a.scale_ld = p.scale_ld;
        a.e5m2 = p.q_dtype == TG_E5M2;
        a.vec_q = host::aligned(p.q, 8) && p.ldq % 8 == 0;
    }
    a.r = p.row_scale;
    a.M = p.M;
    a.K = static_cast<int>(p.K);
    a.eps = p.eps;
    const double inv = 1.0 / static_cast<double>(p.K);
    a.inv_hi = static_cast<float>(inv);
    a.inv_lo = static_cast<float>(inv - a.inv_hi);
    const Spread spread = spread_for(p.K, p.M <= 2 * d.sms);
    const int64_t blocks = spread.rows ? (p.M + 7) / 8 : p.M;
    norm_for(p.x_dtype, residual, p.residual_dtype, spread)<<<static_cast<unsigned>(blocks), spread.rows ? 256 : spread.threads, 0,
                                                              reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host::cuda_fail(e, "norm launch");
    host::count_launches(1);
    return TG_OK;
}

extern "C" tg_status tg_rmsnorm_backward(const tg_rmsnorm_backward_args* args, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    if (!args) return fail(TG_ERR_INVALID_ARG, "args is NULL");
    const tg_rmsnorm_backward_args& p = *args;
    if (!value_type(p.dy_dtype)) return fail(TG_ERR_INVALID_ARG, "bad dy_dtype %d (bf16, fp16 or fp32)", int(p.dy_dtype));
    if (!value_type(p.hidden_dtype))
        return fail(TG_ERR_INVALID_ARG, "bad hidden_dtype %d (bf16, fp16 or fp32)", int(p.hidden_dtype));
    if (p.gain && !value_type(p.gain_dtype)) return fail(TG_ERR_INVALID_ARG, "bad gain_dtype %d (bf16, fp16 or fp32)", int(p.gain_dtype));
    tg_status s = check_sizes(p.M, p.K);
    if (s != TG_OK || p.K == 0) return s;
    if (p.d_gain && !host::aligned(p.d_gain, 4)) return fail(TG_ERR_INVALID_ARG, "d_gain is not 4-byte aligned");
    if (p.M == 0 && !p.d_gain) return TG_OK;
    const int64_t ds = item_bytes(p.dy_dtype), hs = item_bytes(p.hidden_dtype);
    if (p.M > 0) {
        if ((s = check_matrix("dy", p.dy, p.lddy, p.K, ds)) != TG_OK) return s;
        if ((s = check_matrix("hidden", p.hidden, p.ldh, p.K, hs)) != TG_OK) return s;
        if (p.d_hidden && (s = check_matrix("d_hidden", p.d_hidden, p.lddh, p.K, hs)) != TG_OK) return s;
        if ((s = check_matrix("dx", p.dx, p.lddx, p.K, hs)) != TG_OK) return s;
        if (!p.row_scale) return fail(TG_ERR_INVALID_ARG, "row_scale is NULL");
        if (!host::aligned(p.row_scale, 4)) return fail(TG_ERR_INVALID_ARG, "row_scale is not 4-byte aligned");
        if (p.gain && !host::aligned(p.gain, item_bytes(p.gain_dtype)))
            return fail(TG_ERR_INVALID_ARG, "gain is not aligned to its element size");
    }
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (p.M == 0) {                                     // no rows: the gain's gradient is zero
        const cudaError_t e = cudaMemsetAsync(p.d_gain, 0, p.K * sizeof(float), st);
        return e == cudaSuccess ? TG_OK : host::cuda_fail(e, "cudaMemsetAsync(d_gain)");
    }
    NormBackArgs a{};
    a.dy = static_cast<const uint8_t*>(p.dy);
    a.lddy = p.lddy * ds;
    a.h = static_cast<const uint8_t*>(p.hidden);
    a.ldh = p.ldh * hs;
    a.r = p.row_scale;
    a.gain = static_cast<const uint8_t*>(p.gain);
    a.gain_dtype = p.gain_dtype;
    a.d_hidden = static_cast<const uint8_t*>(p.d_hidden);
    a.lddh = p.lddh * hs;
    a.dx = static_cast<uint8_t*>(p.dx);
    a.lddx = p.lddx * hs;
    a.M = p.M;
    a.K = static_cast<int>(p.K);
    a.vec_dy = vectors_of(p.dy, a.lddy);
    a.vec_h = vectors_of(p.hidden, a.ldh);
    a.vec_g = host::aligned(p.gain, 16);
    a.vec_dh = vectors_of(p.d_hidden, a.lddh);
    a.vec_dx = vectors_of(p.dx, a.lddx);
    a.inv_k = 1.0f / static_cast<float>(p.K);
    const Spread spread = spread_for(p.K, false);
    const NormBackKernel kernel = p.dy_dtype == TG_F32 ? back_for<TG_F32>(p.hidden_dtype, spread)
                                : p.dy_dtype == TG_F16 ? back_for<TG_F16>(p.hidden_dtype, spread)
                                                       : back_for<TG_BF16>(p.hidden_dtype, spread);
    // as many blocks as are resident: about 512 threads an SM at these registers
    const int threads = spread.rows ? 256 : spread.threads, per_block = spread.rows ? 8 : 1;
    const int64_t cap = static_cast<int64_t>(d.sms) * (threads >= 512 ? 1 : 512 / threads);
    const int64_t want = (p.M + per_block - 1) / per_block;
    const int64_t blocks = want < cap ? want : cap, units = blocks * per_block;
    void* ws = nullptr;
    if (p.d_gain) {
        if ((s = host::workspace(static_cast<size_t>(units) * p.K * 4, st, "cudaMallocFromPoolAsync(norm's partial sums)", &ws)) != TG_OK)
            return s;
        a.part = static_cast<float*>(ws);
    }
    kernel<<<static_cast<unsigned>(blocks), threads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) host::count_launches(1);
    if (e == cudaSuccess && p.d_gain) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>((p.K + 31) / 32), 1, 1);
        cfg.blockDim = dim3(1024, 1, 1);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, norm_gain_kernel, static_cast<const float*>(a.part), units, a.K, p.d_gain);
        if (e == cudaSuccess) host::count_launches(1);
    }
    s = e == cudaSuccess ? TG_OK : host::cuda_fail(e, "norm backward launch");
    if (ws) {
        e = cudaFreeAsync(ws, st);
        if (e != cudaSuccess && s == TG_OK) s = host::cuda_fail(e, "cudaFreeAsync(norm's partial sums)");
    }
    return s;
}
