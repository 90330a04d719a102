// tg_norm_inst.cu - the norm's kernel for one type of x (TG_NORM_X, a tg_dtype's number), chosen and launched by tg_norm.cu, where the
// mathematics and the reasons stand.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_block_scale.cuh"
#include "tg_norm.cuh"
#include "tg_ptx.cuh"

namespace tg {

namespace norm {

namespace {

// A number as the sum of two fp32 ones, the second what rounding the first lost
struct Pair {
    float hi, lo;
};

// (the error of a rounded sum by Knuth's two-sum, which needs no order of the two)
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
    if (m == 0.0f) return r;
    const float t = __fmul_rn(r, r), tl = __fmaf_rn(r, r, -t);
    const float q = __fmul_rn(m, t), ql = __fmaf_rn(m, t, -q) + (m * tl + ml * t);
    const float e = __fsub_rn(1.0f, q) - ql;          // 1 - m r^2
    return __fmaf_rn(0.5f * r, e, r);
}

// The largest magnitude of a thread's values (NaN is passed over)
template <int DT, int NV>
__device__ __forceinline__ float largest(const Oct<DT> (&h)[NV]) {
    uint32_t w = 0u;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if constexpr (DT == TG_F32) {
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                asm("max.f32 %0, %0, %1, %2;" : "+r"(w) : "r"(h[j].w[i] & 0x7fffffffu), "r"(h[j].w[i + 1] & 0x7fffffffu));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == TG_BF16) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(h[j].w[i]));
                else asm("max.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(w) : "r"(h[j].w[i]));
            }
        }
    }
    if constexpr (DT == TG_F32) return __uint_as_float(w);
    else return fmaxf(fabsf(widen16<DT>(w & 0xffffu)), fabsf(widen16<DT>(w >> 16)));
}

// The sum of a thread's squares, the values times f (1, 2^-80 or 2^100), as a pair.  Two sums run side by side from a power of two above
// the largest square, so that in each addition the sum is the larger number: what the addition adds to it is then an fp32 number,
// and what it leaves of the square is added up by itself (Dekker's fast two-sum, the square being the fused operation's).
template <int DT, int NV>
__device__ __forceinline__ Pair sum_of_squares(const Oct<DT> (&h)[NV], float f) {
    const float top = largest(h) * f;
    // (2^-126 for zeros; where it would pass fp32, -0 or infinity: the sum is infinite or NaN and is not used)
    const float from = __uint_as_float((__float_as_uint(top * top) & 0x7f800000u) + 0x800000u);
    const uint64_t ff = ptx::f32x2_pack(f, f), minus = ptx::f32x2_pack(-1.0f, -1.0f);
    uint64_t hi = ptx::f32x2_pack(from, from), lo = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t v = f == 1.0f ? h[j].pair(i) : ptx::f32x2_mul(h[j].pair(i), ff);
            const uint64_t s = ptx::f32x2_fma(v, v, hi), less = ptx::f32x2_fma(s, minus, hi);
            lo = ptx::f32x2_add(lo, ptx::f32x2_fma(v, v, less));
            hi = s;
        }
    hi = ptx::f32x2_add(hi, ptx::f32x2_pack(-from, -from));       // (exact: a power of two not above the sum)
    Pair a, b;
    ptx::f32x2_unpack(hi, a.hi, b.hi);
    ptx::f32x2_unpack(lo, a.lo, b.lo);
    return pair_add(a, b);
}

// x + residual in the residual's type.  Two 16-bit numbers are added with one rounding, which is the rounding of their fp32 sum: where
// that is not exact, the smaller is below a quarter step of the larger, and both round to the larger.
template <int XT, int HT>
__device__ __forceinline__ void add_rows(Oct<HT>& h, const Oct<XT>& x, const Oct<HT>& residual) {
    if constexpr (XT == HT && HT == TG_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(h.w[i]) : "r"(x.w[i]), "r"(residual.w[i]));
    } else if constexpr (XT == HT && HT == TG_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h.w[i]) : "r"(x.w[i]), "r"(residual.w[i]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h.set2(i, x.value(2 * i) + residual.value(2 * i), x.value(2 * i + 1) + residual.value(2 * i + 1));
    }
}

// The largest magnitude, NaN if one is
__device__ __forceinline__ float max_magnitude(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// Add the parts of a row's warps in a fixed order (every thread gets the sum).  `part` is written anew by each row: two in turn, a
// warp being at most one row ahead of the others.
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

// What a row's thread writes: y in 16 or 32 bits or not at all, and the 8-bit copy
enum : int { Y_NONE = 0, Y_HALF = 1, Y_FLOAT = 2 };

template <int HT, int NV, int FORM, bool STAGED, int Y, bool Q>
__device__ __forceinline__ void finish_row(const NormArgs& a, const Oct<HT> (&h)[NV], float r, int64_t row, int in, int tpr,
                                           const float* gain, const float (&g0)[8]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = in + j * tpr, col = first_of<FORM>(v);
        if ((v & ~31) * 8 >= a.K) return;                // (a whole warp: the shuffles below stay together)
        const int n = count_of<FORM>(col, a.K);          // below 1: nothing here
        float y[8], g[8];
        if constexpr (STAGED) {
            if (n > 0) read_gain<FORM>(g, gain + col, n);
            else {
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = g0[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            ptx::f32x2_unpack(ptx::f32x2_mul(ptx::f32x2_mul(h[j].pair(i), ptx::f32x2_pack(r, r)), ptx::f32x2_pack(g[2 * i], g[2 * i + 1])),
                              y[2 * i], y[2 * i + 1]);
        if constexpr (Y == Y_HALF) {
            Oct<TG_BF16> o;
            if (a.y_dtype == TG_BF16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) o.set2(i, y[2 * i], y[2 * i + 1]);
            } else {
                Oct<TG_F16> f;
#pragma unroll
                for (int i = 0; i < 4; ++i) f.set2(i, y[2 * i], y[2 * i + 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) o.w[i] = f.w[i];
            }
            o.template store<FORM>(a.y + row * a.ldy + col * 2, n);
        } else if constexpr (Y == Y_FLOAT) {
            store8<TG_F32, FORM>(a.y + row * a.ldy + static_cast<int64_t>(col) * 4, y, n);
        }
        if constexpr (Q) {
            // 16 lanes hold a block.  Values past the row's end count as zero (0 times r may be NaN).
            float top = 0.0f;
            if constexpr (FORM == WHOLE) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) top = max_magnitude(top, y[i], y[i + 1]);
                if (n <= 0) top = 0.0f;
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) top = max_magnitude(top, i < n ? y[i] : 0.0f, i + 1 < n ? y[i + 1] : 0.0f);
            }
            uint32_t m = __float_as_uint(top);           // (as integers magnitudes compare alike, NaN above all)
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(FULL, m, d));
            float s, inv;
            block_scale(m, a.e5m2 ? 15 : 8, s, inv);
            if (v % 16 == 0 && n > 0) a.scale[static_cast<int64_t>(v / 16) * a.scale_ld + row] = s;
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ptx::f32x2_unpack(ptx::f32x2_mul(ptx::f32x2_pack(y[2 * i], y[2 * i + 1]), ptx::f32x2_pack(inv, inv)), y[2 * i], y[2 * i + 1]);
            if (a.e5m2) {
#pragma unroll
                for (int i = 0; i < 2; ++i) w[i] = pack8<true>(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) w[i] = pack8<false>(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            }
            if (inv == 0.0f) w[0] = w[1] = 0u;           // a block that is not finite: zeros
            uint8_t* dst = a.q + row * a.ldq + col;
            if (FORM == WHOLE ? n > 0 : FORM == ODD && n >= 8) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            } else if constexpr (FORM != WHOLE) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < n) dst[i * STRIDE<FORM>] = static_cast<uint8_t>(w[i / 4] >> (i % 4 * 8));
            }
        }
    }
}

// The block's rows are blockIdx.x, blockIdx.x + gridDim.x, ..., NV times eight values a thread.  STAGED: the gain waits in shared memory (otherwise, with one vector a thread, in registers).
template <int XT, int RT, int NV, int FORM>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int HT = RT == N_NONE ? XT : RT;
    constexpr bool STAGED = NV > 1;
    extern __shared__ __align__(16) float gain[];
    __shared__ Pair part[2][32];
    const int tpr = blockDim.x, in = threadIdx.x;
    const int64_t units = gridDim.x, unit = blockIdx.x;
    // the next row's values are on their way while a row is finished
    Oct<XT> x[NV];
    Oct<HT> h[NV], add[RT == N_NONE ? 1 : NV];
    auto fetch = [&](int64_t row) {
        const bool wide = row < a.wide;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = first_of<FORM>(in + j * tpr), n = count_of<FORM>(col, a.K);
            x[j].template load<FORM>(a.x + row * a.ldx + static_cast<int64_t>(col) * item_bytes(XT), n, wide);
            if constexpr (RT != N_NONE)
                add[j].template load<FORM>(a.residual + row * a.ldr + static_cast<int64_t>(col) * item_bytes(HT), n, wide);
        }
    };
    if (unit < a.M) fetch(unit);
    float g0[8];
    if constexpr (STAGED) {
        stage_gain(gain, a.gain, a.gain_dtype, a.K);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = first_of<FORM>(in) + i * STRIDE<FORM>;
            g0[i] = col < a.K ? gain_value(a.gain, a.gain_dtype, col) : 0.0f;
        }
    }
    int turn = 0;
    for (int64_t row = unit; row < a.M; row += units, turn ^= 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int n = a.K - (in + j * tpr) * 8;          // (ODD)
            x[j].template cut<FORM>(n);
            if constexpr (RT != N_NONE) {
                add[j].template cut<FORM>(n);
                add_rows(h[j], x[j], add[j]);
            } else {
#pragma unroll
                for (int i = 0; i < Oct<HT>::WORDS; ++i) h[j].w[i] = x[j].w[i];
            }
        }
        if (row + units < a.M) fetch(row + units);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (RT != N_NONE) {
                const int col = first_of<FORM>(in + j * tpr);
                h[j].template store<FORM>(a.hidden + row * a.ldh + static_cast<int64_t>(col) * item_bytes(HT), count_of<FORM>(col, a.K));
            }
        }
        Pair sum = block_sum(sum_of_squares(h, 1.0f), part[turn]);
        float scaled = 1.0f, eps = a.eps;
        const float mean = sum.hi * a.inv_hi + eps;
        if (!(mean < 1.267650600e30f) || mean < 7.888609052e-31f) {       // 2^100, 2^-100
            // a row whose squares or factor's square come near an end of fp32 (or that has an infinity or a NaN, and keeps it): once
            // more, scaled down by 2^-80, with which the squares of 32768 values of 2^128 sum to 2^111, or up by 2^100, with
            // which those of 32768 values sum to 2^115 and that of the smallest number is 2^-98
            scaled = mean < 1.0f ? 1.267650600e30f : 8.271806126e-25f;
            eps = eps * scaled * scaled;
            const Pair again = sum_of_squares(h, scaled);
            __syncthreads();                             // the parts are read above
            sum = block_sum(again, part[turn]);
        }
        const float r = row_factor(sum, a.inv_hi, a.inv_lo, eps) * scaled;
        if (in == 0) a.r[row] = r;
        if (!a.y) {
            finish_row<HT, NV, FORM, STAGED, Y_NONE, true>(a, h, r, row, in, tpr, gain, g0);
        } else if (a.y_dtype == TG_F32) {
            if (a.q) finish_row<HT, NV, FORM, STAGED, Y_FLOAT, true>(a, h, r, row, in, tpr, gain, g0);
            else finish_row<HT, NV, FORM, STAGED, Y_FLOAT, false>(a, h, r, row, in, tpr, gain, g0);
        } else {
            if (a.q) finish_row<HT, NV, FORM, STAGED, Y_HALF, true>(a, h, r, row, in, tpr, gain, g0);
            else finish_row<HT, NV, FORM, STAGED, Y_HALF, false>(a, h, r, row, in, tpr, gain, g0);
        }
    }
}

template <int XT, int RT, int FORM>
NormKernel pick(const Spread& s) {
    return s.nv == 1 ? &norm_kernel<XT, RT, 1, FORM> : s.nv == 2 ? &norm_kernel<XT, RT, 2, FORM>
         : s.nv == 4 ? &norm_kernel<XT, RT, 4, FORM> : &norm_kernel<XT, RT, 8, FORM>;
}

template <int XT, int RT>
NormKernel pick(const Spread& s, Form form) {
    return form == WHOLE ? pick<XT, RT, WHOLE>(s) : form == ODD ? pick<XT, RT, ODD>(s) : pick<XT, RT, APART>(s);
}

}  // namespace

template <>
NormKernel norm_for<TG_NORM_X>(bool residual, tg_dtype rt, const Spread& s, Form form) {
    if (!residual) return pick<TG_NORM_X, N_NONE>(s, form);
    if (TG_NORM_X == TG_F32 || rt == TG_F32) return pick<TG_NORM_X, TG_F32>(s, form);
    return pick<TG_NORM_X, TG_NORM_X>(s, form);
}

}  // namespace norm

}  // namespace tg
