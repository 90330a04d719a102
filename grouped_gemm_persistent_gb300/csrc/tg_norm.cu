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
// Bound by memory: a row is read once, held in registers between the sum and the scaling, and written once.  Blocks are persistent
// (as many as are resident), keep the gain in shared memory and load the next row while they finish one.  65536 x 4096 bf16 with a
// bf16 residual into e4m3 (279 us at the copy rate): a block a row 341 us, 38 instructions a value, with loads and outputs
// chosen inside the loop; persistent, the next row on its way, 326; packed arithmetic (two values an instruction) 296; the gain
// staged by wide loads 285; squares added as pairs 295, 6.4 TB/s.
//
// The row factor.  An 8-bit value next to a rounding border, and a scale next to a power of two, fall on one side or
// the other with the last bit of r, so r is worked out to well below fp32's half step and rounded once: every
// implementation of the definition then gives the same bytes (up to one row in some thousands whose r lies that near a
// border itself).  A thread's squares, and then the lanes' and warps' sums, are added as a pair of fp32 numbers (value and
// what its rounding lost); 1 / sqrt is the hardware's approximation and one Newton step whose residual is worked out in
// such pairs.  Eight neighbours' squares added in plain fp32 in front of the pairs would be 10 us less of 295, but put r a step off in
// 4 % of the rows, 20 % where one column outweighs the others; with Knuth's two-sum of any two numbers instead of an order of
// them it is 316.  Double precision would take 15 cycles a warp instruction on this GPU, about 700 a row, against 1200 that a
// 4096-wide row's bytes take.
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"
#include "tg_norm.cuh"

namespace tg {

namespace norm {

template <>
NormKernel norm_for<TG_BF16>(bool residual, tg_dtype rt, const Spread& s, Form form);
template <>
NormKernel norm_for<TG_F16>(bool residual, tg_dtype rt, const Spread& s, Form form);
template <>
NormKernel norm_for<TG_F32>(bool residual, tg_dtype rt, const Spread& s, Form form);

namespace {

// One vector a thread up to 256 values, two up to 1024 (65536 x 512 into e4m3 41 us, 52 with four).  Longer rows: four of 16-bit streams
// (eight above 16384: a block has 512 threads then); one of 32-bit streams that are not quantised, up to 8192 values, and of few
// rows, so that a row takes one round of loads.  40960 x 4096, x bf16: into e4m3 with a bf16 residual 186 us with four a thread, 205
// with two, 262 with one; into bf16 with an fp32 residual 348, 361 and 318.  Eight spill: up to 232 bytes a thread with 16-bit
// streams, 350 to 1200 with an fp32 x or stream, 3828 with both in odd rows (5000 x 32768 bf16 into e4m3 290 us, 169 at the copy
// rate).
Spread spread_for(int64_t K, bool few, bool wide, bool q) {
    const int64_t vectors = (K + 7) / 8;
    if (vectors <= 32 || (vectors <= 1024 && (few || (wide && !q && vectors > 128)))) return spread(K, 1);
    return spread(K, vectors <= 128 ? 2 : vectors <= 2048 ? 4 : 8);
}

}  // namespace

}  // namespace norm

}  // namespace tg

extern "C" tg_status tg_rmsnorm(const tg_rmsnorm_args* args, tg_stream_t stream) {
    using namespace tg;
    using namespace tg::norm;
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
    bool vec = vectors_of(p.x, a.ldx);
    if (residual) {
        a.residual = static_cast<const uint8_t*>(p.residual);
        a.ldr = p.ldr * hs;
        a.hidden = static_cast<uint8_t*>(p.hidden);
        a.ldh = p.ldh * hs;
        vec = vec && vectors_of(p.residual, a.ldr) && vectors_of(p.hidden, a.ldh);
    }
    if (p.y) {
        a.y = static_cast<uint8_t*>(p.y);
        a.ldy = p.ldy * ys;
        a.y_dtype = p.y_dtype;
        vec = vec && vectors_of(p.y, a.ldy);
    }
    if (p.q) {
        a.q = static_cast<uint8_t*>(p.q);
        a.ldq = p.ldq;
        a.scale = p.scale;
        a.scale_ld = p.scale_ld;
        a.e5m2 = p.q_dtype == TG_E5M2;
        vec = vec && host::aligned(p.q, 8) && p.ldq % 8 == 0;
    }
    const Form form = form_of(vec, p.K);
    a.wide = 0;
    if (vec) {
        a.wide = wide_rows(p.M, p.K, p.ldx);
        if (residual && wide_rows(p.M, p.K, p.ldr) < a.wide) a.wide = wide_rows(p.M, p.K, p.ldr);
    }
    a.r = p.row_scale;
    a.M = p.M;
    a.K = static_cast<int>(p.K);
    a.eps = p.eps;
    const double inv = 1.0 / static_cast<double>(p.K);
    a.inv_hi = static_cast<float>(inv);
    a.inv_lo = static_cast<float>(inv - a.inv_hi);
    const Spread shape = spread_for(p.K, p.M <= 2 * d.sms, ht == TG_F32, p.q != nullptr);
    const NormKernel kernel = p.x_dtype == TG_F32 ? norm_for<TG_F32>(residual, p.residual_dtype, shape, form)
                            : p.x_dtype == TG_F16 ? norm_for<TG_F16>(residual, p.residual_dtype, shape, form)
                                                  : norm_for<TG_BF16>(residual, p.residual_dtype, shape, form);
    const size_t smem = shape.nv == 1 ? 0 : static_cast<size_t>((p.K + 7) / 8) * 32;
    int64_t blocks = p.M;
    cudaError_t e = cudaSuccess;
    if (blocks > 2 * d.sms || smem > FREE_SMEM) {       // (it also lets the kernel have that much)
        int n = 0;
        if ((e = resident(kernel, shape.threads, smem, d.id, &n)) != cudaSuccess) return host::cuda_fail(e, "occupancy of the norm");
        if (blocks > static_cast<int64_t>(n) * d.sms) blocks = static_cast<int64_t>(n) * d.sms;
    }
    kernel<<<static_cast<unsigned>(blocks), shape.threads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return host::cuda_fail(e, "norm launch");
    host::count_launches(1);
    return TG_OK;
}
