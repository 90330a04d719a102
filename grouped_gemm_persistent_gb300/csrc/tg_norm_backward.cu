// tg_norm_backward.cu - the gradients of the norm (tg_rmsnorm_backward in include/tg.h; formulas in tg_norm.cu).
//
// Bound by memory: dy, h and d_hidden are read once, dx written once.  A persistent block keeps the gain in shared memory and the
// sums of its gradient over the block's rows in registers; a second kernel adds the blocks' sums in order.
// 40960 x 4096 bf16 with d_hidden and d_gain: 206 us, 6.5 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"
#include "tg_norm.cuh"
#include "tg_ptx.cuh"

namespace tg {

namespace norm {

namespace {

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
    int64_t wide;                // rows before this one may be read in whole vectors (ODD)
    float inv_k;
};

// Rows as in norm_kernel; the gain waits in shared memory, its gradient is summed in registers over a block's rows.  APART with two
// vectors: held to 64 registers, 32 warps an SM, although fp32 streams spill a few (40970 x 4095: 501 us instead of 594 with 82).
template <int DT, int HT, int NV, int FORM>
__global__ void __launch_bounds__(512, FORM == APART && NV == 2 ? 2 : 0) norm_backward_kernel(const __grid_constant__ NormBackArgs a) {
    ptx::grid_launch_dependents();
    extern __shared__ __align__(16) float gain[];
    __shared__ float part[2][16];
    constexpr int HELD = NV < 8 ? NV : 1;        // vectors of a row that stay in registers
    const int tpr = blockDim.x, in = threadIdx.x;
    const int64_t units = gridDim.x, unit = blockIdx.x;
    stage_gain(gain, a.gain, a.gain_dtype, a.K);
    float acc[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
    int turn = 0;
    for (int64_t row = unit; row < a.M; row += units, turn ^= 1) {
        const bool wide = row < a.wide;
        Oct<DT> dy[HELD];
        Oct<HT> h[HELD], dh[HELD];
        auto fetch = [&](int to, int j) {
            const int col = first_of<FORM>(in + j * tpr), n = count_of<FORM>(col, a.K);
            dy[to].template load<FORM>(a.dy + row * a.lddy + static_cast<int64_t>(col) * item_bytes(DT), n, wide);
            h[to].template load<FORM>(a.h + row * a.ldh + static_cast<int64_t>(col) * item_bytes(HT), n, wide);
        };
        auto fetch_other = [&](int to, int j) {
            const int col = first_of<FORM>(in + j * tpr), n = count_of<FORM>(col, a.K);
            if (a.d_hidden) dh[to].template load<FORM>(a.d_hidden + row * a.lddh + static_cast<int64_t>(col) * item_bytes(HT), n, wide);
            else dh[to].zero();
        };
        if constexpr (HELD == NV) {
#pragma unroll
            for (int j = 0; j < NV; ++j) fetch(j, j);
#pragma unroll
            for (int j = 0; j < NV; ++j) fetch_other(j, j);
        }
        const float r = a.r[row];
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = first_of<FORM>(in + j * tpr), at = j % HELD;
            if (col >= a.K) continue;
            if constexpr (HELD < NV) fetch(at, j);
            dy[at].template cut<FORM>(a.K - col);
            h[at].template cut<FORM>(a.K - col);
            float g[8];
            read_gain<FORM>(g, gain + col, count_of<FORM>(col, a.K));
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = h[at].value(i) * r;
                t = fmaf(dy[at].value(i) * g[i], n, t);
                acc[j][i] = fmaf(dy[at].value(i), n, acc[j][i]);
            }
            s += t;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(FULL, s, d);
        if (blockDim.x > 32) {
            // (two rows' sums in turn: a warp is at most one row ahead of the others)
            if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = s;
            __syncthreads();
            s = part[turn][0];
            for (int w = 1; w < static_cast<int>(blockDim.x / 32); ++w) s += part[turn][w];
        }
        const float c = s * (r * a.inv_k);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = first_of<FORM>(in + j * tpr), at = j % HELD;
            if (col >= a.K) continue;
            if constexpr (HELD < NV) {
                fetch(at, j);
                fetch_other(at, j);
            }
            float g[8], o[8];
            read_gain<FORM>(g, gain + col, count_of<FORM>(col, a.K));
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(dy[at].value(i) * g[i], r, fmaf(-(h[at].value(i) * r), c, dh[at].value(i)));
            store8<HT, FORM>(a.dx + row * a.lddx + static_cast<int64_t>(col) * item_bytes(HT), o, count_of<FORM>(col, a.K));
        }
    }
    if (a.part) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = first_of<FORM>(in + j * tpr);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i * STRIDE<FORM> < a.K) a.part[unit * a.K + col + i * STRIDE<FORM>] = acc[j][i];
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

using NormBackKernel = void (*)(const NormBackArgs);

// Two vectors a thread up to 8192 values, four up to 16384, eight above, which are not held between the row's sum and dx but read again.
// 40960 x 4096 bf16 with d_hidden: two 206 us, four 211, one 264.  10000 x 16383 without padding, fp32 stream: four 604, eight held
// (and spilled) 1738.  5000 x 32768, fp32 stream: read again 504, held 1385 (339 at the copy rate); bf16 424 and 468.
// (Four vectors of fp32 dy and stream spill 144 to 184 bytes a thread, other types none on 16-byte boundaries.)
Spread spread_for(int64_t K) { return spread(K, K <= 8192 ? 2 : K <= 16384 ? 4 : 8); }

template <int DT, int HT, int FORM>
NormBackKernel back_for(const Spread& s) {
    return s.nv == 2 ? &norm_backward_kernel<DT, HT, 2, FORM> : s.nv == 4 ? &norm_backward_kernel<DT, HT, 4, FORM> : &norm_backward_kernel<DT, HT, 8, FORM>;
}

template <int DT, int HT>
NormBackKernel back_for(const Spread& s, Form form) {
    return form == WHOLE ? back_for<DT, HT, WHOLE>(s) : form == ODD ? back_for<DT, HT, ODD>(s) : back_for<DT, HT, APART>(s);
}

template <int DT>
NormBackKernel back_for(tg_dtype h, const Spread& s, Form form) {
    return h == TG_F32 ? back_for<DT, TG_F32>(s, form) : h == TG_F16 ? back_for<DT, TG_F16>(s, form) : back_for<DT, TG_BF16>(s, form);
}

}  // namespace

}  // namespace norm

}  // namespace tg

extern "C" tg_status tg_rmsnorm_backward(const tg_rmsnorm_backward_args* args, tg_stream_t stream) {
    using namespace tg;
    using namespace tg::norm;
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
    const bool vec = vectors_of(p.dy, a.lddy) && vectors_of(p.hidden, a.ldh) &&
                       (!p.d_hidden || vectors_of(p.d_hidden, a.lddh)) && vectors_of(p.dx, a.lddx);
    const Form form = form_of(vec, p.K);
    a.wide = 0;
    if (vec) {
        a.wide = wide_rows(p.M, p.K, p.lddy);
        if (wide_rows(p.M, p.K, p.ldh) < a.wide) a.wide = wide_rows(p.M, p.K, p.ldh);
        if (p.d_hidden && wide_rows(p.M, p.K, p.lddh) < a.wide) a.wide = wide_rows(p.M, p.K, p.lddh);
    }
    a.inv_k = 1.0f / static_cast<float>(p.K);
    const Spread shape = spread_for(p.K);
    const NormBackKernel kernel = p.dy_dtype == TG_F32 ? back_for<TG_F32>(p.hidden_dtype, shape, form)
                                : p.dy_dtype == TG_F16 ? back_for<TG_F16>(p.hidden_dtype, shape, form)
                                                       : back_for<TG_BF16>(p.hidden_dtype, shape, form);
    const size_t smem = static_cast<size_t>((p.K + 7) / 8) * 32;
    int n = 0;
    cudaError_t e = resident(kernel, shape.threads, smem, d.id, &n);
    if (e != cudaSuccess) return host::cuda_fail(e, "occupancy of the norm's backward pass");
    const int64_t cap = static_cast<int64_t>(d.sms) * n, want = p.M;
    const int64_t units = want < cap ? want : cap;
    void* ws = nullptr;
    if (p.d_gain) {
        if ((s = host::workspace(static_cast<size_t>(units) * p.K * 4, st, "cudaMallocFromPoolAsync(norm's partial sums)", &ws)) != TG_OK)
            return s;
        a.part = static_cast<float*>(ws);
    }
    kernel<<<static_cast<unsigned>(units), shape.threads, smem, st>>>(a);
    e = cudaGetLastError();
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
