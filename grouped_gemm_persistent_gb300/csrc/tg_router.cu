// tg_router.cu - the gate of a mixture-of-experts layer: top-k choice, per-expert token
// counts and balance loss, and the gradient of the logits (tg_moe_router and
// tg_moe_router_backward in include/tg.h).
//
// With x[t, :] the logits of token t and p = softmax(x[t, :]):
//   e(t, 0..k-1)   the k experts of largest logit, ties to the lowest index
//   w(t, j)        p of expert e(t, j), or divided by the sum of the k chosen ones
//   counts[g]      how often expert g was chosen
//   loss           G * sum_g f_g P_g,  f_g = counts[g] / (n k),  P_g = (1/n) sum_t p[t, g]
// where n counts the rows with a logit above -infinity.  An expert whose logit is
// -infinity is never chosen; a row of them all chooses none and counts nowhere.
// counts are piecewise constant in the logits, so d loss / d p[t, g] = G f_g / n
// = slope[g], and with w' the gradient of the weights
//   renormalised:  d x = p (u - sum p u) + [chosen] w (w' - sum w w'),   u = d_loss * slope
//   otherwise:     d x = p (u - sum p u - sum w w') + [chosen] w w'.
//
// One warp holds one row: lane l the experts l, l + 32, ...  Everything is summed in a
// fixed order - a lane over its rows, the warps of a block, then the blocks in double -
// so results do not depend on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"
#include "tg_ptx.cuh"

namespace tg {

namespace {

constexpr int R_WARPS = 8;                    // rows in flight per block
constexpr int R_THREADS = 32 * R_WARPS;
constexpr int R_BLOCKS_PER_SM = 2;
constexpr int R_MAX_G = TG_MOE_ROUTER_MAX_EXPERTS;
constexpr int R_MAX_K = TG_MOE_ROUTER_MAX_TOP_K;

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (DT == TG_F32) return __ldg(static_cast<const float*>(p) + i);
    const uint16_t h = __ldg(static_cast<const uint16_t*>(p) + i);
    if constexpr (DT == TG_F16) return __half2float(__ushort_as_half(h));
    else return __uint_as_float(static_cast<uint32_t>(h) << 16);
}

template <int DT>
__device__ __forceinline__ void store_logit(void* p, int64_t i, float v) {
    if constexpr (DT == TG_F32) static_cast<float*>(p)[i] = v;
    else if constexpr (DT == TG_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// An unsigned key that orders like the value: -0 equals +0, NaN is above everything, and 0
// stands for "not to be chosen" (-infinity, or already taken).
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x == __int_as_float(0xff800000)) return 0u;
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Softmax of a row held as v[j] = logit of expert lane + 32 j (-infinity past the last).
// false: the row has no logit above -infinity (p is then 0).
template <int V>
__device__ __forceinline__ bool row_softmax(const float (&v)[V], float (&p)[V]) {
    float m = __int_as_float(0xff800000);
    bool any = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        m = fmaxf(m, v[j]);
        any |= v[j] != __int_as_float(0xff800000);       // true for NaN, too
    }
    m = warp_max(m);
    any = __any_sync(0xffffffffu, any);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        p[j] = any ? expf(v[j] - m) : 0.0f;
        s += p[j];
    }
    s = warp_sum(s);
    const float inv = any ? 1.0f / s : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] *= inv;
    return any;
}

struct RouterArgs {
    const void* logits;
    int64_t ld, T;
    int G, k, renorm;
    int32_t* experts;     // [T, k]
    float* weights;       // [T, k]
    int32_t* counts;      // [G]
    float* loss;
    float* slope;         // [G]
    // per block: probability sums [G], counts [G], then the number of rows
    float* part_p;
    int32_t* part_c;
    int32_t* part_n;
};

template <int DT, int V>
__global__ void __launch_bounds__(R_THREADS) router_kernel(const RouterArgs a) {
    ptx::grid_launch_dependents();
    __shared__ int32_t s_count[32 * V];
    __shared__ float s_sum[R_WARPS][32 * V];
    __shared__ int32_t s_rows[R_WARPS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int i = threadIdx.x; i < 32 * V; i += R_THREADS) s_count[i] = 0;
    __syncthreads();

    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    int rows = 0;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * R_WARPS;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * R_WARPS + warp; t < a.T; t += stride) {
        float v[V], p[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int g = lane + 32 * j;
            v[j] = g < a.G ? load_logit<DT>(a.logits, t * a.ld + g) : __int_as_float(0xff800000);
        }
        rows += row_softmax<V>(v, p) ? 1 : 0;
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += p[j];

        uint32_t key[V];
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = order_key(v[j]);
        int my_e = -1;
        float my_w = 0.0f, total = 0.0f;
        for (int i = 0; i < a.k; ++i) {
            uint32_t best = 0u;
#pragma unroll
            for (int j = 0; j < V; ++j) best = max(best, key[j]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best == 0u) break;
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int j = V - 1; j >= 0; --j)
                if (key[j] == best) at = static_cast<uint32_t>(lane + 32 * j);
            at = __reduce_min_sync(0xffffffffu, at);
            float w = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (static_cast<uint32_t>(lane + 32 * j) == at) {
                    key[j] = 0u;
                    w = p[j];
                }
            w = __shfl_sync(0xffffffffu, w, at % 32);
            total += w;
            if (lane == i) {
                my_e = static_cast<int>(at);
                my_w = w;
                atomicAdd(&s_count[at], 1);
            }
        }
        if (lane < a.k) {
            a.experts[t * a.k + lane] = my_e;
            a.weights[t * a.k + lane] = (a.renorm && my_e >= 0) ? my_w / total : my_w;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s_sum[warp][lane + 32 * j] = sum[j];
    if (lane == 0) s_rows[warp] = rows;
    __syncthreads();
    for (int g = threadIdx.x; g < a.G; g += R_THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < R_WARPS; ++w) s += s_sum[w][g];
        a.part_p[static_cast<int64_t>(blockIdx.x) * a.G + g] = s;
        a.part_c[static_cast<int64_t>(blockIdx.x) * a.G + g] = s_count[g];
    }
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < R_WARPS; ++w) n += s_rows[w];
        a.part_n[blockIdx.x] = n;
    }
}

// Join the blocks' partial sums (in block order, probabilities in double): counts, slope, loss.
constexpr int F_THREADS = 256;

__global__ void __launch_bounds__(F_THREADS) router_join_kernel(const RouterArgs a, int blocks) {
    __shared__ int64_t s_n[F_THREADS];
    __shared__ double s_loss[F_THREADS];
    ptx::grid_dependency_wait();
    int64_t n = 0;
    for (int b = threadIdx.x; b < blocks; b += F_THREADS) n += a.part_n[b];
    s_n[threadIdx.x] = n;
    __syncthreads();
    for (int d = F_THREADS / 2; d > 0; d >>= 1) {
        if (threadIdx.x < d) s_n[threadIdx.x] += s_n[threadIdx.x + d];
        __syncthreads();
    }
    const double rows = s_n[0] > 0 ? static_cast<double>(s_n[0]) : 1.0;
    double loss = 0.0;
    for (int g = threadIdx.x; g < a.G; g += F_THREADS) {
        double s = 0.0;
        int32_t c = 0;
        for (int b = 0; b < blocks; ++b) {
            s += static_cast<double>(a.part_p[static_cast<int64_t>(b) * a.G + g]);
            c += a.part_c[static_cast<int64_t>(b) * a.G + g];
        }
        a.counts[g] = c;
        const double slope = a.G * static_cast<double>(c) / (rows * a.k) / rows;
        a.slope[g] = static_cast<float>(slope);
        loss += slope * s;
    }
    s_loss[threadIdx.x] = loss;
    __syncthreads();
    for (int d = F_THREADS / 2; d > 0; d >>= 1) {
        if (threadIdx.x < d) s_loss[threadIdx.x] += s_loss[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) *a.loss = static_cast<float>(s_loss[0]);
}

struct BackArgs {
    const void* logits;
    int64_t ld, T;
    int G, k, renorm;
    const int32_t* experts;
    const float* weights;
    const float* slope;
    const float* d_weights;   // null: zero
    const float* d_loss;      // null: zero
    void* out;
    int64_t ldo;
};

template <int DT, int V>
__global__ void __launch_bounds__(R_THREADS) router_backward_kernel(const BackArgs a) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float dl = a.d_loss ? __ldg(a.d_loss) : 0.0f;
    float u[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int g = lane + 32 * j;
        u[j] = (a.d_loss && g < a.G) ? dl * __ldg(a.slope + g) : 0.0f;
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * R_WARPS;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * R_WARPS + warp; t < a.T; t += stride) {
        float v[V], p[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int g = lane + 32 * j;
            v[j] = g < a.G ? load_logit<DT>(a.logits, t * a.ld + g) : __int_as_float(0xff800000);
        }
        int e = -1;
        float w = 0.0f, dw = 0.0f;
        if (a.d_weights && lane < a.k) {
            e = __ldg(a.experts + t * a.k + lane);
            w = __ldg(a.weights + t * a.k + lane);
            dw = __ldg(a.d_weights + t * a.k + lane);
            if (e < 0) w = dw = 0.0f;
        }
        row_softmax<V>(v, p);
        float cu = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) cu = fmaf(p[j], u[j], cu);
        cu = warp_sum(cu);
        const float cw = warp_sum(w * dw);
        const float c = a.renorm ? cu : cu + cw;
        const float add = a.renorm ? w * (dw - cw) : w * dw;
        float d[V];
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = p[j] * (u[j] - c);
        for (int i = 0; i < a.k; ++i) {
            const int ei = __shfl_sync(0xffffffffu, e, i);
            const float ai = __shfl_sync(0xffffffffu, add, i);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (lane + 32 * j == ei) d[j] += ai;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int g = lane + 32 * j;
            if (g < a.G) store_logit<DT>(a.out, t * a.ldo + g, d[j]);
        }
    }
}

using RouterKernel = void (*)(const RouterArgs);
using BackKernel = void (*)(const BackArgs);

template <int DT>
RouterKernel router_for(int G) {
    return G <= 32 ? &router_kernel<DT, 1> : G <= 64 ? &router_kernel<DT, 2> : G <= 128 ? &router_kernel<DT, 4>
         : G <= 256 ? &router_kernel<DT, 8> : G <= 512 ? &router_kernel<DT, 16> : &router_kernel<DT, 32>;
}

template <int DT>
BackKernel back_for(int G) {
    return G <= 32 ? &router_backward_kernel<DT, 1> : G <= 64 ? &router_backward_kernel<DT, 2>
         : G <= 128 ? &router_backward_kernel<DT, 4> : G <= 256 ? &router_backward_kernel<DT, 8>
         : G <= 512 ? &router_backward_kernel<DT, 16> : &router_backward_kernel<DT, 32>;
}

tg_status check_router(const void* logits, tg_dtype dt, int64_t ld, int64_t T, int64_t G, int64_t k) {
    using host::fail;
    if (dt != TG_BF16 && dt != TG_F16 && dt != TG_F32)
        return fail(TG_ERR_INVALID_ARG, "bad dtype %d (bf16, fp16 or fp32)", int(dt));
    if (T < 0 || G < 1) return fail(TG_ERR_INVALID_ARG, "bad size T=%lld G=%lld", (long long)T, (long long)G);
    if (k < 1 || k > G) return fail(TG_ERR_INVALID_ARG, "k=%lld is not in [1, G=%lld]", (long long)k, (long long)G);
    if (G > R_MAX_G) return fail(TG_ERR_UNSUPPORTED, "G=%lld experts; the router takes at most %d", (long long)G, R_MAX_G);
    if (k > R_MAX_K) return fail(TG_ERR_UNSUPPORTED, "k=%lld; the router takes at most %d", (long long)k, R_MAX_K);
    if (T > host::MAX_DIM || T * k > host::MAX_DIM)
        return fail(TG_ERR_UNSUPPORTED, "T * k must be below 2^31 (T=%lld, k=%lld)", (long long)T, (long long)k);
    if (T > 0) {
        if (!logits) return fail(TG_ERR_INVALID_ARG, "logits is NULL");
        if (ld < G) return fail(TG_ERR_INVALID_ARG, "ld=%lld < G=%lld", (long long)ld, (long long)G);
        if (ld > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "ld must be below 2^31");
        if (!host::aligned(logits, dt == TG_F32 ? 4 : 2))
            return fail(TG_ERR_INVALID_ARG, "logits is not aligned to its element size");
    }
    return TG_OK;
}

int row_blocks(int64_t T, int sms) {
    const int64_t want = (T + R_WARPS - 1) / R_WARPS, cap = static_cast<int64_t>(sms) * R_BLOCKS_PER_SM;
    return static_cast<int>(want < 1 ? 1 : want > cap ? cap : want);
}

}  // namespace

}  // namespace tg

extern "C" tg_status tg_moe_router(const void* logits, tg_dtype dtype, int64_t ld, int64_t T, int64_t G, int64_t k,
                                   int renormalize, int32_t* experts, float* weights, int32_t* counts, float* loss,
                                   float* slope, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    tg_status s = check_router(logits, dtype, ld, T, G, k);
    if (s != TG_OK) return s;
    if (T > 0 && (!experts || !weights)) return fail(TG_ERR_INVALID_ARG, "%s is NULL", !experts ? "experts" : "weights");
    if (!counts || !loss || !slope)
        return fail(TG_ERR_INVALID_ARG, "%s is NULL", !counts ? "counts" : !loss ? "loss" : "slope");
    if (!host::aligned(experts, 4) || !host::aligned(weights, 4) || !host::aligned(counts, 4) ||
        !host::aligned(loss, 4) || !host::aligned(slope, 4))
        return fail(TG_ERR_INVALID_ARG, "an output is not 4-byte aligned");
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int blocks = row_blocks(T, d.sms);
    void* ws = nullptr;
    const size_t words = static_cast<size_t>(blocks) * (2 * G + 1);
    if ((s = host::workspace(words * 4, st, "cudaMallocFromPoolAsync(router partial sums)", &ws)) != TG_OK) return s;
    RouterArgs a{logits, ld, T, int(G), int(k), renormalize != 0, experts, weights, counts, loss, slope,
                 static_cast<float*>(ws), static_cast<int32_t*>(ws) + blocks * G,
                 static_cast<int32_t*>(ws) + 2 * blocks * G};
    const RouterKernel kern = dtype == TG_F32 ? router_for<TG_F32>(a.G)
                            : dtype == TG_F16 ? router_for<TG_F16>(a.G) : router_for<TG_BF16>(a.G);
    kern<<<blocks, R_THREADS, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        host::count_launches(1);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1, 1, 1);
        cfg.blockDim = dim3(F_THREADS, 1, 1);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, router_join_kernel, static_cast<const RouterArgs&>(a), blocks);
        if (e == cudaSuccess) host::count_launches(1);
    }
    s = e == cudaSuccess ? TG_OK : host::cuda_fail(e, "router launch");
    e = cudaFreeAsync(ws, st);
    if (e != cudaSuccess && s == TG_OK) s = host::cuda_fail(e, "cudaFreeAsync(router partial sums)");
    return s;
}

extern "C" tg_status tg_moe_router_backward(const void* logits, tg_dtype dtype, int64_t ld, int64_t T, int64_t G,
                                            int64_t k, int renormalize, const int32_t* experts, const float* weights,
                                            const float* slope, const float* d_weights, const float* d_loss,
                                            void* d_logits, int64_t ldd, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    tg_status s = check_router(logits, dtype, ld, T, G, k);
    if (s != TG_OK || T == 0) return s;
    if (!d_logits) return fail(TG_ERR_INVALID_ARG, "d_logits is NULL");
    if (d_weights && (!experts || !weights))
        return fail(TG_ERR_INVALID_ARG, "%s is NULL (needed with d_weights)", !experts ? "experts" : "weights");
    if (d_loss && !slope) return fail(TG_ERR_INVALID_ARG, "slope is NULL (needed with d_loss)");
    if (ldd < G) return fail(TG_ERR_INVALID_ARG, "ldd=%lld < G=%lld", (long long)ldd, (long long)G);
    if (ldd > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "ldd must be below 2^31");
    if (!host::aligned(d_logits, dtype == TG_F32 ? 4 : 2))
        return fail(TG_ERR_INVALID_ARG, "d_logits is not aligned to its element size");
    if (!host::aligned(experts, 4) || !host::aligned(weights, 4) || !host::aligned(slope, 4) ||
        !host::aligned(d_weights, 4) || !host::aligned(d_loss, 4))
        return fail(TG_ERR_INVALID_ARG, "an input is not 4-byte aligned");
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    const BackArgs a{logits, ld, T, int(G), int(k), renormalize != 0, experts, weights, slope, d_weights, d_loss,
                     d_logits, ldd};
    const BackKernel kern = dtype == TG_F32 ? back_for<TG_F32>(a.G)
                          : dtype == TG_F16 ? back_for<TG_F16>(a.G) : back_for<TG_BF16>(a.G);
    const int64_t want = (T + R_WARPS - 1) / R_WARPS, cap = static_cast<int64_t>(d.sms) * 8;
    kern<<<static_cast<unsigned>(want < cap ? want : cap), R_THREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host::cuda_fail(e, "router backward launch");
    host::count_launches(1);
    return TG_OK;
}
