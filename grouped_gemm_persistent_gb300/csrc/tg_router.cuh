// tg_router.cuh - what the two gates share (tg_router.cu: softmax alone; tg_router_scored.cu: other scores, a bias and
// groups of experts): a lane's logits, reductions over the lanes of a row, and the joining of the blocks' sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"
#include "tg_ptx.cuh"

namespace tg {
namespace gate {

constexpr int R_WARPS = 16;
constexpr int R_THREADS = 32 * R_WARPS;
constexpr int R_BLOCKS_PER_SM = 2;
constexpr int R_MAX_G = TG_MOE_ROUTER_MAX_EXPERTS;
constexpr int R_MAX_K = TG_MOE_ROUTER_MAX_TOP_K;
constexpr uint32_t FULL = 0xffffffffu;

// ----------------------------------------------------------------------------------------
// a lane's V logits of one row, as they lie in memory

template <int DT, int V>
struct Logits {
    static constexpr int ESIZE = DT == TG_F32 ? 4 : 2;
    static constexpr int WORDS = V * ESIZE / 4;
    static constexpr uint32_t NEG_INF = DT == TG_F32 ? 0xff800000u : DT == TG_F16 ? 0xfc00fc00u : 0xff80ff80u;
    uint32_t w[WORDS];

    __device__ __forceinline__ void load_whole(const uint8_t* p) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            const uint4 t = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
            w[i] = t.x; w[i + 1] = t.y; w[i + 2] = t.z; w[i + 3] = t.w;
        }
    }
    // n of the V are inside the row (the others become -infinity); vec: 16-byte loads allowed
    __device__ __forceinline__ void load(const uint8_t* p, int n, bool vec) {
        if (n == V && vec) {
            load_whole(p);
            return;
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (DT == TG_F32) {
                w[i] = i < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + i) : NEG_INF;
            } else {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
                const uint32_t lo = 2 * i < n ? __ldg(h + 2 * i) : NEG_INF & 0xffffu;
                const uint32_t hi = 2 * i + 1 < n ? __ldg(h + 2 * i + 1) : NEG_INF & 0xffffu;
                w[i] = lo | hi << 16;
            }
        }
    }
    // the same of every STRIDE-th logit
    template <int STRIDE>
    __device__ __forceinline__ void load_apart(const uint8_t* p, int n) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (DT == TG_F32) {
                w[i] = i < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + i * STRIDE) : NEG_INF;
            } else {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
                const uint32_t lo = 2 * i < n ? __ldg(h + 2 * i * STRIDE) : NEG_INF & 0xffffu;
                const uint32_t hi = 2 * i + 1 < n ? __ldg(h + (2 * i + 1) * STRIDE) : NEG_INF & 0xffffu;
                w[i] = lo | hi << 16;
            }
        }
    }
    __device__ __forceinline__ uint32_t bits(int j) const {
        if constexpr (DT == TG_F32) return w[j];
        else return j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu;
    }
    static __device__ __forceinline__ float widen(uint32_t b) {
        if constexpr (DT == TG_F32) return __uint_as_float(b);
        else if constexpr (DT == TG_F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
        else return __uint_as_float(b << 16);
    }
    __device__ __forceinline__ float value(int j) const { return widen(bits(j)); }
    // logit g of the row at p
    static __device__ __forceinline__ float one(const uint8_t* p, int g) {
        if constexpr (DT == TG_F32) return __ldg(reinterpret_cast<const float*>(p) + g);
        else return widen(__ldg(reinterpret_cast<const uint16_t*>(p) + g));
    }
};

constexpr uint32_t KEY_MIN = 0x00800000u;      // keys of -infinity lie below it

// The bits of a value that is not NaN, ordered like an unsigned integer; -0 equals +0.
__device__ __forceinline__ uint32_t order_bits(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// Over the L lanes of a row
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if constexpr (L == 32) {
        return __reduce_max_sync(FULL, v);
    } else {
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(FULL, v, d));
        return v;
    }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
    return v;
}

// NaN if any is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int L>
__device__ __forceinline__ float group_max_nan(float v) {
    if constexpr (L == 32) {
        float r;
        asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
        return r;
    } else {
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(FULL, v, d));
        return v;
    }
}

// e^x, zero below fp32's normal values: for probabilities that are summed.
__device__ __forceinline__ float exp_flush(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

struct RouterArgs {
    const uint8_t* logits;
    int64_t ld_bytes, T;
    int G, k, renorm, vec;
    int32_t* experts;     // [T, k]
    float* weights;       // [T, k]
    int32_t* counts;      // [G]
    float* loss;
    float* slope;         // [G]
    // several blocks: each one's probability sums [G], counts [G] and number of rows
    float* part_p;
    int32_t* part_c;
    int32_t* part_n;
};

// What turns an expert's count into its slope: G / (n k) / n.  Computed once a thread: this GPU's
// double precision is slow, a division a warp and expert cost the join 7 us.
__device__ __forceinline__ double slope_per_count(const RouterArgs& a, int64_t rows) {
    const double n = rows > 0 ? static_cast<double>(rows) : 1.0;
    return a.G / (n * n * a.k);
}

// counts, slope and this expert's term of the loss
__device__ __forceinline__ double finish_expert(const RouterArgs& a, int g, float sum, int32_t count, double per_count) {
    a.counts[g] = count;
    const double slope = per_count * count;
    a.slope[g] = static_cast<float>(slope);
    return slope * sum;
}

// Launch the joining of `blocks` blocks' partial sums after the kernel that writes them, as its programmatic dependent
// (tg_router.cu).
cudaError_t launch_join(const RouterArgs& a, int blocks, cudaStream_t stream);

// The checks of the arguments that the gates share (tg_router.cu).
tg_status check_router(const void* logits, tg_dtype dt, int64_t ld, int64_t T, int64_t G, int64_t k);
tg_status check_backward(int64_t G, tg_dtype dt, const int32_t* experts, const float* weights, bool weights_needed,
                         const float* slope, const float* d_weights, const float* d_loss, const void* d_logits, int64_t ldd);

// Raise a kernel's limit of dynamic shared memory where it needs more than the default.
template <class K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

}  // namespace gate
}  // namespace tg
