// tg_norm.cuh - what the norm (tg_norm.cu) and its gradients (tg_norm_backward.cu) share: eight values of a row, the gain in
// shared memory, how a row is spread over threads, the checks of matrix arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"
#include "tg_ptx.cuh"

namespace tg {

namespace norm {

constexpr uint32_t FULL = 0xffffffffu;
constexpr int N_MAX_K = TG_RMSNORM_MAX_COLUMNS;
constexpr size_t FREE_SMEM = 40 * 1024;       // dynamic shared memory that is there without asking: 48 KB with the kernels' own

constexpr int item_bytes(int dt) { return dt == TG_F32 ? 4 : 2; }

template <int DT>
__device__ __forceinline__ float widen16(uint32_t b) {
    if constexpr (DT == TG_F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
    else return __uint_as_float(b << 16);
}

// How the lanes hold a row.  WHOLE, ODD: eight neighbouring values each, rows on 16-byte boundaries, of whole vectors or not.  APART: rows
// that start elsewhere; the sixteen lanes of a block of 128 values hold every sixteenth value of it, so that a load or a store of a
// warp is two runs of neighbours.  (40970 x 4095 bf16 without padding, bf16 residual: into e4m3 600 us with eight neighbours read
// one by one, 366 apart; gradients 570 and 343.  A row of whole blocks read without checks instead: 543 and 435, the 16-bit
// values being put together, and waited for, inside the branch.)
enum Form : int { ODD, WHOLE, APART };

// The first value of the v-th lane, and how many values it has (eight or more: eight)
template <int FORM>
__device__ __forceinline__ int first_of(int v) { return FORM == APART ? (v & ~15) * 8 + (v & 15) : v * 8; }
template <int FORM>
__device__ __forceinline__ int count_of(int first, int K) { return FORM == APART ? (K - first + 15) >> 4 : K - first; }
template <int FORM>
constexpr int STRIDE = FORM == APART ? 16 : 1;

// Eight values of a row, as they lie in memory
template <int DT>
struct Oct {
    static constexpr int WORDS = DT == TG_F32 ? 8 : 4;
    uint32_t w[WORDS];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    // Plain loads: the memory may be an output of the same call.
    __device__ __forceinline__ void load_whole(const uint8_t* p) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            const uint4 t = *(reinterpret_cast<const uint4*>(p) + i / 4);
            w[i] = t.x; w[i + 1] = t.y; w[i + 2] = t.z; w[i + 3] = t.w;
        }
    }
    // n of the eight are inside the row; WHOLE: eight or none, 16-byte loads; ODD, wide: the same, with values past the row's end
    // that cut() takes away (one by one they would have to be waited for here)
    template <int FORM>
    __device__ __forceinline__ void load(const uint8_t* p, int n, bool wide) {
        zero();
        if (FORM == WHOLE || (FORM == ODD && wide)) {
            if (n > 0) load_whole(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= n) continue;
                if constexpr (DT == TG_F32) w[i] = reinterpret_cast<const uint32_t*>(p)[i * STRIDE<FORM>];
                else w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i * STRIDE<FORM>]) << (i % 2 * 16);
            }
        }
    }
    // the values from n on become zero
    template <int FORM>
    __device__ __forceinline__ void cut(int n) {
        if constexpr (FORM == ODD) {
            if (n >= 8 || n <= 0) return;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                if constexpr (DT == TG_F32) w[i] = i < n ? w[i] : 0u;
                else w[i] &= 2 * i + 1 < n ? 0xffffffffu : 2 * i < n ? 0xffffu : 0u;
            }
        }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (DT == TG_F32) return __uint_as_float(w[i]);
        else if constexpr (DT == TG_BF16) return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else return widen16<DT>(w[i / 2] >> (i % 2 * 16) & 0xffffu);
    }
    // values 2 i and 2 i + 1, side by side for the two-at-once operations
    __device__ __forceinline__ uint64_t pair(int i) const { return ptx::f32x2_pack(value(2 * i), value(2 * i + 1)); }
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
    template <int FORM>
    __device__ __forceinline__ void store(uint8_t* p, int n) const {
        if (FORM == WHOLE ? n > 0 : FORM == ODD && n >= 8) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4)
                reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        } else if constexpr (FORM != WHOLE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= n) continue;
                if constexpr (DT == TG_F32) reinterpret_cast<uint32_t*>(p)[i * STRIDE<FORM>] = w[i];
                else reinterpret_cast<uint16_t*>(p)[i * STRIDE<FORM>] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
            }
        }
    }
};

template <int DT, int FORM>
__device__ __forceinline__ void store8(uint8_t* p, const float (&f)[8], int n) {
    Oct<DT> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.set2(i, f[2 * i], f[2 * i + 1]);
    o.template store<FORM>(p, n);
}

// One value of the gain, or 1
__device__ __forceinline__ float gain_value(const uint8_t* gain, int dt, int64_t col) {
    if (!gain) return 1.0f;
    if (dt == TG_F32) return reinterpret_cast<const float*>(gain)[col];
    const uint32_t b = reinterpret_cast<const uint16_t*>(gain)[col];
    return dt == TG_F16 ? widen16<TG_F16>(b) : widen16<TG_BF16>(b);
}

// The gain as fp32 in shared memory, up to a whole vector: a block's rows all want it.  Loads go ahead of the stores, four a thread.
template <int DT>
__device__ __forceinline__ void stage_values(float* to, const uint8_t* gain, int K) {
    constexpr int AHEAD = 4;
    const int vectors = (K + 7) / 8;
    const bool vec = reinterpret_cast<uintptr_t>(gain) % 16 == 0;
    for (int base = threadIdx.x; base < vectors; base += AHEAD * blockDim.x) {
        Oct<DT> o[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int v = base + i * blockDim.x, n = v < vectors ? K - v * 8 : 0;
            o[i].template load<ODD>(gain + static_cast<int64_t>(v) * 8 * item_bytes(DT), n, vec && n >= 8);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int v = base + i * blockDim.x;
            if (v >= vectors) break;
            float4* at = reinterpret_cast<float4*>(to + v * 8);
            at[0] = make_float4(o[i].value(0), o[i].value(1), o[i].value(2), o[i].value(3));
            at[1] = make_float4(o[i].value(4), o[i].value(5), o[i].value(6), o[i].value(7));
        }
    }
}

__device__ __forceinline__ void stage_gain(float* to, const uint8_t* gain, int dt, int K) {
    if (!gain) {
        for (int i = threadIdx.x; i < (K + 7) / 8 * 8; i += blockDim.x) to[i] = 1.0f;
    } else if (dt == TG_F32) {
        stage_values<TG_F32>(to, gain, K);
    } else if (dt == TG_F16) {
        stage_values<TG_F16>(to, gain, K);
    } else {
        stage_values<TG_BF16>(to, gain, K);
    }
    __syncthreads();
}

// The gain of a lane's values, n of them inside the row
template <int FORM>
__device__ __forceinline__ void read_gain(float (&g)[8], const float* from, int n) {
    if constexpr (FORM == APART) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = i < n ? from[i * STRIDE<FORM>] : 0.0f;
    } else {
        const float4 a = *reinterpret_cast<const float4*>(from), b = *(reinterpret_cast<const float4*>(from) + 1);
        g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
        g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
    }
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
    int64_t wide;                // rows before this one may be read in whole vectors (ODD)
    float eps, inv_hi, inv_lo;
};

constexpr int N_NONE = -1;          // no residual

using NormKernel = void (*)(const NormArgs);

// How a row is spread over a block: its threads, and vectors of eight values a thread
struct Spread {
    int threads, nv;
};

inline Spread spread(int64_t K, int nv) {
    const int64_t vectors = (K + 7) / 8;
    return {static_cast<int>((vectors + 32 * nv - 1) / (32 * nv) * 32), nv};
}

// The kernel for x of type XT and a residual (none, or of x's type or fp32).  Defined in tg_norm_inst.cu, compiled once for each XT.
template <int XT>
NormKernel norm_for(bool residual, tg_dtype rt, const Spread& s, Form form);

// How many blocks of a kernel an SM holds, asked of the driver once for each kernel, block size and device.
template <class K>
cudaError_t resident(K kernel, int threads, size_t smem, int device, int* out) {
    struct Known {
        const void* kernel;
        int threads, device, blocks;
        size_t smem;
    };
    static thread_local Known known[64];
    static thread_local int count = 0;
    for (int i = 0; i < count; ++i)
        if (known[i].kernel == reinterpret_cast<const void*>(kernel) && known[i].threads == threads && known[i].smem == smem && known[i].device == device) {
            *out = known[i].blocks;
            return cudaSuccess;
        }
    if (smem > FREE_SMEM) {
        // the limit of the longest rows, whatever these are: a lower one would take it from rows that were asked for before
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, N_MAX_K * 4);
        if (e != cudaSuccess) return e;
    }
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    *out = n < 1 ? 1 : n;
    known[count < 64 ? count++ : 63] = {reinterpret_cast<const void*>(kernel), threads, device, *out, smem};
    return cudaSuccess;
}

inline bool value_type(tg_dtype t) { return t == TG_BF16 || t == TG_F16 || t == TG_F32; }

// A row-major matrix argument: its pointer, leading dimension and alignment
inline tg_status check_matrix(const char* name, const void* p, int64_t ld, int64_t K, int64_t esize) {
    using host::fail;
    if (!p) return fail(TG_ERR_INVALID_ARG, "%s is NULL", name);
    if (ld < K) return fail(TG_ERR_INVALID_ARG, "the leading dimension of %s, %lld, is below K=%lld", name, (long long)ld, (long long)K);
    if (ld > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "the leading dimension of %s must be below 2^31", name);
    if (!host::aligned(p, esize)) return fail(TG_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    return TG_OK;
}

inline tg_status check_sizes(int64_t M, int64_t K) {
    using host::fail;
    if (M < 0 || K < 0) return fail(TG_ERR_INVALID_ARG, "negative size M=%lld K=%lld", (long long)M, (long long)K);
    if (M > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "M must be below 2^31");
    if (K > N_MAX_K) return fail(TG_ERR_UNSUPPORTED, "K=%lld columns; the norm takes at most %d", (long long)K, N_MAX_K);
    return TG_OK;
}

// How many of a matrix's M rows of K values may be read in whole vectors of eight without passing the end of its last row
inline int64_t wide_rows(int64_t M, int64_t K, int64_t ld) {
    const int64_t past = (K + 7) / 8 * 8 - K, last = (past + ld - 1) / ld;
    return M > last ? M - last : 0;
}

inline Form form_of(bool on_boundaries, int64_t K) { return !on_boundaries ? APART : K % 8 ? ODD : WHOLE; }

inline bool vectors_of(const void* p, int64_t ld_bytes) { return host::aligned(p, 16) && ld_bytes % 16 == 0; }

}  // namespace norm

}  // namespace tg
