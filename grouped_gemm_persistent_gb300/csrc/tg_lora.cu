// tg_lora.cu - low-rank adapters of many requests, added to what a shared projection gave (tg_lora_add in include/tg.h):
//
//   out[t] = base[t] + scale[g] (x[t] A_g^T) B_g^T,   g = adapters[t], A_g [r, K], B_g [N, r]
//
// Bound by memory: x, base and out once, the adapters in use once; the products are 2 r (K + N) operations a row.
//
// Two forms.
//  - Rows (few rows of small rank): a row's u = x A^T is cut along K over blocks of 512, then a block takes a part of a
//    row's columns and adds the cuts.  Every row reads its own adapter, from L2 where rows share one: T r (K + N) 2 bytes.
//    Two launches, the second of which has its part of B and base in registers before it waits for the first.
//  - Tiles (more rows): a block of eight warps takes 16 or 32 rows.  The warps share K, each adding its part with
//    mma.sync (the products are few: tensor memory, which one thread feeds from shared-memory tiles, would have to be
//    refilled for every adapter of a tile); the parts are added in shared memory, u is scaled and cut into two
//    16-bit numbers, and the warps share the columns of the second product.  A tile whose rows have several adapters
//    goes through them one after the other, a row keeping only its own's result: a NaN of another adapter or row does
//    not reach it.
// Operands come straight from global memory in 16-byte loads: the order of k in a product is free, so a lane's eight
// neighbouring values stand for the two pairs that each of two mma.sync instructions wants of it; and the order of
// the columns is free, so a lane's results of four instructions are eight neighbouring columns of a row.
//
// Precision.  u is summed in fp32, times scale, and enters the second product as hi + lo of the operands' type (bf16: 16
// bits, 2^-17; fp16, of the row's power-of-two multiple that brings its largest value to 1..2: 22 bits): a single 16-bit u would
// add half a step of its own type to the adapters' part, as much as rounding the result does.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"
#include "tg_ptx.cuh"

namespace tg {

namespace {

constexpr uint32_t FULL = 0xffffffffu;
constexpr int L_WARPS = 8;
constexpr int L_THREADS = 32 * L_WARPS;
constexpr int ROW_CUT = 512;        // k of a block of the rows form

// Eight neighbouring 16-bit values
struct Half8 {
    uint32_t w[4];

    // n of the eight exist (the others are zero); vec: 16-byte loads allowed
    __device__ __forceinline__ void load(const uint8_t* p, int n, bool vec) {
        if (n >= 8 && vec) {
            const uint4 t = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p) + i)) << (i % 2 * 16);
    }
};

template <int DT>
__device__ __forceinline__ float widen(uint32_t b) {
    if constexpr (DT == TG_F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
    else return __uint_as_float(b << 16);
}

template <int DT>
__device__ __forceinline__ float value(const Half8& h, int i) { return widen<DT>(h.w[i / 2] >> (i % 2 * 16) & 0xffffu); }

template <int DT>
__device__ __forceinline__ uint32_t round16(float f) {
    if constexpr (DT == TG_F16) return __half_as_ushort(__float2half_rn(f));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

__device__ __forceinline__ int type_bytes(int dt) { return dt == TG_F32 ? 4 : 2; }

// One value of base or out
__device__ __forceinline__ float load_value(const uint8_t* p, int dt) {
    if (dt == TG_F32) return *reinterpret_cast<const float*>(p);
    const uint32_t b = *reinterpret_cast<const uint16_t*>(p);
    return dt == TG_F16 ? widen<TG_F16>(b) : widen<TG_BF16>(b);
}

__device__ __forceinline__ void store_value(uint8_t* p, int dt, float f) {
    if (dt == TG_F32) *reinterpret_cast<float*>(p) = f;
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(dt == TG_F16 ? round16<TG_F16>(f) : round16<TG_BF16>(f));
}

// Eight neighbouring values of base or out (plain loads: base may be out)
__device__ __forceinline__ void load_eight(float (&f)[8], const uint8_t* p, int dt, int n, bool vec) {
    if (n >= 8 && vec) {
        const uint4 t = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
        if (dt == TG_F32) {
            const uint4 s = *(reinterpret_cast<const uint4*>(p) + 1);
            const uint32_t v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = __uint_as_float(w[i]);
                f[4 + i] = __uint_as_float(v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = w[i / 2] >> (i % 2 * 16) & 0xffffu;
                f[i] = dt == TG_F16 ? widen<TG_F16>(b) : widen<TG_BF16>(b);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? load_value(p + i * type_bytes(dt), dt) : 0.0f;
}

__device__ __forceinline__ void store_eight(uint8_t* p, const float (&f)[8], int dt, int n, bool vec) {
    if (n >= 8 && vec) {
        if (dt == TG_F32) {
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
            *(reinterpret_cast<float4*>(p) + 1) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = dt == TG_F16 ? round16<TG_F16>(f[2 * i]) | round16<TG_F16>(f[2 * i + 1]) << 16
                                    : round16<TG_BF16>(f[2 * i]) | round16<TG_BF16>(f[2 * i + 1]) << 16;
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) store_value(p + i * type_bytes(dt), dt, f[i]);
}

template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (DT == TG_F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct LoraArgs {
    const uint8_t* x;
    int64_t ldx;                    // strides in bytes
    const uint8_t* a;
    int64_t lda, a_stride;
    const uint8_t* b;
    int64_t ldb, b_stride;
    const int32_t* adapters;
    const float* scale;             // null: ones
    const uint8_t* base;
    int64_t ldbase;
    uint8_t* out;
    int64_t ldo;
    float* part;                    // rows form: [cuts, T, r]
    int64_t T;
    int K, N, r, G, dt, cuts;
    int vec_x, vec_a, vec_b, vec_base, vec_out;
};

__device__ __forceinline__ bool has_adapter(const LoraArgs& p, int g) { return g >= 0 && g < p.G; }

// ----------------------------------------------------------------------------------------------------------- rows

// part[cut][t][j] = sum over the cut's k of x[t][k] A[j][k]: a warp takes every eighth j, a lane eight k of 256
template <int DT>
__global__ void __launch_bounds__(L_THREADS) lora_rows_down_kernel(const LoraArgs p) {
    ptx::grid_launch_dependents();
    const int64_t t = blockIdx.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = p.adapters[t];
    if (!has_adapter(p, g)) return;
    const int k = blockIdx.x * ROW_CUT + lane * 8;
    const uint8_t* xr = p.x + t * p.ldx + static_cast<int64_t>(k) * 2;
    const uint8_t* ar = p.a + g * p.a_stride + static_cast<int64_t>(k) * 2;
    Half8 x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) x[h].load(xr + h * 512, p.K - k - h * 256, p.vec_x);
    float* dst = p.part + (static_cast<int64_t>(blockIdx.x) * p.T + t) * p.r;
#pragma unroll 4
    for (int j = warp; j < p.r; j += L_WARPS) {
        Half8 a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) a[h].load(ar + j * p.lda + h * 512, p.K - k - h * 256, p.vec_a);
        float s = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(value<DT>(x[h], i), value<DT>(a[h], i), s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(FULL, s, d);
        if (lane == 0) dst[j] = s;
    }
}

// out[t][n] = base[t][n] + scale sum_j u[j] B[n][j]: `lanes` lanes take a column's ranks, eight each; four columns a lane
constexpr int UP_STEPS = 4;

template <int DT>
__global__ void __launch_bounds__(L_THREADS) lora_rows_up_kernel(const LoraArgs p, int lanes) {
    __shared__ float u[TG_LORA_MAX_RANK];
    const int64_t t = blockIdx.y;
    const int g = p.adapters[t];
    const bool mine = has_adapter(p, g);
    const int in = threadIdx.x % lanes, per_step = L_THREADS / lanes, size = type_bytes(p.dt);
    const int n0 = blockIdx.x * per_step * UP_STEPS + threadIdx.x / lanes;
    Half8 b[UP_STEPS];
    float base[UP_STEPS];
#pragma unroll
    for (int i = 0; i < UP_STEPS; ++i) {
        const int n = n0 + i * per_step;
        base[i] = in == 0 && n < p.N ? load_value(p.base + t * p.ldbase + static_cast<int64_t>(n) * size, p.dt) : 0.0f;
        b[i].load(p.b + (mine ? g : 0) * p.b_stride + n * p.ldb + in * 16, mine && n < p.N ? p.r - in * 8 : 0, p.vec_b);
    }
    ptx::grid_dependency_wait();
    if (threadIdx.x < TG_LORA_MAX_RANK) {
        float s = 0.0f;
        if (mine && threadIdx.x < p.r) {
#pragma unroll 8
            for (int c = 0; c < p.cuts; ++c) s += p.part[(c * p.T + t) * p.r + threadIdx.x];
            if (p.scale) s *= p.scale[g];
        }
        u[threadIdx.x] = s;
    }
    __syncthreads();
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = u[in * 8 + i];
#pragma unroll
    for (int i = 0; i < UP_STEPS; ++i) {
        const int n = n0 + i * per_step;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(w[j], value<DT>(b[i], j), s);
        for (int d = 1; d < lanes; d <<= 1) s += __shfl_xor_sync(FULL, s, d);
        if (in == 0 && n < p.N)
            store_value(p.out + t * p.ldo + static_cast<int64_t>(n) * size, p.dt, mine ? base[i] + s : base[i]);
    }
}

// ---------------------------------------------------------------------------------------------------------- tiles

// Ranks a block holds: 16, 32, 64 or 128; MT: 16-row parts of its tile
template <int RT, int MT>
struct TileShape {
    static constexpr int ROWS = 16 * MT;
    static constexpr int SUM_LD = RT + 8;                    // floats of a row of a warp's sums: no two rows of a store meet in a bank
    static constexpr int U_LD = RT + 8;                      // 16-bit values of a row of u
    static constexpr int SUM_BYTES = L_WARPS * ROWS * SUM_LD * 4;
    static constexpr int BYTES = SUM_BYTES + 2 * ROWS * U_LD * 2;
};

template <int DT, int RT, int MT>
__global__ void __launch_bounds__(L_THREADS, RT <= 64 ? 2 : 1) lora_tile_kernel(const __grid_constant__ LoraArgs p) {
    using S = TileShape<RT, MT>;
    constexpr int ROWS = S::ROWS, NT = RT / 8;
    extern __shared__ __align__(16) uint8_t dyn[];
    float* sums = reinterpret_cast<float*>(dyn);                                     // [warp][row][rank]
    uint16_t* u_hi = reinterpret_cast<uint16_t*>(dyn + S::SUM_BYTES);                // [row][rank]
    uint16_t* u_lo = u_hi + ROWS * S::U_LD;
    __shared__ int s_id[ROWS], s_adapter[ROWS], s_count;
    __shared__ float s_up[ROWS];                                                     // what takes a row's u back to its size
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, row8 = lane / 4, quad = lane % 4;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * ROWS;
    const int rows = p.T - t0 < ROWS ? static_cast<int>(p.T - t0) : ROWS;
    if (warp == 0) {
        // the rows' adapters, each once, in the order of their first rows
        int g = lane < rows ? p.adapters[t0 + lane] : -1;
        if (!has_adapter(p, g)) g = -1;
        const uint32_t same = __match_any_sync(FULL, g);
        const uint32_t first = __ballot_sync(FULL, g >= 0 && __ffs(same) - 1 == lane);
        if (lane < ROWS) s_id[lane] = g;
        if (first >> lane & 1u) s_adapter[__popc(first & ((1u << lane) - 1u))] = g;
        if (lane == 0) s_count = __popc(first);
    }
    __syncthreads();
    const int count = s_count;

    // this warp's part of K, a multiple of 32
    const int blocks = (p.K + 31) / 32;
    const int k_begin = static_cast<int>(static_cast<int64_t>(blocks) * warp / L_WARPS) * 32;
    const int k_end = static_cast<int>(static_cast<int64_t>(blocks) * (warp + 1) / L_WARPS) * 32;
    const uint8_t* xr[2 * MT];
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m) xr[m] = p.x + (t0 + m * 8 + row8) * p.ldx;
    for (int d = 0; d < count; ++d) {
        const int g = s_adapter[d];
        const uint8_t* ag = p.a + g * p.a_stride + row8 * p.lda;
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
#pragma unroll 2
        for (int k = k_begin; k < k_end; k += 32) {
            const int kl = k + quad * 8, left = p.K - kl;
            Half8 x[2 * MT], a[NT];
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m) x[m].load(xr[m] + static_cast<int64_t>(kl) * 2, m * 8 + row8 < rows ? left : 0, p.vec_x);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                a[j].load(ag + j * 8 * p.lda + static_cast<int64_t>(kl) * 2, j * 8 + row8 < p.r ? left : 0, p.vec_a);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        mma<DT>(acc[m][j], x[2 * m].w[2 * h], x[2 * m + 1].w[2 * h], x[2 * m].w[2 * h + 1], x[2 * m + 1].w[2 * h + 1],
                                a[j].w[2 * h], a[j].w[2 * h + 1]);
        }
        // a row keeps its own adapter's sums
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) {
            const int row = m * 8 + row8;
            if (s_id[row] != g) continue;
            float* dst = sums + (warp * ROWS + row) * S::SUM_LD + quad * 2;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                *reinterpret_cast<float2*>(dst + j * 8) = make_float2(acc[m / 2][j][m % 2 * 2], acc[m / 2][j][m % 2 * 2 + 1]);
        }
    }
    __syncthreads();
    // u of a row: the warps' parts added in order, times scale, as hi + lo
    for (int row = warp; row < ROWS; row += L_WARPS) {
        const int g = s_id[row];
        const float scale = g >= 0 && p.scale ? p.scale[g] : 1.0f;
        constexpr int PER = RT < 32 ? 1 : RT / 32;
        float u[PER];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = lane + 32 * i;
            u[i] = 0.0f;
            if (g >= 0 && j < RT) {
#pragma unroll
                for (int w = 0; w < L_WARPS; ++w) u[i] += sums[(w * ROWS + row) * S::SUM_LD + j];
                u[i] *= scale;
            }
            top = fmaxf(top, fabsf(u[i]));
        }
        float down = 1.0f, up = 1.0f;
        if constexpr (DT == TG_F16) {
            // 2^-e with the largest |u| in [2^e, 2^(e + 1)); left alone where it is zero, tiny or not finite
            const uint32_t e = __reduce_max_sync(FULL, __float_as_uint(top)) >> 23;
            if (e > 10u && e < 245u) {
                down = __uint_as_float((254u - e) << 23);
                up = __uint_as_float(e << 23);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = lane + 32 * i;
            if (j >= RT) continue;
            const float v = u[i] * down;
            const uint32_t hi = round16<DT>(v);
            const float rest = v - widen<DT>(hi);
            u_hi[row * S::U_LD + j] = static_cast<uint16_t>(hi);
            u_lo[row * S::U_LD + j] = static_cast<uint16_t>(fabsf(rest) < __int_as_float(0x7f800000) ? round16<DT>(rest) : 0u);
        }
        if (lane == 0) s_up[row] = up;
    }
    __syncthreads();

    // the columns, 32 a warp and step: a lane has the eight n = quad * 8 and on of its rows
    const int size = type_bytes(p.dt);
    for (int n0 = warp * 32; n0 < p.N; n0 += L_WARPS * 32) {
        const int n = n0 + quad * 8, left = p.N - n;
        float y[2 * MT][8];
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m)
            load_eight(y[m], p.base + (t0 + m * 8 + row8) * p.ldbase + static_cast<int64_t>(n) * size, p.dt,
                       m * 8 + row8 < rows ? left : 0, p.vec_base);
        for (int d = 0; d < count; ++d) {
            const int g = s_adapter[d];
            // column c of instruction i stands for n0 + (c / 2) * 8 + 2 i + c % 2
            const int col = n0 + (row8 / 2) * 8 + row8 % 2;
            const uint8_t* bg = p.b + g * p.b_stride + col * p.ldb;
            float acc[MT][4][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[m][i][c] = 0.0f;
            if constexpr (RT == 16) {
                // one instruction's 16 ranks: a lane's four neighbours
                uint2 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Half8 h;
                    const int have = col + 2 * i < p.N ? p.r - quad * 4 : 0;
                    const uint8_t* at = bg + 2 * i * p.ldb + quad * 8;
                    if (have >= 4 && p.vec_b) b[i] = __ldg(reinterpret_cast<const uint2*>(at));
                    else {
                        h.load(at, have < 4 ? have : 4, false);
                        b[i] = make_uint2(h.w[0], h.w[1]);
                    }
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint16_t* us = part ? u_lo : u_hi;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint2 a = *reinterpret_cast<const uint2*>(us + (m * 16 + row8) * S::U_LD + quad * 4);
                        const uint2 c = *reinterpret_cast<const uint2*>(us + (m * 16 + 8 + row8) * S::U_LD + quad * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma<DT>(acc[m][i], a.x, c.x, a.y, c.y, b[i].x, b[i].y);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < RT; j += 32) {
                    Half8 b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        b[i].load(bg + 2 * i * p.ldb + (j + quad * 8) * 2, col + 2 * i < p.N ? p.r - j - quad * 8 : 0, p.vec_b);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint16_t* us = part ? u_lo : u_hi;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 a = *reinterpret_cast<const uint4*>(us + (m * 16 + row8) * S::U_LD + j + quad * 8);
                            const uint4 c = *reinterpret_cast<const uint4*>(us + (m * 16 + 8 + row8) * S::U_LD + j + quad * 8);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                mma<DT>(acc[m][i], a.x, c.x, a.y, c.y, b[i].w[0], b[i].w[1]);
                                mma<DT>(acc[m][i], a.z, c.z, a.w, c.w, b[i].w[2], b[i].w[3]);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m) {
                const int row = m * 8 + row8;
                if (s_id[row] != g) continue;
                const float up = s_up[row];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[m][2 * i] = fmaf(acc[m / 2][i][m % 2 * 2], up, y[m][2 * i]);
                    y[m][2 * i + 1] = fmaf(acc[m / 2][i][m % 2 * 2 + 1], up, y[m][2 * i + 1]);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m)
            if (m * 8 + row8 < rows)
                store_eight(p.out + (t0 + m * 8 + row8) * p.ldo + static_cast<int64_t>(n) * size, y[m], p.dt, left, p.vec_out);
    }
}

using TileKernel = void (*)(const LoraArgs);
struct TileVariant {
    TileKernel kernel;
    int rows, bytes;
};

template <int DT, int RT, int MT>
TileVariant variant() { return {&lora_tile_kernel<DT, RT, MT>, TileShape<RT, MT>::ROWS, TileShape<RT, MT>::BYTES}; }

// Tiles of 32 rows read an adapter half as often; they are taken once 16-row tiles are more than two a SM.  (128 ranks:
// the sums of 32 rows would fill the registers.)
template <int DT>
TileVariant variant_for(int64_t T, int r, int sms) {
    const bool wide = (T + 15) / 16 > 2 * sms;
    if (r > 64) return variant<DT, 128, 1>();
    if (r > 32) return wide ? variant<DT, 64, 2>() : variant<DT, 64, 1>();
    if (r > 16) return wide ? variant<DT, 32, 2>() : variant<DT, 32, 1>();
    return wide ? variant<DT, 16, 2>() : variant<DT, 16, 1>();
}

// The rows form reads T r (K + N) 16-bit values through L2, whoever shares an adapter; the tile form streams an adapter
// through one SM at a time.
constexpr int64_t ROWS_FORM = 4096;      // largest T * r

tg_status check_operand(const char* name, const void* p, int64_t ld, int64_t cols, int64_t esize) {
    using host::fail;
    if (!p) return fail(TG_ERR_INVALID_ARG, "%s is NULL", name);
    if (ld < cols) return fail(TG_ERR_INVALID_ARG, "the leading dimension of %s, %lld, is below %lld", name, (long long)ld, (long long)cols);
    if (ld > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "the leading dimension of %s must be below 2^31", name);
    if (!host::aligned(p, esize)) return fail(TG_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    return TG_OK;
}

}  // namespace

}  // namespace tg

extern "C" tg_status tg_lora_add(const tg_lora_args* args, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    if (!args) return fail(TG_ERR_INVALID_ARG, "args is NULL");
    const tg_lora_args& p = *args;
    if (p.dtype != TG_BF16 && p.dtype != TG_F16) return fail(TG_ERR_INVALID_ARG, "bad dtype %d (bf16 or fp16)", int(p.dtype));
    if (p.base_dtype != TG_BF16 && p.base_dtype != TG_F16 && p.base_dtype != TG_F32)
        return fail(TG_ERR_INVALID_ARG, "bad base_dtype %d (bf16, fp16 or fp32)", int(p.base_dtype));
    if (p.T < 0 || p.K < 0 || p.N < 0 || p.r < 0 || p.G < 0)
        return fail(TG_ERR_INVALID_ARG, "negative size T=%lld K=%lld N=%lld r=%lld G=%lld", (long long)p.T, (long long)p.K,
                    (long long)p.N, (long long)p.r, (long long)p.G);
    if (p.T > host::MAX_DIM || p.K > host::MAX_DIM - 4096 || p.N > host::MAX_DIM - 4096 || p.G > host::MAX_DIM)
        return fail(TG_ERR_UNSUPPORTED, "sizes must be below 2^31 (K and N by 4096)");
    if (p.r > TG_LORA_MAX_RANK) return fail(TG_ERR_UNSUPPORTED, "r=%lld; adapters have a rank of at most %d", (long long)p.r, TG_LORA_MAX_RANK);
    if (p.T == 0 || p.N == 0) return TG_OK;
    const int64_t bs = p.base_dtype == TG_F32 ? 4 : 2;
    tg_status s = check_operand("base", p.base, p.ldbase, p.N, bs);
    if (s != TG_OK || (s = check_operand("out", p.out, p.ldo, p.N, bs)) != TG_OK) return s;
    if (!p.adapters) return fail(TG_ERR_INVALID_ARG, "adapters is NULL");
    if (!host::aligned(p.adapters, 4) || !host::aligned(p.scale, 4))
        return fail(TG_ERR_INVALID_ARG, "adapters or scale is not 4-byte aligned");
    const bool any = p.G > 0 && p.K > 0 && p.r > 0;          // without an adapter out is base
    if (any) {
        if ((s = check_operand("x", p.x, p.ldx, p.K, 2)) != TG_OK || (s = check_operand("a", p.a, p.lda, p.K, 2)) != TG_OK ||
            (s = check_operand("b", p.b, p.ldb, p.r, 2)) != TG_OK)
            return s;
        if (p.a_stride < 0 || p.b_stride < 0) return fail(TG_ERR_INVALID_ARG, "negative stride between adapters");
    }
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LoraArgs a{};
    a.x = static_cast<const uint8_t*>(p.x);
    a.ldx = p.ldx * 2;
    a.a = static_cast<const uint8_t*>(p.a);
    a.lda = p.lda * 2;
    a.a_stride = p.a_stride * 2;
    a.b = static_cast<const uint8_t*>(p.b);
    a.ldb = p.ldb * 2;
    a.b_stride = p.b_stride * 2;
    a.adapters = p.adapters;
    a.scale = p.scale;
    a.base = static_cast<const uint8_t*>(p.base);
    a.ldbase = p.ldbase * bs;
    a.out = static_cast<uint8_t*>(p.out);
    a.ldo = p.ldo * bs;
    a.T = p.T;
    a.K = static_cast<int>(p.K);
    a.N = static_cast<int>(p.N);
    a.r = static_cast<int>(p.r);
    a.G = any ? static_cast<int>(p.G) : 0;
    a.dt = p.base_dtype;
    auto vec = [](const void* q, int64_t ld, int64_t stride) { return host::aligned(q, 16) && ld % 16 == 0 && stride % 16 == 0; };
    a.vec_x = vec(p.x, a.ldx, 0);
    a.vec_a = vec(p.a, a.lda, a.a_stride);
    a.vec_b = vec(p.b, a.ldb, a.b_stride);
    a.vec_base = vec(p.base, a.ldbase, 0);
    a.vec_out = vec(p.out, a.ldo, 0);
    cudaError_t e;
    if (any && p.T * p.r <= ROWS_FORM) {
        a.cuts = (a.K + ROW_CUT - 1) / ROW_CUT;
        void* ws = nullptr;
        const size_t bytes = static_cast<size_t>(a.cuts) * p.T * p.r * 4;
        if ((s = host::workspace(bytes, st, "cudaMallocFromPoolAsync(adapters' sums)", &ws)) != TG_OK) return s;
        a.part = static_cast<float*>(ws);
        const dim3 grid(static_cast<unsigned>(a.cuts), static_cast<unsigned>(p.T), 1);
        if (p.dtype == TG_F16) lora_rows_down_kernel<TG_F16><<<grid, L_THREADS, 0, st>>>(a);
        else lora_rows_down_kernel<TG_BF16><<<grid, L_THREADS, 0, st>>>(a);
        e = cudaGetLastError();
        if (e == cudaSuccess) {
            host::count_launches(1);
            int lanes = 1;
            while (lanes * 8 < a.r) lanes *= 2;
            const int cols = L_THREADS / lanes * UP_STEPS;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>((a.N + cols - 1) / cols), static_cast<unsigned>(p.T), 1);
            cfg.blockDim = dim3(L_THREADS, 1, 1);
            cfg.stream = st;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = p.dtype == TG_F16 ? cudaLaunchKernelEx(&cfg, lora_rows_up_kernel<TG_F16>, static_cast<const LoraArgs&>(a), lanes)
                                  : cudaLaunchKernelEx(&cfg, lora_rows_up_kernel<TG_BF16>, static_cast<const LoraArgs&>(a), lanes);
            if (e == cudaSuccess) host::count_launches(1);
        }
        s = e == cudaSuccess ? TG_OK : host::cuda_fail(e, "adapters launch");
        e = cudaFreeAsync(ws, st);
        if (e != cudaSuccess && s == TG_OK) s = host::cuda_fail(e, "cudaFreeAsync(adapters' sums)");
        return s;
    }
    const TileVariant v = p.dtype == TG_F16 ? variant_for<TG_F16>(p.T, a.r, d.sms) : variant_for<TG_BF16>(p.T, a.r, d.sms);
    e = v.bytes > 48 * 1024 ? cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.bytes) : cudaSuccess;
    if (e == cudaSuccess) {
        v.kernel<<<static_cast<unsigned>((p.T + v.rows - 1) / v.rows), L_THREADS, v.bytes, st>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return host::cuda_fail(e, "adapters launch");
    host::count_launches(1);
    return TG_OK;
}
