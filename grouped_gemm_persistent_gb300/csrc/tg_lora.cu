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
//  - Tiles (more rows).  A kernel of one cluster orders the rows by adapter, each adapter's filled up to whole tiles, so that
//    any order of the rows reads an adapter once a tile.  A cluster takes a tile: its blocks share k, add their parts of u over
//    distributed shared memory, and share the columns.  x and A go through a ring of stages (cp.async: the rows are gathered) into
//    mma.sync; u is cut into two 16-bit numbers for the second product, whose B and base come through the same ring.  (mma.sync
//    and not tcgen05.mma: the operations take 16 % of its rate, 605 TFLOP/s measured, and an accumulator of 16 to 128 columns
//    would be read back after a few thousand cycles, for every adapter of a tile anew.)  A tile may hold several adapters (more
//    than 512 of them share buckets): it goes through them one after the other, a row keeping only its own's result, so that a
//    NaN of another adapter or row does not reach it.
// The order of the second product's columns is free: B's rows are laid out so that a lane's results are neighbouring columns.
//
// What it took, 8191 rows of K 4096, N 1536, rank 64, 16 adapters (19 us at the copy rate): operands from global memory to
// registers, tiles of neighbouring rows 131 us (tiles of several adapters took as many times as long); rows ordered, k through the
// ring, clusters 81; fewer instructions a stage 54; the order by a cluster instead of a block 52; B and base through the ring and u
// put together by rows 49; whole stages copied without checks, a stage's operands loaded before its products 43.  Now about 10 us of
// it go before the first stage (the order, two launches), 19 into the first product (141 MB through L2: A is read once a tile)
// and 14 into the second.
//
// Precision.  u is summed in fp32, times scale, and enters the second product as hi + lo of the operands' type (bf16: 16
// bits, 2^-17, of a multiple next to the ends of its range; fp16, of the row's power-of-two multiple that brings its largest value to
// 1..2: 22 bits): a single 16-bit u would add half a step of its own type to the adapters' part, as much as rounding the result does.
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
constexpr int FREE_SMEM = 40 * 1024;       // dynamic shared memory that is there without asking: 48 KB with the kernels' own

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

// Neighbouring values of a row of base and then of out, as they lie in memory
template <int BT, int COUNT>
struct Columns {
    static constexpr int SIZE = BT == TG_F32 ? 4 : 2, WORDS = COUNT * SIZE / 4;
    uint32_t w[WORDS];

    // from column `col` of a row in shared memory whose 16-byte pieces are where piece ^ key says
    __device__ __forceinline__ void read(uint32_t row, int col, int key) {
        if constexpr (WORDS == 2) {
            const int at = col * SIZE;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(row + (((at / 16) ^ key) * 16) + at % 16));
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                             : "r"(row + (((col * SIZE / 16 + i / 4) ^ key) * 16)));
        }
    }
    // a and b added to values 2 i and 2 i + 1, in fp32, rounded to the type
    __device__ __forceinline__ void add2(int i, float a, float b) {
        if constexpr (BT == TG_F32) {
            w[2 * i] = __float_as_uint(__uint_as_float(w[2 * i]) + a);
            w[2 * i + 1] = __float_as_uint(__uint_as_float(w[2 * i + 1]) + b);
        } else if constexpr (BT == TG_F16) {
            const __half2 h = __floats2half2_rn(widen<TG_F16>(w[i] & 0xffffu) + a, widen<TG_F16>(w[i] >> 16) + b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) + a, __uint_as_float(w[i] & 0xffff0000u) + b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    // n of them exist; vec: whole vectors, n a multiple of their count
    __device__ __forceinline__ void store(uint8_t* p, int n, bool vec) const {
        if (vec) {
            if (n <= 0) return;
            if constexpr (WORDS == 2) {
                *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int i = 0; i < WORDS; i += 4) reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            if (i >= n) continue;
            if constexpr (BT == TG_F32) reinterpret_cast<uint32_t*>(p)[i] = w[i];
            else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
        }
    }
};

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

// Where the tiles' rows are: an adapter's rows side by side in their own order, each bucket of adapters (those that agree
// modulo `buckets`; the rows without one are a bucket of their own) filled up to whole tiles with -1.
struct Plan {
    int2* rows;         // [tiles * tile_rows]: a row, and its adapter or -1
    int32_t* tiles;
    int buckets, tile_rows;
};

constexpr int PLAN_WARPS = 32;
constexpr int PLAN_BATCH = 8;          // rows of a lane in registers
constexpr int MAX_BUCKETS = 512;
constexpr int MAX_CTAS = 8;            // of a tile's cluster

// A cluster's blocks, and a block's warps, take neighbouring rows: two passes, counting and placing.  A warp's 32 rows are most
// often one bucket's, which a vote sees; only others take match.any, which is slow.  (One block of 32 warps is short of issue
// slots: 9 us for 8191 rows.)
constexpr int PLAN_CTAS = 8;

__global__ void __cluster_dims__(PLAN_CTAS, 1, 1) __launch_bounds__(32 * PLAN_WARPS)
    lora_plan_kernel(const int32_t* __restrict__ adapters, int64_t T, int G, const Plan plan) {
    ptx::grid_launch_dependents();
    extern __shared__ int32_t place[];                           // [warp][bucket], buckets + 1 of them
    __shared__ int32_t s_scan[PLAN_WARPS], s_total[MAX_BUCKETS + 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, count = plan.buckets + 1;
    const uint32_t rank = ptx::cluster_ctarank();
    int32_t* mine = place + warp * count;
    for (int i = threadIdx.x; i < PLAN_WARPS * count; i += 32 * PLAN_WARPS) place[i] = 0;
    __syncthreads();
    constexpr int CHUNK = 32 * PLAN_WARPS * PLAN_CTAS;
    const int64_t each = (T + CHUNK - 1) / CHUNK * 32;
    const int64_t begin = (static_cast<int64_t>(rank) * PLAN_WARPS + warp) * each, end = begin + each < T ? begin + each : T;
    auto pass = [&](bool write) {
        for (int64_t base = begin; base < end; base += 32 * PLAN_BATCH) {
            int id[PLAN_BATCH];
#pragma unroll
            for (int i = 0; i < PLAN_BATCH; ++i) {
                const int64_t row = base + 32 * i + lane;
                id[i] = row < end ? adapters[row] : -1;
            }
#pragma unroll
            for (int i = 0; i < PLAN_BATCH; ++i) {
                const int64_t row = base + 32 * i + lane;
                if (base + 32 * i >= end) break;
                const bool valid = id[i] >= 0 && id[i] < G;
                const int key = row >= end ? -1 : !valid ? plan.buckets : G > plan.buckets ? id[i] % plan.buckets : id[i];
                const uint32_t same = __all_sync(FULL, key == __shfl_sync(FULL, key, 0)) ? FULL : __match_any_sync(FULL, key);
                const int at = key >= 0 ? mine[key] : 0;
                const int before = __popc(same & ((1u << lane) - 1u));
                if (write && key >= 0) plan.rows[at + before] = make_int2(static_cast<int>(row), valid ? id[i] : -1);
                __syncwarp();
                if (key >= 0 && before == 0) mine[key] = at + __popc(same);
                __syncwarp();
            }
        }
    };
    pass(false);
    __syncthreads();
    // a thread a bucket: its rows, and where it starts
    const int b = threadIdx.x;
    int n[PLAN_WARPS], total = 0, ahead = 0;
    if (b < count) {
#pragma unroll
        for (int w = 0; w < PLAN_WARPS; ++w) n[w] = place[w * count + b];
#pragma unroll
        for (int w = 0; w < PLAN_WARPS; ++w) total += n[w];
        s_total[b] = total;
    }
    ptx::cluster_sync();
    if (b < count) {
        const uint32_t here = ptx::smem_u32(s_total + b);
        total = 0;
#pragma unroll
        for (uint32_t c = 0; c < PLAN_CTAS; ++c) {
            const int other = static_cast<int>(ptx::ld_cluster_u32(ptx::mapa(here, c)));
            total += other;
            ahead += c < rank ? other : 0;
        }
    }
    ptx::cluster_arrive();                                       // (no block leaves before the others have read its totals)
    const int padded = (total + plan.tile_rows - 1) / plan.tile_rows * plan.tile_rows;
    int start = padded;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(FULL, start, d);
        if (lane >= d) start += o;
    }
    if (lane == 31) s_scan[warp] = start;
    __syncthreads();
    for (int w = 0; w < warp; ++w) start += s_scan[w];
    start -= padded;
    if (b < count) {
        int at = start + ahead;
#pragma unroll
        for (int w = 0; w < PLAN_WARPS; ++w) {
            place[w * count + b] = at;
            at += n[w];
        }
        if (rank == 0) {
            for (int i = total; i < padded; ++i) plan.rows[start + i] = make_int2(-1, -1);
            if (b == count - 1) *plan.tiles = (start + padded) / plan.tile_rows;
        }
    }
    __syncthreads();
    pass(true);
    ptx::cluster_wait();
}

// A block: RT ranks (16, 32, 64 or 128) and ROWS rows.  Eight warps.  First product: WM along the rows, two along the ranks, WK
// along k.  Second: WM along the rows, the others along the columns, TILES instructions of eight columns each.
template <int RT, int ROWS, int SIZE>
struct Tile {
    static constexpr int WM = ROWS / 16, WN = 2, WK = L_WARPS / (WM * WN);
    static constexpr int NW = RT / 8 / WN;                       // instructions' columns of a warp in the first product
    static constexpr int STAGE = (ROWS + RT) * 128;              // 64 k: 128 bytes of each row of x and of A
    static constexpr int STAGES = STAGE > 18432 ? 3 : STAGE > 12288 ? 4 : STAGE > 6144 ? 6 : 8;
    static constexpr int TILES = WM == 4 ? 4 : 2, COLS = L_WARPS / WM * TILES * 8;
    static constexpr int BASE_ROW = COLS * SIZE;                 // bytes of a row's part of base
    static constexpr int OUT_STAGE = COLS * RT * 2 + ROWS * BASE_ROW;
    static constexpr int FIT = STAGES * STAGE / OUT_STAGE;
    static constexpr int OUT_STAGES = FIT < 2 ? 2 : FIT > 6 ? 6 : FIT;
    static constexpr int RING = STAGES * STAGE > OUT_STAGES * OUT_STAGE ? STAGES * STAGE : OUT_STAGES * OUT_STAGE;
    static constexpr int SUM_LD = RT + 8;                        // floats: no two rows of a store meet in a bank
    static constexpr int U_LD = RT + 8;                          // 16-bit values of a row of u
    static constexpr int SUM_BYTES = WK * ROWS * SUM_LD * 4;
    static constexpr int BYTES = RING + SUM_BYTES + 2 * ROWS * U_LD * 2;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}

__device__ __forceinline__ void ldmatrix2(uint32_t& r0, uint32_t& r1, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(at));
}

// Sixteen bytes of a row into shared memory, n values of them (the rest zero), where they are not copied whole
__device__ __forceinline__ void copy_values(uint32_t dst, const uint8_t* src, int n) {
    Half8 h;
    h.load(src, n, false);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(dst), "r"(h.w[0]), "r"(h.w[1]), "r"(h.w[2]), "r"(h.w[3]) : "memory");
}

// The same of values of SIZE bytes: 16 bytes, n values of them
template <int SIZE>
__device__ __forceinline__ void copy_piece(uint32_t dst, const uint8_t* src, int n) {
    if constexpr (SIZE == 2) {
        copy_values(dst, src, n);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = i < n ? reinterpret_cast<const uint32_t*>(src)[i] : 0u;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
}

template <int DT, int BT, int RT, int ROWS>
__global__ void __launch_bounds__(L_THREADS, 2) lora_tile_kernel(const __grid_constant__ LoraArgs p, const Plan plan) {
    constexpr int SIZE = BT == TG_F32 ? 4 : 2;
    using S = Tile<RT, ROWS, SIZE>;
    extern __shared__ __align__(128) uint8_t dyn[];
    float* sums = reinterpret_cast<float*>(dyn + S::RING);                           // [WK][row][rank]
    uint16_t* u_hi = reinterpret_cast<uint16_t*>(dyn + S::RING + S::SUM_BYTES);      // [row][rank], and u_lo behind it
    __shared__ int s_row[ROWS], s_id[ROWS], s_adapter[ROWS], s_count;
    __shared__ float s_up[ROWS];                                                     // what takes a row's u back to its size
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, row8 = lane / 4, quad = lane % 4;
    const int ctas = static_cast<int>(ptx::cluster_nctarank()), rank = static_cast<int>(ptx::cluster_ctarank());
    const int tile = blockIdx.x / ctas;
    ptx::grid_dependency_wait();
    int2 own = make_int2(-1, -1);
    if (threadIdx.x < ROWS) own = plan.rows[static_cast<int64_t>(tile) * ROWS + threadIdx.x];
    if (tile >= *plan.tiles) return;                 // (the whole cluster)
    if (threadIdx.x < ROWS) {
        s_row[threadIdx.x] = own.x;
        s_id[threadIdx.x] = own.y;
    }
    __syncthreads();
    if (warp == 0) {
        // the rows' adapters, each once, in the order of their first rows
        int count = 0;
#pragma unroll
        for (int i = 0; i < ROWS; i += 32) {
            const int g = i + lane < ROWS ? s_id[i + lane] : -1;
            bool seen = g < 0;
            for (int j = 0; j < count; ++j) seen |= s_adapter[j] == g;
            const uint32_t same = __match_any_sync(FULL, g);
            const uint32_t first = __ballot_sync(FULL, !seen && __ffs(same) - 1 == lane);
            __syncwarp();
            if (first >> lane & 1u) s_adapter[count + __popc(first & ((1u << lane) - 1u))] = g;
            count += __popc(first);
            __syncwarp();
        }
        if (lane == 0) s_count = count;
    }
    __syncthreads();
    const int count = s_count;

    // ---- u = x A^T: this block's part of k, 64 at a time through a ring of stages.  A thread copies the same 16 bytes of a row's
    // 128 in every stage.
    constexpr int XN = (ROWS * 8 + L_THREADS - 1) / L_THREADS, AN = (RT * 8 + L_THREADS - 1) / L_THREADS;
    const int blocks = (p.K + 63) / 64;
    const int first_block = static_cast<int>(static_cast<int64_t>(blocks) * rank / ctas);
    const int steps = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / ctas) - first_block;
    const int wm = warp % S::WM, wn = warp / S::WM % S::WN, wk = warp / (S::WM * S::WN);
    const uint32_t ring = ptx::smem_u32(dyn);
    const int my_row = threadIdx.x / 8, k_mine = first_block * 64 + threadIdx.x % 8 * 8;
    const uint32_t copy_at = ring + my_row * 128 + ((threadIdx.x ^ my_row) & 7) * 16;     // (the same place in every 32nd row on)
    const uint32_t x_at = ring + (wm * 16 + lane % 16) * 128 + ((lane / 16) ^ lane % 8) * 16;
    const uint32_t a_at = ring + ROWS * 128 + (wn * S::NW * 8 + lane % 8 + (S::NW > 1 ? lane / 16 * 8 : 0)) * 128 + ((lane / 8 % 2) ^ lane % 8) * 16;
    for (int d = 0; d < count; ++d) {
        const int g = s_adapter[d];
        const uint8_t *xp[XN], *ap[AN];
        int x_size[XN], a_size[AN];                  // bytes of a whole copy: 16, or none
#pragma unroll
        for (int i = 0; i < XN; ++i) {
            const int row = my_row + 32 * i;
            x_size[i] = row < ROWS && s_id[row < ROWS ? row : 0] == g ? 16 : 0;
            xp[i] = p.x + (x_size[i] ? s_row[row] * p.ldx + static_cast<int64_t>(k_mine) * 2 : 0);
        }
#pragma unroll
        for (int i = 0; i < AN; ++i) {
            const int row = my_row + 32 * i;
            a_size[i] = row < p.r ? 16 : 0;
            ap[i] = p.a + (a_size[i] ? g * p.a_stride + row * p.lda + static_cast<int64_t>(k_mine) * 2 : 0);
        }
        // stages are fetched one after the other: the pointers go along
        const int whole = p.vec_x && p.vec_a ? p.K / 64 - first_block : 0;       // stages before this one are whole
        auto fetch = [&](int step, uint32_t slot) {
            const uint32_t to = copy_at + slot * S::STAGE;
            if (step < whole) {
#pragma unroll
                for (int i = 0; i < XN; ++i) {
                    if (ROWS >= 32 || threadIdx.x < ROWS * 8) ptx::cp_async_16_part(to + i * 4096, xp[i], x_size[i]);
                    xp[i] += x_size[i] * 8;
                }
#pragma unroll
                for (int i = 0; i < AN; ++i) {
                    if (RT >= 32 || threadIdx.x < RT * 8) ptx::cp_async_16_part(to + ROWS * 128 + i * 4096, ap[i], a_size[i]);
                    ap[i] += a_size[i] * 8;
                }
                return;
            }
            const int left = p.K - k_mine - step * 64, n = left < 0 ? 0 : left < 8 ? left : 8;
#pragma unroll
            for (int i = 0; i < XN; ++i) {
                if (ROWS < 32 && threadIdx.x >= ROWS * 8) break;
                const uint8_t* src = n > 0 && x_size[i] ? xp[i] : p.x;
                if (p.vec_x) ptx::cp_async_16_part(to + i * 4096, src, x_size[i] ? 2 * n : 0);
                else copy_values(to + i * 4096, src, x_size[i] ? n : 0);
                xp[i] += x_size[i] * 8;
            }
#pragma unroll
            for (int i = 0; i < AN; ++i) {
                if (RT < 32 && threadIdx.x >= RT * 8) break;
                const uint8_t* src = n > 0 && a_size[i] ? ap[i] : p.a;
                if (p.vec_a) ptx::cp_async_16_part(to + ROWS * 128 + i * 4096, src, a_size[i] ? 2 * n : 0);
                else copy_values(to + ROWS * 128 + i * 4096, src, a_size[i] ? n : 0);
                ap[i] += a_size[i] * 8;
            }
        };
        float acc[S::NW][4];
#pragma unroll
        for (int j = 0; j < S::NW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i) {
            if (i < steps) fetch(i, i);
            ptx::cp_async_commit();
        }
        uint32_t slot = 0, next = S::STAGES - 1;
        for (int step = 0; step < steps; ++step) {
            ptx::cp_async_wait<S::STAGES - 2>();
            __syncthreads();
            if (step + S::STAGES - 1 < steps) fetch(step + S::STAGES - 1, next);
            ptx::cp_async_commit();
            const uint32_t xs = x_at + slot * S::STAGE, as = a_at + slot * S::STAGE;
            slot = slot + 1 == S::STAGES ? 0 : slot + 1;
            next = next + 1 == S::STAGES ? 0 : next + 1;
            // the operands of as many k as fit, then their products: the loads' latencies lie over one another
            // (a stage's products are added up by themselves: an instruction's sum is cut off, not rounded, and a chain of them along
            // the whole of k would drift)
            constexpr int KS = 4 / S::WK, BATCH = S::NW > 4 && KS > 2 ? 2 : KS;
            float part[S::NW][4];
#pragma unroll
            for (int n = 0; n < S::NW; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[n][i] = 0.0f;
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += BATCH) {
                uint32_t a[BATCH][4], b[BATCH][S::NW * 2];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const uint32_t flip = static_cast<uint32_t>((k0 + k) * S::WK + wk) * 32;   // (chunk ^ row: its low bit with the row, then its others)
                    ldmatrix4(a[k], xs ^ flip);
                    if constexpr (S::NW == 1) {
                        ldmatrix2(b[k][0], b[k][1], as ^ flip);
                    } else {
#pragma unroll
                        for (int n = 0; n < S::NW; n += 2)
                            ldmatrix4(*reinterpret_cast<uint32_t(*)[4]>(b[k] + 2 * n), (as ^ flip) + n * 1024);
                    }
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k)
#pragma unroll
                    for (int n = 0; n < S::NW; ++n)
                        mma<DT>(part[n], a[k][0], a[k][1], a[k][2], a[k][3], b[k][2 * n], b[k][2 * n + 1]);
            }
#pragma unroll
            for (int n = 0; n < S::NW; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] += part[n][i];
        }
        // a row keeps its own adapter's sums
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = wm * 16 + h * 8 + row8;
            if (s_id[row] != g) continue;
            float* dst = sums + (wk * ROWS + row) * S::SUM_LD + wn * S::NW * 8 + quad * 2;
#pragma unroll
            for (int j = 0; j < S::NW; ++j) *reinterpret_cast<float2*>(dst + j * 8) = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
        }
        __syncthreads();                             // the next adapter's first stages, and u, go where these were
    }
    // ---- out = base + u B^T: this block's columns, COLS at a time through the same ring (its first stages are on their way while u
    // is put together).  With several adapters a part of the columns takes a step for each of them, base coming with the first.
    const int groups = (p.N + S::COLS - 1) / S::COLS;
    const int first_group = static_cast<int>(static_cast<int64_t>(groups) * rank / ctas);
    const int turns = count > 0 ? count : 1;         // (no adapter: base alone)
    const int out_steps = (static_cast<int>(static_cast<int64_t>(groups) * (rank + 1) / ctas) - first_group) * turns;
    constexpr int CHUNKS = RT / 8;                   // 16 bytes of a row of B
    constexpr int COPIES = S::COLS * CHUNKS, BN = (COPIES + L_THREADS - 1) / L_THREADS, YN = ROWS * S::BASE_ROW / 16 / L_THREADS;
    static_assert(YN > 0 && (COPIES < L_THREADS || COPIES % L_THREADS == 0) && ROWS * S::BASE_ROW / 16 % L_THREADS == 0, "whole copies");
    constexpr int KEYS = CHUNKS < 8 ? CHUNKS : 8, KEY_SHIFT = CHUNKS == 2 ? 2 : CHUNKS == 4 ? 1 : 0;
    constexpr int GROUP = S::TILES * 8, LANE = S::TILES * 2;     // columns of a warp, and of a lane (neighbours)
    constexpr int PIECES = S::BASE_ROW / 16;
    // where a thread's copies go, and for whole groups of columns and one adapter where they come from (the pointers go along)
    uint32_t b_to[BN], y_to[YN];
    const uint8_t *bp[BN], *yp[YN];
    int b_size[BN], y_size[YN];
#pragma unroll
    for (int i = 0; i < BN; ++i) {
        // a row of B goes where ldmatrix wants it: column c of instruction i of a warp stands for its column
        // (c / 2) * LANE + 2 i + c % 2, so that a lane's results are neighbours
        const int c = threadIdx.x + i * L_THREADS, chunk = c % CHUNKS, col = c / CHUNKS, in = col % GROUP;
        const int at = col - in + in % LANE / 2 * 8 + in / LANE * 2 + in % 2;
        b_to[i] = ring + at * (RT * 2) + ((chunk ^ (at >> KEY_SHIFT & (KEYS - 1))) * 16);
        b_size[i] = count > 0 && chunk * 8 < p.r ? 16 : 0;
        bp[i] = p.b + (b_size[i] ? s_adapter[0] * p.b_stride + (static_cast<int64_t>(first_group) * S::COLS + col) * p.ldb + chunk * 16 : 0);
    }
#pragma unroll
    for (int i = 0; i < YN; ++i) {
        const int c = threadIdx.x + i * L_THREADS, piece = c % PIECES, at = c / PIECES, row = s_row[at];
        y_to[i] = ring + S::COLS * RT * 2 + at * S::BASE_ROW + ((piece ^ (at & 7)) * 16);
        y_size[i] = row >= 0 ? 16 : 0;
        yp[i] = p.base + (row >= 0 ? row * p.ldbase + static_cast<int64_t>(first_group) * S::BASE_ROW + piece * 16 : 0);
    }
    const int64_t b_step = S::COLS * p.ldb;
    const int whole_out = p.vec_b && p.vec_base && turns == 1 ? p.N / S::COLS - first_group : 0;
    int fetch_turn = 0, fetch_group = 0;             // of the next step to be fetched
    auto fetch_out = [&](uint32_t slot) {
        const uint32_t shift = slot * S::OUT_STAGE;
        if (fetch_group < whole_out) {
#pragma unroll
            for (int i = 0; i < BN; ++i) {
                if (COPIES >= L_THREADS || threadIdx.x < COPIES) ptx::cp_async_16_part(b_to[i] + shift, bp[i], b_size[i]);
                bp[i] += b_size[i] ? b_step : 0;
            }
#pragma unroll
            for (int i = 0; i < YN; ++i) {
                ptx::cp_async_16_part(y_to[i] + shift, yp[i], y_size[i]);
                yp[i] += y_size[i] * (S::BASE_ROW / 16);
            }
            ++fetch_group;
            return;
        }
        const int n0 = (first_group + fetch_group) * S::COLS;
        if (count > 0) {
            const uint8_t* bg = p.b + s_adapter[fetch_turn] * p.b_stride;
#pragma unroll
            for (int i = 0; i < BN; ++i) {
                const int c = threadIdx.x + i * L_THREADS, chunk = c % CHUNKS, n = n0 + c / CHUNKS;
                if (COPIES < L_THREADS && c >= COPIES) break;
                const int have = n < p.N ? p.r - chunk * 8 : 0;
                const uint8_t* src = have > 0 ? bg + n * p.ldb + chunk * 16 : p.b;
                if (p.vec_b) ptx::cp_async_16_part(b_to[i] + shift, src, have > 0 ? 16 : 0);       // (r is a multiple of 8)
                else copy_values(b_to[i] + shift, src, have);
            }
        }
        if (fetch_turn == 0) {
#pragma unroll
            for (int i = 0; i < YN; ++i) {
                const int c = threadIdx.x + i * L_THREADS, row = s_row[c / PIECES], n = n0 + c % PIECES * (16 / SIZE);
                const bool wanted = row >= 0 && n < p.N;
                const uint8_t* src = wanted ? p.base + row * p.ldbase + static_cast<int64_t>(n) * SIZE : p.base;
                if (p.vec_base) ptx::cp_async_16_part(y_to[i] + shift, src, wanted ? 16 : 0);      // (N is a multiple of 8)
                else copy_piece<SIZE>(y_to[i] + shift, src, wanted ? p.N - n : 0);
            }
        }
        if (++fetch_turn == turns) {
            fetch_turn = 0;
            ++fetch_group;
        }
    };
#pragma unroll
    for (int i = 0; i < S::OUT_STAGES - 1; ++i) {
        if (i < out_steps) fetch_out(i);
        ptx::cp_async_commit();
    }
    if constexpr (S::WK > 1) {
        for (int i = threadIdx.x; i < ROWS * RT; i += L_THREADS) {
            float* at = sums + i / RT * S::SUM_LD + i % RT;
            float s = at[0];
#pragma unroll
            for (int w = 1; w < S::WK; ++w) s += at[w * ROWS * S::SUM_LD];
            at[0] = s;
        }
    }
    if (ctas > 1) ptx::cluster_sync();
    else __syncthreads();
    // u of a row: the blocks' parts added in order, times scale, as hi + lo.  A block does its share of the rows for the whole
    // cluster.
    constexpr int PER = RT < 64 ? 2 : RT / 32;       // neighbouring ranks of a lane
    for (int row = ROWS * static_cast<int>(rank) / ctas + warp; row < ROWS * (static_cast<int>(rank) + 1) / ctas; row += L_WARPS) {
        const int g = s_id[row];
        const bool on = lane * PER < RT;
        const float scale = g >= 0 && p.scale ? p.scale[g] : 1.0f;
        float u[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) u[i] = 0.0f;
        if (g >= 0 && on) {
            const uint32_t here = ptx::smem_u32(sums + row * S::SUM_LD + lane * PER);
            if (ctas == 1) {
#pragma unroll
                for (int i = 0; i < PER; ++i) u[i] = sums[row * S::SUM_LD + lane * PER + i];
            } else {
                float part[MAX_CTAS][PER];
#pragma unroll
                for (int c = 0; c < MAX_CTAS; ++c)
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        part[c][i] = c < ctas ? __uint_as_float(ptx::ld_cluster_u32(ptx::mapa(here, c) + 4 * i)) : 0.0f;
#pragma unroll
                for (int c = 0; c < MAX_CTAS; ++c)
#pragma unroll
                    for (int i = 0; i < PER; ++i) u[i] += part[c][i];
            }
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            // (the ranks that fill up to RT are zeros of A: with an infinity in x they would be NaN)
            u[i] = lane * PER + i < p.r ? u[i] * scale : 0.0f;
            if (fabsf(u[i]) < __int_as_float(0x7f800000)) top = fmaxf(top, fabsf(u[i]));
        }
        // fp16: 2^-e with the largest finite |u| in [2^e, 2^(e + 1)) (beside an infinity the others stay numbers).  bf16 has fp32's range:
        // 2^64 or 2^-64 where u or what is left of it would pass an end of that, which keeps the products with any B inside.
        const uint32_t e = __reduce_max_sync(FULL, __float_as_uint(top)) >> 23;
        const uint32_t to = DT == TG_F16 ? (e < 1u ? 1u : e > 253u ? 253u : e) : e < 32u ? 63u : e > 252u ? 191u : 127u;
        const float down = __uint_as_float((254u - to) << 23), up = __uint_as_float(to << 23);      // (both normal numbers)
        uint32_t hi[PER / 2], lo[PER / 2];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float v = u[i] * down;
            const uint32_t h = round16<DT>(v);
            const float rest = v - widen<DT>(h);
            const uint32_t l = fabsf(rest) < __int_as_float(0x7f800000) ? round16<DT>(rest) : 0u;
            hi[i / 2] = i % 2 ? hi[i / 2] | h << 16 : h;
            lo[i / 2] = i % 2 ? lo[i / 2] | l << 16 : l;
        }
        const uint32_t at = ptx::smem_u32(u_hi + row * S::U_LD + lane * PER), scale_at = ptx::smem_u32(s_up + row);
        for (int c = 0; c < ctas; ++c) {
            const uint32_t there = ptx::mapa(at, c);
            if (on) {
#pragma unroll
                for (int i = 0; i < PER / 2; ++i) {
                    ptx::st_cluster_u32(there + 4 * i, hi[i]);
                    ptx::st_cluster_u32(there + ROWS * S::U_LD * 2 + 4 * i, lo[i]);
                }
            }
            if (lane == 0) ptx::st_cluster_u32(ptx::mapa(scale_at, c), __float_as_uint(up));
        }
    }
    if (ctas > 1) {
        ptx::cluster_arrive();
        ptx::cluster_wait();
    } else {
        __syncthreads();
    }
    // this warp's 16 rows of u, for all of its columns: k = 16 j and on of part h
    uint32_t u[2][RT / 16][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < RT / 16; ++j)
            ldmatrix4(u[h][j], ptx::smem_u32(u_hi + (h * ROWS + wm * 16 + lane % 16) * S::U_LD + j * 16 + lane / 16 * 8));
    const int group = warp / S::WM;                  // of columns
    const int low = wm * 16 + row8, row[2] = {s_row[low], s_row[low + 8]}, id[2] = {s_id[low], s_id[low + 8]};
    const float up[2] = {s_up[low], s_up[low + 8]};
    const uint32_t b_row = group * GROUP + lane % 8 + lane / 16 * 8;
    const uint32_t b_at = ring + b_row * (RT * 2), b_key = b_row >> KEY_SHIFT & (KEYS - 1);
    const uint32_t y_at = ring + S::COLS * RT * 2 + low * S::BASE_ROW;
    Columns<BT, LANE> y[2];
    uint8_t* out[2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
        out[m] = p.out + (row[m] < 0 ? 0 : row[m]) * p.ldo + (static_cast<int64_t>(first_group) * S::COLS + group * GROUP + quad * LANE) * SIZE;
    int turn = 0, left = p.N - first_group * S::COLS - group * GROUP - quad * LANE;      // columns from this lane's first on
    uint32_t slot = 0, next = S::OUT_STAGES - 1;
    for (int step = 0; step < out_steps; ++step) {
        ptx::cp_async_wait<S::OUT_STAGES - 2>();
        __syncthreads();
        if (step + S::OUT_STAGES - 1 < out_steps) fetch_out(next);
        ptx::cp_async_commit();
        const uint32_t shift = slot * S::OUT_STAGE;
        slot = slot + 1 == S::OUT_STAGES ? 0 : slot + 1;
        next = next + 1 == S::OUT_STAGES ? 0 : next + 1;
        if (turn == 0) {
            y[0].read(y_at + shift, group * GROUP + quad * LANE, low & 7);
            y[1].read(y_at + shift + 8 * S::BASE_ROW, group * GROUP + quad * LANE, low & 7);
        }
        if (count > 0) {
            float acc[S::TILES][4];
#pragma unroll
            for (int i = 0; i < S::TILES; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
            constexpr int KS = RT / 16, BATCH = S::TILES == 4 && KS > 2 ? 2 : KS < 4 ? KS : 4;
#pragma unroll
            for (int j0 = 0; j0 < KS; j0 += BATCH) {
                uint32_t b[BATCH][S::TILES * 2];
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
#pragma unroll
                    for (int i = 0; i < S::TILES; i += 2)
                        ldmatrix4(*reinterpret_cast<uint32_t(*)[4]>(b[j] + 2 * i),
                                  b_at + shift + i * 8 * (RT * 2) + (((2 * (j0 + j) + lane / 8 % 2) ^ b_key) * 16));
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < S::TILES; ++i)
                            mma<DT>(acc[i], u[h][j0 + j][0], u[h][j0 + j][1], u[h][j0 + j][2], u[h][j0 + j][3], b[j][2 * i], b[j][2 * i + 1]);
            }
            const int g = s_adapter[turn];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (id[m] != g) continue;
#pragma unroll
                for (int i = 0; i < S::TILES; ++i)
                    y[m].add2(i, acc[i][2 * m] * up[m], acc[i][2 * m + 1] * up[m]);
            }
        }
        if (++turn == turns) {
            turn = 0;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (row[m] >= 0) y[m].store(out[m], left, p.vec_out);
                out[m] += S::COLS * SIZE;
            }
            left -= S::COLS;
        }
    }
}

using TileKernel = void (*)(const LoraArgs, const Plan);
struct TileVariant {
    TileKernel kernel;
    int rows, bytes;
};

template <int DT, int BT, int RT, int ROWS>
TileVariant variant() { return {&lora_tile_kernel<DT, BT, RT, ROWS>, ROWS, Tile<RT, ROWS, BT == TG_F32 ? 4 : 2>::BYTES}; }

// Tiles of 64 rows (32 above 64 ranks, for their sums' room) read an adapter less often; tiles of 16 where an adapter has fewer than 32
// rows on average, if all of them are in use.  8191 rows, K 4096, N 1536, rank 64, 64-row against 16-row tiles, us: one adapter
// 43 / 56, 16 adapters 44 / 57, 64 66 / 57, 128 78 / 59, 200 73 / 72, 300 80 / 87, 512 144 / 99.  (Between a few adapters and the border
// neither is better throughout: 16384 rows at rank 128 over 600 adapters take 108 us in 32-row tiles and 160 in 16-row ones.  It goes by
// the adapters there are, the host not knowing which are in use: 512 of them, of which the rows name 10, 51 / 57.)
template <int DT, int BT>
TileVariant variant_for(int64_t T, int G, int r) {
    const bool tall = T >= 32 * static_cast<int64_t>(G);
    if (r > 64) return tall ? variant<DT, BT, 128, 32>() : variant<DT, BT, 128, 16>();
    if (r > 32) return tall ? variant<DT, BT, 64, 64>() : variant<DT, BT, 64, 16>();
    if (r > 16) return tall ? variant<DT, BT, 32, 64>() : variant<DT, BT, 32, 16>();
    return tall ? variant<DT, BT, 16, 64>() : variant<DT, BT, 16, 16>();
}

template <int DT>
TileVariant variant_for(tg_dtype base, int64_t T, int G, int r) {
    return base == TG_F32 ? variant_for<DT, TG_F32>(T, G, r) : base == TG_F16 ? variant_for<DT, TG_F16>(T, G, r)
                                                                              : variant_for<DT, TG_BF16>(T, G, r);
}

// The rows form reads T r (K + N) 16-bit values through L2, whoever shares an adapter; the tile form takes 10 to 14 us however few the
// rows are.  Rows / tiles, us, at the nearest measured sizes below and above the border (T r (K + N) in millions of 2^20):
//   K = N = 4096, r 16  16 M: 10.6 / 12.0   24 M: 14.2 / 12.1      K = N = 4096, r 64  16 M: 11.7 / 12.8   32 M: 17.9 / 13.7
//   K = N = 1024, r 16  16 M: 10.0 / 12.2   32 M: 17.2 / 13.3      K = N = 512, r 64   16 M: 10.7 / 10.4   24 M: 13.4 / 10.5
//   K 8192, N 1024, r 8 18 M: 11.9 / 11.9   27 M: 15.0 / 12.2      K 1024, N 8192, r 32 18 M: 14.0 / 14.4  36 M: 23.0 / 14.7
constexpr int64_t ROWS_FORM = 21 << 20, ROWS_FORM_T = 4096;      // largest T r (K + N), and T

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
    a.vec_b = vec(p.b, a.ldb, a.b_stride) && a.r % 8 == 0;          // (whole vectors only, as of base and out)
    a.vec_base = vec(p.base, a.ldbase, 0) && a.N % 8 == 0;
    a.vec_out = vec(p.out, a.ldo, 0) && a.N % 8 == 0;
    cudaError_t e;
    if (any && p.T <= ROWS_FORM_T && p.T * p.r * (p.K + p.N) <= ROWS_FORM) {
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
    const TileVariant v = p.dtype == TG_F16 ? variant_for<TG_F16>(p.base_dtype, p.T, a.G, a.r)
                                               : variant_for<TG_BF16>(p.base_dtype, p.T, a.G, a.r);
    // at most one tile a bucket is not full
    const int64_t buckets = a.G < 1 ? 1 : a.G < MAX_BUCKETS ? a.G : MAX_BUCKETS;
    const int64_t used = p.T < buckets + 1 ? p.T : buckets + 1, tiles = (p.T + v.rows - 1) / v.rows + used;
    if (tiles * v.rows > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "T=%lld rows are too many", (long long)p.T);
    void* ws = nullptr;
    if ((s = host::workspace(static_cast<size_t>(tiles * v.rows + 2) * 8, st, "cudaMallocFromPoolAsync(adapters' plan)", &ws)) != TG_OK) return s;
    const Plan plan{static_cast<int2*>(ws) + 2, static_cast<int32_t*>(ws), int(buckets), v.rows};
    // Few tiles share each one's k and columns among the blocks of a cluster, up to about two blocks an SM.
    const int64_t likely = (p.T + v.rows - 1) / v.rows > used - 1 ? (p.T + v.rows - 1) / v.rows : used - 1;
    int ctas = 1;
    while (ctas < MAX_CTAS && likely * ctas * 2 <= 2 * d.sms && a.K >= ctas * 512) ctas *= 2;
    const int plan_bytes = PLAN_WARPS * int(buckets + 1) * 4;
    // (the limit of the most buckets, whatever these are: another thread's call may be between here and its launch)
    constexpr int MOST_PLAN_BYTES = PLAN_WARPS * (MAX_BUCKETS + 1) * 4;
    e = plan_bytes > FREE_SMEM ? cudaFuncSetAttribute(lora_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_PLAN_BYTES) : cudaSuccess;
    if (e == cudaSuccess && v.bytes > FREE_SMEM)
        e = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.bytes);
    if (e == cudaSuccess) {
        lora_plan_kernel<<<PLAN_CTAS, 32 * PLAN_WARPS, plan_bytes, st>>>(p.adapters, p.T, a.G, plan);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) {
        host::count_launches(1);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(tiles * ctas), 1, 1);
        cfg.blockDim = dim3(L_THREADS, 1, 1);
        cfg.dynamicSmemBytes = v.bytes;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, v.kernel, static_cast<const LoraArgs&>(a), plan);
        if (e == cudaSuccess) host::count_launches(1);
    }
    s = e == cudaSuccess ? TG_OK : host::cuda_fail(e, "adapters launch");
    e = cudaFreeAsync(ws, st);
    if (e != cudaSuccess && s == TG_OK) s = host::cuda_fail(e, "cudaFreeAsync(adapters' plan)");
    return s;
}
