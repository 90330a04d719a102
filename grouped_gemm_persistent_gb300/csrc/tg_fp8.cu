// tg_fp8.cu - host side of the 8-bit products (tg_gemm_scaled and tg_moe_gemm_scaled in
// include/tg.h): argument checks, tensor maps, the choice of tile and the launch.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "tg.h"
#include "tg_fp8.cuh"
#include "tg_host.cuh"

namespace tg {

namespace {

using host::fail;

template <class Cfg>
cudaError_t launch_fp8(const Params& p, const Fp8Params& x, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(F8_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = Cfg::SPLIT ? static_cast<unsigned>(x.splits) : Cfg::CTA_GROUP;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, &fp8_kernel<Cfg>, p, x);
}

// Clusters of `cluster` CTAs (single CTAs, pairs, or the CTAs that share a tile) that can be resident
// at once; asked once per device, kernel and size, before the first launch there, and sets the
// kernel's shared memory limit.
template <class Cfg>
cudaError_t units_fp8(int cluster, int* units) {
    auto kern = &fp8_kernel<Cfg>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster), 1, 1);
    cfg.blockDim = dim3(F8_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(units, kern, &cfg);
}

struct Fp8Variant {
    cudaError_t (*launch)(const Params&, const Fp8Params&, int, cudaStream_t);
    cudaError_t (*units)(int, int*);
    int cta_group;
};

template <int CG, bool SBC, bool MOE, bool SPLIT = false>
constexpr Fp8Variant fp8_variant() {
    using C = Fp8Config<CG, SBC, MOE, SPLIT>;
    return Fp8Variant{&launch_fp8<C>, &units_fp8<C>, CG};
}

enum : int { FORM_BLOCK = 0, FORM_COLUMN = 1, FORM_MOE = 2, FORM_BLOCK_SPLIT = 3, FORM_COLUMN_SPLIT = 4, FORMS = 5 };

// [form][CTA pair]; split tiles are single CTAs'
const Fp8Variant kFp8[FORMS][2] = {
    {fp8_variant<1, false, false>(), fp8_variant<2, false, false>()},
    {fp8_variant<1, true, false>(), fp8_variant<2, true, false>()},
    {fp8_variant<1, false, true>(), fp8_variant<2, false, true>()},
    {fp8_variant<1, false, false, true>(), {}},
    {fp8_variant<1, true, false, true>(), {}},
};

constexpr int kMaxDevices = 64;
constexpr int kMaxSplitLog = 3;                // at most 8 CTAs share a tile
std::mutex g_units_mu;
int g_units[kMaxDevices][FORMS][kMaxSplitLog + 1];      // [log2 of the cluster's size]

// Resident clusters of 2^log CTAs of a form's kernel
tg_status resident(const host::Device& d, int form, int log, int* units) {
    std::lock_guard<std::mutex> lock(g_units_mu);
    int& u = g_units[d.id][form][log];
    if (u <= 0) {
        const bool split = form == FORM_BLOCK_SPLIT || form == FORM_COLUMN_SPLIT;
        const cudaError_t e = kFp8[form][split ? 0 : log].units(1 << log, &u);
        if (e != cudaSuccess) return host::cuda_fail(e, "occupancy query");
    }
    *units = u;
    return TG_OK;
}

// One operand: `rows` x K with its scales, rows being A's rows or B's columns.
tg_status check_operand(const tg_scaled_operand* o, const char* name, int64_t rows, int64_t K, tg_layout k_major) {
    if (o->dtype != TG_E4M3 && o->dtype != TG_E5M2)
        return fail(TG_ERR_INVALID_ARG, "%s: bad dtype %d (e4m3 or e5m2)", name, int(o->dtype));
    if (o->layout != TG_ROW_MAJOR && o->layout != TG_COL_MAJOR)
        return fail(TG_ERR_INVALID_ARG, "%s: bad layout %d", name, int(o->layout));
    if (o->block != 1 && o->block != 128) return fail(TG_ERR_INVALID_ARG, "%s: bad block %d (1 or 128)", name, o->block);
    if (K == 0 || rows == 0) return TG_OK;
    if (!o->data) return fail(TG_ERR_INVALID_ARG, "%s: data is NULL", name);
    if (!o->scale) return fail(TG_ERR_INVALID_ARG, "%s: scale is NULL", name);
    const int64_t inner = o->layout == k_major ? K : rows;
    if (o->ld < inner) return fail(TG_ERR_INVALID_ARG, "%s: ld=%lld < %lld", name, (long long)o->ld, (long long)inner);
    if (o->scale_stride < 0 || o->scale_k_stride < 0) return fail(TG_ERR_INVALID_ARG, "%s: negative scale stride", name);
    if (o->ld > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "%s: ld must be below 2^31", name);
    if (!host::aligned(o->scale, 4)) return fail(TG_ERR_INVALID_ARG, "%s: scale is not 4-byte aligned", name);
    if (!host::aligned(o->data, 16) || o->ld % 16)
        return fail(TG_ERR_UNSUPPORTED, "%s: data must be 16-byte aligned with ld a multiple of 16 (TMA)", name);
    return TG_OK;
}

tg_status check_output(const void* C, tg_dtype cd, int64_t ldc, int64_t M, int64_t N, int64_t K, tg_epilogue epi,
                       const void* bias) {
    if (cd != TG_BF16 && cd != TG_F32 && cd != TG_F16) return fail(TG_ERR_INVALID_ARG, "bad c_dtype %d", int(cd));
    if (epi != TG_EPI_NONE && epi != TG_EPI_BIAS && epi != TG_EPI_BIAS_GELU)
        return fail(TG_ERR_INVALID_ARG, "bad epilogue %d", int(epi));
    if (M < 0 || N < 0 || K < 0)
        return fail(TG_ERR_INVALID_ARG, "negative size M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
    if (M > host::MAX_DIM || N > host::MAX_DIM || K > host::MAX_DIM)
        return fail(TG_ERR_UNSUPPORTED, "sizes must be below 2^31");
    if (M == 0 || N == 0) return TG_OK;
    if (!C) return fail(TG_ERR_INVALID_ARG, "C is NULL");
    if (ldc < N) return fail(TG_ERR_INVALID_ARG, "ldc=%lld < N=%lld", (long long)ldc, (long long)N);
    if (ldc > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "ldc must be below 2^31");
    if (!host::aligned(C, cd == TG_F32 ? 4 : 2)) return fail(TG_ERR_INVALID_ARG, "C is not aligned to its element size");
    if (epi != TG_EPI_NONE && !bias) return fail(TG_ERR_INVALID_ARG, "epilogue needs a bias");
    if (bias && !host::aligned(bias, 2)) return fail(TG_ERR_INVALID_ARG, "bias is not 2-byte aligned");
    return TG_OK;
}

// Everything both forms fill alike.  rows: rows of A; experts: 0 for the dense form.
struct Fp8Call {
    const tg_scaled_operand *A, *B;
    int64_t rows, N, K;
    void* C;
    tg_dtype c_dtype;
    int64_t ldc;
    tg_epilogue epi;
    const void* bias;
    int64_t experts, expert_stride, scale_stride;
    const int32_t* counts;
};

// log2 of the CTAs that share each 128 x 128 tile of a dense launch with fewer tiles than SMs: the
// largest, at most 3, with every cluster resident and at least two k-blocks a CTA.  A cluster lies
// within one part of the GPU, so fewer fit than SMs would: 15 of eight CTAs and 36 of four, and one
// more costs a second wave (a row, K 4096: 15 tiles 7.5 us, 16 tiles 12.4 in clusters of eight and
// 8.0 in clusters of four).  1 x 4096 x 4096: 16.5 us with one CTA a tile (32 of them), 8.7 with four.
// TG_STREAM_K=0 keeps tiles whole.
tg_status pick_splits(const Fp8Call& c, const host::Device& d, int form, int* log) {
    *log = 0;
    const char* env = std::getenv("TG_STREAM_K");
    if (env && env[0] == '0') return TG_OK;
    const int64_t tiles = ((c.rows + 127) / 128) * ((c.N + 127) / 128), kb = (c.K + F8_BK - 1) / F8_BK;
    while (*log < kMaxSplitLog && tiles << (*log + 1) <= d.sms && kb >= int64_t(4) << *log) {
        int units = 0;
        const tg_status s = resident(d, form, *log + 1, &units);
        if (s != TG_OK) return s;
        if (tiles > units) break;
        ++*log;
    }
    return TG_OK;
}

tg_status run_fp8(const Fp8Call& c, cudaStream_t stream) {
    host::Device d;
    tg_status s = host::device(&d);
    if (s != TG_OK || (s = host::encoder()) != TG_OK) return s;
    const bool moe = c.experts > 0;
    int form = moe ? FORM_MOE : c.B->block == 1 ? FORM_COLUMN : FORM_BLOCK;

    // CTA pairs (256 x 256 tiles) once there are more 128 x 128 tiles than SMs.  4096 columns, K 4096:
    // 512 rows 17.1 us in pairs and 15.2 us in single CTAs, 768 rows 21.1 and 26.0.  Experts fill pair
    // tiles from an average of 256 rows on: 64 of them, K 1536, N 4096, 2048 rows 93 us in pairs and
    // 72 us in single CTAs, 8192 rows 124 and 115, 16384 rows 182 and 184.
    const int64_t tiles = ((c.rows + 127) / 128) * ((c.N + 127) / 128);
    int pair = tiles > d.sms && (!moe || c.rows >= 256 * c.experts) ? 1 : 0;
    if (const char* env = std::getenv("TG_TILE")) {
        int cg = 0, bn = 0;
        if (std::sscanf(env, "%dx%d", &cg, &bn) == 2 && (cg == 1 || cg == 2)) pair = cg - 1;
    }
    int log = 0, units = 0;
    if (!moe && !pair) {
        const int split_form = form == FORM_COLUMN ? FORM_COLUMN_SPLIT : FORM_BLOCK_SPLIT;
        if ((s = pick_splits(c, d, split_form, &log)) != TG_OK) return s;
        if (log > 0) form = split_form;
    }
    const int splits = 1 << log;
    const Fp8Variant& v = kFp8[form][pair];
    if ((s = resident(d, form, log + pair, &units)) != TG_OK) return s;
    if (units <= 0) return fail(TG_ERR_UNSUPPORTED, "the 8-bit kernel cannot be resident on this device");

    const int tile = 128 * v.cta_group;
    Params p;
    std::memset(&p, 0, sizeof p);
    Fp8Params x;
    std::memset(&x, 0, sizeof x);
    Problem& q = p.dense;
    const bool a_mn = c.A->layout == TG_COL_MAJOR, b_mn = c.B->layout == TG_ROW_MAJOR;
    if (c.K > 0) {
        const uint64_t K = static_cast<uint64_t>(c.K), M = static_cast<uint64_t>(c.rows), N = static_cast<uint64_t>(c.N);
        const uint32_t box[3] = {128, 128, 1};
        // A row-major A of fewer than 128 rows is loaded in boxes of that many (the rows of shared
        // memory past them hold anything: they only feed rows of the product that are not stored).
        // Boxes with 127 rows outside the matrix made 1 x 19456 x 8192 take 48 us.
        const uint32_t a_rows = a_mn || c.rows >= 128 ? 128u : static_cast<uint32_t>((c.rows + 7) / 8 * 8);
        const uint32_t a_box[2] = {128, a_rows};
        x.a_bytes = 128 * a_rows;
        const uint64_t ad[2] = {a_mn ? M : K, a_mn ? K : M}, as[1] = {static_cast<uint64_t>(c.A->ld)};
        if ((s = host::encode_bytes(&q.tma_a, c.A->data, 2, ad, as, a_box, "A")) != TG_OK) return s;
        const uint64_t bd[3] = {b_mn ? N : K, b_mn ? K : N, static_cast<uint64_t>(moe ? c.experts : 1)};
        const uint64_t bs[2] = {static_cast<uint64_t>(c.B->ld), static_cast<uint64_t>(c.expert_stride)};
        if ((s = host::encode_bytes(&q.tma_b, c.B->data, moe ? 3 : 2, bd, bs, box, "B")) != TG_OK) return s;
    }
    q.bias = c.epi != TG_EPI_NONE ? c.bias : nullptr;
    q.M = static_cast<int32_t>(c.rows);
    q.N = static_cast<int32_t>(c.N);
    q.K = static_cast<int32_t>(c.K);
    q.epi = static_cast<int32_t>(c.epi);
    q.tiles_m = static_cast<int32_t>((c.rows + tile - 1) / tile);
    q.tiles_n = static_cast<int32_t>((c.N + tile - 1) / tile);
    q.k_blocks = static_cast<int32_t>((c.K + F8_BK - 1) / F8_BK);
    q.replicas = 1;
    q.idesc = ptx::idesc_f8(tile, tile, a_mn, b_mn, c.A->dtype == TG_E5M2, c.B->dtype == TG_E5M2);
    q.flags = c.c_dtype == TG_F32 ? FLAG_C_F32 : c.c_dtype == TG_F16 ? FLAG_C_F16 : 0u;
    if (static_cast<int64_t>(q.tiles_m) * q.tiles_n > host::MAX_DIM / 2)
        return fail(TG_ERR_UNSUPPORTED, "C has more than 2^30 tiles of %d x %d", tile, tile);
    p.num_problems = 1;
    p.total_tiles = moe ? 0 : static_cast<int64_t>(q.tiles_m) * q.tiles_n;
    int band = 1;
    while (band * band * 2 <= units && band < 16) band *= 2;
    p.band = band < q.tiles_n ? band : q.tiles_n;
    p.moe_counts = c.counts;
    p.moe_groups = static_cast<int32_t>(c.experts);
    p.moe_rows = c.rows;
    x.sa = c.A->scale;
    x.sa_mn = c.A->scale_stride;
    x.sa_k = c.A->scale_k_stride;
    x.sa_shift = c.A->block == 128 ? 7 : 0;
    x.sb = c.B->scale;
    x.sb_mn = c.B->scale_stride;
    x.sb_k = c.B->scale_k_stride;
    x.sb_g = c.scale_stride;
    x.a_mn = a_mn;
    x.b_mn = b_mn;
    x.splits = splits;
    const char* env = std::getenv("TG_STREAM_K");
    x.halves = env && env[0] == '0' ? 0u : 1u;
    x.c = c.C;
    x.ldc = c.ldc;
    x.vec_c = host::aligned(c.C, 16) && (c.ldc * (c.c_dtype == TG_F32 ? 4 : 2)) % 16 == 0;
    host::launch_params(&p, d.err);
    // every resident unit, or fewer when there are fewer tiles (half tiles) than units
    int64_t want = pair && x.halves ? 2 * p.total_tiles : p.total_tiles;
    if (moe || want > units) want = units;
    if (splits > 1) want = p.total_tiles * splits;
    const cudaError_t e = v.launch(p, x, static_cast<int>(want) * v.cta_group, stream);
    if (e != cudaSuccess) return host::cuda_fail(e, "8-bit kernel launch");
    host::count_launches(1);
    return TG_OK;
}

}  // namespace

}  // namespace tg

extern "C" tg_status tg_gemm_scaled(const tg_scaled_operand* A, const tg_scaled_operand* B, void* C, tg_dtype c_dtype,
                                 int64_t ldc, int64_t M, int64_t N, int64_t K, tg_epilogue epi, const void* bias,
                                 tg_stream_t stream) {
    using namespace tg;
    if (!A || !B) return fail(TG_ERR_INVALID_ARG, "%s is NULL", !A ? "A" : "B");
    tg_status s = check_output(C, c_dtype, ldc, M, N, K, epi, bias);
    if (s != TG_OK || (s = check_operand(A, "A", M, K, TG_ROW_MAJOR)) != TG_OK ||
        (s = check_operand(B, "B", N, K, TG_COL_MAJOR)) != TG_OK)
        return s;
    if (M == 0 || N == 0) return TG_OK;
    const Fp8Call c{A, B, M, N, K, C, c_dtype, ldc, epi, bias, 0, 0, 0, nullptr};
    return run_fp8(c, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" tg_status tg_moe_gemm_scaled(const tg_scaled_operand* A, int64_t T, int64_t K, const tg_scaled_operand* B,
                                     int64_t expert_stride, int64_t scale_stride, int64_t G, int64_t N, void* C,
                                     tg_dtype c_dtype, int64_t ldc, const int32_t* counts, tg_epilogue epi,
                                     const void* bias, tg_stream_t stream) {
    using namespace tg;
    if (!A || !B) return fail(TG_ERR_INVALID_ARG, "%s is NULL", !A ? "A" : "B");
    if (G < 0) return fail(TG_ERR_INVALID_ARG, "negative G=%lld", (long long)G);
    tg_status s = check_output(C, c_dtype, ldc, T, N, K, epi, bias);
    if (s != TG_OK || (s = check_operand(A, "A", T, K, TG_ROW_MAJOR)) != TG_OK ||
        (s = check_operand(B, "B", G > 0 ? N : 0, K, TG_COL_MAJOR)) != TG_OK)
        return s;
    if (A->layout != TG_ROW_MAJOR) return fail(TG_ERR_INVALID_ARG, "A must be row-major");
    if (A->block != 1) return fail(TG_ERR_INVALID_ARG, "A needs a scale per row (block 1)");
    if (B->block != 128) return fail(TG_ERR_INVALID_ARG, "B needs a scale per 128 x 128 block (block 128)");
    if (T == 0 || N == 0 || G == 0) return TG_OK;
    if (G > TG_MOE_MAX_EXPERTS)
        return fail(TG_ERR_UNSUPPORTED, "G=%lld experts; the device-counts form takes at most %d", (long long)G,
                    TG_MOE_MAX_EXPERTS);
    if (!counts) return fail(TG_ERR_INVALID_ARG, "counts is NULL");
    if (!host::aligned(counts, 4)) return fail(TG_ERR_INVALID_ARG, "counts is not 4-byte aligned");
    if (K > 0) {
        const int64_t least = (B->layout == TG_ROW_MAJOR ? K : N) * B->ld;
        if (expert_stride < least)
            return fail(TG_ERR_INVALID_ARG, "expert_stride=%lld < %lld (one expert's B)", (long long)expert_stride,
                        (long long)least);
        if (scale_stride < 0) return fail(TG_ERR_INVALID_ARG, "negative scale_stride");
        if (expert_stride % 16 || expert_stride > (int64_t(1) << 39))
            return fail(TG_ERR_UNSUPPORTED, "expert_stride must be a multiple of 16 below 2^39 (TMA)");
    }
    const Fp8Call c{A, B, T, N, K, C, c_dtype, ldc, epi, bias, G, expert_stride, scale_stride, counts};
    return run_fp8(c, reinterpret_cast<cudaStream_t>(stream));
}
