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
// L lanes of a warp hold one row (L = 8, 16 or 32, at least k and G / 8), each V
// neighbouring experts; a warp works on 32 / L rows at once, with the next rows' logits on
// their way.  Everything is summed in a fixed order - a lane over its rows, a warp's row
// slots, the warps of a block, then the blocks - so results do not depend on
// timing.
//
// Selection.  An expert's key is its logit's bits made to order like an unsigned integer, the
// lowest 8 (9, 10 above 256, 512 experts) replaced by the expert's index counted down, so that
// keys are unique and equal logits go to the lowest index.  Keys come out in decreasing order,
// so those still to come are the ones below the last one, t: the largest of (key - t) modulo
// 2^32, one fused add-and-maximum a key.  For 16-bit logits the replaced bits are zeros anyway;
// fp32 logits that agree in all the others, at the top of a row, send that row through an exact
// selection (choose_exactly).  131072 x 256 fp32, k = 8: 152 us with a rescan of (value, index)
// pairs after every choice, 1018 warp instructions a row, against the read's 20 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_host.cuh"
#include "tg_ptx.cuh"
#include "tg_router.cuh"

namespace tg {

using namespace gate;

namespace {

// The k choices of a row from its logits alone, in order of value (NaN first) and index: lane i
// gets the i-th expert, or -1.  Every lane of the warp calls it; a row that need not choose
// (!wanted) takes part and gets nothing.
template <int DT, int L, int V>
__device__ __noinline__ int choose_exactly(const Logits<DT, V>& x, int first, int k, bool wanted) {
    const int lane = threadIdx.x % 32, in = lane % L;
    uint32_t taken = wanted ? 0u : (V == 32 ? FULL : (1u << V % 32) - 1u);
    int my_e = -1;
    for (int i = 0; i < k; ++i) {
        // this lane's best: the key of its value (1 and up; NaN on top), then the lowest index
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float v = x.value(j);
            const uint32_t key = (taken >> j & 1u) || v == __int_as_float(0xff800000) ? 0u : v != v ? FULL : order_bits(v);
            if (key > best) { best = key; at = j; }
        }
        const uint32_t top = group_max<L>(best);
        const uint32_t has = __ballot_sync(FULL, best == top) >> (lane - in) & (L == 32 ? FULL : (1u << L % 32) - 1u);
        const int who = __ffs(has) - 1;          // the lowest lane holds the lowest indices
        const int e = __shfl_sync(FULL, first + at, who, L);
        if (top != 0u) {
            if (in == i) my_e = e;
            if (in == who) taken |= 1u << at;
        }
    }
    return my_e;
}

template <int DT, int L, int V>
__global__ void __launch_bounds__(R_THREADS, V == 8 ? 2 : 1) router_kernel(const RouterArgs a) {
    ptx::grid_launch_dependents();
    constexpr int SPAN = L * V;                   // experts a row's lanes cover
    constexpr int ROWS = 32 / L;                  // rows of a warp at once
    extern __shared__ __align__(16) uint8_t dyn[];
    float* s_sum = reinterpret_cast<float*>(dyn);                              // [warps][SPAN]
    int32_t* s_count = reinterpret_cast<int32_t*>(s_sum + R_WARPS * SPAN);     // [SPAN]
    __shared__ int32_t s_rows[R_WARPS];
    __shared__ double s_loss[R_WARPS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, in = lane % L;
    for (int i = threadIdx.x; i < SPAN; i += R_THREADS) s_count[i] = 0;
    __syncthreads();

    const int first = in * V;                     // this lane's experts [first, first + V)
    const int n = a.G - first < 0 ? 0 : a.G - first < V ? a.G - first : V;
    const int64_t step = static_cast<int64_t>(gridDim.x) * R_WARPS * ROWS;
    // (a warp's rows are neighbours; lanes past the last row keep -infinity and store nothing)
    int64_t t = (static_cast<int64_t>(blockIdx.x) * R_WARPS + warp) * ROWS + lane / L;
    const int64_t warp_first = t - lane / L;
    Logits<DT, V> next;
    const bool whole = a.vec && a.G == SPAN;      // every lane of every row loads V logits
    auto fetch = [&](int64_t row) {
        const uint8_t* at = a.logits + row * a.ld_bytes + first * Logits<DT, V>::ESIZE;
        if (whole && row - lane / L + ROWS <= a.T) next.load_whole(at);
        else next.load(at, row < a.T ? n : 0, a.vec != 0);
    };
    fetch(t);
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    int rows = 0;
    for (int64_t base = warp_first; base < a.T; base += step, t += step) {
        const Logits<DT, V> x = next;
        if (base + step < a.T) fetch(t + step);
        float m = x.value(0);                     // the row's largest logit, NaN if it has one
#pragma unroll
        for (int j = 1; j < V; ++j) m = max_nan(m, x.value(j));
        m = group_max_nan<L>(m);
        const bool any = m != __int_as_float(0xff800000);
        m = any ? m : 0.0f;                       // (e^(-infinity - 0) = 0)
        float p[V];
        float total = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            p[j] = exp_flush(x.value(j) - m);
            total += p[j];
        }
        total = group_sum<L>(total);
        const float inv = any ? 1.0f / total : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = fmaf(p[j], inv, sum[j]);
        rows += any && in == 0 ? 1 : 0;

        // the i-th choice ends up with lane i of the row; one more is looked at, to see that the
        // last one is apart from it
        constexpr uint32_t LOW = L * V - 1 > 255 ? L * V - 1 : 255;
        uint32_t key[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
            key[j] = (order_bits(x.value(j)) & ~LOW) | (LOW - static_cast<uint32_t>(first + j));
        uint32_t mine = 0u, top = 0u;
        for (int i = 0; i <= a.k; ++i) {
            uint32_t best = 0u;
#pragma unroll
            for (int j = 0; j < V; ++j) best = __viaddmax_u32(key[j], 0u - top, best);
            top += group_max<L>(best);
            if (in == i) mine = top;
        }
        // lane k (or, when there is none, every lane) has the first key left out
        int my_e = mine >= KEY_MIN ? static_cast<int>(LOW - (mine & LOW)) : -1;
        bool redo = m != m;
        if constexpr (DT == TG_F32) {
            uint32_t after = __shfl_down_sync(FULL, mine, 1, L);
            if (in == L - 1) after = top;
            const bool close = in < a.k && after >= KEY_MIN && ((mine ^ after) & ~LOW) == 0u;
            if (__any_sync(FULL, close)) {
                // do the row's values differ in the bits that the keys leave out?
                uint32_t low = 0u;
#pragma unroll
                for (int j = 0; j < V; ++j) low |= x.bits(j);
                const uint32_t group = L == 32 ? FULL : (1u << L % 32) - 1u;
                const uint32_t c = __ballot_sync(FULL, close) >> (lane - in) & group;
                const uint32_t o = __ballot_sync(FULL, (low & LOW) != 0u) >> (lane - in) & group;
                redo |= c != 0u && o != 0u;
            }
        }
        if (__any_sync(FULL, redo)) {
            const int e = choose_exactly<DT, L, V>(x, first, a.k, redo);
            if (redo) my_e = e;
        }
        float my_w = 0.0f;
        if (in >= a.k) my_e = -1;
        if (my_e >= 0) {
            my_w = __expf(Logits<DT, V>::one(a.logits + t * a.ld_bytes, my_e) - m) * inv;
            atomicAdd(&s_count[my_e], 1);
        }
        const float chosen = a.renorm ? group_sum<L>(my_w) : 1.0f;
        if (in < a.k && t < a.T) {
            a.experts[t * a.k + in] = my_e;
            a.weights[t * a.k + in] = my_e >= 0 ? my_w / chosen : 0.0f;
        }
    }
    // the row slots of a warp, then the warps of the block
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int d = L; d < 32; d <<= 1) sum[j] += __shfl_xor_sync(FULL, sum[j], d);
        if (lane < L) s_sum[warp * SPAN + first + j] = sum[j];
    }
    rows = __reduce_add_sync(FULL, rows);
    if (lane == 0) s_rows[warp] = rows;
    __syncthreads();
    int block_rows = 0;
#pragma unroll
    for (int w = 0; w < R_WARPS; ++w) block_rows += s_rows[w];
    double loss = 0.0, per_count = 0.0;
    if (!a.part_p && warp * 32 < a.G) per_count = slope_per_count(a, block_rows);
    for (int g = threadIdx.x; g < a.G; g += R_THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < R_WARPS; ++w) s += s_sum[w * SPAN + g];
        if (a.part_p) {
            a.part_p[static_cast<int64_t>(blockIdx.x) * a.G + g] = s;
            a.part_c[static_cast<int64_t>(blockIdx.x) * a.G + g] = s_count[g];
        } else {
            loss += finish_expert(a, g, s, s_count[g], per_count);
        }
    }
    if (a.part_p) {
        if (threadIdx.x == 0) a.part_n[blockIdx.x] = block_rows;
        return;
    }
    // the only block finishes the loss itself
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) loss += __shfl_xor_sync(FULL, loss, d);
    if (lane == 0) s_loss[warp] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < R_WARPS; ++w) loss += s_loss[w];
        *a.loss = static_cast<float>(loss);
    }
}

// Join the blocks' partial sums: a cluster of JOIN_CTAS blocks, each taking every JOIN_CTAS-th
// group of 32 experts, first with a lane an expert and the warps spread over the partial sums,
// then with a warp an expert; one warp finishes them, and the first block adds the loss's terms.  (One block reading one
// partial sum after the other took 70 us for 304 of them.)
constexpr int JOIN_CTAS = 8;
constexpr int JOIN_WARPS = 32;

__global__ void __cluster_dims__(JOIN_CTAS, 1, 1) __launch_bounds__(32 * JOIN_WARPS)
    router_join_kernel(const RouterArgs a, int blocks) {
    __shared__ float s_p[JOIN_WARPS][33];
    __shared__ int32_t s_c[JOIN_WARPS][33];
    __shared__ float s_sum[32];
    __shared__ int32_t s_count[32];
    __shared__ int32_t s_n[JOIN_WARPS];
    __shared__ double s_loss[JOIN_CTAS];           // in block 0: every block's share
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank();
    // block 0's shared memory takes the others' shares below: it may be written once every block of
    // the cluster has started (with few experts nothing else stands between the two)
    ptx::cluster_sync();
    ptx::grid_dependency_wait();
    int n = 0;
    for (int b = threadIdx.x; b < blocks; b += 32 * JOIN_WARPS) n += a.part_n[b];
    n = __reduce_add_sync(FULL, n);
    if (lane == 0) s_n[warp] = n;
    double loss = 0.0, per_count = -1.0;
    for (int g0 = static_cast<int>(rank) * 32; g0 < a.G; g0 += 32 * JOIN_CTAS) {
        float s = 0.0f;
        int32_t c = 0;
        if (g0 + lane < a.G) {
#pragma unroll 10
            for (int b = warp; b < blocks; b += JOIN_WARPS) {
                s += a.part_p[static_cast<int64_t>(b) * a.G + g0 + lane];
                c += a.part_c[static_cast<int64_t>(b) * a.G + g0 + lane];
            }
        }
        s_p[warp][lane] = s;
        s_c[warp][lane] = c;
        __syncthreads();
        s = group_sum<32>(s_p[lane][warp]);
        c = __reduce_add_sync(FULL, s_c[lane][warp]);
        if (lane == 0) {
            s_sum[warp] = s;
            s_count[warp] = c;
        }
        __syncthreads();
        if (warp == 0) {
            if (per_count < 0.0) per_count = slope_per_count(a, __reduce_add_sync(FULL, s_n[lane]));
            if (g0 + lane < a.G) loss += finish_expert(a, g0 + lane, s_sum[lane], s_count[lane], per_count);
        }
        __syncthreads();
    }
    if (warp == 0) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) loss += __shfl_xor_sync(FULL, loss, d);
        if (lane == 0) {
            const uint32_t dst = ptx::mapa(ptx::smem_u32(&s_loss[rank]), 0);
            asm volatile("st.shared::cluster.f64 [%0], %1;" :: "r"(dst), "d"(loss) : "memory");
        }
    }
    ptx::cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        double sum = 0.0;
        for (int r = 0; r < JOIN_CTAS; ++r) sum += s_loss[r];
        *a.loss = static_cast<float>(sum);
    }
}

struct BackArgs {
    const uint8_t* logits;
    int64_t ld_bytes, T;
    int G, k, renorm, vec_in, vec_out;
    const int32_t* experts;
    const float* weights;
    const float* slope;
    const float* d_weights;   // null: zero
    const float* d_loss;      // null: zero
    uint8_t* out;
    int64_t ldo_bytes;
};

template <int DT, int L, int V>
__global__ void __launch_bounds__(R_THREADS, V == 8 ? 2 : 1) router_backward_kernel(const BackArgs a) {
    using X = Logits<DT, V>;
    constexpr int ROWS = 32 / L;
    // per warp: what the chosen experts of its rows get on top, by expert; zero elsewhere
    extern __shared__ __align__(16) uint8_t dyn[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, in = lane % L;
    float* extra = reinterpret_cast<float*>(dyn) + warp * 32 * V + (lane / L) * L * V;
    const int first = in * V;
    const int n = a.G - first < 0 ? 0 : a.G - first < V ? a.G - first : V;
    const float dl = a.d_loss ? __ldg(a.d_loss) : 0.0f;
    float u[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        u[j] = (a.d_loss && j < n) ? dl * __ldg(a.slope + first + j) : 0.0f;
        extra[first + j] = 0.0f;
    }
    __syncwarp();
    const int64_t step = static_cast<int64_t>(gridDim.x) * R_WARPS * ROWS;
    int64_t t = (static_cast<int64_t>(blockIdx.x) * R_WARPS + warp) * ROWS + lane / L;
    const int64_t warp_first = t - lane / L;
    const bool choice = a.d_weights != nullptr && in < a.k;
    X next;
    int e_next = -1;
    float w_next = 0.0f, dw_next = 0.0f;
    auto fetch = [&](int64_t row) {
        next.load(a.logits + row * a.ld_bytes + first * X::ESIZE, row < a.T ? n : 0, a.vec_in != 0);
        e_next = -1;
        if (choice && row < a.T) {
            e_next = __ldg(a.experts + row * a.k + in);
            w_next = __ldg(a.weights + row * a.k + in);
            dw_next = __ldg(a.d_weights + row * a.k + in);
        }
        if (e_next < 0 || e_next >= a.G) {       // no choice (-1): nothing of it counts
            e_next = -1;
            w_next = dw_next = 0.0f;
        }
    };
    fetch(t);
    for (int64_t base = warp_first; base < a.T; base += step, t += step) {
        const X x = next;
        const int e = e_next;
        const float w = w_next, dw = dw_next;
        if (base + step < a.T) fetch(t + step);
        float m = x.value(0);
#pragma unroll
        for (int j = 1; j < V; ++j) m = max_nan(m, x.value(j));
        m = group_max_nan<L>(m);
        const bool any = m != __int_as_float(0xff800000);
        m = any ? m : 0.0f;                       // (e^(-infinity - 0) = 0)
        float p[V];
        float total = 0.0f, pu = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            p[j] = exp_flush(x.value(j) - m);
            total += p[j];
            pu = fmaf(p[j], u[j], pu);
        }
        total = group_sum<L>(total);
        const float inv = any ? 1.0f / total : 0.0f;
        const float cu = group_sum<L>(pu) * inv;
        float c = cu;
        if (a.d_weights) {
            const float cw = group_sum<L>(w * dw);
            if (!a.renorm) c += cw;
            if (e >= 0) extra[e] = a.renorm ? w * (dw - cw) : w * dw;
            __syncwarp();
        }
        float d[V];
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = p[j] * inv * (u[j] - c);
        if (a.d_weights) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(extra + first + j);
                d[j] += f.x; d[j + 1] += f.y; d[j + 2] += f.z; d[j + 3] += f.w;
            }
            __syncwarp();
            if (e >= 0) extra[e] = 0.0f;
            __syncwarp();
        }
        if (t >= a.T) continue;
        uint8_t* dst = a.out + t * a.ldo_bytes + first * X::ESIZE;
        uint32_t o[X::WORDS];
#pragma unroll
        for (int i = 0; i < X::WORDS; ++i) {
            if constexpr (DT == TG_F32) {
                o[i] = __float_as_uint(d[i]);
            } else if constexpr (DT == TG_F16) {
                const __half2 h = __floats2half2_rn(d[2 * i], d[2 * i + 1]);
                o[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(d[2 * i], d[2 * i + 1]);
                o[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        if (n == V && a.vec_out) {
#pragma unroll
            for (int i = 0; i < X::WORDS; i += 4)
                reinterpret_cast<uint4*>(dst)[i / 4] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (j >= n) continue;
                if constexpr (DT == TG_F32) reinterpret_cast<uint32_t*>(dst)[j] = o[j];
                else reinterpret_cast<uint16_t*>(dst)[j] = static_cast<uint16_t>(o[j / 2] >> ((j & 1) * 16));
            }
        }
    }
}

using RouterKernel = void (*)(const RouterArgs);
using BackKernel = void (*)(const BackArgs);

// The kernel for G experts and k choices: L lanes a row, V experts a lane.  (32 a lane spill: 232 bytes a thread with
// fp32 logits, 20 with 16-bit ones.)
struct RouterVariant {
    RouterKernel forward;
    BackKernel backward;
    int lanes, per_lane;
};

template <int DT>
RouterVariant variant_for(int G, int k) {
    const int need = (G + 7) / 8 > k ? (G + 7) / 8 : k;
    if (G > 512) return {&router_kernel<DT, 32, 32>, &router_backward_kernel<DT, 32, 32>, 32, 32};
    if (G > 256) return {&router_kernel<DT, 32, 16>, &router_backward_kernel<DT, 32, 16>, 32, 16};
    if (need > 16) return {&router_kernel<DT, 32, 8>, &router_backward_kernel<DT, 32, 8>, 32, 8};
    if (need > 8) return {&router_kernel<DT, 16, 8>, &router_backward_kernel<DT, 16, 8>, 16, 8};
    return {&router_kernel<DT, 8, 8>, &router_backward_kernel<DT, 8, 8>, 8, 8};
}

RouterVariant variant_for(tg_dtype dt, int G, int k) {
    return dt == TG_F32 ? variant_for<TG_F32>(G, k) : dt == TG_F16 ? variant_for<TG_F16>(G, k) : variant_for<TG_BF16>(G, k);
}

}  // namespace

namespace gate {

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

tg_status check_backward(int64_t G, tg_dtype dt, const int32_t* experts, const float* weights, bool weights_needed,
                         const float* slope, const float* d_weights, const float* d_loss, const void* d_logits, int64_t ldd) {
    using host::fail;
    if (!d_logits) return fail(TG_ERR_INVALID_ARG, "d_logits is NULL");
    if (d_weights && (!experts || (weights_needed && !weights)))
        return fail(TG_ERR_INVALID_ARG, "%s is NULL (needed with d_weights)", !experts ? "experts" : "weights");
    if (d_loss && !slope) return fail(TG_ERR_INVALID_ARG, "slope is NULL (needed with d_loss)");
    if (ldd < G) return fail(TG_ERR_INVALID_ARG, "ldd=%lld < G=%lld", (long long)ldd, (long long)G);
    if (ldd > host::MAX_DIM) return fail(TG_ERR_UNSUPPORTED, "ldd must be below 2^31");
    if (!host::aligned(d_logits, dt == TG_F32 ? 4 : 2))
        return fail(TG_ERR_INVALID_ARG, "d_logits is not aligned to its element size");
    if (!host::aligned(experts, 4) || !host::aligned(weights, 4) || !host::aligned(slope, 4) ||
        !host::aligned(d_weights, 4) || !host::aligned(d_loss, 4))
        return fail(TG_ERR_INVALID_ARG, "an input is not 4-byte aligned");
    return TG_OK;
}

cudaError_t launch_join(const RouterArgs& a, int blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(JOIN_CTAS, 1, 1);
    cfg.blockDim = dim3(32 * JOIN_WARPS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, router_join_kernel, a, blocks);
}

}  // namespace gate

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
    const RouterVariant v = variant_for(dtype, static_cast<int>(G), static_cast<int>(k));
    const int64_t esize = dtype == TG_F32 ? 4 : 2;
    const int64_t block_rows = R_WARPS * (32 / v.lanes);
    // One block (which then needs no second kernel and no workspace) while it has at most four rows
    // a slot; beyond that every SM.
    const int64_t want = (T + block_rows - 1) / block_rows, cap = static_cast<int64_t>(d.sms) * R_BLOCKS_PER_SM;
    const int blocks = want <= 4 ? 1 : static_cast<int>(want < cap ? want : cap);
    void* ws = nullptr;
    RouterArgs a{static_cast<const uint8_t*>(logits), ld * esize, T, int(G), int(k), renormalize != 0,
                 host::aligned(logits, 16) && ld * esize % 16 == 0, experts, weights, counts, loss, slope,
                 nullptr, nullptr, nullptr};
    if (blocks > 1) {
        const size_t words = static_cast<size_t>(blocks) * (2 * G + 1);
        if ((s = host::workspace(words * 4, st, "cudaMallocFromPoolAsync(router partial sums)", &ws)) != TG_OK) return s;
        a.part_p = static_cast<float*>(ws);
        a.part_c = static_cast<int32_t*>(ws) + blocks * G;
        a.part_n = static_cast<int32_t*>(ws) + 2 * blocks * G;
    }
    const size_t smem = static_cast<size_t>(R_WARPS + 1) * v.lanes * v.per_lane * 4;
    cudaError_t e = allow_smem(v.forward, smem);
    if (e == cudaSuccess) {
        v.forward<<<blocks, R_THREADS, smem, st>>>(a);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) {
        host::count_launches(1);
        if (blocks > 1) {
            e = launch_join(a, blocks, st);
            if (e == cudaSuccess) host::count_launches(1);
        }
    }
    s = e == cudaSuccess ? TG_OK : host::cuda_fail(e, "router launch");
    if (ws) {
        e = cudaFreeAsync(ws, st);
        if (e != cudaSuccess && s == TG_OK) s = host::cuda_fail(e, "cudaFreeAsync(router partial sums)");
    }
    return s;
}

extern "C" tg_status tg_moe_router_backward(const void* logits, tg_dtype dtype, int64_t ld, int64_t T, int64_t G,
                                            int64_t k, int renormalize, const int32_t* experts, const float* weights,
                                            const float* slope, const float* d_weights, const float* d_loss,
                                            void* d_logits, int64_t ldd, tg_stream_t stream) {
    using namespace tg;
    tg_status s = check_router(logits, dtype, ld, T, G, k);
    if (s != TG_OK || T == 0) return s;
    if ((s = check_backward(G, dtype, experts, weights, true, slope, d_weights, d_loss, d_logits, ldd)) != TG_OK) return s;
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    const RouterVariant v = variant_for(dtype, static_cast<int>(G), static_cast<int>(k));
    const int64_t esize = dtype == TG_F32 ? 4 : 2;
    const BackArgs a{static_cast<const uint8_t*>(logits), ld * esize, T, int(G), int(k), renormalize != 0,
                     host::aligned(logits, 16) && ld * esize % 16 == 0,
                     host::aligned(d_logits, 16) && ldd * esize % 16 == 0, experts, weights, slope, d_weights, d_loss,
                     static_cast<uint8_t*>(d_logits), ldd * esize};
    const int64_t block_rows = R_WARPS * (32 / v.lanes);
    const int64_t want = (T + block_rows - 1) / block_rows, cap = static_cast<int64_t>(d.sms) * R_BLOCKS_PER_SM;
    const size_t smem = static_cast<size_t>(R_WARPS) * 32 * v.per_lane * 4;
    cudaError_t e = allow_smem(v.backward, smem);
    if (e == cudaSuccess) {
        v.backward<<<static_cast<unsigned>(want < cap ? want : cap), R_THREADS, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return host::cuda_fail(e, "router backward launch");
    host::count_launches(1);
    return TG_OK;
}
