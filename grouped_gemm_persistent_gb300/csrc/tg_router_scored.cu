// tg_router_scored.cu - the gate with sigmoid or softmax scores, a bias for balance, groups of experts and a factor on the
// weights (tg_moe_router_scored and tg_moe_router_scored_backward in include/tg.h).
//
//   s(t, g)     sigmoid(x) or softmax(x)                    v = s + bias[g]: what is chosen by
//   group       its score is the sum of its group_top (1 or 2) largest v; the top_groups best are kept
//   e(t, j)     the k experts of largest v in the kept groups; without a bias by x itself, of which v is a rising function
//   w(t, j)     factor * s, over the sum of the chosen s when renormalised
//   loss        G sum_g f_g P_g as in tg_router.cu, with P_g the mean of s / sum_g s
// and, counts being constant, with u = d_loss * slope and c' the gradient of the chosen s through w
//   sigmoid:    d x = s (1 - s) ((u - sum s u / sum s) / sum s + c')
//   softmax:    d x = s (u - sum s u + c' - sum s c')
// where, with w' the factor's product with the gradient of w, s c' is s w' or, renormalised, w (w' - sum w w') (whose sum is 0).
//
// Choosing.  A choice by v is one of real numbers: with fp32 scores two experts next to each other in the order would change
// places with the last bits of exp.  The kernel works in fp32 with a bound E on a score's error and sees where that does not decide:
// two neighbours among the first k + 1 whose keys are within the bound, or two groups at the border of the kept ones.  Then the k + 1
// candidates, or the groups' largest experts, are worked out in 64 bits, each by a lane, and put in order; a row whose next
// candidate is within the bound too is done again as a whole (choose_in_64).  Double precision is slow here (a row of 256 takes the
// SM some 5 us): with the whole row always, sigmoid scores of 131072 x 256 fp32 take 109 us instead of 95, of 8191 rows 28 instead of 18.
// Neighbours whose logit and bias are both the same are a true tie, which the index decides: with 16-bit logits and a bias of zeros
// they are common.
//   sigmoid  e^-x: 2^-22 of itself and |x| 2^-24 for its argument, which s (1 - s) <= 1/4 takes down to 7.3e-8; 1 + e^-x and the
//            reciprocal 1.5 * 2^-23 of s: E = 3e-7.
//   softmax  of the row's largest score: 3.4e-7 for its own exponential, twice in a pair; the sum's terms, up to 36 additions and its
//            reciprocal 3.1e-6, the same for all of the row and so once in a pair: E = 2e-6.
//
// Keys.  Without a bias as in tg_router.cu: the logit's ordered bits, the lowest ones replaced by the position counted down.
// With one: v - lo + 4 is a number from 4 to 8, whose bits below the exponent are a fixed-point number of 21 binary places (about
// what the scores are known to); they and the position below them are the key, one shift and add.  lo is the smallest bias, or the
// largest minus 2.5 where they spread further: what then lies below lo is left out, and a row whose k-th choice is not clear of lo
// goes to 64 bits.  Above 256 positions the key has room for a bit or two less.
// The groups are chosen the same way, by their scores' bits and their indices, while each has its group_top experts to choose
// from and none below lo; otherwise, and without a bias by the largest logit itself, by counting the groups that come before each.
//
// Bound by instruction issue: 594 warp instructions a row of 256 with 8 groups and k = 8, 73 % of the issue rate, 95 us for 131072
// rows whose logits are read in 20 us; a choice more costs 2.6 us, the groups 17.  The gradient: 317 instructions a row, 52 us (40 us
// at the copy rate).
//
// Positions.  A row is L lanes of V positions.  Each group has a power of two of positions, V at least, so that
// a group is whole lanes and its sums are a few exchanges; the positions past its experts hold -infinity.
//
// Registers.  Eight positions a lane are held to 64 for two blocks an SM (softmax spills 112 to 164 bytes a thread, sigmoid at most
// 68); 16 and 32 positions take 126 and 128, one block an SM, so that a grid cut for two runs in two waves; 32 spill 136 to 564.
//
// Weights come from the hardware's 2^x and 1 / x: next to 1e-7 of themselves around logits of zero, about 1e-5 at 88 from it (softmax:
// from the row's largest), where the rounding of the exponent's argument is that large.
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

constexpr float MINUS_INF = -__builtin_huge_valf();
constexpr int MAX_CTAS = 8;

struct ScoredArgs {
    RouterArgs r;
    const float* bias;        // null: none
    int each;                 // experts of a group
    int shift;                // log2 of a group's positions (31: one group)
    int groups, top_groups, group_top;
    float factor;
};

// 2^x and 1 / x, zero below fp32's normal values
__device__ __forceinline__ float ex2_flush(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_flush(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// (a subnormal score would have an infinite reciprocal)
__device__ __forceinline__ float mul_flush(float x, float y) {
    float r;
    asm("mul.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float sigmoid_approx(float x) { return rcp_flush(1.0f + ex2_flush(x * -1.4426950408889634f)); }

template <int L>
__device__ __forceinline__ float group_max_plain(float v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, d));
    return v;
}

// The votes of a row's lanes
template <int L>
__device__ __forceinline__ uint32_t row_ballot(bool v, int lane, int in) {
    return __ballot_sync(FULL, v) >> (lane - in) & (L == 32 ? FULL : (1u << L % 32) - 1u);
}

// A double's place in the order: NaN above all, -infinity (what may not be chosen) 0
__device__ __forceinline__ unsigned long long order64(double v) {
    if (v != v) return ~0ull;
    if (v == -__builtin_huge_val()) return 0ull;
    const long long b = __double_as_longlong(v + 0.0);
    return static_cast<unsigned long long>(b) ^ (static_cast<unsigned long long>(b >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ double value64(unsigned long long o) {
    if (o == ~0ull) return __longlong_as_double(0x7ff8000000000000ll);
    return __longlong_as_double(static_cast<long long>(o >> 63 ? o ^ 0x8000000000000000ull : ~o));
}

__device__ __forceinline__ unsigned long long max64(unsigned long long a, unsigned long long b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned long long min64(unsigned long long a, unsigned long long b) { return a < b ? a : b; }

// What a row's softmax scores are made of, in 64 bits: the largest logit (0 in a row of -infinity) and 1 / sum of e^(x - it)
struct Softmax64 {
    double m, inv;
};

// The row at `row`, of which this lane has experts e0, e0 + 1, ... (n of them).  Every lane of the warp calls it.
template <int DT, int L, int V>
__device__ __noinline__ Softmax64 softmax64(const uint8_t* row, int e0, int n) {
    auto top = [](double p, double q) { return p != p ? p : q != q ? q : p > q ? p : q; };
    double m = -__builtin_huge_val(), total = 0.0;
    for (int j = 0; j < n; ++j) m = top(m, Logits<DT, V>::one(row, e0 + j));
    for (int d = L / 2; d > 0; d >>= 1) m = top(m, __shfl_xor_sync(FULL, m, d));
    if (m == -__builtin_huge_val()) m = 0.0;
#pragma unroll 4
    for (int j = 0; j < V; ++j)
        if (j < n) total += exp(Logits<DT, V>::one(row, e0 + j) - m);
    for (int d = L / 2; d > 0; d >>= 1) total += __shfl_xor_sync(FULL, total, d);
    return {m, 1.0 / total};
}

// A score with its bias, in 64 bits (sigmoid: `of` is not used)
template <bool SIGMOID>
__device__ __forceinline__ double value_of(double x, const Softmax64& of, const float* bias, int e) {
    const double v = SIGMOID ? 1.0 / (1.0 + exp(-x)) : exp(x - of.m) * of.inv;
    return bias ? v + static_cast<double>(__ldg(bias + e)) : v;
}

// The k choices of the row at `row` in 64 bits: lane i gets the i-th expert, or -1.  Every lane of the warp calls it; a row
// that need not choose (!wanted) takes part and gets nothing.  n: this lane's experts e0, e0 + 1, ...
template <int DT, int L, int V, bool SIGMOID>
__device__ __noinline__ int choose_in_64(const ScoredArgs& a, const uint8_t* row, int e0, int n, bool wanted) {
    const int lane = threadIdx.x % 32, in = lane % L;
    if (!wanted) n = 0;
    const bool by_logit = a.bias == nullptr;
    Softmax64 of{0.0, 0.0};
    if constexpr (!SIGMOID) of = softmax64<DT, L, V>(row, e0, n);
    unsigned long long key[V];
    unsigned long long first = 0ull, second = 0ull;           // the lane's largest v
#pragma unroll 4
    for (int j = 0; j < V; ++j) {
        key[j] = 0ull;
        if (j >= n) continue;
        const double x = Logits<DT, V>::one(row, e0 + j);
        // (a bias of -infinity forbids an expert whose score is NaN too)
        if (x == -__builtin_huge_val() || (a.bias && __ldg(a.bias + e0 + j) == MINUS_INF)) continue;
        const unsigned long long by_v = order64(value_of<SIGMOID>(x, of, a.bias, e0 + j)), by_x = order64(x);
        key[j] = by_logit ? by_x : by_v;
        const unsigned long long o = by_logit && a.group_top == 1 ? by_x : by_v;
        second = max64(second, min64(first, o));
        first = max64(first, o);
    }
    if (a.groups > 1) {
        const int lanes = (1 << a.shift) / V;
        for (int d = 1; d < lanes; d <<= 1) {
            const unsigned long long f = __shfl_xor_sync(FULL, first, d), g = __shfl_xor_sync(FULL, second, d);
            second = max64(min64(first, f), max64(second, g));
            first = max64(first, f);
        }
        unsigned long long score = first;
        if (a.group_top == 2 && second != 0ull) score = order64(value64(first) + value64(second));
        const int mine = in * V >> a.shift;
        int before = 0;
        for (int h = 0; h < a.groups; ++h) {
            const unsigned long long o = __shfl_sync(FULL, score, h * lanes, L);
            before += o > score || (o == score && h < mine) ? 1 : 0;
        }
        if (score == 0ull || before >= a.top_groups)
            for (int j = 0; j < V; ++j) key[j] = 0ull;
    }
    int my_e = -1;
    for (int i = 0; i < a.r.k; ++i) {
        unsigned long long best = 0ull;
        int at = 0;
        for (int j = 0; j < V; ++j)
            if (key[j] > best) { best = key[j]; at = j; }
        unsigned long long top = best;
        for (int d = L / 2; d > 0; d >>= 1) top = max64(top, __shfl_xor_sync(FULL, top, d));
        const int who = __ffs(row_ballot<L>(best == top, lane, in)) - 1;     // the lowest lane holds the lowest indices
        const int e = __shfl_sync(FULL, e0 + at, who, L);
        if (top != 0ull) {
            if (in == i) my_e = e;
            if (in == who) key[at] = 0ull;
        }
    }
    return my_e;
}

template <int DT, int L, int V, bool SIGMOID>
__global__ void __launch_bounds__(R_THREADS, V == 8 ? 2 : 1) scored_kernel(const __grid_constant__ ScoredArgs s) {
    ptx::grid_launch_dependents();
    const RouterArgs& a = s.r;
    using X = Logits<DT, V>;
    constexpr int SPAN = L * V;                   // positions of a row
    constexpr int ROWS = 32 / L;                  // rows of a warp at once
    constexpr uint32_t LOW = SPAN - 1 > 255 ? SPAN - 1 : 255;      // a key's bits of the position
    constexpr int LOW_BITS = SPAN > 512 ? 10 : SPAN > 256 ? 9 : 8;
    constexpr float E = SIGMOID ? 3.0e-7f : 2.0e-6f;               // a score's error
    constexpr float U = 5.9604645e-8f;                             // 2^-24
    // How far a computed v may be off: the score (softmax: E of itself, and so of the row's largest, 1 / whole), and the roundings of
    // b - lo, of 4 more and of v itself (2^-23, 2^-22 and 2^-22).  Keys that are nearer than twice that, in their steps of 2^-21, are
    // not told apart; nor are groups' scores, of one such v or of two, whose sum is rounded by 2^-21 and has steps of 2^-20.
    constexpr int CUT = LOW_BITS - 8;                              // bits of v that a key leaves out
    auto steps_of = [](float off) { return static_cast<uint32_t>(2097152.0f * 2.0f * off) + 2; };
    auto pair_steps_of = [](float off) { return static_cast<uint32_t>(1048576.0f * 2.0f * (2.0f * off + 8.0f * U)) + 2; };
    extern __shared__ __align__(16) uint8_t dyn[];
    float* s_sum = reinterpret_cast<float*>(dyn);                              // [warps][SPAN]
    int32_t* s_count = reinterpret_cast<int32_t*>(s_sum + R_WARPS * SPAN);     // [SPAN], by expert
    __shared__ int32_t s_rows[R_WARPS], s_block_rows;
    __shared__ double s_per_count, s_loss[R_WARPS], s_share[MAX_CTAS];          // s_share: in block 0 every block's part of the loss
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, in = lane % L;
    for (int i = threadIdx.x; i < SPAN; i += R_THREADS) s_count[i] = 0;
    __syncthreads();

    const int first = in * V;                     // this lane's positions [first, first + V): experts e0 and on, n of them
    const int group = first >> s.shift, off = first & ((1u << s.shift) - 1u);
    const int e0 = group * s.each + off;
    const int n = group >= s.groups || s.each <= off ? 0 : s.each - off < V ? s.each - off : V;
    auto expert_of = [&](uint32_t key) {
        const uint32_t p = LOW - (key & LOW);
        return static_cast<int>((p >> s.shift) * s.each + (p & ((1u << s.shift) - 1u)));
    };
    const bool biased = s.bias != nullptr;
    float lo = 0.0f;
    float* s_bias = reinterpret_cast<float*>(s_count + SPAN) + first;          // this lane's: the bias - lo + 4
    bool odd = false, below = false;              // a bias of NaN or +infinity (64 bits sort it out), or below lo
    if (biased) {
        float small = __int_as_float(0x7f800000), large = MINUS_INF, b[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            b[j] = j < n ? __ldg(s.bias + e0 + j) : 0.0f;
            odd |= b[j] != b[j] || b[j] == __int_as_float(0x7f800000);
            if (j < n && fabsf(b[j]) < __int_as_float(0x7f800000)) {
                small = fminf(small, b[j]);
                large = fmaxf(large, b[j]);
            }
        }
        odd = __any_sync(FULL, odd);
        small = -group_max_plain<L>(-small);
        large = group_max_plain<L>(large);
        if (large > MINUS_INF) lo = fmaxf(small, large - 2.5f);
        below = small < lo;
        // (every row of the block writes the same)
#pragma unroll
        for (int j = 0; j < V; ++j) s_bias[j] = b[j] - lo + 4.0f;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) s_bias[j] = 4.0f;
    }
    __syncwarp();
    // (a warp's rows are neighbours; lanes past the last row keep -infinity and store nothing.  T * k is below 2^31.)
    const uint32_t rows_in = static_cast<uint32_t>(a.T), step = gridDim.x * R_WARPS * ROWS;
    const uint32_t warp_first = (blockIdx.x * R_WARPS + warp) * ROWS;
    uint32_t t = warp_first + lane / L;
    const int64_t ahead = step * a.ld_bytes;
    const uint8_t* row = a.logits + t * a.ld_bytes;                // row t
    X next;
    const bool whole_rows = a.vec && a.G == SPAN;      // every lane of every row loads V logits
    // row `first` + lane / L, the warp's rows beginning at `first`, at `from`
    auto fetch = [&](uint32_t first, const uint8_t* from) {
        const uint8_t* at = from + e0 * X::ESIZE;
        if (whole_rows && first + ROWS <= rows_in) next.load_whole(at);
        else next.load(at, first + lane / L < rows_in ? n : 0, a.vec != 0);
    };
    fetch(warp_first, row);
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    int rows = 0;
    for (uint32_t base = warp_first; base < rows_in; base += step, t += step, row += ahead) {
        const X x = next;
        if (base + step < rows_in) fetch(base + step, row + ahead);
        float v[V];                               // the scores, then v - lo + 4, -infinity for what may not be chosen
        float m = 0.0f, whole = 0.0f;
        bool any;
        if constexpr (SIGMOID) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = sigmoid_approx(x.value(j));
                whole += v[j];
            }
            whole = group_sum<L>(whole);
            any = whole != 0.0f;
            if (__any_sync(FULL, !any)) {         // padding, or scores that are all 0 in fp32
                bool live = false;
#pragma unroll
                for (int j = 0; j < V; ++j) live |= x.value(j) != MINUS_INF;
                any = row_ballot<L>(live, lane, in) != 0u;
            }
        } else {
            m = x.value(0);                       // the row's largest logit, NaN if it has one
#pragma unroll
            for (int j = 1; j < V; ++j) m = max_nan(m, x.value(j));
            m = group_max_nan<L>(m);
            any = m != MINUS_INF;
            m = any ? m : 0.0f;                   // (e^(-infinity - 0) = 0)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = exp_flush(x.value(j) - m);
                whole += v[j];
            }
            whole = group_sum<L>(whole);
        }
        const float inv = whole != 0.0f ? rcp_flush(whole) : 0.0f;          // (whole is a normal number: so are scores that are not 0)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (SIGMOID) {
                sum[j] = fmaf(v[j], inv, sum[j]);
            } else {
                v[j] *= inv;
                sum[j] += v[j];
            }
        }
        rows += any && in == 0 ? 1 : 0;
        const float off = (SIGMOID ? E : E * fminf(inv, 1.0f)) + 10.0f * U;
        const uint32_t steps = steps_of(off), apart_from = (steps >> CUT) + 1;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 b = *reinterpret_cast<const float4*>(s_bias + j);
            v[j] = x.value(j) == MINUS_INF ? MINUS_INF : v[j] + b.x;
            v[j + 1] = x.value(j + 1) == MINUS_INF ? MINUS_INF : v[j + 1] + b.y;
            v[j + 2] = x.value(j + 2) == MINUS_INF ? MINUS_INF : v[j + 2] + b.z;
            v[j + 3] = x.value(j + 3) == MINUS_INF ? MINUS_INF : v[j + 3] + b.w;
        }

        bool redo = whole != whole || (odd && any), kept = true;
        if (s.groups > 1) {
            const int lanes = (1 << s.shift) / V;
            const bool exact = !biased && s.group_top == 1;        // the largest logit: nothing is rounded
            float one, two = MINUS_INF;
            if (exact) {
                one = x.value(0);
#pragma unroll
                for (int j = 1; j < V; ++j) one = fmaxf(one, x.value(j));
                for (int d = 1; d < lanes; d <<= 1) one = fmaxf(one, __shfl_xor_sync(FULL, one, d));
            } else {
                one = v[0];
#pragma unroll
                for (int j = 1; j < V; ++j) {
                    two = fmaxf(two, fminf(one, v[j]));
                    one = fmaxf(one, v[j]);
                }
                for (int d = 1; d < lanes; d <<= 1) {
                    const float o = __shfl_xor_sync(FULL, one, d), p = __shfl_xor_sync(FULL, two, d);
                    two = fmaxf(fminf(one, o), fmaxf(two, p));
                    one = fmaxf(one, o);
                }
            }
            const int mine = first >> s.shift;
            const float least = s.group_top == 2 ? two : one;
            if (!exact && __all_sync(FULL, least >= 4.0f || group >= s.groups || !any)) {
                // scores from 4 to 8, or of two from 8 to 16: their bits below the exponent, and the group counted down
                const float score = s.group_top == 2 ? one + two : one;
                const uint32_t key = group < s.groups && any
                                         ? __float_as_uint(score) << 8 | 0x80000000u | static_cast<uint32_t>(31 - mine) : 0u;
                uint32_t edge = 0u, after = 0u;
                for (int i = 0; i <= s.top_groups; ++i) {
                    edge = after;
                    after += group_max<L>(__viaddmax_u32(key, 0u - after, 0u));
                }
                kept = key >= edge;
                const bool open = after >= 0x80000000u && (edge >> 8) - (after >> 8) <= (s.group_top == 2 ? pair_steps_of(off) : steps);
                if (__any_sync(FULL, open)) {
                    // the groups at the border are not told apart.  A group's score in 64 bits needs its largest experts alone, if
                    // they are apart from the next.
                    bool clear = true;
                    int e[2] = {0, 0};
                    uint32_t last = 0u;
                    for (int i = 0; i <= s.group_top; ++i) {
                        uint32_t best = 0u;
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const uint32_t low = LOW - static_cast<uint32_t>(first + j);
                            best = __viaddmax_u32(v[j] >= 4.0f ? (__float_as_uint(v[j]) << 8 & ~LOW) + low : low, 0u - last, best);
                        }
                        for (int d = 1; d < lanes; d <<= 1) best = max(best, __shfl_xor_sync(FULL, best, d));
                        const uint32_t now = last + best;
                        if (i < s.group_top) e[i] = expert_of(now);
                        else clear &= now < 0x80000000u || (last >> LOW_BITS) - (now >> LOW_BITS) > apart_from;
                        last = now;
                    }
                    const uint32_t all_clear = row_ballot<L>(clear || group >= s.groups, lane, in);
                    const bool whole_row = all_clear == (L == 32 ? FULL : (1u << L % 32) - 1u);
                    redo |= open && !whole_row;
                    double score64 = 0.0;
                    Softmax64 of{0.0, 0.0};
                    if constexpr (!SIGMOID) {
                        if (__any_sync(FULL, open && whole_row)) of = softmax64<DT, L, V>(row, e0, open && whole_row ? n : 0);
                    }
                    if (open && whole_row && group < s.groups) {
                        score64 = value_of<SIGMOID>(X::one(row, e[0]), of, s.bias, e[0]);
                        if (s.group_top == 2) score64 += value_of<SIGMOID>(X::one(row, e[1]), of, s.bias, e[1]);
                    }
                    int before = 0;
                    for (int h = 0; h < s.groups; ++h) {
                        const double o = __shfl_sync(FULL, score64, h * lanes, L);
                        before += o > score64 || (o == score64 && h < mine) ? 1 : 0;
                    }
                    if (open && whole_row) kept = before < s.top_groups;
                }
            } else {
                float score = one, near = 0.0f;
                if (!exact) {
                    if (s.group_top == 2) score += two > MINUS_INF ? two : 4.0f - lo;    // (of sums less 2 lo and 8 more)
                    // twice a sum's error: scores, biases less lo, the sum itself, and lo where it stands alone
                    near = 4.0f * off + 8.0f * U * (8.0f + fabsf(score)) + 4.0f * U * fabsf(lo);
                    if (!(near < __int_as_float(0x7f800000))) near = 0.0f;              // (no expert that may be chosen)
                }
                int before = 0, maybe = 0;        // groups that come first for certain, and possibly
                for (int h = 0; h < s.groups; ++h) {
                    const float o = __shfl_sync(FULL, score, h * lanes, L);
                    if (exact) {
                        before += o > score || (o == score && h < mine) ? 1 : 0;
                    } else {
                        const float gap = o - score;
                        // (near goes with this score; the other's error is as large only where it is as large itself)
                        before += gap > 2.0f * near ? 1 : 0;
                        maybe += h != mine && o > MINUS_INF && gap >= -2.0f * near ? 1 : 0;
                    }
                }
                const bool none = !(score > MINUS_INF);
                kept = !none && before < s.top_groups;
                if (!exact)
                    redo |= row_ballot<L>(!none && group < s.groups && before < s.top_groups && maybe >= s.top_groups, lane, in) != 0u;
            }
        }

        // the i-th choice ends up with lane i of the row; one more is looked at, to see that the last one is apart from it
        const uint32_t key_min = biased ? 0x80000000u : KEY_MIN;
        uint32_t key[V];
        if (biased) {
            const float least = kept ? 4.0f : __int_as_float(0x7f800000);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t low = LOW - static_cast<uint32_t>(first + j);
                const uint32_t bits = CUT == 0 ? __float_as_uint(v[j]) << 8 : __float_as_uint(v[j]) << 8 & ~LOW;
                key[j] = v[j] >= least ? bits + low : low;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                key[j] = (kept ? order_bits(x.value(j)) & ~LOW : 0u) | (LOW - static_cast<uint32_t>(first + j));
        }
        uint32_t mine = 0u, top = 0u;
        for (int i = 0; i <= a.k; ++i) {
            uint32_t best = 0u;
#pragma unroll
            for (int j = 0; j < V; ++j) best = __viaddmax_u32(key[j], 0u - top, best);
            top += group_max<L>(best);
            if (in == i) mine = top;
        }
        // lane k (or, when there is none, every lane) has the first key left out
        int my_e = mine >= key_min ? expert_of(mine) : -1;
        if (DT == TG_F32 || biased) {
            uint32_t after = __shfl_down_sync(FULL, mine, 1, L);
            if (in == L - 1) after = top;
            const uint32_t apart = (mine >> LOW_BITS) - (after >> LOW_BITS);
            // the last choice has to be clear of what lies below lo
            if (below) redo |= row_ballot<L>(in == a.k - 1 && any && mine < (0x80000000u | (apart_from << LOW_BITS)), lane, in) != 0u;
            bool close = in < a.k && after >= key_min && (biased ? apart <= apart_from : apart == 0u);
            if (__any_sync(FULL, close)) {
                if (close) {
                    const int e = expert_of(after);
                    const bool tie = X::one(row, my_e) == X::one(row, e) && (!biased || __ldg(s.bias + my_e) == __ldg(s.bias + e));
                    close = !tie;
                }
                // The first k + 1 in 64 bits, each by its lane, and put in order: enough if the one after them is apart from them.
                const bool some = row_ballot<L>(close, lane, in) != 0u;
                uint32_t best = 0u;
#pragma unroll
                for (int j = 0; j < V; ++j) best = __viaddmax_u32(key[j], 0u - top, best);
                const uint32_t past = top + group_max<L>(best);
                const uint32_t gap = (top >> LOW_BITS) - (past >> LOW_BITS);
                const bool clear = past >= top || past < key_min || gap > (biased ? apart_from : 0u);
                const bool order = some && clear && a.k < L;
                redo |= some && !order;
                if (__any_sync(FULL, order)) {
                    unsigned long long my_v = 0ull;
                    Softmax64 of{0.0, 0.0};
                    if constexpr (!SIGMOID) {
                        if (biased) of = softmax64<DT, L, V>(row, e0, order ? n : 0);
                    }
                    if (order && in <= a.k && my_e >= 0) {
                        const double z = X::one(row, my_e);
                        my_v = order64(biased ? value_of<SIGMOID>(z, of, s.bias, my_e) : z);
                    }
                    int place = 0, got = -1;
                    for (int i = 0; i <= a.k; ++i) {
                        const unsigned long long o = __shfl_sync(FULL, my_v, i, L);
                        const int e = __shfl_sync(FULL, my_e, i, L);
                        place += o > my_v || (o == my_v && e < my_e) ? 1 : 0;
                    }
                    for (int i = 0; i <= a.k; ++i) {
                        const int to = __shfl_sync(FULL, place, i, L), e = __shfl_sync(FULL, my_e, i, L);
                        if (e >= 0 && to == in) got = e;          // (those there are come first, before and after)
                    }
                    if (order) my_e = got;
                }
            }
        }
        if (__any_sync(FULL, redo)) {
            const int e = choose_in_64<DT, L, V, SIGMOID>(s, row, e0, n, redo);
            if (redo) my_e = e;
        }
        float my_s = 0.0f;
        if (in >= a.k) my_e = -1;
        if (my_e >= 0) {
            const float z = X::one(row, my_e);
            my_s = SIGMOID ? sigmoid_approx(z) : mul_flush(exp_flush(z - m), inv);
            atomicAdd(&s_count[my_e], 1);
        }
        const float chosen = a.renorm ? group_sum<L>(my_s) : 1.0f;
        if (in < a.k && t < rows_in) {
            const uint32_t at = t * a.k + in;
            a.experts[at] = my_e;
            a.weights[at] = my_s != 0.0f ? my_s * rcp_flush(chosen) * s.factor : 0.0f;
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
    // an expert's sum over the block's warps, where its place in the first warp's sums is
    auto place_of = [&](int g) { return s.groups > 1 ? (g / s.each << s.shift) + g % s.each : g; };
    for (int g = threadIdx.x; g < a.G; g += R_THREADS) {
        const int p = place_of(g);
        float f = 0.0f;
#pragma unroll
        for (int w = 0; w < R_WARPS; ++w) f += s_sum[w * SPAN + p];
        if (a.part_p) {
            a.part_p[static_cast<int64_t>(blockIdx.x) * a.G + g] = f;
            a.part_c[static_cast<int64_t>(blockIdx.x) * a.G + g] = s_count[g];
        } else {
            s_sum[p] = f;
        }
    }
    if (a.part_p) {
        if (threadIdx.x == 0) a.part_n[blockIdx.x] = block_rows;
        return;
    }
    // the blocks of the only cluster (or the only block) share the experts, each adding all blocks' sums in their order
    const int ctas = static_cast<int>(ptx::cluster_nctarank()), rank = static_cast<int>(ptx::cluster_ctarank());
    if (threadIdx.x == 0) s_block_rows = block_rows;
    __syncthreads();
    if (ctas > 1) {
        ptx::cluster_sync();
        block_rows = 0;
        for (int c = 0; c < ctas; ++c) block_rows += static_cast<int>(ptx::ld_cluster_u32(ptx::mapa(ptx::smem_u32(&s_block_rows), c)));
    }
    // (one thread's division: double precision is slow, and warps without experts have none of it to do)
    if (threadIdx.x == 0) s_per_count = slope_per_count(a, block_rows);
    __syncthreads();
    const int chunk = (a.G + 32 * ctas - 1) / (32 * ctas) * 32, begin = rank * chunk, end = begin + chunk < a.G ? begin + chunk : a.G;
    double loss = 0.0;
    for (int g = begin + threadIdx.x; g < end; g += R_THREADS) {
        float f = s_sum[place_of(g)];
        int32_t count = s_count[g];
        if (ctas > 1) {
            const uint32_t sum_at = ptx::smem_u32(s_sum + place_of(g)), count_at = ptx::smem_u32(s_count + g);
            float fs[MAX_CTAS];
            int32_t counts[MAX_CTAS];
#pragma unroll
            for (int c = 0; c < MAX_CTAS; ++c) {
                fs[c] = c < ctas ? __uint_as_float(ptx::ld_cluster_u32(ptx::mapa(sum_at, c))) : 0.0f;
                counts[c] = c < ctas ? static_cast<int32_t>(ptx::ld_cluster_u32(ptx::mapa(count_at, c))) : 0;
            }
            f = 0.0f;
            count = 0;
#pragma unroll
            for (int c = 0; c < MAX_CTAS; ++c) {
                f += fs[c];
                count += counts[c];
            }
        }
        loss += finish_expert(a, g, f, count, s_per_count);
    }
    if (begin + warp * 32 < end) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) loss += __shfl_xor_sync(FULL, loss, d);
    }
    if (lane == 0) s_loss[warp] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < R_WARPS && begin + w * 32 < end; ++w) loss += s_loss[w];
        const uint32_t to = ptx::mapa(ptx::smem_u32(s_share + rank), 0);
        asm volatile("st.shared::cluster.f64 [%0], %1;" :: "r"(to), "d"(loss) : "memory");
    }
    if (ctas > 1) {
        ptx::cluster_arrive();                       // (nor does a block leave before the others have read its sums)
        ptx::cluster_wait();
    }
    if (rank == 0 && threadIdx.x == 0) {
        loss = 0.0;
        for (int c = 0; c < ctas; ++c) loss += s_share[c];
        *a.loss = static_cast<float>(loss);
    }
}

struct ScoredBackArgs {
    const uint8_t* logits;
    int64_t ld_bytes, T;
    int G, k, renorm;
    const int32_t* experts;
    const float* slope;
    const float* d_weights;   // null: zero
    const float* d_loss;      // null: zero
    uint8_t* out;
    int64_t ldo_bytes;
    float factor;
};

// CLOSE: a lane has V neighbouring experts of a row, moved in 16-byte vectors; otherwise every L-th expert, moved one by one, a line at a time
// over the lanes, wherever the row starts.  65536 rows, us, neighbours / apart:
//   bf16  64: 7.6 / 9.6   256: 23.8 / 24.8   512: 56 / 62   1024: 147 / 113     (neighbours up to 512, off the boundaries apart)
//   fp32  64: 8.4 / 9.1   128: 14.8 / 13.4   256: 31.4 / 30.2   512: 72 / 63   1024: 252 / 122     (apart)
// 255 fp32 off the boundaries: neighbours, read one by one, 46.6, apart 29.1.
template <int DT, int L, int V, bool SIGMOID, bool CLOSE>
__global__ void __launch_bounds__(R_THREADS, V == 8 ? 2 : 1) scored_backward_kernel(const ScoredBackArgs a) {
    using X = Logits<DT, V>;
    constexpr int ROWS = 32 / L;
    // per warp: the part of the chosen experts' gradients that comes through their weights, by expert; zero elsewhere
    extern __shared__ __align__(16) uint8_t dyn[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, in = lane % L;
    float* extra = reinterpret_cast<float*>(dyn) + warp * 32 * V + (lane / L) * L * V;
    constexpr int STRIDE = CLOSE ? 1 : L;
    const int first = CLOSE ? in * V : in, have = (a.G - first + STRIDE - 1) / STRIDE, n = have < 0 ? 0 : have < V ? have : V;
    const float dl = a.d_loss ? __ldg(a.d_loss) : 0.0f;
    float u[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        u[j] = (a.d_loss && j < n) ? dl * __ldg(a.slope + first + j * STRIDE) : 0.0f;
        extra[first + j * STRIDE] = 0.0f;
    }
    __syncwarp();
    // (T * k is below 2^31)
    const uint32_t rows_in = static_cast<uint32_t>(a.T), step = gridDim.x * R_WARPS * ROWS;
    const uint32_t warp_first = (blockIdx.x * R_WARPS + warp) * ROWS;
    uint32_t t = warp_first + lane / L;
    const int64_t ahead = step * a.ld_bytes, out_ahead = step * a.ldo_bytes;
    const uint8_t* row = a.logits + t * a.ld_bytes;
    uint8_t* out = a.out + t * a.ldo_bytes + first * X::ESIZE;
    const bool choice = a.d_weights != nullptr && in < a.k;
    X next;
    int e_next = -1;
    float z_next = 0.0f, dw_next = 0.0f;
    auto fetch = [&](uint32_t from, const uint8_t* at) {
        const uint32_t r = from + lane / L;
        if constexpr (CLOSE) next.load(at + first * X::ESIZE, r < rows_in ? n : 0, true);
        else next.template load_apart<STRIDE>(at + first * X::ESIZE, r < rows_in ? n : 0);
        e_next = -1;
        if (choice && r < rows_in) {
            e_next = __ldg(a.experts + r * a.k + in);
            dw_next = __ldg(a.d_weights + r * a.k + in);
        }
        if (e_next < 0 || e_next >= a.G) {       // no choice (-1): nothing of it counts
            e_next = -1;
            dw_next = 0.0f;
        } else {
            z_next = X::one(at, e_next);
        }
    };
    fetch(warp_first, row);
    for (uint32_t base = warp_first; base < rows_in; base += step, t += step, row += ahead, out += out_ahead) {
        const X x = next;
        const int e = e_next;
        const float z = z_next, dw = dw_next;
        if (base + step < rows_in) fetch(base + step, row + ahead);
        float p[V];                              // sigmoid: s (1 - s); softmax: s
        float m = 0.0f, whole = 0.0f, pu = 0.0f;
        if constexpr (SIGMOID) {
            // with e = e^-|x| and t = 1 / (1 + e): s is t or e t, s (1 - s) is e t^2 on either side of zero, 0 at both infinities
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = ex2_flush(fabsf(x.value(j)) * -1.4426950408889634f), q = rcp_flush(1.0f + f), r = f * q;
                const float score = x.value(j) < 0.0f ? r : q;
                p[j] = r * q;
                // (past the row's end the logit is -infinity: nothing)
                whole += score;
                pu = fmaf(score, u[j], pu);
            }
        } else {
            m = x.value(0);
#pragma unroll
            for (int j = 1; j < V; ++j) m = max_nan(m, x.value(j));
            m = group_max_nan<L>(m);
            m = m != MINUS_INF ? m : 0.0f;        // (e^(-infinity - 0) = 0)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                p[j] = exp_flush(x.value(j) - m);
                whole += p[j];
                pu = fmaf(p[j], u[j], pu);
            }
        }
        whole = group_sum<L>(whole);
        const float inv = whole != 0.0f ? 1.0f / whole : 0.0f;
        float c = group_sum<L>(pu) * inv;
        float d[V];
        if (a.d_weights) {
            // by the weight w = s / sum of the chosen: g / sum by itself has no room in 32 bits where the sum is small
            float my = 0.0f, rest = 1.0f;        // s and, of a sigmoid, 1 - s
            if (e >= 0) {
                if constexpr (SIGMOID) {
                    const float f = ex2_flush(fabsf(z) * -1.4426950408889634f), q = rcp_flush(1.0f + f), r = mul_flush(f, q);
                    my = z < 0.0f ? r : q;
                    rest = z < 0.0f ? q : r;
                } else {
                    my = mul_flush(exp_flush(z - m), inv);
                }
            }
            float g = a.factor * dw;
            if (a.renorm) {
                const float chosen = group_sum<L>(my);
                my *= chosen != 0.0f ? 1.0f / chosen : 0.0f;
                g -= group_sum<L>(my * g);
            } else if (!SIGMOID) {
                c += group_sum<L>(my * g);
            }
            g *= my * rest;
            if (e >= 0) extra[e] = g;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = extra[first + j * STRIDE];
            __syncwarp();
            if (e >= 0) extra[e] = 0.0f;
            __syncwarp();
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = fmaf(p[j] * inv, u[j] - c, d[j]);
        if (t >= rows_in) continue;
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
        if (CLOSE && n == V) {
#pragma unroll
            for (int i = 0; i < X::WORDS; i += 4)
                reinterpret_cast<uint4*>(out)[i / 4] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            continue;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j >= n) continue;
            if constexpr (DT == TG_F32) reinterpret_cast<uint32_t*>(out)[j * STRIDE] = o[j];
            else reinterpret_cast<uint16_t*>(out)[j * STRIDE] = static_cast<uint16_t>(o[j / 2] >> ((j & 1) * 16));
        }
    }
}

using ScoredKernel = void (*)(const ScoredArgs);
using ScoredBackKernel = void (*)(const ScoredBackArgs);

// Positions a lane and lanes a row
struct Shape {
    int lanes, per_lane, shift;
};

// The narrowest row that holds the groups (each in a power of two of positions, a lane's at least) and k choices; false
// when none does.
bool shape_for(int64_t groups, int64_t each, int64_t k, Shape* out) {
    for (int v = 8; v <= 32; v *= 2) {
        int64_t span = each;
        int shift = 31;
        if (groups > 1) {
            for (shift = 3; (int64_t(1) << shift) < each || (1 << shift) < v; ++shift) {}
            span = groups << shift;
        }
        if (span > 32 * v) continue;
        int lanes = v == 8 ? 8 : 32;
        while (lanes * v < span || lanes < k) lanes *= 2;
        *out = {lanes, v, shift};
        return true;
    }
    return false;
}

template <int DT, bool SIGMOID>
ScoredKernel scored_for(const Shape& s) {
    if (s.per_lane == 32) return &scored_kernel<DT, 32, 32, SIGMOID>;
    if (s.per_lane == 16) return &scored_kernel<DT, 32, 16, SIGMOID>;
    return s.lanes == 32 ? &scored_kernel<DT, 32, 8, SIGMOID> : s.lanes == 16 ? &scored_kernel<DT, 16, 8, SIGMOID>
                                                                             : &scored_kernel<DT, 8, 8, SIGMOID>;
}

ScoredKernel scored_for(tg_dtype dt, bool sigmoid, const Shape& s) {
    if (sigmoid)
        return dt == TG_F32 ? scored_for<TG_F32, true>(s) : dt == TG_F16 ? scored_for<TG_F16, true>(s) : scored_for<TG_BF16, true>(s);
    return dt == TG_F32 ? scored_for<TG_F32, false>(s) : dt == TG_F16 ? scored_for<TG_F16, false>(s) : scored_for<TG_BF16, false>(s);
}

template <int DT, bool SIGMOID>
ScoredBackKernel back_for(bool on_boundaries, const Shape& s) {
    if constexpr (DT != TG_F32) {
        if (on_boundaries && s.per_lane <= 16) {
            if (s.per_lane == 16) return &scored_backward_kernel<DT, 32, 16, SIGMOID, true>;
            if (s.lanes == 32) return &scored_backward_kernel<DT, 32, 8, SIGMOID, true>;
            return s.lanes == 16 ? &scored_backward_kernel<DT, 16, 8, SIGMOID, true> : &scored_backward_kernel<DT, 8, 8, SIGMOID, true>;
        }
    }
    if (s.per_lane == 32) return &scored_backward_kernel<DT, 32, 32, SIGMOID, false>;
    if (s.per_lane == 16) return &scored_backward_kernel<DT, 32, 16, SIGMOID, false>;
    if (s.lanes == 32) return &scored_backward_kernel<DT, 32, 8, SIGMOID, false>;
    return s.lanes == 16 ? &scored_backward_kernel<DT, 16, 8, SIGMOID, false> : &scored_backward_kernel<DT, 8, 8, SIGMOID, false>;
}

template <bool SIGMOID>
ScoredBackKernel back_for(tg_dtype dt, bool on_boundaries, const Shape& s) {
    return dt == TG_F32 ? back_for<TG_F32, SIGMOID>(on_boundaries, s) : dt == TG_F16 ? back_for<TG_F16, SIGMOID>(on_boundaries, s)
                                                                                     : back_for<TG_BF16, SIGMOID>(on_boundaries, s);
}

tg_status check_scores(tg_score score, float factor) {
    using host::fail;
    if (score != TG_SCORE_SOFTMAX && score != TG_SCORE_SIGMOID) return fail(TG_ERR_INVALID_ARG, "bad score %d", int(score));
    if (!(factor > 0.0f) || factor > 3.0e38f) return fail(TG_ERR_INVALID_ARG, "weight_scale must be finite and positive");
    return TG_OK;
}

}  // namespace

}  // namespace tg

extern "C" tg_status tg_moe_router_scored(const tg_router_args* args, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    if (!args) return fail(TG_ERR_INVALID_ARG, "args is NULL");
    const tg_router_args& p = *args;
    tg_status s = check_router(p.logits, p.dtype, p.ld, p.T, p.G, p.k);
    if (s != TG_OK || (s = check_scores(p.score, p.weight_scale)) != TG_OK) return s;
    if (p.groups < 1 || p.groups > p.G || p.G % p.groups != 0)
        return fail(TG_ERR_INVALID_ARG, "groups=%lld does not divide G=%lld", (long long)p.groups, (long long)p.G);
    const int64_t each = p.G / p.groups;
    if (p.top_groups < 1 || p.top_groups > p.groups)
        return fail(TG_ERR_INVALID_ARG, "top_groups=%lld is not in [1, groups=%lld]", (long long)p.top_groups, (long long)p.groups);
    if (p.group_top < 1 || p.group_top > 2 || p.group_top > each)
        return fail(TG_ERR_INVALID_ARG, "group_top=%lld is not 1 or 2, or above the %lld experts of a group", (long long)p.group_top,
                    (long long)each);
    if (p.k > p.top_groups * each)
        return fail(TG_ERR_INVALID_ARG, "k=%lld choices from %lld experts in the groups kept", (long long)p.k,
                    (long long)(p.top_groups * each));
    if (p.T > 0 && (!p.experts || !p.weights)) return fail(TG_ERR_INVALID_ARG, "%s is NULL", !p.experts ? "experts" : "weights");
    if (!p.counts || !p.loss || !p.slope)
        return fail(TG_ERR_INVALID_ARG, "%s is NULL", !p.counts ? "counts" : !p.loss ? "loss" : "slope");
    if (!host::aligned(p.experts, 4) || !host::aligned(p.weights, 4) || !host::aligned(p.counts, 4) || !host::aligned(p.loss, 4) ||
        !host::aligned(p.slope, 4) || !host::aligned(p.bias, 4))
        return fail(TG_ERR_INVALID_ARG, "bias or an output is not 4-byte aligned");
    Shape shape;
    if (!shape_for(p.groups, each, p.k, &shape))
        return fail(TG_ERR_UNSUPPORTED, "%lld groups of %lld experts: groups rounded up to powers of two of 8 at least hold at most %d",
                    (long long)p.groups, (long long)each, R_MAX_G);
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t esize = p.dtype == TG_F32 ? 4 : 2;
    const int64_t block_rows = R_WARPS * (32 / shape.lanes);
    // One cluster of up to eight blocks, which needs no second kernel and no workspace, while they have at most four rows a slot;
    // beyond that every SM.  64 x 256 fp32 in 8 groups: 13 us by one block, 8.3 by a cluster of four.
    const int64_t want = (p.T + block_rows - 1) / block_rows, cap = static_cast<int64_t>(d.sms) * R_BLOCKS_PER_SM;
    const bool cluster = want <= 4 * MAX_CTAS;
    const int blocks = cluster ? static_cast<int>(want < 1 ? 1 : want < MAX_CTAS ? want : MAX_CTAS) : static_cast<int>(want < cap ? want : cap);
    const int vec = host::aligned(p.logits, 16) && p.ld * esize % 16 == 0 && (p.groups == 1 || each * esize % 16 == 0);
    ScoredArgs a{{static_cast<const uint8_t*>(p.logits), p.ld * esize, p.T, int(p.G), int(p.k), p.renormalize != 0, vec, p.experts,
                  p.weights, p.counts, p.loss, p.slope, nullptr, nullptr, nullptr},
                 p.bias, int(each), shape.shift, int(p.groups), int(p.top_groups), int(p.group_top), p.weight_scale};
    void* ws = nullptr;
    if (!cluster) {
        const size_t words = static_cast<size_t>(blocks) * (2 * p.G + 1);
        if ((s = host::workspace(words * 4, st, "cudaMallocFromPoolAsync(router partial sums)", &ws)) != TG_OK) return s;
        a.r.part_p = static_cast<float*>(ws);
        a.r.part_c = static_cast<int32_t*>(ws) + blocks * p.G;
        a.r.part_n = static_cast<int32_t*>(ws) + 2 * blocks * p.G;
    }
    const ScoredKernel kernel = scored_for(p.dtype, p.score == TG_SCORE_SIGMOID, shape);
    const size_t smem = static_cast<size_t>(R_WARPS + 2) * shape.lanes * shape.per_lane * 4;
    cudaError_t e = allow_smem(kernel, smem);
    if (e == cudaSuccess && cluster && blocks > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
        cfg.blockDim = dim3(R_THREADS, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const ScoredArgs&>(a));
    } else if (e == cudaSuccess) {
        kernel<<<blocks, R_THREADS, smem, st>>>(a);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) {
        host::count_launches(1);
        if (!cluster) {
            e = launch_join(a.r, blocks, st);
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

extern "C" tg_status tg_moe_router_scored_backward(const tg_router_backward_args* args, tg_stream_t stream) {
    using namespace tg;
    using host::fail;
    if (!args) return fail(TG_ERR_INVALID_ARG, "args is NULL");
    const tg_router_backward_args& p = *args;
    tg_status s = check_router(p.logits, p.dtype, p.ld, p.T, p.G, p.k);
    if (s != TG_OK || (s = check_scores(p.score, p.weight_scale)) != TG_OK || p.T == 0) return s;
    if ((s = check_backward(p.G, p.dtype, p.experts, nullptr, false, p.slope, p.d_weights, p.d_loss, p.d_logits, p.ldd)) != TG_OK) return s;
    host::Device d;
    if ((s = host::device(&d)) != TG_OK) return s;
    Shape shape;
    shape_for(1, p.G, p.k, &shape);
    const int64_t esize = p.dtype == TG_F32 ? 4 : 2;
    const ScoredBackArgs a{static_cast<const uint8_t*>(p.logits), p.ld * esize, p.T, int(p.G), int(p.k), p.renormalize != 0, p.experts, p.slope,
                           p.d_weights, p.d_loss, static_cast<uint8_t*>(p.d_logits), p.ldd * esize, p.weight_scale};
    const bool on_boundaries = host::aligned(p.logits, 16) && p.ld * esize % 16 == 0 && host::aligned(p.d_logits, 16) &&
                               p.ldd * esize % 16 == 0;
    const ScoredBackKernel kernel = p.score == TG_SCORE_SIGMOID ? back_for<true>(p.dtype, on_boundaries, shape)
                                                                : back_for<false>(p.dtype, on_boundaries, shape);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t block_rows = R_WARPS * (32 / shape.lanes);
    const int64_t want = (p.T + block_rows - 1) / block_rows, cap = static_cast<int64_t>(d.sms) * R_BLOCKS_PER_SM;
    const size_t smem = static_cast<size_t>(R_WARPS) * 32 * shape.per_lane * 4;
    cudaError_t e = allow_smem(kernel, smem);
    if (e == cudaSuccess) {
        kernel<<<static_cast<unsigned>(want < cap ? want : cap), R_THREADS, smem, st>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return host::cuda_fail(e, "router backward launch");
    host::count_launches(1);
    return TG_OK;
}
