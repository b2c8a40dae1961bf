// Expert choice from router logits by softmax or sigmoid scores, with a
// selection bias, expert groups and renormalised, scaled gate weights.
//
//   s_e = sigmoid(z_e), or softmax(z)_e;  c_e = s_e + bias_e
//   group score = sum of the group_top largest c of the group; the topk_groups
//   best groups stay (ties to the lower group)
//   the k largest c of those groups, ties to the lower expert
//   w_j = s of the chosen expert (the bias only selects), / their sum when
//   renormalised, times scale
//
// The choice must not depend on rounding: with E scores in [0, 1] two
// neighbours are often closer than fp32 can tell.  The exact form of a token
// (one warp, scores in fp64) does not need to run for most of them: the fast
// form finds the k best by coarse scores (16 significant bits, with the expert
// in the low bits of the same word), proves that the set is right by the gap
// behind the k-th, and orders the k by their logits or fp32 scores.  Where that
// gap, or one among the k, is within the scores' error, up to 16 contenders are
// settled by fp64 scores; tokens with masked, infinite, far or tiny logits, and
// those whose groups are not told apart, take the exact form.
//
// What bounds it: the sorting networks (minimum and maximum at half the rate of
// an add) and, in a launch of a few waves, the tail of its last blocks; memory
// asks for a tenth of the time.  Measured (replayed in a graph):
//   128 tokens, 64 experts, fp32, bias               4.3 us
//   36,992 tokens, 64 experts, fp32, 8 groups       13.6 us  (0.83 TB/s)
//   8,191 tokens, 256 experts, fp32, bias, groups   15.9 us  (0.56 TB/s)
//   36,992 tokens, 256 experts, bf16, bias, groups  29.0 us  (0.73 TB/s)
// (The parameters are __grid_constant__: the exact form takes them by reference,
// and a copy of them in every thread's local memory costs 6 % of that.)
#include <limits.h>
#include <math.h>

#include "ms_common.cuh"

namespace ms {

constexpr int RG_MAXE = 256;
constexpr int RG_WARPS = 8;
constexpr double kMaskedScore = -1e300;   // masked experts of a chosen group rank behind every other one

struct RouteGroupedArgs {
    const void* logits;   // [T, E]
    const float* bias;    // [E] or NULL
    int T, E, groups, topk_groups, group_top, k, sigmoid, renorm;
    float scale;
    int32_t* idx;
    float* w;
};

__device__ __forceinline__ float rg_load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float rg_load(const __nv_bfloat16* p) {
    return bf16_to_f32(__ldg(reinterpret_cast<const uint16_t*>(p)));
}

// The two larger of (b1 >= b2) and (o1 >= o2).
template <typename T>
__device__ __forceinline__ void merge_two(T& b1, T& b2, T o1, T o2) {
    const T lo = o1 < b1 ? o1 : b1;
    const T second = b2 < o2 ? o2 : b2;
    b1 = o1 < b1 ? b1 : o1;
    b2 = lo < second ? second : lo;
}

// e^x for x <= 0, about 1e-14 relative, underflowing like exp: 2^k times the
// Taylor polynomial of degree 12 of 2^f, |f| <= 1/2.  Straight code, so that a
// lane's independent values overlap.
__constant__ double kExp2[13] = {1.0,
                                 6.9314718055994531e-1,
                                 2.4022650695910071e-1,
                                 5.5504108664821580e-2,
                                 9.6181291076284772e-3,
                                 1.3333558146428443e-3,
                                 1.5403530393381610e-4,
                                 1.5252733804059841e-5,
                                 1.3215486790144309e-6,
                                 1.0178086009239700e-7,
                                 7.0549116208011233e-9,
                                 4.4455382718708116e-10,
                                 2.5678435993488205e-11};
__device__ __forceinline__ double rg_exp(double x) {
    x = fmax(x, -800.0);   // 0 from -745.2 on
    const double t = x * 1.4426950408889634, k = rint(t);
    // the product is rounded: its remainder goes into f
    const double f = (t - k) + fma(x, 1.4426950408889634, -t);
    double p = kExp2[12];
#pragma unroll
    for (int i = 11; i >= 0; --i) p = fma(p, f, kExp2[i]);
    const int n = static_cast<int>(k), h = n >> 1;
    return p * __hiloint2double((h + 1023) << 20, 0) * __hiloint2double((n - h + 1023) << 20, 0);
}
// 1/d for d >= 1, by two Newton steps from the fp32 reciprocal.
__device__ __forceinline__ double rg_reciprocal(double d) {
    double y = static_cast<double>(1.f / static_cast<float>(d));
    y = y * fma(-d, y, 2.0);
    return y * fma(-d, y, 2.0);
}

// The exact form of one token, by one warp; lane l holds experts l, l + 32, ...
// sel, score: this warp's scratch, E doubles each.
template <typename TL>
__device__ __noinline__ void route_token_exact(const RouteGroupedArgs& a, int t, double* sel, double* score) {
    constexpr int kPer = RG_MAXE / 32;
    const int lane = threadIdx.x & 31;
    const TL* zr = static_cast<const TL*>(a.logits) + static_cast<size_t>(t) * a.E;
    float z[kPer];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        z[i] = e < a.E ? rg_load(zr + e) : -INFINITY;
        m = fmaxf(m, z[i]);   // a NaN operand is ignored
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double s[kPer], sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        // NaN and -inf are masked; +inf is 1 by sigmoid, and shares the weight with its like by softmax
        const double x = a.sigmoid ? -fabs(static_cast<double>(z[i])) : z[i] == m ? 0.0 : static_cast<double>(z[i]) - static_cast<double>(m);
        const double e = rg_exp(x);
        s[i] = z[i] > -INFINITY ? e : 0.0;
        if (a.sigmoid && z[i] > -INFINITY) s[i] = rg_reciprocal(1.0 + e) * (z[i] >= 0.f ? 1.0 : e);
        sum += s[i];
    }
    double norm = 1.0;
    if (!a.sigmoid) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        norm = sum > 0.0 ? rg_reciprocal(sum) : 0.0;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.E) break;
        const bool on = z[i] > -INFINITY;
        const double v = s[i] * norm;
        score[e] = v;
        const double c = on ? (a.bias ? v + static_cast<double>(__ldg(a.bias + e)) : v) : -INFINITY;
        sel[e] = c == c ? c : -INFINITY;   // (a NaN bias)
    }
    __syncwarp();
    const int gs = a.E / a.groups;
    unsigned chosen = 0xffffffffu;
    if (a.topk_groups < a.groups) {
        // W lanes per group, neighbours of each other; lane g ends up with group g
        int W = 1;
        while (2 * W * a.groups <= 32) W *= 2;
        double b1 = -INFINITY, b2 = -INFINITY;
        const int lw = 31 - __clz(W), first = (lane >> lw) * gs;
        if ((lane >> lw) < a.groups)
            for (int j = lane & (W - 1); j < gs; j += W) merge_two(b1, b2, sel[first + j], -static_cast<double>(INFINITY));
        for (int o = 1; o < W; o <<= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            merge_two(b1, b2, o1, o2);
        }
        double g = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        g = __shfl_sync(0xffffffffu, g, (lane * W) & 31);
        if (lane >= a.groups) g = -INFINITY;
        int better = 0;
        for (int o = 0; o < a.groups; ++o) {
            const double v = __shfl_sync(0xffffffffu, g, o);
            better += v > g || (v == g && o < lane);
        }
        chosen = __ballot_sync(0xffffffffu, lane < a.groups && better < a.topk_groups);
    }
    // scores as integers in their order; 64-bit maxima in two 32-bit reductions
    long long v[kPer];
    const float per_group = 1.f / static_cast<float>(gs);   // (e + 1/2) / gs is a half away from whole numbers over gs
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        v[i] = LLONG_MIN;
        if (e < a.E && ((chosen >> static_cast<int>((static_cast<float>(e) + 0.5f) * per_group)) & 1u)) {
            const long long b = __double_as_longlong(fmax(sel[e], kMaskedScore) + 0.0);
            v[i] = b ^ ((b >> 63) & 0x7fffffffffffffffll);
        }
    }
    double wsel = 0.0, wsum = 0.0;
    int isel = 0;
    for (int j = 0; j < a.k; ++j) {
        long long best = LLONG_MIN;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            at = v[i] > best ? i : at;
            best = v[i] > best ? v[i] : best;
        }
        const int hi = static_cast<int>(best >> 32);
        const int hi_max = __reduce_max_sync(0xffffffffu, hi);
        const uint32_t lo = hi == hi_max ? static_cast<uint32_t>(best) : 0u;
        const uint32_t lo_max = __reduce_max_sync(0xffffffffu, lo);
        const uint32_t e = hi == hi_max && lo == lo_max ? static_cast<uint32_t>(lane + 32 * at) : 0xffffffffu;
        const uint32_t be = __reduce_min_sync(0xffffffffu, e);   // equal scores: the lower expert
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (e == be && i == at) v[i] = LLONG_MIN;
        const double w = score[be];
        wsum += w;
        if (lane == j) {
            wsel = w;
            isel = static_cast<int>(be);
        }
    }
    if (lane < a.k) {
        double w = wsel;
        if (a.renorm) w = wsum > 0.0 ? w / wsum : 0.0;
        a.idx[static_cast<size_t>(t) * a.k + lane] = isel;
        a.w[static_cast<size_t>(t) * a.k + lane] = static_cast<float>(w * static_cast<double>(a.scale));
    }
    __syncwarp();   // the scratch may be used again
}

// Any shape, in the exact form: one warp per token.  It is for the shapes that
// the fast form cannot take: 36,992 tokens of 64 and of 256 experts took 62 and
// 121 us by it, 14 and 29 by the other.
template <typename TL>
__global__ void __launch_bounds__(RG_WARPS * 32) route_grouped_kernel(const __grid_constant__ RouteGroupedArgs a) {
    __shared__ double sel[RG_WARPS][RG_MAXE];
    __shared__ double score[RG_WARPS][RG_MAXE];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, t = blockIdx.x * RG_WARPS + warp;
    if (t < a.T) route_token_exact<TL>(a, t, sel[warp], score[warp]);
}

// ---------------------------------------------------------------- fast form
// Signed integers in the order of the floats, and back.
__device__ __forceinline__ int rg_order(float v) {
    const int b = __float_as_int(v);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float rg_value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }
__device__ __forceinline__ float rg_ex2(float x) {   // 2^x, about 2^-22 relative
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rg_rcp(float x) {   // 1/x, about 2^-23 relative
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^(a - b) to a few fp32 roundings whatever the difference: the rounding of
// a - b and of its product with log2(e) go into a second factor.
__device__ __forceinline__ float rg_exp_diff(float a, float b) {
    const float d = a - b, bb = d - a;
    const float lost = (a - (d - bb)) - (b + bb);
    const float t = d * 1.4426950408889634f;
    const float rest = fmaf(d, 1.4426950408889634f, -t) + fmaf(d, 1.925963033500e-8f, lost * 1.4426950408889634f);
    const float y = exp2f(t);
    return fmaf(y, rest * 0.6931471805599453f, y);
}
constexpr int kNoKey = static_cast<int>(0x80000000u);

// Without a bias the logits order the scores, as long as different logits have
// different fp64 scores.  They may not among logits under kTiny (above it fp32
// neighbours are 2^-44 apart, 2^-46 in their scores) and, by sigmoid, where
// 1 - s is small: at 20 neighbours of fp32 are 3.9e-15 apart, 35 steps of fp64,
// at 24 often none; at 30 neighbours of bf16 are 1e-14 apart.  Ties of scores go
// to the lower expert, which the exact form sees to.
constexpr float kTiny = 0x1p-20f;

__device__ __forceinline__ void rg_swap(int& a, int& b) {   // larger first
    const int hi = max(a, b), lo = min(a, b);
    a = hi;
    b = lo;
}
// Batcher's odd-even merge network for 8 keys, descending.
__device__ __forceinline__ void rg_sort8(int (&v)[8]) {
    rg_swap(v[0], v[1]); rg_swap(v[2], v[3]); rg_swap(v[4], v[5]); rg_swap(v[6], v[7]);
    rg_swap(v[0], v[2]); rg_swap(v[1], v[3]); rg_swap(v[4], v[6]); rg_swap(v[5], v[7]);
    rg_swap(v[1], v[2]); rg_swap(v[5], v[6]);
    rg_swap(v[0], v[4]); rg_swap(v[1], v[5]); rg_swap(v[2], v[6]); rg_swap(v[3], v[7]);
    rg_swap(v[2], v[4]); rg_swap(v[3], v[5]);
    rg_swap(v[1], v[2]); rg_swap(v[3], v[4]); rg_swap(v[5], v[6]);
}
// The 8 largest of two descending lists into v, descending; rest: the largest
// key left behind by any merge (REST: for k = 8, whose next key is not listed).
template <bool REST>
__device__ __forceinline__ void rg_merge8(int (&v)[8], const int (&w)[8], int& rest) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        if (REST) rest = __vimax3_s32(rest, min(v[i], w[7 - i]), min(v[i + 1], w[6 - i]));
        v[i] = max(v[i], w[7 - i]);
        v[i + 1] = max(v[i + 1], w[6 - i]);
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)   // a bitonic sequence
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) rg_swap(v[i], v[i + d]);
}

// Scratch of a token whose k best are not told apart by coarse scores.
struct RouteClose {
    double c[16];
    int e[16];
};
static_assert(sizeof(RouteClose) <= RG_MAXE / 4 * sizeof(double), "four of them share a warp's scratch");

// Eight lanes per token, four tokens per warp: a group is one or more whole
// lanes, and a list of 8 keys per lane is sorted in registers.  Three blocks per
// SM at 256 experts (80 registers): with two 40, with four (64 registers) 41 us
// against 36 then; four at 64 experts: 14.2 us, with five 14.6.  Lane l holds the P = E / 8 neighbours from l P on, as
// NL lists of 8.  E a multiple of 8, at most 8 groups (a power of two), k <= 8.
// FULL: P = 8 NL, aligned for vector loads.
template <typename TL, int NL, bool REST, bool FULL>
__global__ void __launch_bounds__(RG_WARPS * 32, NL == 4 ? 3 : 4)
    route_grouped_fast_kernel(const __grid_constant__ RouteGroupedArgs a) {
    __shared__ double sel[RG_WARPS][RG_MAXE];
    __shared__ double score[RG_WARPS][RG_MAXE];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7;
    const int t0 = (blockIdx.x * (blockDim.x >> 5) + warp) * 4;
    if (t0 >= a.T) return;
    const int t = min(t0 + (lane >> 3), a.T - 1);   // (the last warp's spare lanes repeat a token)
    const int P = a.E >> 3, e0 = sub * P;
    const TL* zr = static_cast<const TL*>(a.logits) + static_cast<size_t>(t) * a.E + e0;
    // the logits as they come; FULL: in vectors, unpacked at each use
    constexpr int V = 16 / sizeof(TL), NQ = NL * 8 / V;
    uint4 raw[FULL ? NQ : 1];
    float zs[FULL ? 1 : NL * 8];
    if (FULL) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) raw[FULL ? q : 0] = __ldg(reinterpret_cast<const uint4*>(zr) + q);
    } else {
#pragma unroll
        for (int i = 0; i < NL * 8; ++i) zs[FULL ? 0 : i] = i < P ? rg_load(zr + i) : 0.f;
    }
    auto zval = [&](int i) -> float {
        if (!FULL) return zs[FULL ? 0 : i];
        const uint4& u = raw[FULL ? i / V : 0];
        const int j = i % V;
        if (sizeof(TL) == 4) return __uint_as_float(j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w);
        const uint32_t x = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
        return __uint_as_float(j & 1 ? x & 0xffff0000u : x << 16);
    };
    float zero = 0.f;   // becomes NaN by a masked or infinite logit
#pragma unroll
    for (int i = 0; i < NL * 8; ++i) zero = fmaf(zval(i), 0.f, zero);
    bool odd = !(zero == 0.f);   // the exact form
    bool close = false;          // the k best, or their order, not told apart by coarse scores
    constexpr float kLog2e = 1.4426950408889634f;
    float m = 0.f, sum = 1.f, norm = 1.f;
    if (!a.sigmoid) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NL * 8; ++i)
            if (FULL || i < P) m = fmaxf(m, zval(i));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < NL * 8; ++i)
            if (FULL || i < P) sum += rg_ex2((zval(i) - m) * kLog2e);   // (the difference first: exact for near ones)
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        norm = rg_rcp(sum);
    }
    // Coarse keys: 16 significant bits of the selection score, the expert below them (lower experts first).  Without
    // a bias the logits order the scores, and 16 bits of a bf16 logit are all of it.  The fp32 score of the lane's
    // expert i with its bias:
    auto biased = [&](float zi, int i) -> float {
        const float sc = a.sigmoid ? rg_rcp(1.f + rg_ex2(zi * -kLog2e)) : rg_ex2((zi - m) * kLog2e) * norm;
        return sc + __ldg(a.bias + e0 + i);
    };
    int rest = kNoKey, best[8];
#pragma unroll
    for (int l = 0; l < NL; ++l) {
        int key[8];
        if (!a.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) key[i] = rg_order(zval(8 * l + i) + 0.f);   // (-0 as +0)
        } else if (FULL) {
            const float4 b0 = __ldg(reinterpret_cast<const float4*>(a.bias + e0 + 8 * l));
            const float4 b1 = __ldg(reinterpret_cast<const float4*>(a.bias + e0 + 8 * l) + 1);
            const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float zi = zval(8 * l + i);
                key[i] = rg_order((a.sigmoid ? rg_rcp(1.f + rg_ex2(zi * -kLog2e)) : rg_ex2((zi - m) * kLog2e) * norm) + b[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) key[i] = 8 * l + i < P ? rg_order(biased(zval(8 * l + i), 8 * l + i)) : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) key[i] = FULL || 8 * l + i < P ? (key[i] & ~255) | (255 - e0 - 8 * l - i) : kNoKey;
        rg_sort8(key);
        if (l == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) best[i] = key[i];
        } else {
            rg_merge8<REST>(best, key, rest);
        }
    }

    // groups: the two best of each, their rank among the groups
    bool inside = true, ties = false;   // ties: equal fp64 scores of different logits may matter
    constexpr float kFar = sizeof(TL) == 4 ? 20.f : 30.f;
    if (a.topk_groups < a.groups) {
        const int L = 8 / a.groups, mine = sub / L;
        bool& in = inside;
        if (!a.bias && (a.group_top == 1 || a.E == a.groups)) {   // by the best logit; equal ones to the lower expert
            int g = best[0];
            for (int o = 1; o < L; o <<= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
            int better = 0;
#pragma unroll
            for (int o = 0; o < 8; ++o) better += __shfl_sync(0xffffffffu, g, (lane & 24) + ((o * L) & 7)) > g && o < a.groups ? 1 : 0;
            in = better < a.topk_groups;
            int low = in ? g : 0x7fffffff, high = in ? kNoKey : g;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) {
                low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
                high = max(high, __shfl_xor_sync(0xffffffffu, high, o));
            }
            odd |= sizeof(TL) == 4 && ((low ^ high) & ~255) == 0;
            const float lowest = rg_value(low & ~255);
            odd |= a.sigmoid ? lowest > kFar || lowest < -30.f : lowest - m < -80.f;
            ties = fabsf(lowest) < kTiny;
        } else {
            // The scores of the lane's two best, in fp32 from their logits, then of its group's, in every lane of it.
            // Errors: a score's own, 2.6e-7 by sigmoid, by softmax 3e-7 of itself and 5e-8 of the largest; the fp32
            // sum's, 3.4e-6 of a score by softmax (without a bias the same for all); a rounding of every sum.  Where
            // the second and third keys of a lane are not told apart, the third and fourth may be the larger ones,
            // each by at most disp, a step of the keys (2^-15 relative).  A comparison has four scores, and the group
            // left out may lack two displaced ones.  r: for groups of errors x and y and displacement d of the second,
            // max(2 x, 2 y + 4 d) >= x + y + 2 d, so the largest r of all lanes covers two groups; doubled where the
            // scores' part varies as well.
            const TL* row = static_cast<const TL*>(a.logits) + static_cast<size_t>(t) * a.E;
            const int e1 = 255 - (best[0] & 255), e2 = P > 1 ? 255 - (best[1] & 255) : e1;
            const float z1 = rg_load(row + e1), z2 = rg_load(row + e2);
            odd |= a.sigmoid ? fabsf(z1) > 30.f : z1 - m < -80.f;
            float c1 = a.sigmoid ? rg_rcp(1.f + rg_ex2(z1 * -kLog2e)) : rg_ex2((z1 - m) * kLog2e) * norm;
            float c2 = a.sigmoid ? rg_rcp(1.f + rg_ex2(z2 * -kLog2e)) : rg_ex2((z2 - m) * kLog2e) * norm;
            float err = a.sigmoid ? 1.04e-6f : a.bias ? fmaf(fmaxf(c1, c2), 1.7e-5f, 4e-7f * norm) : 2e-7f * norm;
            float disp = 0.f;
            if (a.bias) {
                c1 += __ldg(a.bias + e1);
                c2 += __ldg(a.bias + e2);
                odd |= !(c1 == c1);   // a NaN bias: the lane's first key, and comparisons with it would lose its group
            }
            if (P > 2 && rg_value(best[1] & ~255) - rg_value(best[2] & ~255) <= fabsf(rg_value(best[1] & ~255)) * 4e-5f + 8e-6f) {
                // (by softmax with a bias their scores may be any, and so their part of the sum's error)
                disp = a.bias ? fmaf(fabsf(c2), 3.2e-5f, a.sigmoid ? 0.f : 2e-6f)
                              : fabsf(z2) * (a.sigmoid ? 1e-5f : 4e-5f * c2);
                odd |= !(fabsf(z2) < 1e4f);   // a step of the logit is more than a small part of its weight
            }
            if (P == 1) c2 = -INFINITY;
            // equal keys come to the lower expert first, which may have the smaller score
            const float larger = fmaxf(c1, c2);
            c2 = fminf(c1, c2);
            c1 = larger;
            for (int o = 1; o < L; o <<= 1) {
                const float o1 = __shfl_xor_sync(0xffffffffu, c1, o), o2 = __shfl_xor_sync(0xffffffffu, c2, o);
                merge_two(c1, c2, o1, o2);
            }
            const float both = fabsf(c1) + (a.E == a.groups ? 0.f : fabsf(c2));
            const float r = fmaf(both, a.sigmoid || a.bias ? 2.4e-7f : 7.2e-7f, 4.f * disp);
            err += a.sigmoid || !a.bias ? r : 2.f * r;
            const float g = a.group_top == 2 && c2 > -INFINITY ? c1 + c2 : c1;
            int better = 0;
#pragma unroll
            for (int o = 0; o < 8; ++o) {
                const float v = __shfl_sync(0xffffffffu, g, (lane & 24) + ((o * L) & 7));
                better += o < a.groups && (v > g || (v == g && o < mine)) ? 1 : 0;
            }
            in = better < a.topk_groups;
            float low = in ? g : INFINITY, high = in ? -INFINITY : g;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) {
                low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
                err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, o));
            }
            odd |= !(low - high > err);
        }
        if (!in) {
#pragma unroll
            for (int i = 0; i < 8; ++i) best[i] = kNoKey;
            rest = kNoKey;
        }
    }
    // the token's 8 best, in every lane
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        int w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __shfl_xor_sync(0xffffffffu, best[i], o);
        if (REST) rest = max(rest, __shfl_xor_sync(0xffffffffu, rest, o));
        rg_merge8<REST>(best, w, rest);
    }
    // the k-th must be clear of the next by the same errors
    int kth = best[0], next = REST ? rest : kNoKey, own = best[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i == a.k - 1) kth = best[i];
        if (i == a.k) next = best[i];
        if (i == sub) own = best[i];
    }
    if (!a.bias) {
        close |= sizeof(TL) == 4 && next != kNoKey && ((kth ^ next) & ~255) == 0;
        ties |= fabsf(rg_value(kth & ~255)) < kTiny;
        if (ties) {   // (seldom: read again)
#pragma unroll 1
            for (int i = 0; i < P; ++i) {
                const float zi = rg_load(zr + i);
                odd |= fabsf(zi) < kTiny && zi != 0.f;
            }
        }
    } else if (next != kNoKey) {
        const float vk = rg_value(kth & ~255), vn = rg_value(next & ~255);
        close |= !(vk - vn > fmaxf(fabsf(vk), fabsf(vn)) * 4e-5f + 8e-6f);
    }
    // the k, their order and weights: lane j of the token has candidate j.  Without a bias the logits order the
    // scores (but for tiny and far ones), with one, scores closer than their error are settled below.
    const bool has = sub < a.k && own != kNoKey;
    const int e = has ? 255 - (own & 255) : 0;
    const float ze = rg_load(static_cast<const TL*>(a.logits) + static_cast<size_t>(t) * a.E + e);
    const float x = a.sigmoid ? rg_exp_diff(0.f, ze) : rg_exp_diff(ze, m);
    float w = a.sigmoid ? 1.f / (1.f + x) : x / sum;
    const float c = a.bias ? w + __ldg(a.bias + e) : ze;
    // far scores need fp64's range
    odd |= has && (a.sigmoid ? ze > (a.bias ? 30.f : kFar) || ze < -30.f : ze - m < -80.f);
    odd |= has && !a.bias && fabsf(ze) < kTiny && ze != 0.f;
    // two scores' errors: 1.9e-7 each by sigmoid; by softmax the fp32 sum's comes on top, at most 3.4e-6 of the two
    // scores' difference (32 terms in sequence and three levels of lanes, 2.1e-6; the terms' own, 1.3e-6)
    const float apart = a.sigmoid ? 1.2e-6f : 4.6e-6f;
    int rank = 0;
    float wsum = 0.f;
#pragma unroll
    for (int o = 0; o < 8; ++o) {
        const float co = __shfl_sync(0xffffffffu, c, (lane & 24) + o), wo = __shfl_sync(0xffffffffu, w, (lane & 24) + o);
        const int eo = __shfl_sync(0xffffffffu, e, (lane & 24) + o);
        if (o < a.k) {
            rank += co > c || (co == c && eo < e) ? 1 : 0;
            wsum += wo;
            if (a.bias) close |= has && eo != e && fabsf(co - c) < apart + fabsf(c) * 3e-7f;
        }
    }
    odd |= (sub < a.k && !has) || !(c == c);
    unsigned odds = __ballot_sync(0xffffffffu, odd);
    const unsigned closes = __ballot_sync(0xffffffffu, close);
    const unsigned mine = 0xffu << (lane & 24);
    if (has && !((odds | closes) & mine) && t0 + (lane >> 3) < a.T) {
        if (a.renorm) w = w / wsum;
        a.idx[static_cast<size_t>(t) * a.k + rank] = e;
        a.w[static_cast<size_t>(t) * a.k + rank] = w * a.scale;
    }
    if (closes & ~odds) {
        // every expert that may be among the k, at most 16 of a token, by fp64 scores; all four tokens at once
        RouteClose& sc = *reinterpret_cast<RouteClose*>(&sel[warp][(lane >> 3) * (RG_MAXE / 4)]);
        const float vk = rg_value(kth & ~255);
        const float least = a.bias ? vk - fabsf(vk) * 4e-5f - 8e-6f : vk;
        double dsum = 0.0;
        uint32_t may = 0;
#pragma unroll
        for (int i = 0; i < NL * 8; ++i) {
            if (!(FULL || i < P)) continue;
            const float c0 = a.bias ? biased(zval(i), i) : zval(i);
            may |= (inside && c0 >= least ? 1u : 0u) << i;
        }
        if (!a.sigmoid && a.bias)
            for (int i = 0; i < P; ++i) dsum += rg_exp(static_cast<double>(rg_load(zr + i)) - static_cast<double>(m));
        int at = __popc(may), n = at;
        if (!a.sigmoid) {
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) dsum += __shfl_xor_sync(0xffffffffu, dsum, o);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, at, o, 8);
            if (sub >= o) at += v;
        }
        const int total = __shfl_sync(0xffffffffu, at, (lane & 24) + 7);
        at -= n;
        const bool fits = total <= 16 && total >= a.k;   // (fewer: infinite or NaN scores by the bias)
        odds |= __ballot_sync(0xffffffffu, !fits && ((closes & mine) != 0));
        if (fits)
            for (uint32_t b = may; b; b &= b - 1) sc.e[at++] = e0 + __ffs(b) - 1;
        __syncwarp();
        double cc[2], ww[2];
        int ee[2], rr[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool on = fits && sub + 8 * h < total;
            ee[h] = on ? sc.e[sub + 8 * h] : 0;
            const double x0 = static_cast<double>(rg_load(static_cast<const TL*>(a.logits) + static_cast<size_t>(t) * a.E + ee[h]));
            const double x1 = rg_exp(a.sigmoid ? -fabs(x0) : x0 - static_cast<double>(m));
            ww[h] = a.sigmoid ? rg_reciprocal(1.0 + x1) * (x0 >= 0.0 ? 1.0 : x1) : x1 / (a.bias ? dsum : static_cast<double>(sum));
            cc[h] = a.bias ? ww[h] + static_cast<double>(__ldg(a.bias + ee[h])) : x0 + 0.0;
            if (on) sc.c[sub + 8 * h] = cc[h];
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const double cj = sc.c[j];
            const int ej = sc.e[j];
#pragma unroll
            for (int h = 0; h < 2; ++h) rr[h] += j < total && (cj > cc[h] || (cj == cc[h] && ej < ee[h])) ? 1 : 0;
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (fits && sub + 8 * h < total && rr[h] < a.k) sc.c[rr[h]] = ww[h];
        __syncwarp();
        if (fits && (closes & mine) && !(odds & mine) && t0 + (lane >> 3) < a.T) {
            double all = 0.0;
            for (int j = 0; j < a.k; ++j) all += sc.c[j];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (sub + 8 * h < total && rr[h] < a.k) {
                    const double x = a.renorm ? ww[h] / all : ww[h];
                    a.idx[static_cast<size_t>(t) * a.k + rr[h]] = ee[h];
                    a.w[static_cast<size_t>(t) * a.k + rr[h]] = static_cast<float>(x * static_cast<double>(a.scale));
                }
        }
        __syncwarp();
    }
    for (int j = 0; j < 4; ++j)
        if (((odds >> (8 * j)) & 0xffu) && t0 + j < a.T) route_token_exact<TL>(a, t0 + j, sel[warp], score[warp]);
}

template <typename TL>
static ms_status route_grouped_launch(const RouteGroupedArgs& a, cudaStream_t s) {
    const bool fast = a.E % 8 == 0 && a.k <= 8 && a.groups <= 8 && (a.groups & (a.groups - 1)) == 0;
    if (!fast)
        return launch(K_ROUTE_GROUPED, route_grouped_kernel<TL>, dim3((a.T + RG_WARPS - 1) / RG_WARPS), dim3(RG_WARPS * 32),
                      0, s, a);
    const int P = a.E / 8;
    // warps per block: fewer for small batches, so that more SMs have some (128 tokens: 4.5 us, with 8 warps 4.6)
    int warps = RG_WARPS;
    while (warps > 1 && (a.T + 4 * warps - 1) / (4 * warps) < num_sms()) warps /= 2;
    const dim3 grid((a.T + 4 * warps - 1) / (4 * warps)), block(32 * warps);
    const bool vec = aligned16(a.logits) && aligned16(a.bias), rest = a.k == 8;
#define ROUTE_FAST(NL)                                                                                               \
    return launch(K_ROUTE_GROUPED,                                                                                   \
                  P == 8 * NL && vec ? (rest ? route_grouped_fast_kernel<TL, NL, true, true>                         \
                                             : route_grouped_fast_kernel<TL, NL, false, true>)                       \
                                     : (rest ? route_grouped_fast_kernel<TL, NL, true, false>                        \
                                             : route_grouped_fast_kernel<TL, NL, false, false>),                     \
                  grid, block, 0, s, a)
    if (P <= 8) ROUTE_FAST(1);
    if (P <= 16) ROUTE_FAST(2);
    ROUTE_FAST(4);
#undef ROUTE_FAST
}

}  // namespace ms

extern "C" ms_status moe_route_grouped(const void* logits, ms_dtype logits_dtype, const float* select_bias, int T,
                                       int E, ms_score score, int n_groups, int topk_groups, int group_top, int k,
                                       int renormalize, float scale, int32_t* topk_idx, float* topk_w, void* stream) {
    if (!logits || !topk_idx || !topk_w) return MS_ERR_INVALID_ARG;
    if (logits_dtype != MS_F32 && logits_dtype != MS_BF16) return MS_ERR_INVALID_ARG;
    if (score != MS_SOFTMAX && score != MS_SIGMOID) return MS_ERR_INVALID_ARG;
    if (T <= 0 || E <= 0 || n_groups <= 0 || E % n_groups != 0) return MS_ERR_INVALID_ARG;
    if (topk_groups <= 0 || topk_groups > n_groups || group_top < 1 || group_top > 2) return MS_ERR_INVALID_ARG;
    if (k <= 0 || k > topk_groups * (E / n_groups)) return MS_ERR_INVALID_ARG;
    if (!ms::element_aligned(logits, logits_dtype)) return MS_ERR_INVALID_ARG;
    if (!ms::words_aligned(select_bias, topk_idx, topk_w)) return MS_ERR_INVALID_ARG;
    if (E > ms::RG_MAXE || n_groups > 32 || k > 32) return MS_ERR_UNSUPPORTED;
    ms::RouteGroupedArgs a{logits,       select_bias,  T,     E,        n_groups, topk_groups, group_top, k,
                           score == MS_SIGMOID, renormalize != 0, scale, topk_idx, topk_w};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return logits_dtype == MS_BF16 ? ms::route_grouped_launch<__nv_bfloat16>(a, s) : ms::route_grouped_launch<float>(a, s);
}
