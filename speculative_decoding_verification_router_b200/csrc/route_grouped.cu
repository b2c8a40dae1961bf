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
// Scores are held in fp64: with E scores in [0, 1] two neighbours are often
// closer than fp32 rounding, and the choice must not depend on it.
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

__device__ __forceinline__ void argmax_merge_f64(double& v, int& i, double v2, int i2) {
    if (v2 > v || (v2 == v && i2 < i)) {
        v = v2;
        i = i2;
    }
}

// One warp per token; lane l holds experts l, l + 32, ...
template <typename TL>
__global__ void __launch_bounds__(RG_WARPS * 32) route_grouped_kernel(const RouteGroupedArgs a) {
    constexpr int kPer = RG_MAXE / 32;
    __shared__ double sel_s[RG_WARPS][RG_MAXE];
    __shared__ double score_s[RG_WARPS][RG_MAXE];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * RG_WARPS + warp;
    if (t >= a.T) return;
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
        const bool on = z[i] > -INFINITY;   // NaN and -inf: masked
        if (!on) s[i] = 0.0;
        else if (a.sigmoid) s[i] = 1.0 / (1.0 + exp(-static_cast<double>(z[i])));
        else s[i] = z[i] == m ? 1.0 : exp(static_cast<double>(z[i]) - static_cast<double>(m));
        sum += s[i];
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    double* sel = sel_s[warp];
    double* score = score_s[warp];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.E) break;
        const bool on = z[i] > -INFINITY;
        const double v = !on ? 0.0 : a.sigmoid ? s[i] : s[i] / sum;
        score[e] = v;
        sel[e] = on ? (a.bias ? v + static_cast<double>(__ldg(a.bias + e)) : v) : -INFINITY;
    }
    __syncwarp();
    const int gs = a.E / a.groups;
    unsigned chosen = 0xffffffffu;
    if (a.topk_groups < a.groups) {
        double g = -INFINITY;
        if (lane < a.groups) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int j = 0; j < gs; ++j) {
                const double v = sel[lane * gs + j];
                if (v > b1) {
                    b2 = b1;
                    b1 = v;
                } else if (v > b2) {
                    b2 = v;
                }
            }
            g = b1;
            if (a.group_top == 2 && b2 > -INFINITY) g += b2;
        }
        int better = 0;
        for (int o = 0; o < a.groups; ++o) {
            const double v = __shfl_sync(0xffffffffu, g, o);
            better += v > g || (v == g && o < lane);
        }
        chosen = __ballot_sync(0xffffffffu, lane < a.groups && better < a.topk_groups);
    }
    double v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        v[i] = -INFINITY;
        if (e < a.E && ((chosen >> (e / gs)) & 1u)) v[i] = fmax(sel[e], kMaskedScore);
    }
    double wsel = 0.0, wsum = 0.0;
    int isel = 0;
    for (int j = 0; j < a.k; ++j) {
        double bv = -INFINITY;
        int bi = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < kPer; ++i) argmax_merge_f64(bv, bi, v[i], v[i] > -INFINITY ? lane + 32 * i : 0x7fffffff);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double v2 = __shfl_xor_sync(0xffffffffu, bv, o);
            const int i2 = __shfl_xor_sync(0xffffffffu, bi, o);
            argmax_merge_f64(bv, bi, v2, i2);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i == bi) v[i] = -INFINITY;
        const double w = score[bi];
        wsum += w;
        if (lane == j) {
            wsel = w;
            isel = bi;
        }
    }
    if (lane < a.k) {
        double w = wsel;
        if (a.renorm) w = wsum > 0.0 ? w / wsum : 0.0;
        a.idx[static_cast<size_t>(t) * a.k + lane] = isel;
        a.w[static_cast<size_t>(t) * a.k + lane] = static_cast<float>(w * static_cast<double>(a.scale));
    }
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
    if (E > ms::RG_MAXE || n_groups > 32 || k > 32) return MS_ERR_UNSUPPORTED;
    ms::RouteGroupedArgs a{logits,       select_bias,  T,     E,        n_groups, topk_groups, group_top, k,
                           score == MS_SIGMOID, renormalize != 0, scale, topk_idx, topk_w};
    const dim3 grid((T + ms::RG_WARPS - 1) / ms::RG_WARPS), block(ms::RG_WARPS * 32);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (logits_dtype == MS_BF16)
        return ms::launch(ms::K_ROUTE_GROUPED, ms::route_grouped_kernel<__nv_bfloat16>, grid, block, 0, s, a);
    return ms::launch(ms::K_ROUTE_GROUPED, ms::route_grouped_kernel<float>, grid, block, 0, s, a);
}
