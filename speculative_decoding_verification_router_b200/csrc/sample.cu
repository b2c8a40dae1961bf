// Sampling from logits rows by temperature, min-p, top-k and top-p, and
// speculative verification that keeps the sampled distribution.
//
// A row's weights are w_i = exp((l_i - max l) / T); NaN counts as -inf, and
// weights under 2^-64 of the largest (or under min_p) as zero.  Top-k keeps
// the first k tokens of the order (larger logit, lower index), top-p the
// shortest prefix of those whose weights reach p times their sum.  The token
// is the first index whose cumulative weight, in index order, exceeds u times
// the sum S of the kept weights.
//
// A decision (is the prefix long enough, does the cumulative sum pass u S)
// must not depend on rounding: with 10^5 tokens of similar weight the
// borders of the cumulative sum are 10^-5 apart, so an error of 10^-7 (fp32)
// would move one draw in a hundred.  Weights are therefore computed to ~10^-13
// and summed in fp64 in a fixed order; sums that pass through integer
// histograms are fixed point (2^-45), so that their order cannot matter.
//
// One thread-block cluster per row: each CTA copies its part of the row into
// shared memory once, and every later pass (maximum, selection, sums, the
// draw) reads it from there; partial results cross the cluster through
// distributed shared memory.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "ms_common.cuh"

namespace ms {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_MAXC = 8;              // CTAs of a row's cluster
constexpr int SP_MAX_CHUNK = 32768;     // elements of a row per CTA (bounds the histogram limbs)
constexpr int SP_BINS = 1024;
constexpr int32_t SP_ACCEPTED = -2;
constexpr int SP_MAX_V = SP_MAXC * SP_MAX_CHUNK;
constexpr int SP_FIX = 45;              // fixed point of histogram masses: 2^18 weights of 1 fit 63 bits
constexpr int SP_LIMB = 15;             // 3 limbs; 2^15 elements x 2^15 fit a 32-bit counter
constexpr int SP_CAP = 2048;            // candidates of a row that the leader finishes from a list
static_assert(SP_BINS == 2 * SP_THREADS, "the bin scan gives every thread two bins");

struct SampleArgs {
    const void* logits;         // [rows, V]
    int V, rows, chunk, cluster;
    int per;                    // rows that share one entry of the parameters (K + 1; 1 for plain sampling)
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    const int32_t* draft;       // verify: [rows / per, per - 1]
    const float* q;             // verify: [rows / per, per - 1, V] or NULL (the draft is certain)
    int32_t* token;             // [rows]; verify: SP_ACCEPTED where the row's draft is accepted
    float* probs;               // sample: [rows, V] or NULL
};

// ---------------------------------------------------------------- small helpers
__device__ __forceinline__ uint32_t sp_mapa(const void* local, uint32_t rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
    return ra;
}
__device__ __forceinline__ void st_cluster_u64(const void* local, uint32_t rank, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(sp_mapa(local, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f64(const void* local, uint32_t rank, double v) {
    st_cluster_u64(local, rank, static_cast<unsigned long long>(__double_as_longlong(v)));
}
__device__ __forceinline__ void red_cluster_u32(const void* local, uint32_t rank, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(sp_mapa(local, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void red_cluster_u64(const void* local, uint32_t rank, unsigned long long v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(sp_mapa(local, rank)), "l"(v) : "memory");
}

// The bits of a float as a double.  Zero and subnormals become about 2^-127,
// which no difference of logits can see; infinities become +-2^128 (masked
// tokens are sorted out by comparisons on the float itself).
__device__ __forceinline__ double bits_to_f64(uint32_t u) {
    const uint32_t hi = (u & 0x80000000u) | (((u & 0x7fffffffu) >> 3) + 0x38000000u);
    return __hiloint2double(static_cast<int>(hi), static_cast<int>(u << 29));
}

// Floats in ascending order as unsigned integers (-0 equal to +0).
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// 2^t for -65 < t <= 0, relative error about 2e-13: 2^(k/16) from a table of
// 16 doubles (one per pair of shared-memory banks: no conflicts whatever the
// lanes ask for) times the Taylor polynomial of degree 5 of 2^r, |r| <= 1/32.
__device__ __forceinline__ double exp2_64(double t, const double* tab) {
    constexpr double kMagic = 422212465065984.0;   // 1.5 * 2^48: adding it rounds t to multiples of 1/16
    const double z = t + kMagic;
    const int k = __double2loint(z);
    const double r = t - (z - kMagic);
    double p = fma(r, 1.3333558146428443e-3, 9.6181291076284772e-3);   // ln2^5/5!, ln2^4/4!
    p = fma(p, r, 5.5504108664821580e-2);                              // ln2^3/3!
    p = fma(p, r, 2.4022650695910071e-1);                              // ln2^2/2!
    p = fma(p, r, 6.9314718055994531e-1);                              // ln2
    const double base = tab[k & 15];
    const double v = fma(base, p * r, base);
    return __hiloint2double(__double2hiint(v) + ((k >> 4) << 20), __double2loint(v));
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

template <typename TL>
struct SpElem;
template <>
struct SpElem<float> {
    static constexpr int VEC = 4;
    static constexpr int KSH = 0;
    static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ float load(const float* p) { return __ldg(p); }
    static __device__ __forceinline__ float ninf() { return -INFINITY; }
};
template <>
struct SpElem<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static constexpr int KSH = 16;   // the low half of a widened bf16 carries nothing
    static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
        const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
        return bf16_to_f32(__ldg(reinterpret_cast<const uint16_t*>(p)));
    }
    static __device__ __forceinline__ __nv_bfloat16 ninf() { return __ushort_as_bfloat16(0xff80); }
};

// Row masses by logit interval, and the candidate lists; never in use together.
struct SampleSmem {
    double tab[16];
    double wsum[SP_MAXC * SP_WARPS];          // every warp's sum, of every CTA of the cluster
    double rsum[SP_MAXC * SP_WARPS];          // the same for the residual
    double dscan[SP_WARPS];
    unsigned long long scan[SP_WARPS];
    unsigned long long sel_above, sel_total;  // broadcast results of a selection round
    unsigned long long list_cut;              // broadcast results of a list: composite key of the last token kept,
    double list_sum;                          // and the sum of the kept weights
    double wx;
    union {
        struct {
            unsigned long long mass[SP_BINS];   // leader: masses pushed by the other CTAs
            uint32_t limb[3][SP_BINS];
        } h;
        struct {
            unsigned long long lst[SP_CAP];     // leader: the row's candidates in index order
            unsigned long long loc[SP_CAP];     // this CTA's candidates; leader, later: the list in descending order
        } l;
    };
    uint32_t cnt[SP_BINS];
    float cmax[SP_MAXC];
    uint32_t ccnt[SP_MAXC];
    uint32_t tie[SP_MAXC];
    float wmax[SP_WARPS];
    uint32_t wcnt[SP_WARPS];
    uint32_t sel_bin, sel_cnt, sel_cabove;
    uint32_t cut_idx;                         // broadcast: index of the last tied token kept
    int last;
    uint32_t keep;
};

// Where a CTA's part of the row sits: element i (row index begin + i) is
// buf[mis + i]; positions outside [mis, mis + n) hold -inf.
template <typename TL>
struct SpChunk {
    TL* buf;
    int mis, n, nvec, begin;
    __device__ __forceinline__ int index(int vec, int e) const { return begin + vec * SpElem<TL>::VEC + e - mis; }
    __device__ __forceinline__ void load(int vec, float (&v)[SpElem<TL>::VEC]) const {
        SpElem<TL>::unpack(reinterpret_cast<const uint4*>(buf)[vec], v);
    }
};

// The row's weights: w(l) = 2^((l - max) c), c = log2(e) / T.
struct SpScale {
    float m;        // max l
    double md, c;
    const double* tab;
    __device__ __forceinline__ double weight(float l) const {
        return exp2_64((bits_to_f64(__float_as_uint(l)) - md) * c, tab);
    }
};

// A kept set: logits above tau, and those equal to it up to index icut.
struct SpCut {
    float tau;
    int icut;
    __device__ __forceinline__ bool keeps(float l, int idx) const { return l > tau || (l == tau && idx <= icut); }
};

// Tokens in descending order: (logit, lower index first) as one integer.
__device__ __forceinline__ unsigned long long composite(float l, int idx) {
    return (static_cast<unsigned long long>(order_key(l)) << 32) | (0xffffffffu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ float composite_value(unsigned long long k) { return key_value(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int composite_index(unsigned long long k) {
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
}

// Index range of a warp's part of the chunk, in 16-byte vectors: contiguous,
// so that (warp, step, lane, element) runs in index order.
__device__ __forceinline__ void warp_segment(int nvec, int warp, int& q0, int& q1) {
    const int per = ((nvec + SP_WARPS - 1) / SP_WARPS + 31) & ~31;
    q0 = min(nvec, warp * per);
    q1 = min(nvec, q0 + per);
}

// ---------------------------------------------------------------- selection
// Logit intervals of equal width below the maximum; the last one takes the rest.
struct SpBins {
    float m, s;
    __device__ __forceinline__ uint32_t of(float l) const {
        return min(static_cast<uint32_t>((m - l) * s), static_cast<uint32_t>(SP_BINS - 1));   // NaN (inf - inf): 0
    }
};

struct SpBin {
    uint32_t b, cnt, cabove;            // the interval, its tokens, the tokens above it
    unsigned long long above, total;    // masses (or counts) above it, and of the row
};

// The leader's part of a selection round: merges the tables, scans them from
// the top and broadcasts the first interval where `above` + the running total
// reaches the target (`frac` of the round's total where target < 0).
template <bool MASS>
__device__ void select_bin(SampleSmem& sm, uint32_t C, unsigned long long above, uint32_t cabove, double target,
                           double frac) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned long long v[2];
    uint32_t n[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = 2 * tid + j;
        n[j] = sm.cnt[i];
        v[j] = n[j];
        if (MASS)
            v[j] = sm.h.mass[i] + sm.h.limb[0][i] + (static_cast<unsigned long long>(sm.h.limb[1][i]) << SP_LIMB) +
                   (static_cast<unsigned long long>(sm.h.limb[2][i]) << (2 * SP_LIMB));
        if (n[j]) atomicMax(&sm.last, i);
    }
    const unsigned long long own = v[0] + v[1];
    const unsigned long long inc = warp_scan(own, lane);
    const uint32_t cown = n[0] + n[1];
    const uint32_t cinc = warp_scan(cown, lane);
    if (lane == 31) {
        sm.scan[warp] = inc;
        sm.wcnt[warp] = cinc;
    }
    __syncthreads();
    unsigned long long ex = above + inc - own, tot = above;
    uint32_t cex = cabove + cinc - cown;
    for (int w = 0; w < SP_WARPS; ++w) {
        if (w < warp) {
            ex += sm.scan[w];
            cex += sm.wcnt[w];
        }
        tot += sm.scan[w];
    }
    if (target < 0.0) target = fmax(frac * static_cast<double>(tot), 0.5);
    // the last occupied interval where rounding left the target above the total
    const bool never = static_cast<double>(tot) < target;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const bool hit = never ? 2 * tid + j == sm.last
                               : n[j] && static_cast<double>(ex) < target && static_cast<double>(ex + v[j]) >= target;
        if (hit)
            for (uint32_t r = 0; r < C; ++r) {
                st_cluster_s32(&sm.sel_bin, r, 2 * tid + j);
                st_cluster_s32(&sm.sel_cnt, r, static_cast<int>(n[j]));
                st_cluster_s32(&sm.sel_cabove, r, static_cast<int>(cex));
                st_cluster_u64(&sm.sel_above, r, ex);
                st_cluster_u64(&sm.sel_total, r, tot);
            }
        ex += v[j];
        cex += n[j];
    }
}

// One selection round over the cluster's part of the row: a histogram of the
// elements that bin_of() accepts (counts always, fixed-point masses when MASS),
// merged and scanned by the leader.  Elements of the last interval are summed
// in registers when LAST: it takes the bulk of a peaked row.
template <typename TL, bool MASS, bool LAST, typename F>
__device__ SpBin select_round(SampleSmem& sm, const SpChunk<TL>& ck, const SpScale& sc, uint32_t rank, uint32_t C,
                              unsigned long long above, uint32_t cabove, double target, double frac, F bin_of) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < SP_BINS; i += SP_THREADS) {
        sm.cnt[i] = 0;
        if (MASS) {
            sm.h.limb[0][i] = sm.h.limb[1][i] = sm.h.limb[2][i] = 0;
            sm.h.mass[i] = 0;
        }
    }
    if (tid == 0) sm.last = 0;
    cluster_sync_all();   // the leader's tables are clear before anyone adds to them
    uint32_t rest_n = 0;
    unsigned long long rest = 0;
    for (int q = tid; q < ck.nvec; q += SP_THREADS) {
        float v[VEC];
        ck.load(q, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            uint32_t bin;
            if (!bin_of(v[e], bin)) continue;
            unsigned long long W = 0;
            if (MASS) {
                // adding 2^7 leaves the weight as an integer of 2^-45 in the low mantissa bits
                const double z = sc.weight(v[e]) + 128.0;
                W = static_cast<unsigned long long>(__double_as_longlong(z)) & 0xfffffffffffffull;
            }
            if (LAST && bin == SP_BINS - 1) {
                ++rest_n;
                rest += W;
                continue;
            }
            atomicAdd(&sm.cnt[bin], 1u);
            if (MASS) {
                atomicAdd(&sm.h.limb[0][bin], static_cast<uint32_t>(W) & ((1u << SP_LIMB) - 1));
                atomicAdd(&sm.h.limb[1][bin], static_cast<uint32_t>(W >> SP_LIMB) & ((1u << SP_LIMB) - 1));
                atomicAdd(&sm.h.limb[2][bin], static_cast<uint32_t>(W >> (2 * SP_LIMB)));
            }
        }
    }
    if (LAST) {
        rest_n = __reduce_add_sync(0xffffffffu, rest_n);
        if (MASS) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
        }
        if (lane == 0 && rest_n) {
            atomicAdd(&sm.cnt[SP_BINS - 1], rest_n);
            if (MASS) {
                atomicAdd(&sm.h.limb[0][SP_BINS - 1], static_cast<uint32_t>(rest) & ((1u << SP_LIMB) - 1));
                atomicAdd(&sm.h.limb[1][SP_BINS - 1], static_cast<uint32_t>(rest >> SP_LIMB) & ((1u << SP_LIMB) - 1));
                atomicAdd(&sm.h.limb[2][SP_BINS - 1], static_cast<uint32_t>(rest >> (2 * SP_LIMB)));
            }
        }
    }
    __syncthreads();
    if (rank != 0) {
        for (int i = tid; i < SP_BINS; i += SP_THREADS) {
            if (sm.cnt[i] == 0) continue;
            if (MASS)
                red_cluster_u64(&sm.h.mass[i], 0,
                                sm.h.limb[0][i] + (static_cast<unsigned long long>(sm.h.limb[1][i]) << SP_LIMB) +
                                    (static_cast<unsigned long long>(sm.h.limb[2][i]) << (2 * SP_LIMB)));
            red_cluster_u32(&sm.cnt[i], 0, sm.cnt[i]);
        }
    }
    cluster_sync_all();
    if (rank == 0) select_bin<MASS>(sm, C, above, cabove, target, frac);
    cluster_sync_all();
    return SpBin{sm.sel_bin, sm.sel_cnt, sm.sel_cabove, sm.sel_above, sm.sel_total};
}

// First round: intervals of the logit itself over the 24 binary orders of
// magnitude below the largest weight, or down to `lo` where that is nearer.
__device__ __forceinline__ SpBins first_bins(const SpScale& sc, float lo) {
    const float width = fminf(sc.m - lo, static_cast<float>(24.0 / sc.c));
    return SpBins{sc.m, width > 0.f && width < 1e30f ? static_cast<float>(SP_BINS - 1) / width : 0.f};
}

template <typename TL, bool MASS>
__device__ SpBin select_first(SampleSmem& sm, const SpChunk<TL>& ck, const SpScale& sc, uint32_t rank, uint32_t C,
                              float lo, double target, double frac) {
    const SpBins bins = first_bins(sc, lo);
    return select_round<TL, MASS, true>(sm, ck, sc, rank, C, 0ull, 0u, target, frac, [&](float l, uint32_t& bin) {
        bin = bins.of(l);
        return l >= lo;
    });
}

// Later rounds: the ordered keys of one interval, SP_BINS ranges at a time, down
// to a single key.  Returns that key; `at` becomes its entry.
template <typename TL, bool MASS>
__device__ uint32_t select_key(SampleSmem& sm, const SpChunk<TL>& ck, const SpScale& sc, uint32_t rank, uint32_t C,
                               float lo, double target, SpBin& at) {
    constexpr int KSH = SpElem<TL>::KSH;
    const SpBins bins = first_bins(sc, lo);
    const uint32_t b0 = at.b;
    // bounds of the interval's logits, widened by more than the rounding of SpBins::of
    float top = sc.m, bot = lo;
    if (bins.s > 0.f) {
        const float slack = fabsf(sc.m) * 3e-7f;
        if (b0 > 0) top = fminf(sc.m, sc.m - static_cast<float>(b0) / bins.s * (1.f - 1e-6f) + slack);
        if (b0 < SP_BINS - 1) bot = fmaxf(lo, sc.m - static_cast<float>(b0 + 1) / bins.s * (1.f + 1e-6f) - slack);
    }
    uint32_t khi = order_key(top) >> KSH, klo = order_key(bot) >> KSH;
    const unsigned long long total = at.total;
    while (khi > klo) {
        int sh = 0;
        while (((khi - klo) >> sh) >= SP_BINS) ++sh;
        at = select_round<TL, MASS, false>(sm, ck, sc, rank, C, at.above, at.cabove, target, 0.0,
                                           [&](float l, uint32_t& bin) {
                                               const uint32_t key = order_key(l) >> KSH;
                                               bin = (khi - key) >> sh;
                                               return l >= lo && key >= klo && key <= khi && bins.of(l) == b0;
                                           });
        khi -= at.b << sh;
        const uint32_t span = (1u << sh) - 1;
        klo = khi - klo > span ? khi - span : klo;
    }
    at.total = total;
    return khi;
}

// The logit that a key stands for.
template <typename TL>
__device__ __forceinline__ float key_logit(uint32_t key) {
    constexpr int KSH = SpElem<TL>::KSH;
    return key_value(KSH ? (key << KSH) | ((key >> 15) ? 0u : 0xffffu) : key);
}

// This CTA's elements that keep() accepts as composite keys in sm.l.loc, in
// index order, and the count of every CTA in sm.ccnt.  Returns the cluster's
// count; where it exceeds SP_CAP the lists are not complete.
template <typename TL, typename F>
__device__ uint32_t gather(SampleSmem& sm, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, F keep) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    uint32_t n = 0;
    for (int q = q0 + lane; q < q1; q += 32) {
        float v[VEC];
        ck.load(q, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) n += keep(v[e]) ? 1u : 0u;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sm.wcnt[warp] = n;
    __syncthreads();
    uint32_t at = 0, tot = 0;
#pragma unroll
    for (int w = 0; w < SP_WARPS; ++w) {
        const uint32_t x = sm.wcnt[w];
        if (w < warp) at += x;
        tot += x;
    }
    if (tid < static_cast<int>(C)) st_cluster_s32(&sm.ccnt[rank], tid, static_cast<int>(tot));
    if (tot <= SP_CAP && n > 0) {
        for (int v0 = q0; v0 < q1; v0 += 32) {
            uint32_t mask = 0;
            float v[VEC];
            if (v0 + lane < q1) {
                ck.load(v0 + lane, v);
#pragma unroll
                for (int e = 0; e < VEC; ++e) mask |= (keep(v[e]) ? 1u : 0u) << e;
            }
            if (!__any_sync(0xffffffffu, mask)) continue;
            const uint32_t mine = __popc(mask);
            const uint32_t in = warp_scan(mine, lane);
            uint32_t w = at + in - mine;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (mask & (1u << e)) sm.l.loc[w++] = composite(v[e], ck.index(v0 + lane, e));
            at += __shfl_sync(0xffffffffu, in, 31);
        }
    }
    cluster_sync_all();
    uint32_t all = 0;
    for (uint32_t r = 0; r < C; ++r) all += sm.ccnt[r];
    return all;
}

// A lower bound of the k-th largest logit: the k-th largest of the threads'
// maxima (each of k threads holds an element at least that large), to within
// an interval.  -inf where fewer than k threads hold an element above lo.
__device__ float kth_bound(SampleSmem& sm, const SpScale& sc, uint32_t C, float lo, float mine, uint32_t k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const SpBins bins = first_bins(sc, lo);
    if (mine >= lo) atomicAdd(&sm.cnt[bins.of(mine)], 1u);   // cleared before the first cluster barrier
    cluster_sync_all();
    uint32_t n[2] = {0, 0};
#pragma unroll 8
    for (uint32_t r = 0; r < C; ++r) {
        uint32_t x, y;
        asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(sp_mapa(&sm.cnt[2 * tid], r)) : "memory");
        n[0] += x;
        n[1] += y;
    }
    if (tid == 0) sm.last = SP_BINS;
    const uint32_t own = n[0] + n[1];
    const uint32_t inc = warp_scan(own, lane);
    if (lane == 31) sm.wcnt[warp] = inc;
    __syncthreads();
    uint32_t ex = inc - own;
    for (int w = 0; w < warp; ++w) ex += sm.wcnt[w];
    if (ex < k && ex + own >= k) sm.last = ex + n[0] >= k ? 2 * tid : 2 * tid + 1;
    __syncthreads();
    const int b = sm.last;
    __syncthreads();   // wcnt and last are free again
    if (b >= SP_BINS - 1 || !(bins.s > 0.f)) return lo;
    return fmaxf(lo, sc.m - static_cast<float>(b + 1) / bins.s * (1.f + 1e-6f) - fabsf(sc.m) * 3e-7f);
}

// ---------------------------------------------------------------- the draw from a list (leader)
// Sums over per-thread runs: start of this thread's run and the total.  A
// thread's end is the next one's start exactly.
__device__ __forceinline__ void block_runs(SampleSmem& sm, double own, int nwarps, double& start, double& end,
                                           double& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const double inc = warp_scan(own, lane);
    double prev = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) prev = 0.0;
    __syncthreads();
    if (lane == 31) sm.dscan[warp] = inc;
    __syncthreads();
    double base = 0.0, sum = 0.0;
    for (int w = 0; w < nwarps; ++w) {
        if (w == warp) base = sum;
        sum += sm.dscan[w];
    }
    start = base + prev;
    end = base + inc;
    total = sum;
}

// Descending order of n composite keys from lst into srt.
__device__ void sort_list(SampleSmem& sm, const unsigned long long* lst, unsigned long long* srt, int n) {
    const int tid = threadIdx.x;
    if (n <= 128) {   // each key's rank by counting, four threads a key
        uint32_t* rk = sm.cnt;
        for (int i = tid; i < 128; i += SP_THREADS) rk[i] = 0;
        __syncthreads();
        const int i = tid & 127, part = tid >> 7;
        if (i < n) {
            const unsigned long long k = lst[i];
            const int per = (n + 3) / 4;
            uint32_t r = 0;
#pragma unroll 4
            for (int j = part * per; j < min(n, part * per + per); ++j) r += lst[j] > k;
            atomicAdd(&rk[i], r);
        }
        __syncthreads();
        if (tid < n) srt[rk[tid]] = lst[tid];
        __syncthreads();
        return;
    }
    int p2 = 256;
    while (p2 < n) p2 *= 2;
    for (int i = tid; i < p2; i += SP_THREADS) srt[i] = i < n ? lst[i] : 0ull;
    __syncthreads();
    for (int size = 2; size <= p2; size *= 2)
        for (int step = size / 2; step > 0; step /= 2) {
            for (int i = tid; i < p2 / 2; i += SP_THREADS) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const unsigned long long x = srt[a], y = srt[b];
                const bool desc = (a & size) == 0;
                if ((x < y) == desc) {
                    srt[a] = y;
                    srt[b] = x;
                }
            }
            __syncthreads();
        }
}

constexpr int SP_PER = SP_CAP / SP_THREADS;

// Index of the entry of the list where the running sum of w (this thread's
// run starts at `start`) passes the target, in the one thread it falls to; -1
// elsewhere.
__device__ __forceinline__ int run_hit(const double (&w)[SP_PER], double start, double end, double target) {
    if (!(start <= target && target < end)) return -1;
    int at = -1;
    double acc = start;
#pragma unroll
    for (int e = 0; e < SP_PER; ++e) {
        if (w[e] > 0.0 && (at < 0 || acc <= target)) at = e;   // the first that passes, else the last with weight
        acc += w[e];
    }
    return at;
}

struct SpRow {
    bool by_k, by_p;
    int k;
    double p;
    int x;              // the draft, or -1
    bool has_draft;
    const float* q;     // its distribution, or NULL
    double ua, us;
};

// The leader's end of a row whose kept tokens all lie in the list lst[0..n):
// filters, acceptance of the draft, the draw.  S_all: the row's sum before
// top-p, or negative where the list is the whole row.
template <bool VERIFY>
__device__ void draw_from_list(SampleSmem& sm, int n, const SpScale& sc, const SpRow& r, double S_all, int32_t* token) {
    const int tid = threadIdx.x;
    const unsigned long long* lst = sm.l.lst;
    unsigned long long* srt = sm.l.loc;
    const int per = (n + SP_THREADS - 1) / SP_THREADS;
    const int nwarps = min(SP_WARPS, (n + 32 * per - 1) / (32 * per));
    int nk = r.by_k ? min(r.k, n) : n;
    unsigned long long cut = 0;
    if (nk < n || r.by_p) {
        sort_list(sm, lst, srt, n);
        if (r.by_p) {
            if (tid == 0) sm.keep = nk;
            double w[SP_PER], own = 0.0, start, end, total;
#pragma unroll
            for (int e = 0; e < SP_PER; ++e) {
                const int j = tid * per + e;
                w[e] = e < per && j < nk ? sc.weight(composite_value(srt[j])) : 0.0;
                own += w[e];
            }
            block_runs(sm, own, nwarps, start, end, total);
            const double target = fmax(r.p * (r.by_k || S_all < 0.0 ? total : S_all), 1e-9);
            // the prefix ends with the first token at which the running sum reaches the target
            if (start < target && end >= target) {
                double acc = start;
                int at = -1;
#pragma unroll
                for (int e = 0; e < SP_PER; ++e) {
                    if (w[e] > 0.0 && (at < 0 || acc < target)) at = e;
                    acc += w[e];
                }
                sm.keep = tid * per + at + 1;
            }
            __syncthreads();
            nk = sm.keep;
        }
        cut = srt[nk - 1];
    }
    if (tid == 0) sm.wx = 0.0;
    __syncthreads();
    double w[SP_PER], own = 0.0, start, end, total;
#pragma unroll
    for (int e = 0; e < SP_PER; ++e) {
        const int j = tid * per + e;
        w[e] = 0.0;
        if (e < per && j < n && lst[j] >= cut) {
            w[e] = sc.weight(composite_value(lst[j]));
            if (VERIFY && r.has_draft && composite_index(lst[j]) == r.x) {
                sm.wx = w[e];
                if (!r.q) w[e] = 0.0;   // a certain draft leaves the others
            }
        }
        own += w[e];
    }
    block_runs(sm, own, nwarps, start, end, total);
    double S = total;
    if (VERIFY && r.has_draft) {
        const double wx = sm.wx;
        if (!r.q) S = total + wx;
        const double qx = r.q ? (r.x >= 0 ? static_cast<double>(__ldg(r.q + r.x)) : 0.0) : 1.0;
        if (wx > 0.0 && r.ua * qx * S < wx) {
            if (tid == 0) *token = SP_ACCEPTED;
            return;
        }
        if (r.q) {
            double rw[SP_PER], rown = 0.0, rs, re, rt;
#pragma unroll
            for (int e = 0; e < SP_PER; ++e) {
                rw[e] = 0.0;
                if (w[e] > 0.0)
                    rw[e] = fmax(0.0, w[e] - static_cast<double>(__ldg(r.q + composite_index(lst[tid * per + e]))) * S);
                rown += rw[e];
            }
            block_runs(sm, rown, nwarps, rs, re, rt);
            if (rt > 0.0) {
#pragma unroll
                for (int e = 0; e < SP_PER; ++e) w[e] = rw[e];
                start = rs;
                end = re;
                total = rt;
            }
        }
    }
    if (tid == 0) {
        sm.list_cut = cut;
        sm.list_sum = S;
    }
    if (!(total > 0.0)) {   // the draft is the only token kept
        if (tid == 0) *token = r.x;
        return;
    }
    const int e = run_hit(w, start, end, r.us * total);
    if (e >= 0) *token = composite_index(lst[tid * per + e]);
}

// ---------------------------------------------------------------- the draw from the whole row
// A warp's kept weights in index order; with q, the residual max(w - q S, 0).
template <typename TL>
__device__ __forceinline__ double kept_weight(float l, int idx, const SpCut& cut, const SpScale& sc, int skip,
                                              const float* q, double S) {
    double w = 0.0;
    if (cut.keeps(l, idx) && idx != skip) {
        w = sc.weight(l);
        if (q) w = fmax(0.0, w - static_cast<double>(__ldg(q + idx)) * S);
    }
    return w;
}

// Sum of every warp's kept weights into sums[cta][warp] of every CTA (one
// cluster barrier).
template <typename TL>
__device__ void segment_sums(double* sums, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, const SpCut& cut,
                             const SpScale& sc, int skip, const float* q, double S) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    double s = 0.0;
    for (int v0 = q0 + lane; v0 < q1; v0 += 32) {
        float v[VEC];
        ck.load(v0, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += kept_weight<TL>(v[e], ck.index(v0, e), cut, sc, skip, q, S);
    }
    s = warp_sum_f64(s);
    if (lane < static_cast<int>(C)) st_cluster_f64(&sums[rank * SP_WARPS + warp], lane, s);
    cluster_sync_all();
}

// Sum of the table, the same in every thread of the cluster.
__device__ double table_sum(const double* sums, uint32_t C, int lane) {
    double s = 0.0;
    for (int i = lane; i < static_cast<int>(C) * SP_WARPS; i += 32) s += sums[i];
    return warp_sum_f64(s);
}

// The first index whose cumulative weight exceeds u times the total.  Returns
// the token in the warp that owns it, -1 elsewhere.
template <typename TL>
__device__ int draw_token(const double* sums, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, const SpCut& cut,
                          const SpScale& sc, int skip, const float* q, double S, double u) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nseg = static_cast<int>(C) * SP_WARPS;
    const int per = (nseg + 31) / 32;
    // every warp finds the owning segment: lane l scans segments [l per, l per + per)
    double own = 0.0;
    for (int j = 0; j < per; ++j)
        if (lane * per + j < nseg) own += sums[lane * per + j];
    const double inc = warp_scan(own, lane);
    const double total = __shfl_sync(0xffffffffu, inc, 31);
    const double target = u * total;
    double base = inc - own;
    int seg = -1, lastseg = -1;
    double seg_base = 0.0, last_base = 0.0;
    for (int j = 0; j < per; ++j) {
        const int s = lane * per + j;
        if (s >= nseg) break;
        if (sums[s] > 0.0) {
            lastseg = s;
            last_base = base;
            if (seg < 0 && base + sums[s] > target) {
                seg = s;
                seg_base = base;
            }
        }
        base += sums[s];
    }
    const unsigned any = __ballot_sync(0xffffffffu, seg >= 0);
    const unsigned some = __ballot_sync(0xffffffffu, lastseg >= 0);
    const int src = any ? __ffs(any) - 1 : 31 - __clz(some);   // rounding left u S above the total: the last segment
    if (!any) {
        seg = lastseg;
        seg_base = last_base;
    }
    seg = __shfl_sync(0xffffffffu, seg, src);
    base = __shfl_sync(0xffffffffu, seg_base, src);
    if (seg != static_cast<int>(rank) * SP_WARPS + warp) return -1;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    int last = -1;
    for (int v0 = q0; v0 < q1; v0 += 32) {
        double w[VEC], s = 0.0;
        const int vq = v0 + lane;
        int mine = -1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = 0.0;
        if (vq < q1) {
            float v[VEC];
            ck.load(vq, v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                w[e] = kept_weight<TL>(v[e], ck.index(vq, e), cut, sc, skip, q, S);
                s += w[e];
                if (w[e] > 0.0) mine = ck.index(vq, e);
            }
        }
        const double in = warp_scan(s, lane);
        const unsigned pass = __ballot_sync(0xffffffffu, s > 0.0 && base + in > target);
        if (pass) {
            int tok = mine;
            double acc = base + in - s;
            bool found = false;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                acc += w[e];
                if (!found && w[e] > 0.0 && acc > target) {
                    tok = ck.index(vq, e);
                    found = true;
                }
            }
            return __shfl_sync(0xffffffffu, tok, __ffs(pass) - 1);
        }
        const unsigned have = __ballot_sync(0xffffffffu, mine >= 0);
        if (have) last = __shfl_sync(0xffffffffu, mine, 31 - __clz(have));
        base += __shfl_sync(0xffffffffu, in, 31);
    }
    return last;
}

// Index of the keep-th token with logit tau, in index order, of `ties` in the
// row (two cluster barriers).
template <typename TL>
__device__ int tie_index(SampleSmem& sm, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, float tau, uint32_t keep) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    uint32_t n = 0;
    for (int q = q0 + lane; q < q1; q += 32) {
        float v[VEC];
        ck.load(q, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) n += v[e] == tau ? 1u : 0u;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sm.wcnt[warp] = n;
    __syncthreads();
    uint32_t tot = 0, before = 0;
    for (int w = 0; w < SP_WARPS; ++w) {
        if (w < warp) before += sm.wcnt[w];
        tot += sm.wcnt[w];
    }
    if (tid < static_cast<int>(C)) st_cluster_s32(&sm.tie[rank], tid, static_cast<int>(tot));
    cluster_sync_all();
    for (uint32_t r = 0; r < rank; ++r) before += sm.tie[r];
    if (keep > before && keep <= before + n) {
        uint32_t left = keep - before;   // 1-based
        for (int v0 = q0; v0 < q1; v0 += 32) {
            uint32_t mask = 0;
            if (v0 + lane < q1) {
                float v[VEC];
                ck.load(v0 + lane, v);
#pragma unroll
                for (int e = 0; e < VEC; ++e) mask |= (v[e] == tau ? 1u : 0u) << e;
            }
            const uint32_t mine = __popc(mask);
            const uint32_t in = warp_scan(mine, lane);
            if (in >= left && in - mine < left) {
                uint32_t skip = left - (in - mine) - 1;
                while (skip--) mask &= mask - 1;
                for (uint32_t r = 0; r < C; ++r) st_cluster_s32(&sm.cut_idx, r, ck.index(v0 + lane, __ffs(mask) - 1));
            }
            const uint32_t t = __shfl_sync(0xffffffffu, in, 31);
            if (t >= left) break;
            left -= t;
        }
    }
    cluster_sync_all();
    return static_cast<int>(sm.cut_idx);
}

template <typename TL, bool VERIFY>
__global__ void __launch_bounds__(SP_THREADS, 2) sample_kernel(const SampleArgs a) {
    constexpr int VEC = SpElem<TL>::VEC;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ SampleSmem sm;
    const uint32_t rank = cluster_rank(), C = a.cluster;
    const int row = blockIdx.x / a.cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 16) sm.tab[tid] = exp2(static_cast<double>(tid) / 16.0);
    for (int i = tid; i < SP_BINS; i += SP_THREADS) sm.cnt[i] = 0;
    grid_dep_wait();
    grid_dep_launch();

    // ---- the row's part into shared memory, and its maximum
    SpChunk<TL> ck;
    ck.buf = reinterpret_cast<TL*>(dyn);
    ck.begin = static_cast<int>(rank) * a.chunk;
    ck.n = max(0, min(a.chunk, a.V - ck.begin));
    const TL* rowp = static_cast<const TL*>(a.logits) + static_cast<size_t>(row) * a.V;
    const TL* g = rowp + ck.begin;
    ck.mis = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(TL));
    ck.nvec = ck.n > 0 ? (ck.mis + ck.n + VEC - 1) / VEC : 0;
    float mine = -INFINITY;
    for (int q0 = tid; q0 < ck.nvec; q0 += 4 * SP_THREADS) {
        uint4 r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s0 = (q0 + j * SP_THREADS) * VEC;
            if (s0 >= ck.mis && s0 + VEC <= ck.mis + ck.n)
                r[j] = __ldg(reinterpret_cast<const uint4*>(g + (s0 - ck.mis)));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = q0 + j * SP_THREADS, s0 = q * VEC;
            if (q >= ck.nvec) break;
            if (!(s0 >= ck.mis && s0 + VEC <= ck.mis + ck.n)) {   // a ragged end of the part
                TL t[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    t[e] = s0 + e >= ck.mis && s0 + e < ck.mis + ck.n ? g[s0 + e - ck.mis] : SpElem<TL>::ninf();
                memcpy(&r[j], t, 16);
            }
            reinterpret_cast<uint4*>(ck.buf)[q] = r[j];
            float v[VEC];
            SpElem<TL>::unpack(r[j], v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) mine = fmaxf(mine, v[e]);   // a NaN operand is ignored
        }
    }
    float m = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sm.wmax[warp] = m;
    __syncthreads();
    if (warp == 0) {
        m = lane < SP_WARPS ? sm.wmax[lane] : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane < static_cast<int>(C)) st_cluster_f32(&sm.cmax[rank], lane, m);
    }

    // ---- the row's parameters
    const int seq = row / a.per, pj = row % a.per;
    double T = a.temperature ? static_cast<double>(__ldg(a.temperature + seq)) : 1.0;
    SpRow r;
    r.k = a.top_k ? __ldg(a.top_k + seq) : 0;
    r.p = a.top_p ? static_cast<double>(__ldg(a.top_p + seq)) : 2.0;
    double mp = a.min_p ? static_cast<double>(__ldg(a.min_p + seq)) : 0.0;
    if (!(T > 0.0)) {   // greedy
        T = 1.0;
        r.k = 1;
        r.p = 2.0;
        mp = 0.0;
    }
    r.by_k = r.k > 0 && r.k < a.V;
    r.by_p = r.p < 1.0;
    r.has_draft = VERIFY && pj < a.per - 1;
    r.x = -1;
    r.q = nullptr;
    r.ua = 0.0;
    if (r.has_draft) {
        r.x = __ldg(a.draft + static_cast<size_t>(seq) * (a.per - 1) + pj);
        if (r.x < 0 || r.x >= a.V) r.x = -1;
        if (a.q) r.q = a.q + (static_cast<size_t>(seq) * (a.per - 1) + pj) * a.V;
        r.ua = static_cast<double>(__ldg(a.u + static_cast<size_t>(seq) * a.per + pj));
    }
    r.us = static_cast<double>(__ldg(a.u + (VERIFY ? static_cast<size_t>(seq) * a.per + a.per - 1 : static_cast<size_t>(row))));
    r.us = fmin(r.us, 1.0 - 0x1p-24);

    cluster_sync_all();
    m = -INFINITY;
    for (uint32_t i = 0; i < C; ++i) m = fmaxf(m, sm.cmax[i]);
    const SpScale sc{m, bits_to_f64(__float_as_uint(m)), 1.4426950408889634 / T, sm.tab};
    double dmin = -44.361419555836498 * T;   // 64 ln 2
    if (mp > 0.0) dmin = fmax(dmin, T * log(fmin(mp, 1.0)));
    const float lcut = fmaxf(__double2float_ru(static_cast<double>(m) + dmin), -FLT_MAX);

    if (m == -INFINITY) {   // nothing can be drawn
        if (rank == 0 && tid == 0) a.token[row] = -1;
        if (!VERIFY && a.probs)
            for (int i = tid; i < ck.n; i += SP_THREADS) a.probs[static_cast<size_t>(row) * a.V + ck.begin + i] = 0.f;
        return;
    }

    // ---- few candidates: a list of them, finished by the leader
    uint32_t n = 0xffffffffu;
    double S_all = -1.0;
    float list_lo = lcut;
    SpBin at{};
    if (mp > 0.0) n = gather<TL>(sm, ck, rank, C, [&](float l) { return l >= lcut; });
    if (n > SP_CAP && r.by_k && r.k <= SP_CAP) {
        list_lo = kth_bound(sm, sc, C, lcut, mine, static_cast<uint32_t>(r.k));
        n = gather<TL>(sm, ck, rank, C, [&](float l) { return l >= list_lo; });
    }
    if (n > SP_CAP && r.by_p && !r.by_k) {
        at = select_first<TL, true>(sm, ck, sc, rank, C, lcut, -1.0, r.p);
        S_all = static_cast<double>(at.total) / static_cast<double>(1ull << SP_FIX);
        if (at.cabove + at.cnt <= SP_CAP) {
            const SpBins bins = first_bins(sc, lcut);
            n = gather<TL>(sm, ck, rank, C, [&](float l) { return l >= lcut && bins.of(l) <= at.b; });
        }
    }
    if (n <= SP_CAP) {
        if (rank == 0) {
            for (int i = tid; i < static_cast<int>(n); i += SP_THREADS) {
                uint32_t j = i, c = 0;
                while (j >= sm.ccnt[c]) j -= sm.ccnt[c++];
                unsigned long long k;
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(sp_mapa(&sm.l.loc[j], c)) : "memory");
                sm.l.lst[i] = k;
            }
        }
        cluster_sync_all();   // the other CTAs' lists have been read
        if (rank == 0)
            draw_from_list<VERIFY>(sm, static_cast<int>(n), sc, r, S_all, a.token + row);
        if (VERIFY || !a.probs) return;
        if (rank == 0) {
            __syncthreads();
            if (tid < static_cast<int>(C)) {
                st_cluster_u64(&sm.list_cut, tid, sm.list_cut);
                st_cluster_f64(&sm.list_sum, tid, sm.list_sum);
            }
        }
        cluster_sync_all();
    }

    // ---- many: the border of the kept set by selection over the whole row
    SpCut cut{lcut, INT_MAX};
    double S = 0.0;
    if (n <= SP_CAP) {
        S = sm.list_sum;
        cut.tau = list_lo;   // the whole list is kept where it has no cut
        if (sm.list_cut) {
            cut.tau = composite_value(sm.list_cut);
            cut.icut = composite_index(sm.list_cut);
        }
    } else {
        if (r.by_k || r.by_p) {
            unsigned long long keep = 0;   // how many of the tokens at the border are kept
            uint32_t key = 0;
            float lo = lcut;
            if (r.by_k) {
                at = select_first<TL, false>(sm, ck, sc, rank, C, lcut, static_cast<double>(r.k), 0.0);
                key = select_key<TL, false>(sm, ck, sc, rank, C, lcut, static_cast<double>(r.k), at);
                const unsigned long long want = static_cast<unsigned long long>(r.k) - min(at.above, static_cast<unsigned long long>(r.k));
                keep = min(want, static_cast<unsigned long long>(at.cnt));
                lo = key_logit<TL>(key);
            }
            if (r.by_p) {
                const float kth = lo;
                const unsigned long long kkeep = keep;
                double target;
                if (r.by_k) {
                    // the sum over the top-k tokens: everything above the border, and its kept ties
                    segment_sums<TL>(sm.wsum, ck, rank, C, SpCut{kth, -1}, sc, -1, nullptr, 0.0);
                    target = fmax(r.p * (table_sum(sm.wsum, C, lane) + static_cast<double>(keep) * sc.weight(kth)), 1e-9);
                    at = select_first<TL, true>(sm, ck, sc, rank, C, kth, target * static_cast<double>(1ull << SP_FIX), 0.0);
                } else {
                    target = fmax(r.p * S_all, 1e-9);
                }
                key = select_key<TL, true>(sm, ck, sc, rank, C, lo, target * static_cast<double>(1ull << SP_FIX), at);
                lo = key_logit<TL>(key);
                const double need =
                    ceil((target - static_cast<double>(at.above) / static_cast<double>(1ull << SP_FIX)) / sc.weight(lo));
                keep = need < 1.0 ? 1 : need >= static_cast<double>(at.cnt) ? at.cnt : static_cast<unsigned long long>(need);
                if (r.by_k && lo == kth) keep = min(keep, kkeep);
            }
            cut.tau = lo;
            if (keep < at.cnt) cut.icut = tie_index<TL>(sm, ck, rank, C, lo, static_cast<uint32_t>(keep));
        }
        // ---- sums, acceptance of the draft, the draw
        double wx = 0.0;
        if (r.x >= 0) wx = kept_weight<TL>(SpElem<TL>::load(rowp + r.x), r.x, cut, sc, -1, nullptr, 0.0);
        const int skip = r.has_draft && !r.q ? r.x : -1;   // a certain draft leaves the others
        segment_sums<TL>(sm.wsum, ck, rank, C, cut, sc, skip, nullptr, 0.0);
        const double rest = table_sum(sm.wsum, C, lane);
        S = skip >= 0 ? rest + wx : rest;
        if (r.has_draft) {
            const double qx = r.q ? (r.x >= 0 ? static_cast<double>(__ldg(r.q + r.x)) : 0.0) : 1.0;
            if (wx > 0.0 && r.ua * qx * S < wx) {
                if (rank == 0 && tid == 0) a.token[row] = SP_ACCEPTED;
                return;
            }
        }
        int tok = -1;
        if (r.q) {
            segment_sums<TL>(sm.rsum, ck, rank, C, cut, sc, -1, r.q, S);
            if (table_sum(sm.rsum, C, lane) > 0.0) tok = draw_token<TL>(sm.rsum, ck, rank, C, cut, sc, -1, r.q, S, r.us);
            else tok = draw_token<TL>(sm.wsum, ck, rank, C, cut, sc, -1, nullptr, 0.0, r.us);
        } else if (rest > 0.0) {
            tok = draw_token<TL>(sm.wsum, ck, rank, C, cut, sc, skip, nullptr, 0.0, r.us);
        } else if (rank == 0 && warp == 0) {
            tok = r.x;   // the draft is the only token kept
        }
        if (tok >= 0 && lane == 0) a.token[row] = tok;
    }
    if (!VERIFY && a.probs) {
        float* out = a.probs + static_cast<size_t>(row) * a.V + ck.begin;
        const double inv = 1.0 / S;
        for (int i = tid; i < ck.n; i += SP_THREADS) {
            const float l = static_cast<float>(ck.buf[ck.mis + i]);
            out[i] = static_cast<float>(kept_weight<TL>(l, ck.begin + i, cut, sc, -1, nullptr, 0.0) * inv);
        }
    }
}

// The verification's last step, one thread per sequence: the rows' results in
// committed become the accepted drafts up to the first rejection, the token
// drawn there, and padding.
__global__ void __launch_bounds__(128) sample_commit_kernel(const int32_t* __restrict__ draft, int B, int K,
                                                            int32_t* __restrict__ committed,
                                                            int32_t* __restrict__ n_committed) {
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= B) return;
    int32_t* row = committed + static_cast<size_t>(b) * (K + 1);
    int n = 0;
    while (n < K && row[n] == SP_ACCEPTED) {
        row[n] = draft[static_cast<size_t>(b) * K + n];
        ++n;
    }
    for (int j = n + 1; j <= K; ++j) row[j] = -1;
    n_committed[b] = n + (row[n] >= 0 ? 1 : 0);
}

// ---------------------------------------------------------------- host side
template <typename TL, bool VERIFY>
static ms_status sample_launch_t(const SampleArgs& a, cudaStream_t s) {
    static PerDevice set;
    set.get([] {
        cudaFuncSetAttribute(sample_kernel<TL, VERIFY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SP_MAX_CHUNK * static_cast<int>(sizeof(TL)) + 32);
        return 1;
    });
    const size_t smem = static_cast<size_t>(a.chunk) * sizeof(TL) + 32;
    return launch_cluster(VERIFY ? K_SAMPLE_VERIFY : K_SAMPLE, sample_kernel<TL, VERIFY>,
                          dim3(static_cast<unsigned>(a.rows) * a.cluster), dim3(SP_THREADS), smem, s, a.cluster, a);
}

static ms_status sample_launch(SampleArgs a, ms_dtype dt, bool verify, cudaStream_t s) {
    int C = 1;
    while (C < SP_MAXC && a.V > 1024 * C) C *= 2;
    a.cluster = C;
    a.chunk = ((a.V + C - 1) / C + 7) / 8 * 8;
    if (dt == MS_BF16)
        return verify ? sample_launch_t<__nv_bfloat16, true>(a, s) : sample_launch_t<__nv_bfloat16, false>(a, s);
    return verify ? sample_launch_t<float, true>(a, s) : sample_launch_t<float, false>(a, s);
}

// Rows and vocabulary that one launch can take.
static bool sample_size_ok(long rows, int V) { return V <= SP_MAX_V && rows <= (1L << 24); }

}  // namespace ms

extern "C" ms_status spec_sample(const void* logits, ms_dtype logits_dtype, int T, int V, const float* temperature,
                                 const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                                 int32_t* token, float* probs, void* stream) {
    if (!logits || !u || !token) return MS_ERR_INVALID_ARG;
    if (T <= 0 || V <= 0) return MS_ERR_INVALID_ARG;
    if (logits_dtype != MS_F32 && logits_dtype != MS_BF16) return MS_ERR_INVALID_ARG;
    if (!ms::element_aligned(logits, logits_dtype)) return MS_ERR_INVALID_ARG;
    if (!ms::sample_size_ok(T, V)) return MS_ERR_UNSUPPORTED;
    ms::SampleArgs a{};
    a.logits = logits;
    a.V = V;
    a.rows = T;
    a.per = 1;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.token = token;
    a.probs = probs;
    return ms::sample_launch(a, logits_dtype, false, static_cast<cudaStream_t>(stream));
}

extern "C" ms_status spec_verify_sample(const void* logits, ms_dtype logits_dtype, const int32_t* draft,
                                        const float* draft_probs, const float* temperature, const int32_t* top_k,
                                        const float* top_p, const float* min_p, const float* u, int B, int K, int V,
                                        int32_t* committed, int32_t* n_committed, void* stream) {
    if (!logits || (K > 0 && !draft) || !u || !committed || !n_committed) return MS_ERR_INVALID_ARG;
    if (B <= 0 || V <= 0 || K < 0) return MS_ERR_INVALID_ARG;
    if (logits_dtype != MS_F32 && logits_dtype != MS_BF16) return MS_ERR_INVALID_ARG;
    if (!ms::element_aligned(logits, logits_dtype)) return MS_ERR_INVALID_ARG;
    if (K > 8 || !ms::sample_size_ok(static_cast<long>(B) * (K + 1), V)) return MS_ERR_UNSUPPORTED;
    ms::SampleArgs a{};
    a.logits = logits;
    a.V = V;
    a.rows = B * (K + 1);
    a.per = K + 1;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.draft = draft;
    a.q = K > 0 ? draft_probs : nullptr;
    a.token = committed;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const ms_status st = ms::sample_launch(a, logits_dtype, true, s);
    if (st != MS_OK) return st;
    return ms::launch(ms::K_SAMPLE_COMMIT, ms::sample_commit_kernel, dim3((B + 127) / 128), dim3(128), 0, s,
                      draft, B, K, committed, n_committed);
}
