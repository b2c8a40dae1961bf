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
// would move one draw in a hundred.  Weights are therefore computed in fp64 to
// about 2e-13 and summed in a fixed order; histograms hold counts, whose order
// cannot matter, and sums of a count times a weight.
//
// One thread-block cluster per row: each CTA copies its part of the row into
// shared memory once, and every later pass (maximum, selection, sums, the
// draw) reads it from there; partial results cross the cluster through
// distributed shared memory.  A row takes one of three ways:
//  - few tokens kept (top-k of up to SP_CAP, a top-p or min-p set as small):
//    they are listed, in index order, and one CTA sorts, cuts and draws;
//  - a bf16 row that keeps more: every value of the row is counted (a bf16 row
//    has few), which gives its borders exactly by one scan;
//  - other rows that keep more: counts over 1024 intervals of the logit bracket
//    the border, the tokens of the bracket are listed and refined by their bits.
// A row without filters needs the sums alone.
//
// What bounds it: one row's time is the chain of cluster barriers (0.25 us each
// at 1.9 GHz) and block scans; many rows are bound by instructions, 21 per
// element and fp64 pass, 11 of them fp64 at two issue cycles.  Memory is not the
// bound: the row is read once.  Measured at V = 129,280 (replayed in a graph):
//   1 bf16 row, all filters                       7.7 us
//   32 fp32 rows, top-p (3 of them wide)           52 us
//   64 bf16 rows, temperature, probs written       39 us  (1.3 TB/s)
//   512 bf16 rows, filters of every kind          129 us  (1.0 TB/s)
//   verification of 32 x 4 bf16 rows, top-p        88 us
//   the same by temperature with draft probs       62 us  (0.8 TB/s)
#include <float.h>
#include <limits.h>
#include <math.h>

#include "ms_common.cuh"

namespace ms {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_MAXC = 8;              // CTAs of a row's cluster
constexpr int SP_MAX_CHUNK = 32768;     // elements of a row per CTA
constexpr int SP_BINS = 1024;
constexpr int32_t SP_ACCEPTED = -2;
constexpr int SP_MAX_V = SP_MAXC * SP_MAX_CHUNK;
constexpr int SP_CAP = 2048;            // candidates that a CTA lists, and that the leader finishes a row from
constexpr int SP_BPT = SP_BINS / SP_THREADS;   // bins per thread of a bin scan

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
// A float times 2^-896 as a double: its bits shifted into place, without the
// exponent's bias.  Infinities become +-2^-768 (masked tokens are sorted out by
// comparisons on the float itself).
__device__ __forceinline__ double scaled_f64(float l) {
    const int u = __float_as_int(l);
    return __hiloint2double((u >> 3) & static_cast<int>(0x8fffffffu), u << 29);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The cluster barrier where only warp 0 has stored to other CTAs since the last
// one (the others' stores to their own CTA's shared memory are ordered by the
// block barrier): one warp's fence instead of every warp's.
__device__ __forceinline__ void cluster_sync_warp0() {
    __syncthreads();
    if (threadIdx.x < 32) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    cluster_wait();
}

// Floats in ascending order as unsigned integers (-0 equal to +0).
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// A row's weights w(l) = 2^((l - max) c), c = log2(e) / T, for -65 < (l - max) c
// <= 0, to about 2e-13 relative and exactly 1 at the maximum: t = k/16 + r,
// 2^(k/16) from a table of 16 doubles (one per pair of shared-memory banks: no
// conflicts whatever the lanes ask for) times the Taylor polynomial of degree 5
// of 2^r, |r| <= 1/32.  11 fp64 instructions with the sum, 20 in all.
// The coefficients come from constant memory as operands of the fp64
// instructions; as literals each took two moves per use.
__constant__ double kPow2[6] = {1.5 * 281474976710656.0, 6.9314718055994531e-1, 2.4022650695910071e-1,
                                5.5504108664821580e-2,   9.6181291076284772e-3, 1.3333558146428443e-3};
struct SpScale {
    float m;          // max l
    double md, cs;    // max l times 2^-896, c times 2^896
    double c;
    const double* tab;
    __device__ __forceinline__ double weight(float l) const { return weight(scaled_f64(l), tab); }
    // the same from a scaled logit; a table times x gives weights times x
    __device__ __forceinline__ double weight(double l, const double* tab) const {
        const double kMagic = kPow2[0];   // 1.5 * 2^48: adding it rounds t to multiples of 1/16
        const double d = l - md;
        const double z = fma(d, cs, kMagic);
        const int k = __double2loint(z);
        const double r = fma(d, cs, kMagic - z);
        double p = fma(r, kPow2[5], kPow2[4]);   // ln2^5/5!, ln2^4/4!
        p = fma(p, r, kPow2[3]);                 // ln2^3/3!
        p = fma(p, r, kPow2[2]);                 // ln2^2/2!
        p = fma(p, r, kPow2[1]);                 // ln2
        // the table's high words lack j << 16, which k << 16 brings besides the exponent
        const double b = tab[k & 15];
        const double base = __hiloint2double(__double2hiint(b) + (k << 16), __double2loint(b));
        return fma(base * r, p, base);
    }
};

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

// Sum of the lower lanes' v <= 15, and of all lanes': a ballot per bit, which do
// not wait for one another as the steps of a scan do.
__device__ __forceinline__ uint32_t lanes_before(uint32_t v, int lane, uint32_t& all) {
    uint32_t before = 0;
    all = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t bits = __ballot_sync(0xffffffffu, (v >> i) & 1u);
        before += __popc(bits & ((1u << lane) - 1u)) << i;
        all += __popc(bits) << i;
    }
    return before;
}

// The elements of a 16-byte vector.
template <typename TL>
struct SpElem;
template <>
struct SpElem<float> {
    static constexpr int VEC = 4;
    static constexpr int KSH = 0;
    static constexpr double OCTAVES = 20.0;
    using Bound = float;   // a threshold as the comparisons below want it
    static __device__ __forceinline__ Bound bound(float t) { return t; }
    static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ double scaled(const uint4& r, int e) {
        return scaled_f64(__uint_as_float(e == 0 ? r.x : e == 1 ? r.y : e == 2 ? r.z : r.w));
    }
    // NaN elements are ignored in any_ge and fail all_ge
    static __device__ __forceinline__ bool any_ge(const uint4& r, Bound t) {
        return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                     fmaxf(__uint_as_float(r.z), __uint_as_float(r.w))) >= t;
    }
    static __device__ __forceinline__ bool all_ge(const uint4& r, Bound t) {
        return __uint_as_float(r.x) >= t && __uint_as_float(r.y) >= t && __uint_as_float(r.z) >= t &&
               __uint_as_float(r.w) >= t;
    }
    static __device__ __forceinline__ bool any_eq(const uint4& r, float t) {
        return __uint_as_float(r.x) == t || __uint_as_float(r.y) == t || __uint_as_float(r.z) == t ||
               __uint_as_float(r.w) == t;
    }
    struct Max {
        float m = -INFINITY;
        __device__ __forceinline__ void add(const uint4& r) {
            m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(r.x), __uint_as_float(r.y))),
                      fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
        }
        __device__ __forceinline__ float get() const { return m; }
    };
    static __device__ __forceinline__ float ninf() { return -INFINITY; }
};
template <>
struct SpElem<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static constexpr int KSH = 16;   // the low half of a widened bf16 carries nothing
    static constexpr double OCTAVES = 16.0;
    using Bound = __nv_bfloat162;
    // l >= t for bf16 l holds exactly where l >= t rounded up to bf16
    static __device__ __forceinline__ Bound bound(float t) {
        const __nv_bfloat16 b = __float2bfloat16_ru(t);
        return __halves2bfloat162(b, b);
    }
    static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t q) {
        __nv_bfloat162 x;
        memcpy(&x, &q, 4);
        return x;
    }
    static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
        const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ double scaled(const uint4& r, int e) {
        const uint32_t q = e < 2 ? r.x : e < 4 ? r.y : e < 6 ? r.z : r.w;
        const int u = static_cast<int>(e & 1 ? q : q << 16);
        return __hiloint2double((u >> 3) & static_cast<int>(0x8fffe000u), 0);
    }
    static __device__ __forceinline__ bool any_ge(const uint4& r, Bound t) {
        const __nv_bfloat162 m = __hmax2(__hmax2(pair(r.x), pair(r.y)), __hmax2(pair(r.z), pair(r.w)));
        return __hge(__low2bfloat16(m), __low2bfloat16(t)) || __hge(__high2bfloat16(m), __low2bfloat16(t));
    }
    static __device__ __forceinline__ bool all_ge(const uint4& r, Bound t) {
        return __hbge2(__hmin2_nan(__hmin2_nan(pair(r.x), pair(r.y)), __hmin2_nan(pair(r.z), pair(r.w))), t);
    }
    static __device__ __forceinline__ bool any_eq(const uint4& r, float t) {
        const __nv_bfloat162 x = __float2bfloat162_rn(t);
        return (__heq2_mask(pair(r.x), x) | __heq2_mask(pair(r.y), x) | __heq2_mask(pair(r.z), x) |
                __heq2_mask(pair(r.w), x)) != 0;
    }
    struct Max {
        __nv_bfloat162 m = __halves2bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
        __device__ __forceinline__ void add(const uint4& r) {
            m = __hmax2(m, __hmax2(__hmax2(pair(r.x), pair(r.y)), __hmax2(pair(r.z), pair(r.w))));
        }
        __device__ __forceinline__ float get() const {
            return fmaxf(__bfloat162float(__low2bfloat16(m)), __bfloat162float(__high2bfloat16(m)));
        }
    };
    static __device__ __forceinline__ __nv_bfloat16 ninf() { return __ushort_as_bfloat16(0xff80); }
};

struct SampleSmem {
    double tab[16], ptab[16];                 // 2^(j/16), and the same over the row's sum
    double wsum[SP_MAXC * SP_WARPS];          // every warp's sum, of every CTA of the cluster
    double rsum[SP_MAXC * SP_WARPS];          // the same for the residual
    double dscan[2][SP_WARPS];
    float fscan[2][SP_WARPS];
    unsigned long long scan[SP_WARPS];
    unsigned long long sel_key;
    double sel_before, sel_w;                 // a selection round's border: the sum before it, its weight
    unsigned long long list_cut;              // broadcast results of a list: composite key of the last token kept,
    double list_sum;                          // and the sum of the kept weights
    double wx;
    unsigned long long lst[SP_CAP];           // leader: the row's candidates in index order
    unsigned long long loc[SP_CAP];           // this CTA's candidates; leader, later: scratch for sorting
    uint32_t cnt[SP_BINS];                    // counts by interval
    float cmax[SP_MAXC], cmin[SP_MAXC];       // every CTA's maximum, and the least of its threads' maxima
    uint32_t ccnt[4][SP_MAXC];                // every CTA's count, of each of up to four gathers
    uint32_t tie[SP_MAXC];
    unsigned long long few[32];               // a window's last tokens, this CTA's
    uint32_t nfew;
    float wmax[SP_WARPS], wmin[SP_WARPS];
    uint16_t order[SP_CAP];                   // leader: list entries by bucket
    uint32_t wcnt[SP_WARPS];
    uint32_t sel_cnt;
    uint32_t nb0, nb1, nn;                    // the border's intervals and their tokens
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
    // a vector, of -inf at and behind `end`
    __device__ __forceinline__ uint4 raw_to(int vec, int end) const {
        constexpr uint32_t kNone = sizeof(TL) == 2 ? 0xff80ff80u : 0xff800000u;
        return vec < end ? reinterpret_cast<const uint4*>(buf)[vec] : make_uint4(kNone, kNone, kNone, kNone);
    }
    __device__ __forceinline__ void load_to(int vec, int end, float (&v)[SpElem<TL>::VEC]) const {
        SpElem<TL>::unpack(raw_to(vec, end), v);
    }
    // leaves element idx of the row out of every later pass
    __device__ __forceinline__ void mask(int idx) const {
        const int i = idx - begin;
        if (i >= 0 && i < n) buf[mis + i] = SpElem<TL>::ninf();
    }
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

// This CTA's warp sums into row `rank` of the table of every CTA (one cluster
// barrier).
__device__ void share_sums(double* sums, double s, uint32_t rank, uint32_t C) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    s = warp_sum_f64(s);
    double* own = sums + rank * SP_WARPS;
    if (lane == 0) own[warp] = s;
    __syncthreads();
    if (warp == 0)
        for (int i = lane; i < static_cast<int>(C) * SP_WARPS; i += 32)
            if (static_cast<uint32_t>(i) / SP_WARPS != rank) st_cluster_f64(own + i % SP_WARPS, i / SP_WARPS, own[i % SP_WARPS]);
    cluster_sync_warp0();
}

// The same for two tables at once.
__device__ void share_two(double* ta, double a, double* tb, double b, uint32_t rank, uint32_t C) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = warp_sum_f64(a);
    b = warp_sum_f64(b);
    ta += rank * SP_WARPS;
    tb += rank * SP_WARPS;
    if (lane == 0) {
        ta[warp] = a;
        tb[warp] = b;
    }
    __syncthreads();
    if (warp == 0)
        for (int i = lane; i < static_cast<int>(C) * SP_WARPS; i += 32)
            if (static_cast<uint32_t>(i) / SP_WARPS != rank) {
                st_cluster_f64(ta + i % SP_WARPS, i / SP_WARPS, ta[i % SP_WARPS]);
                st_cluster_f64(tb + i % SP_WARPS, i / SP_WARPS, tb[i % SP_WARPS]);
            }
    cluster_sync_warp0();
}

// Sum of the table, the same in every thread of the cluster.
__device__ double table_sum(const double* sums, uint32_t C, int lane) {
    double s = 0.0;
    for (int i = lane; i < static_cast<int>(C) * SP_WARPS; i += 32) s += sums[i];
    return warp_sum_f64(s);
}

// ---------------------------------------------------------------- selection
// Logit intervals of equal width below the maximum; the last one takes the rest.
struct SpBins {
    float m, s;
    // a bound above every logit of intervals b and later
    __device__ __forceinline__ float upper(uint32_t b) const {
        if (b == 0 || !(s > 0.f)) return m;
        return fminf(m, m - (static_cast<float>(b) - 0.5f) / s * (1.f - 1e-6f) + fabsf(m) * 3e-7f);
    }
    // a bound below every logit of intervals 0..b that is at least lo, by more than the rounding of of()
    __device__ __forceinline__ float lower(uint32_t b, float lo) const {
        if (b >= SP_BINS - 1 || !(s > 0.f)) return lo;
        return fmaxf(lo, m - (static_cast<float>(b) + 0.5f) / s * (1.f + 1e-6f) - fabsf(m) * 3e-7f);
    }
    __device__ __forceinline__ uint32_t raw(float l) const {
        return __float_as_uint(fmaf(m - l, s, 8388608.f)) - 0x4b000000u;
    }
    __device__ __forceinline__ uint32_t of(float l) const {
        // adding 2^23 leaves the rounded product in the low bits; infinities and NaN (inf - inf) end in the last one
        return min(raw(l), static_cast<uint32_t>(SP_BINS - 1));
    }
};

// First round: intervals of the logit itself over the OCTAVES binary orders of
// magnitude below the largest weight, or down to `lo` where that is nearer.
template <typename TL>
__device__ __forceinline__ SpBins first_bins(const SpScale& sc, float lo) {
    const float width = fminf(sc.m - lo, static_cast<float>(SpElem<TL>::OCTAVES / sc.c));
    return SpBins{sc.m, width > 0.f && width < 1e30f ? static_cast<float>(SP_BINS - 1) / width : 0.f};
}

// Sum of the weights of a vector's elements at or above tau, into two running
// sums.  A warp that keeps all of its elements sums them without a test, others
// skip pairs of elements that none of their lanes keeps.
template <typename TL>
__device__ __forceinline__ void add_weights(const uint4& r, float tau, typename SpElem<TL>::Bound tb, const SpScale& sc,
                                            double& s0, double& s1) {
    constexpr int VEC = SpElem<TL>::VEC;
    if (__all_sync(0xffffffffu, SpElem<TL>::all_ge(r, tb))) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            s0 += sc.weight(SpElem<TL>::scaled(r, e), sc.tab);
            s1 += sc.weight(SpElem<TL>::scaled(r, e + 1), sc.tab);
        }
    } else if (__any_sync(0xffffffffu, SpElem<TL>::any_ge(r, tb))) {
        float v[VEC];
        SpElem<TL>::unpack(r, v);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const bool in0 = v[e] >= tau, in1 = v[e + 1] >= tau;
            if (!__any_sync(0xffffffffu, in0 || in1)) continue;
            const double w0 = sc.weight(v[e]), w1 = sc.weight(v[e + 1]);
            if (in0) s0 += w0;
            if (in1) s1 += w1;
        }
    }
}

// This thread's bins of the cluster's count table, summed over the CTAs.
__device__ __forceinline__ void pull_counts(SampleSmem& sm, uint32_t C, uint32_t (&n)[SP_BPT]) {
#pragma unroll
    for (int j = 0; j < SP_BPT; ++j) n[j] = 0;
#pragma unroll 8
    for (uint32_t r = 0; r < C; ++r)
#pragma unroll
        for (int j = 0; j < SP_BPT; j += 2) {
            uint32_t x, y;
            asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                         : "=r"(x), "=r"(y)
                         : "r"(sp_mapa(&sm.cnt[SP_BPT * threadIdx.x + j], r))
                         : "memory");
            n[j] += x;
            n[j + 1] += y;
        }
}

// Counts a vector's elements at or above lo by interval, but for the last one:
// that takes the bulk of a peaked row, where a border seldom lies.
template <typename TL>
__device__ __forceinline__ void count_vector(SampleSmem& sm, const uint4& raw, float lo, const SpBins& bins) {
    float v[SpElem<TL>::VEC];
    SpElem<TL>::unpack(raw, v);
#pragma unroll
    for (int e = 0; e < SpElem<TL>::VEC; ++e) {
        const uint32_t b = bins.raw(v[e]);
        if (v[e] >= lo && b < SP_BINS - 1) atomicAdd(&sm.cnt[b], 1u);
    }
}

// Top-p over the elements at or above lo, first step: their sum S (less
// `minus`), exactly, and from a histogram of counts the intervals b0..b1 that
// hold the border of the shortest prefix reaching p S.  An interval's tokens
// weigh between its ends' weights (2^(1/43) apart), so counts bound the running
// sums from both sides.  Clears nothing: sm.cnt is zero in every CTA when called.
struct SpNucleus {
    double S;
    uint32_t b0, b1, n;   // n: tokens down to b1, at most
};
template <typename TL>
__device__ SpNucleus nucleus(SampleSmem& sm, const SpChunk<TL>& ck, const SpScale& sc, uint32_t rank, uint32_t C,
                             int V, float lo, double p, double minus) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const SpBins bins = first_bins<TL>(sc, lo);
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    double s0 = 0.0, s1 = 0.0;
    const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(lo);
    for (int v0 = q0; v0 < q1; v0 += 32) {
        const uint4 raw = ck.raw_to(v0 + lane, q1);
        count_vector<TL>(sm, raw, lo, bins);
        add_weights<TL>(raw, lo, tb, sc, s0, s1);
    }
    __syncthreads();
    share_sums(sm.wsum, s0 + s1, rank, C);
    SpNucleus r;
    r.S = table_sum(sm.wsum, C, lane) - minus;
    // every CTA evaluates the whole table; the margins of 1e-4 cover fp32 sums and exp2f
    const float step = bins.s > 0.f ? static_cast<float>(sc.c) / bins.s : 0.f;   // -log2 of the weight, per interval
    const float target = static_cast<float>(fmax(p * r.S, 1e-9));
    uint32_t n[SP_BPT], nown = 0;
    pull_counts(sm, C, n);
    float lo2[SP_BPT], hi2[SP_BPT], hown = 0.f, lown = 0.f;
#pragma unroll
    for (int j = 0; j < SP_BPT; ++j) {
        const int b = SP_BPT * tid + j;
        const float cn = static_cast<float>(n[j]);
        hi2[j] = cn * fminf(1.f, exp2f(-step * (static_cast<float>(b) - 0.5f))) * 1.0001f;
        lo2[j] = b == SP_BINS - 1 || !(bins.s > 0.f) ? 0.f : cn * exp2f(-step * (static_cast<float>(b) + 0.5f)) * 0.9999f;
        hown += hi2[j];
        lown += lo2[j];
        nown += n[j];
    }
    float h = warp_scan(hown, lane), l = warp_scan(lown, lane);
    uint32_t nex = warp_scan(nown, lane);
    if (lane == 31) {
        sm.fscan[0][warp] = h;
        sm.fscan[1][warp] = l;
        sm.wcnt[warp] = nex;
    }
    if (tid == 0) {
        sm.nb0 = SP_BINS - 1;
        sm.nb1 = SP_BINS - 1;
    }
    h -= hown;
    l -= lown;
    nex -= nown;
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        h += sm.fscan[0][w];
        l += sm.fscan[1][w];
        nex += sm.wcnt[w];
    }
    uint32_t f0 = SP_BINS - 1, f1 = SP_BINS - 1, run[SP_BPT];
#pragma unroll
    for (int j = 0; j < SP_BPT; ++j) {
        h += hi2[j];
        l += lo2[j];
        nex += n[j];
        run[j] = nex;
        if (h >= target) f0 = min(f0, static_cast<uint32_t>(SP_BPT * tid + j));
        if (l >= target) f1 = min(f1, static_cast<uint32_t>(SP_BPT * tid + j));
    }
    f0 = __reduce_min_sync(0xffffffffu, f0);
    f1 = __reduce_min_sync(0xffffffffu, f1);
    if (lane == 0) {
        atomicMin(&sm.nb0, f0);
        atomicMin(&sm.nb1, f1);
    }
    __syncthreads();
    r.b0 = sm.nb0;
    r.b1 = sm.nb1;
#pragma unroll
    for (int j = 0; j < SP_BPT; ++j)
        if (r.b1 == static_cast<uint32_t>(SP_BPT * tid + j)) sm.nn = run[j];
    __syncthreads();
    r.n = r.b1 < SP_BINS - 1 ? sm.nn : V;
    return r;
}

// Top-k over the elements at or above lo, first step: the interval that holds
// the k-th (the last one where the others hold fewer), and the tokens above it.
// Clears nothing: sm.cnt is zero in every CTA when called.
struct SpKth {
    uint32_t b, above;
};
template <typename TL>
__device__ SpKth kth_interval(SampleSmem& sm, const SpChunk<TL>& ck, const SpScale& sc, uint32_t C, float lo,
                              uint32_t k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const SpBins bins = first_bins<TL>(sc, lo);
    for (int q = tid; q < ck.nvec; q += SP_THREADS)
        count_vector<TL>(sm, reinterpret_cast<const uint4*>(ck.buf)[q], lo, bins);
    cluster_sync_warp0();
    uint32_t n[SP_BPT], own = 0;
    pull_counts(sm, C, n);
#pragma unroll
    for (int j = 0; j < SP_BPT; ++j) own += n[j];
    const uint32_t inc = warp_scan(own, lane);
    if (lane == 31) sm.wcnt[warp] = inc;
    __syncthreads();
    uint32_t ex = inc - own, tot = 0;
    for (int w = 0; w < SP_WARPS; ++w) {
        if (w < warp) ex += sm.wcnt[w];
        tot += sm.wcnt[w];
    }
    if (tot < k) {
        __syncthreads();   // wcnt has been read: the caller's gather() writes it
        return SpKth{SP_BINS - 1, tot};
    }
#pragma unroll
    for (int j = 0; j < SP_BPT; ++j) {
        if (ex < k && ex + n[j] >= k) {
            sm.nb0 = SP_BPT * tid + j;
            sm.nb1 = ex;
        }
        ex += n[j];
    }
    __syncthreads();
    return SpKth{sm.nb0, sm.nb1};
}

// The logit that a key stands for.
template <typename TL>
__device__ __forceinline__ float key_logit(uint32_t key) {
    constexpr int KSH = SpElem<TL>::KSH;
    return key_value(KSH ? (key << KSH) | ((key >> 15) ? 0u : 0xffffu) : key);
}

// This CTA's elements at or above `floor` that keep() accepts as composite keys
// in sm.loc, in index order, and the count of every CTA in ccnt (not used
// before).  Returns the cluster's count; a CTA with more than SP_CAP lists none.
// This warp's entries are loc[start, start + count).
template <typename TL, typename F>
__device__ uint32_t gather(SampleSmem& sm, uint32_t* ccnt, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, float floor,
                           F keep, uint32_t* start = nullptr, uint32_t* count = nullptr) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    constexpr uint32_t kRoom = SP_CAP / SP_WARPS;
    const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(floor);
    // this warp's entries from loc[from] on, as far as `room`; returns their number
    auto list = [&](uint32_t from, uint32_t room) {
        uint32_t n = 0;
        for (int v0 = q0; v0 < q1; v0 += 32) {
            const uint4 raw = ck.raw_to(v0 + lane, q1);
            if (!__any_sync(0xffffffffu, SpElem<TL>::any_ge(raw, tb))) continue;
            uint32_t mask = 0, all;
            float v[VEC];
            SpElem<TL>::unpack(raw, v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) mask |= (v[e] >= floor && keep(v[e]) ? 1u : 0u) << e;
            uint32_t w = n + lanes_before(__popc(mask), lane, all);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (mask & (1u << e)) {
                    if (w < room) sm.loc[from + w] = composite(v[e], ck.index(v0 + lane, e));
                    ++w;
                }
            n += all;
        }
        return n;
    };
    // into a part of loc for each warp, then together; a second pass where one has more than that
    const uint32_t n = list(warp * kRoom, kRoom);
    if (lane == 0) sm.wcnt[warp] = n;
    __syncthreads();
    uint32_t at = 0, tot = 0, most = 0;
#pragma unroll
    for (int w = 0; w < SP_WARPS; ++w) {
        const uint32_t x = sm.wcnt[w];
        if (w < warp) at += x;
        tot += x;
        most = max(most, x);
    }
    if (tid < static_cast<int>(C)) st_cluster_s32(&ccnt[rank], tid, static_cast<int>(tot));
    if (start) {
        *start = at;
        *count = n;
    }
    if (tot <= SP_CAP) {
        if (most <= kRoom) {
            unsigned long long k[kRoom / 32];
#pragma unroll
            for (uint32_t i = 0; i < kRoom / 32; ++i)
                if (lane + 32 * i < n) k[i] = sm.loc[warp * kRoom + lane + 32 * i];
            __syncthreads();
#pragma unroll
            for (uint32_t i = 0; i < kRoom / 32; ++i)
                if (lane + 32 * i < n) sm.loc[at + lane + 32 * i] = k[i];
        } else {
            list(at, n);
        }
    }
    cluster_sync_warp0();
    uint32_t all = 0;
    for (uint32_t r = 0; r < C; ++r) all += ccnt[r];
    return all;
}

// A lower bound of the k-th largest of the elements at or above lo: the k-th
// largest of the threads' maxima (each of k threads holds an element at least
// that large), to within one of SP_THREADS intervals between low and high, the
// least and the largest of those maxima.  lo where fewer than k threads hold an
// element that large.
__device__ float kth_bound(SampleSmem& sm, uint32_t C, float lo, float low, float high, float mine, uint32_t k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    low = fmaxf(low, lo);
    const float width = high - low;
    const SpBins bins{high, width > 0.f && width < 1e30f ? static_cast<float>(SP_THREADS - 1) / width : 0.f};
    if (mine >= lo) atomicAdd(&sm.cnt[min(bins.raw(mine), SP_THREADS - 1u)], 1u);   // the table is clear when called
    cluster_sync_warp0();
    uint32_t n = 0;
#pragma unroll 8
    for (uint32_t r = 0; r < C; ++r) {
        uint32_t x;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(sp_mapa(&sm.cnt[tid], r)) : "memory");
        n += x;
    }
    if (tid == 0) sm.last = SP_THREADS;
    uint32_t in = warp_scan(n, lane);
    if (lane == 31) sm.wcnt[warp] = in;
    __syncthreads();
    for (int w = 0; w < warp; ++w) in += sm.wcnt[w];
    if (in - n < k && in >= k) sm.last = tid;
    __syncthreads();
    const int b = sm.last;
    __syncthreads();   // wcnt and last are free again
    if (b < SP_THREADS - 1 || !(bins.s > 0.f)) return bins.lower(b, lo);
    return b < SP_THREADS ? low : lo;   // all of the maxima, or too few
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
    if (lane == 31) sm.dscan[0][warp] = inc;
    __syncthreads();
    double base = 0.0, sum = 0.0;
    for (int w = 0; w < nwarps; ++w) {
        if (w == warp) base = sum;
        sum += sm.dscan[0][w];
    }
    start = base + prev;
    end = base + inc;
    total = sum;
}

// The starts of two sets of runs at once.
__device__ __forceinline__ void block_starts(SampleSmem& sm, double a, double b, double& sa, double& sb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const double ia = warp_scan(a, lane), ib = warp_scan(b, lane);
    double pa = __shfl_up_sync(0xffffffffu, ia, 1), pb = __shfl_up_sync(0xffffffffu, ib, 1);
    if (lane == 0) pa = pb = 0.0;
    if (lane == 31) {
        sm.dscan[0][warp] = ia;
        sm.dscan[1][warp] = ib;
    }
    __syncthreads();
    sa = sb = 0.0;
    for (int w = 0; w < warp; ++w) {
        sa += sm.dscan[0][w];
        sb += sm.dscan[1][w];
    }
    sa += pa;
    sb += pb;
}

constexpr int SP_PER = SP_CAP / SP_THREADS;

// Descending order of n composite keys from lst into srt.
__device__ void sort_list(SampleSmem& sm, const unsigned long long* lst, unsigned long long* srt, int n) {
    const int tid = threadIdx.x;
    if (n <= 128) {   // each key's rank by counting, SP_THREADS / 128 threads a key
        uint32_t* rk = sm.cnt;
        for (int i = tid; i < 128; i += SP_THREADS) rk[i] = 0;
        __syncthreads();
        const int i = tid & 127, part = tid >> 7;
        if (i < n) {
            const unsigned long long k = lst[i];
            const int per = (n + SP_THREADS / 128 - 1) / (SP_THREADS / 128);
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
    // into SP_BINS buckets by logit, then each key's rank within its bucket
    const int lane = tid & 31, warp = tid >> 5;
    unsigned long long k[SP_PER];
    uint32_t least = 0xffffffffu, most = 0;
#pragma unroll
    for (int e = 0; e < SP_PER; ++e) {
        const int i = tid + e * SP_THREADS;
        k[e] = i < n ? lst[i] : 0ull;
        if (i < n) {
            least = min(least, static_cast<uint32_t>(k[e] >> 32));
            most = max(most, static_cast<uint32_t>(k[e] >> 32));
        }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        sm.wcnt[warp] = least;
        sm.scan[warp] = most;
    }
    for (int i = tid; i < SP_BINS; i += SP_THREADS) sm.cnt[i] = 0;
    __syncthreads();
    for (int w = 0; w < SP_WARPS; ++w) {
        least = min(least, sm.wcnt[w]);
        most = max(most, static_cast<uint32_t>(sm.scan[w]));
    }
    const float high = key_value(most), width = high - key_value(least);
    const SpBins bins{high, width > 0.f && width < 1e30f ? static_cast<float>(SP_BINS - 1) / width : 0.f};
    uint32_t b[SP_PER], at[SP_PER];
#pragma unroll
    for (int e = 0; e < SP_PER; ++e) {
        if (tid + e * SP_THREADS >= n) continue;
        b[e] = bins.of(key_value(static_cast<uint32_t>(k[e] >> 32)));
        at[e] = atomicAdd(&sm.cnt[b[e]], 1u);
    }
    __syncthreads();
    uint32_t c[SP_BPT], own = 0, big = 0;
#pragma unroll
    for (int j = 0; j < SP_BPT; ++j) {
        c[j] = sm.cnt[SP_BPT * tid + j];
        own += c[j];
        big = max(big, c[j]);
    }
    const uint32_t inc = warp_scan(own, lane);
    if (lane == 31) sm.wcnt[warp] = inc;
    const bool crowded = __syncthreads_or(big > 96);   // (a barrier either way)
    if (!crowded) {
        uint32_t ex = inc - own;
        for (int w = 0; w < warp; ++w) ex += sm.wcnt[w];
#pragma unroll
        for (int j = 0; j < SP_BPT; ++j) {
            sm.cnt[SP_BPT * tid + j] = ex;
            ex += c[j];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < SP_PER; ++e)
            if (tid + e * SP_THREADS < n) sm.order[sm.cnt[b[e]] + at[e]] = static_cast<uint16_t>(tid + e * SP_THREADS);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < SP_PER; ++e) {
            if (tid + e * SP_THREADS >= n) continue;
            const uint32_t i0 = sm.cnt[b[e]], i1 = b[e] + 1 < SP_BINS ? sm.cnt[b[e] + 1] : static_cast<uint32_t>(n);
            uint32_t r = i0;
            for (uint32_t i = i0; i < i1; ++i) r += lst[sm.order[i]] > k[e];
            srt[r] = k[e];
        }
        __syncthreads();
        return;
    }
    // many equal logits: a bitonic network
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

// The cluster's gathered candidates into the leader's lst, in index order.
__device__ void pull_list(SampleSmem& sm, const uint32_t* ccnt, int n) {
    for (int i = threadIdx.x; i < n; i += SP_THREADS) {
        uint32_t j = i, c = 0;
        while (j >= ccnt[c]) j -= ccnt[c++];
        unsigned long long k;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(sp_mapa(&sm.loc[j], c)) : "memory");
        sm.lst[i] = k;
    }
}

// The border token of a list in index order: the k-th of the descending order
// (k > 0), or the first at which the running weight reaches the target
// (entries under `least` weigh nothing).  Returns its composite key, with a
// zero index part where no tie of it stays behind.  srt is scratch for n keys.
// All threads of the leader call it.
__device__ unsigned long long border_of(SampleSmem& sm, const unsigned long long* lst, unsigned long long* srt, int n,
                                        int ksh, const SpScale& sc, unsigned long long least, uint32_t k, double want) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n + SP_THREADS - 1) / SP_THREADS;
    const int nwarps = min(SP_WARPS, (n + 32 * per - 1) / (32 * per));
    if (n > 128) {
        // few distinct logits (bf16): count each, and take the border's ties in index order
        uint32_t kmin = 0xffffffffu, kmax = 0;
        for (int i = tid; i < n; i += SP_THREADS) {
            const uint32_t x = static_cast<uint32_t>(lst[i] >> 32) >> ksh;
            kmin = min(kmin, x);
            kmax = max(kmax, x);
        }
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        __syncthreads();
        if (lane == 0) {
            sm.wcnt[warp] = kmin;
            sm.scan[warp] = kmax;
        }
        for (int i = tid; i < SP_BINS; i += SP_THREADS) sm.cnt[i] = 0;
        __syncthreads();
        for (int w = 0; w < SP_WARPS; ++w) {
            kmin = min(kmin, sm.wcnt[w]);
            kmax = max(kmax, static_cast<uint32_t>(sm.scan[w]));
        }
        if (kmax - kmin < SP_BINS) {
            for (int i = tid; i < n; i += SP_THREADS) atomicAdd(&sm.cnt[kmax - (static_cast<uint32_t>(lst[i] >> 32) >> ksh)], 1u);
            if (tid == 0) {
                sm.nb0 = kmax - kmin;
                sm.keep = n;
            }
            __syncthreads();
            uint32_t c[SP_BPT];
            double m[SP_BPT], own = 0.0, start, end, total;
#pragma unroll
            for (int j = 0; j < SP_BPT; ++j) {
                const uint32_t b = SP_BPT * tid + j;
                c[j] = sm.cnt[b];
                m[j] = c[j];
                if (k == 0 && c[j]) {
                    const uint32_t okey = ((kmax - b) << ksh) | (ksh && !((kmax - b) >> 15) ? 0xffffu : 0u);
                    m[j] = (static_cast<unsigned long long>(okey) << 32 | 0xffffffffu) >= least ? c[j] * sc.weight(key_value(okey)) : 0.0;
                }
                own += m[j];
            }
            block_runs(sm, own, SP_WARPS, start, end, total);
            const double goal = k > 0 ? static_cast<double>(min(k, static_cast<uint32_t>(n))) : want;
            if (start < goal && end >= goal) {
                int at = -1;
                double acc = start, before = start;
#pragma unroll
                for (int j = 0; j < SP_BPT; ++j) {
                    if (c[j] && m[j] > 0.0 && (at < 0 || acc < goal)) {
                        at = j;
                        before = acc;
                    }
                    acc += m[j];
                }
                if (at >= 0) {
#pragma unroll
                    for (int j = 0; j < SP_BPT; ++j)
                        if (j == at) {
                            const double need = ceil((goal - before) / (m[j] / c[j]));
                            sm.nb0 = SP_BPT * tid + j;
                            sm.keep = need < 1.0 ? 1u : need > c[j] ? c[j] : static_cast<uint32_t>(need);
                        }
                }
            }
            __syncthreads();
            // the keep-th entry of that logit
            const uint32_t key = kmax - sm.nb0, ties = sm.cnt[sm.nb0], keep = min(sm.keep, ties);
            uint32_t mine = 0;
            for (int e = 0; e < per; ++e) {
                const int i = tid * per + e;
                mine += i < n && (static_cast<uint32_t>(lst[i] >> 32) >> ksh) == key ? 1u : 0u;
            }
            const uint32_t inc = warp_scan(mine, lane);
            if (lane == 31) sm.wcnt[warp] = inc;
            __syncthreads();
            uint32_t ex = inc - mine;
            for (int w = 0; w < warp; ++w) ex += sm.wcnt[w];
            for (int e = 0; e < per; ++e) {
                const int i = tid * per + e;
                if (i < n && (static_cast<uint32_t>(lst[i] >> 32) >> ksh) == key && ++ex == keep) sm.sel_key = lst[i];
            }
            __syncthreads();
            const unsigned long long cut = sm.sel_key;
            __syncthreads();
            return keep < ties ? cut : cut & 0xffffffff00000000ull;
        }
    }
    __syncthreads();
    sort_list(sm, lst, srt, n);
    if (tid == 0) sm.keep = k > 0 ? min(k, static_cast<uint32_t>(n)) : n;
    if (k == 0) {
        double w[SP_PER], own = 0.0, start, end, total;
#pragma unroll
        for (int e = 0; e < SP_PER; ++e) {
            const int j = tid * per + e;
            w[e] = e < per && j < n && srt[j] >= least ? sc.weight(composite_value(srt[j])) : 0.0;
            own += w[e];
        }
        block_runs(sm, own, nwarps, start, end, total);
        // the first token at which the running sum reaches the target
        if (start < want && end >= want) {
            double acc = start;
            int at = -1;
#pragma unroll
            for (int e = 0; e < SP_PER; ++e) {
                if (w[e] > 0.0 && (at < 0 || acc < want)) at = e;
                acc += w[e];
            }
            sm.keep = tid * per + at + 1;
        }
    }
    __syncthreads();
    const int at = max(0, static_cast<int>(sm.keep) - 1);
    const unsigned long long cut = srt[at];
    bool behind = false;
    for (int j = tid; j < n; j += SP_THREADS) behind |= j > at && srt[j] >> 32 == cut >> 32;
    return __syncthreads_or(behind) ? cut : cut & 0xffffffff00000000ull;
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
// filters, acceptance of the draft, the draw.  Entries under lcut carry no
// weight.  S_all: the row's sum before top-p, or negative where the list has
// all of the row's weight.
template <bool VERIFY>
__device__ void draw_from_list(SampleSmem& sm, int n, int ksh, float lcut, const SpScale& sc, const SpRow& r, double S_all,
                               int32_t* token) {
    const int tid = threadIdx.x;
    if (n <= 0) return;   // (the list holds the maximum)
    const unsigned long long* lst = sm.lst;
    unsigned long long* srt = sm.loc;
    const int per = (n + SP_THREADS - 1) / SP_THREADS;
    const int nwarps = min(SP_WARPS, (n + 32 * per - 1) / (32 * per));
    const unsigned long long least = static_cast<unsigned long long>(order_key(lcut)) << 32;
    unsigned long long cut = least;
    if (n <= 128 && (r.by_k || r.by_p)) {   // one short sort serves both filters
        int nk = r.by_k ? min(r.k, n) : n;
        sort_list(sm, lst, srt, n);
        if (r.by_p) {
            if (tid == 0) sm.keep = nk;
            double w[SP_PER], own = 0.0, start, end, total;
#pragma unroll
            for (int e = 0; e < SP_PER; ++e) {
                const int j = tid * per + e;
                w[e] = e < per && j < nk && srt[j] >= least ? sc.weight(composite_value(srt[j])) : 0.0;
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
        cut = max(least, srt[nk - 1]);
    } else if (r.by_k || r.by_p) {
        if (r.by_k) cut = max(least, border_of(sm, lst, srt, n, ksh, sc, least, static_cast<uint32_t>(r.k), 0.0));
        if (r.by_p) {
            double S = S_all;
            if (r.by_k || S_all < 0.0) {
                double own = 0.0, start, end;
                for (int e = 0; e < per; ++e) {
                    const int j = tid * per + e;
                    if (j < n && lst[j] >= cut) own += sc.weight(composite_value(lst[j]));
                }
                block_runs(sm, own, nwarps, start, end, S);
            }
            // tokens that top-k left out come behind the border in the order
            cut = max(cut, border_of(sm, lst, srt, n, ksh, sc, least, 0, fmax(r.p * S, 1e-9)));
        }
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
                if (w[e] > 0.0) {
                    const double q = fabs(static_cast<double>(__ldg(r.q + composite_index(lst[tid * per + e]))));
                    rw[e] = fmax(0.0, w[e] - q * S);   // (NaN: 0)
                }
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

// ---------------------------------------------------------------- borders by counting every value (bf16)
// A bf16 row has few distinct values: between the smallest and the largest that
// carry weight there are at most some thousands, but for the many tiny ones
// around zero.  One pass counts each (the values of magnitude at most m0 as one,
// their weights summed apart); counts times weights are then exact sums in the
// order of the selection, and the borders of top-k and top-p follow by a scan.
// The pass is bound by shared-memory atomics (35 cycles per 32 elements and
// quarter of an SM, as much as an fp64 pass), so it replaces the later passes of
// rows that keep many tokens and not the first of every row: by intervals and
// refinement the 512 mixed rows take 154 us instead of 131, the 32 x 4 rows of
// a top-p verification 101 instead of 91.
constexpr int SP_KEYS = 4096;
static_assert(SP_KEYS * sizeof(uint32_t) <= sizeof(SampleSmem::lst), "the counts share the candidates' memory");
constexpr int SP_KPT = SP_KEYS / SP_THREADS;

struct SpKeys {
    int m0, top, n;   // value of rank r below the maximum: signed magnitude top - r, less the collapsed ones
    static __device__ __forceinline__ int signed_mag(float l) {
        const int b = __float_as_int(l) >> 16;   // (sign-extended)
        return b < 0 ? -(b & 0x7fff) : b;
    }
    __device__ __forceinline__ int squeeze(int s) const { return s > m0 ? s - m0 : s < -m0 ? s + m0 : 0; }
    // NaN and what lies below the smallest get ranks of n and more (as unsigned)
    __device__ __forceinline__ uint32_t rank(uint32_t bits, uint32_t sign) const {   // 15 bits, 0 or ~0
        const uint32_t a = max(static_cast<int>(bits) - m0, 0);
        return top + sign - (a ^ sign);
    }
    __device__ __forceinline__ uint32_t rank(float l) const { return static_cast<uint32_t>(top - squeeze(signed_mag(l))); }
    __device__ __forceinline__ bool mixed(uint32_t r) const { return m0 > 0 && static_cast<int>(r) == top; }
    __device__ __forceinline__ float value(uint32_t r) const {
        const int c = top - static_cast<int>(r), s = c > 0 ? c + m0 : c < 0 ? c - m0 : 0;
        return __uint_as_float(static_cast<uint32_t>(s < 0 ? 0x8000 - s : s) << 16);
    }
};
// The values from m down to lo, bf16 both; the smallest m0 that fits.
__device__ __forceinline__ SpKeys make_keys(float m, float lo) {
    const int a = SpKeys::signed_mag(m), b = SpKeys::signed_mag(lo);
    SpKeys k{a - b < SP_KEYS ? 0 : max((a - b + 2 - SP_KEYS) >> 1, max(a, -b) + 1 - SP_KEYS), 0, 0};
    k.top = k.squeeze(a);
    k.n = k.top - k.squeeze(b) + 1;
    return k;
}

struct SpBorder {
    bool ok;               // false: a border among the collapsed values
    uint32_t r;            // rank of the border's value,
    uint32_t above, ties;  // tokens above it and with it,
    uint32_t keep;         // and how many of the latter are kept
    double zsum;           // this thread's part of the collapsed values' weights
};

// The border of the first k tokens (k > 0) and, p < 1, of the prefix of those
// that reaches p times their sum; S > 0: p times S instead.  The border is at or
// above the smallest of the keys.  All threads of the cluster call it.
__device__ SpBorder key_border(SampleSmem& sm, const SpChunk<__nv_bfloat16>& ck, const SpScale& sc, const SpKeys& keys,
                               uint32_t rank, uint32_t C, float lo, uint32_t k, double p, double S) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t* hist = reinterpret_cast<uint32_t*>(sm.lst);
    for (int i = tid; i < keys.n; i += SP_THREADS) hist[i] = 0;
    if (tid == 0) {
        sm.nb0 = SP_KEYS;
        sm.nb1 = SP_KEYS;
        sm.last = 0;
    }
    __syncthreads();
    SpBorder o;
    o.zsum = 0.0;
    const __nv_bfloat162 small = __halves2bfloat162(__ushort_as_bfloat16(keys.m0), __ushort_as_bfloat16(keys.m0));
    for (int q = tid; q < ck.nvec; q += SP_THREADS) {
        const uint4 raw = reinterpret_cast<const uint4*>(ck.buf)[q];
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r0 = keys.rank(w[i] & 0x7fffu, static_cast<uint32_t>(static_cast<int>(w[i] << 16) >> 31));
            const uint32_t r1 = keys.rank((w[i] >> 16) & 0x7fffu, static_cast<uint32_t>(static_cast<int>(w[i]) >> 31));
            if (r0 < keys.n) atomicAdd(&hist[r0], 1u);
            if (r1 < keys.n) atomicAdd(&hist[r1], 1u);
        }
        if (keys.m0 > 0) {
            const __nv_bfloat162 a = __hmin2(__hmin2(__habs2(SpElem<__nv_bfloat16>::pair(raw.x)), __habs2(SpElem<__nv_bfloat16>::pair(raw.y))),
                                             __hmin2(__habs2(SpElem<__nv_bfloat16>::pair(raw.z)), __habs2(SpElem<__nv_bfloat16>::pair(raw.w))));
            if (__hle2_mask(a, small)) {
                float v[8];
                SpElem<__nv_bfloat16>::unpack(raw, v);
                for (int e = 0; e < 8; ++e)
                    if (keys.rank(v[e]) == static_cast<uint32_t>(keys.top) && v[e] >= lo) o.zsum += sc.weight(v[e]);
            }
        }
    }
    double z = 0.0;
    if (keys.m0 > 0) {
        share_sums(sm.rsum, o.zsum, rank, C);
        z = table_sum(sm.rsum, C, lane);
    } else {
        cluster_sync_warp0();
    }
    // the cluster's counts, then this thread's ranks, in order
    uint32_t* sum = reinterpret_cast<uint32_t*>(sm.loc);
    for (int i = tid; i < keys.n; i += SP_THREADS) {
        uint32_t x[SP_MAXC], t = 0;
#pragma unroll
        for (uint32_t c = 0; c < SP_MAXC; ++c) {
            x[c] = 0;
            if (c < C) asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x[c]) : "r"(sp_mapa(&hist[i], c)) : "memory");
        }
#pragma unroll
        for (uint32_t c = 0; c < SP_MAXC; ++c) t += x[c];
        sum[i] = t;
    }
    __syncthreads();
    const int per = (keys.n + SP_THREADS - 1) / SP_THREADS, r0 = tid * per;
    uint32_t n[SP_KPT], own = 0;
    double w[SP_KPT], wown = 0.0, start, end, total;
#pragma unroll
    for (int j = 0; j < SP_KPT; ++j) {
        n[j] = j < per && r0 + j < keys.n ? sum[r0 + j] : 0u;
        own += n[j];
    }
    uint32_t last = 0;
#pragma unroll
    for (int j = 0; j < SP_KPT; ++j) {
        w[j] = 0.0;
        if (n[j]) {
            w[j] = keys.mixed(r0 + j) ? z : n[j] * sc.weight(keys.value(r0 + j));
            last = r0 + j;
        }
        wown += w[j];
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) atomicMax(&sm.last, static_cast<int>(last));
    uint32_t ex = warp_scan(own, lane);
    if (lane == 31) sm.wcnt[warp] = ex;
    block_runs(sm, wown, SP_WARPS, start, end, total);
    ex -= own;
    uint32_t all = 0;
    for (int i = 0; i < SP_WARPS; ++i) {
        if (i < warp) ex += sm.wcnt[i];
        all += sm.wcnt[i];
    }
    // the k-th token: its value, how many of that value are kept, the sum of the tokens kept
    uint32_t kr = SP_KEYS, kkeep = 0;
    if (!(S > 0.0)) S = total;
    if (k > 0 && k < all) {
        uint32_t c = ex;
        double run = start;
#pragma unroll
        for (int j = 0; j < SP_KPT; ++j) {
            if (c < k && c + n[j] >= k) {
                sm.nb0 = r0 + j;
                sm.nn = k - c;
                sm.sel_w = run + w[j] / n[j] * (k - c);
            }
            c += n[j];
            run += w[j];
        }
        __syncthreads();
        kr = sm.nb0;
        kkeep = sm.nn;
        S = sm.sel_w;
        __syncthreads();   // they are written again below
    }
    double target = 0.0;
    uint32_t r = min(kr, static_cast<uint32_t>(sm.last));
    if (p < 1.0) {
        target = fmax(p * S, 1e-9);
        double run = start;
        uint32_t f = SP_KEYS;
#pragma unroll
        for (int j = 0; j < SP_KPT; ++j) {
            run += w[j];
            if (n[j] && run >= target) f = min(f, static_cast<uint32_t>(r0 + j));
        }
        f = __reduce_min_sync(0xffffffffu, f);
        if (lane == 0) atomicMin(&sm.nb1, f);
        __syncthreads();
        r = min(r, sm.nb1);
    }
    double run = start;
#pragma unroll
    for (int j = 0; j < SP_KPT; ++j) {
        if (j < per && r == static_cast<uint32_t>(r0 + j)) {
            sm.sel_before = run;
            sm.sel_w = w[j] / n[j];
            sm.sel_cnt = ex;
            sm.nn = n[j];
        }
        ex += n[j];
        run += w[j];
    }
    __syncthreads();
    o.r = r;
    o.above = sm.sel_cnt;
    o.ties = sm.nn;
    o.keep = r == kr ? kkeep : o.ties;
    if (p < 1.0) {
        const double need = ceil((target - sm.sel_before) / sm.sel_w);
        if (need < static_cast<double>(o.keep)) o.keep = need < 1.0 ? 1u : static_cast<uint32_t>(need);
    }
    o.ok = !keys.mixed(r) && !(kr < SP_KEYS && keys.mixed(kr));
    return o;
}

// This thread's part of the kept weights of its CTA: the counted values above
// the border, `ties` of the border's, without the certain draft's (rank rx).
__device__ double key_sum(const SampleSmem& sm, const SpScale& sc, const SpKeys& keys, const SpBorder& b, uint32_t ties,
                          uint32_t rx) {
    const uint32_t* hist = reinterpret_cast<const uint32_t*>(sm.lst);
    double s = keys.m0 > 0 && static_cast<uint32_t>(keys.top) < b.r ? b.zsum : 0.0;
    for (uint32_t r = threadIdx.x; r <= b.r; r += SP_THREADS) {
        if (keys.mixed(r)) continue;
        const uint32_t n = (r == b.r ? ties : hist[r]) - (r == rx ? 1u : 0u);
        if (n) s += n * sc.weight(keys.value(r));
    }
    return s;
}

// ---------------------------------------------------------------- the draw from the whole row
// This thread's part of its warp's weights at or above tau.
template <typename TL>
__device__ double segment_part(const SpChunk<TL>& ck, float tau, const SpScale& sc) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    double s0 = 0.0, s1 = 0.0;
    const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(tau);
    for (int v0 = q0; v0 < q1; v0 += 32) add_weights<TL>(ck.raw_to(v0 + lane, q1), tau, tb, sc, s0, s1);
    return s0 + s1;
}

// w - |q| S, S as S 2^896.  An infinite or NaN q becomes 2^128 or more and leaves nothing; without its sign, which a
// NaN may have (0/0 on the host) and which would leave all of the row's weight to its token.
__device__ __forceinline__ double residual(double w, float q, double S896) {
    const int u = __float_as_int(q);
    return fma(-__hiloint2double((u >> 3) & 0x0fffffff, u << 29), S896, w);
}

// One element of the residual max(w - q S, 0) of the weights at or above tau
// (q NULL: of the weights).
template <typename TL>
__device__ __forceinline__ double left_weight(float l, int idx, float tau, const SpScale& sc, const float* q, double S896) {
    if (!(l >= tau)) return 0.0;
    const double w = sc.weight(l);
    return q ? fmax(0.0, residual(w, __ldg(q + idx), S896)) : w;
}

template <typename TL>
__device__ void residual_sums(double* sums, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, float tau,
                              const SpScale& sc, const float* q, double S896) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    double s = 0.0;
    const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(tau);
    const float* qp = q + ck.begin - ck.mis;   // of the part's first vector
    const bool wide = ck.mis == 0 && (reinterpret_cast<uintptr_t>(qp) & 15u) == 0;
    for (int v0 = q0 + lane; v0 < q1; v0 += 32) {
        const uint4 raw = reinterpret_cast<const uint4*>(ck.buf)[v0];
        if (wide && (v0 + 1) * VEC <= ck.n && SpElem<TL>::all_ge(raw, tb)) {
            float4 f[VEC / 4];
#pragma unroll
            for (int e = 0; e < VEC / 4; ++e) f[e] = __ldg(reinterpret_cast<const float4*>(qp + v0 * VEC) + e);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float4& g = f[e / 4];
                const double d = residual(sc.weight(SpElem<TL>::scaled(raw, e), sc.tab),
                                          e % 4 == 0 ? g.x : e % 4 == 1 ? g.y : e % 4 == 2 ? g.z : g.w, S896);
                if (d > 0.0) s += d;
            }
        } else if (SpElem<TL>::any_ge(raw, tb)) {
            float v[VEC];
            SpElem<TL>::unpack(raw, v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += left_weight<TL>(v[e], ck.index(v0, e), tau, sc, q, S896);
        }
    }
    share_sums(sums, s, rank, C);
}

// The first index whose cumulative weight exceeds the target, given the sums of
// nseg segments, of which this warp has segment `own_seg`.  Returns the token in
// the warp that owns it, -1 elsewhere.
template <typename TL>
__device__ int draw_token(const double* sums, int nseg, int own_seg, const SpChunk<TL>& ck, float tau, const SpScale& sc,
                          const float* q, double S896, double target) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (nseg + 31) / 32;
    // every warp finds the owning segment: lane l scans segments [l per, l per + per)
    double own = 0.0;
    for (int j = 0; j < per; ++j)
        if (lane * per + j < nseg) own += sums[lane * per + j];
    double base = warp_scan(own, lane) - own;
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
    if (seg != own_seg) return -1;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    int last = -1;
    for (int v0 = q0; v0 < q1; v0 += 32) {
        double w[VEC], s = 0.0;
        const int vq = v0 + lane;
        int mine = -1;
        float v[VEC];
        ck.load_to(vq, q1, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[e] = left_weight<TL>(v[e], ck.index(vq, e), tau, sc, q, S896);
            s += w[e];
            if (w[e] > 0.0) mine = ck.index(vq, e);
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

// The elements of the border's intervals b0..b1: listed in every CTA's loc, or,
// where one CTA has too many, found by passes over the row.
struct SpWindow {
    bool listed;
    uint32_t all, mine;            // the cluster's entries, this CTA's;
    uint32_t start, count;         // this warp's range of them
    float bot, top;                // bounds of the intervals' logits
    SpBins bins;
    uint32_t b0, b1;
};
template <typename TL, typename F>
__device__ __forceinline__ void each_in(const SampleSmem& sm, const SpChunk<TL>& ck, const SpWindow& w, F f) {
    if (w.listed) {
        for (uint32_t i = threadIdx.x; i < w.mine; i += SP_THREADS) f(composite_value(sm.loc[i]));
        return;
    }
    constexpr int VEC = SpElem<TL>::VEC;
    const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(w.bot);
    for (int q = threadIdx.x; q < ck.nvec; q += SP_THREADS) {
        const uint4 raw = reinterpret_cast<const uint4*>(ck.buf)[q];
        if (!SpElem<TL>::any_ge(raw, tb)) continue;
        float v[VEC];
        SpElem<TL>::unpack(raw, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (!(v[e] >= w.bot && v[e] <= w.top)) continue;
            const uint32_t b = w.bins.of(v[e]);
            if (b >= w.b0 && b <= w.b1) f(v[e]);
        }
    }
}
template <typename TL>
__device__ SpWindow make_window(SampleSmem& sm, uint32_t* ccnt, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, float lo,
                                const SpBins& bins, uint32_t b0, uint32_t b1) {
    SpWindow w;
    w.bins = bins;
    w.b0 = b0;
    w.b1 = b1;
    w.bot = bins.lower(b1, lo);
    w.top = bins.upper(b0);
    w.all = gather<TL>(sm, ccnt, ck, rank, C, w.bot, [&](float l) { const uint32_t b = bins.of(l); return b >= b0 && b <= b1; },
               &w.start, &w.count);
    uint32_t most = 0;
    for (uint32_t r = 0; r < C; ++r) most = max(most, ccnt[r]);
    w.listed = most <= SP_CAP;
    w.mine = ccnt[rank];
    return w;
}

// A bit per element of vector i that equals tau.
template <typename TL>
__device__ __forceinline__ uint32_t tie_mask(const SpChunk<TL>& ck, int i, float tau) {
    constexpr int VEC = SpElem<TL>::VEC;
    const uint4 raw = reinterpret_cast<const uint4*>(ck.buf)[i];
    uint32_t mask = 0;
    if (SpElem<TL>::any_eq(raw, tau)) {
        float v[VEC];
        SpElem<TL>::unpack(raw, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) mask |= (v[e] == tau ? 1u : 0u) << e;
    }
    return mask;
}

// Index of the keep-th token with logit tau, in index order (two cluster
// barriers).
template <typename TL>
__device__ int tie_index(SampleSmem& sm, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, const SpWindow& win, float tau,
                         uint32_t keep) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    // this warp's ties, in index order along lanes and steps of 32 entries or vectors
    const int first = win.listed ? static_cast<int>(win.start) : q0;
    const int last = win.listed ? static_cast<int>(win.start + win.count) : q1;
    auto ties_at = [&](int i) -> uint32_t {   // a bit per element of entry or vector i
        if (i >= last) return 0;
        if (win.listed) return composite_value(sm.loc[i]) == tau ? 1u : 0u;
        return tie_mask<TL>(ck, i, tau);
    };
    uint32_t n = 0;
    for (int i = first + lane; i < last; i += 32) n += __popc(ties_at(i));
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sm.wcnt[warp] = n;
    __syncthreads();
    uint32_t tot = 0, before = 0;
    for (int w = 0; w < SP_WARPS; ++w) {
        if (w < warp) before += sm.wcnt[w];
        tot += sm.wcnt[w];
    }
    if (tid < static_cast<int>(C)) st_cluster_s32(&sm.tie[rank], tid, static_cast<int>(tot));
    cluster_sync_warp0();
    for (uint32_t r = 0; r < rank; ++r) before += sm.tie[r];
    if (keep > before && keep <= before + n) {
        uint32_t left = keep - before;   // 1-based
        for (int i0 = first; i0 < last; i0 += 32) {
            uint32_t mask = ties_at(i0 + lane);
            const uint32_t mine = __popc(mask);
            uint32_t t;
            const uint32_t ex = lanes_before(mine, lane, t);
            if (ex + mine >= left && ex < left) {
                uint32_t skip = left - ex - 1;
                while (skip--) mask &= mask - 1;
                const int idx = win.listed ? composite_index(sm.loc[i0 + lane]) : ck.index(i0 + lane, __ffs(mask) - 1);
                for (uint32_t r = 0; r < C; ++r) st_cluster_s32(&sm.cut_idx, r, idx);
            }
            if (t >= left) break;
            left -= t;
        }
    }
    cluster_sync_all();
    return static_cast<int>(sm.cut_idx);
}

// The border of a window, as border_of() returns one: with by_count the token
// at which the count A of the tokens above the window plus the running count
// reaches the target, else the one at which the weight A above it plus the
// running weight does.  SP_BINS key ranges at a time: counts times the weights
// of a range's ends bound its running sums, so that exact sums are needed of one
// range only; a range of a single key is exact, and one of up to 32 tokens is
// sorted (without that the 32 fp32 rows of top-p took 56 us instead of 50).
// dropped: the ties behind the border.  All threads of the cluster call it.
template <typename TL>
__device__ unsigned long long refine(SampleSmem& sm, const SpChunk<TL>& ck, const SpScale& sc, uint32_t rank, uint32_t C,
                           const SpWindow& w, bool by_count, double A, double target, uint32_t& dropped) {
    constexpr int KSH = SpElem<TL>::KSH;
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t khi = order_key(w.top) >> KSH, klo = order_key(w.bot) >> KSH;
    while (true) {
        int sh = 0;
        while (((khi - klo) >> sh) >= SP_BINS) ++sh;
        const uint32_t span = (1u << sh) - 1;
        for (int i = tid; i < SP_BINS; i += SP_THREADS) sm.cnt[i] = 0;
        if (tid == 0) {
            sm.nb0 = SP_BINS;
            sm.nb1 = SP_BINS;
            sm.last = 0;
        }
        __syncthreads();
        each_in<TL>(sm, ck, w, [&](float l) {
            const uint32_t key = order_key(l) >> KSH;
            if (key >= klo && key <= khi) atomicAdd(&sm.cnt[(khi - key) >> sh], 1u);
        });
        cluster_sync_warp0();
        uint32_t n[SP_BPT];
        pull_counts(sm, C, n);
        double hi[SP_BPT], low[SP_BPT], hown = 0.0, lown = 0.0, hs, ls;
#pragma unroll
        for (int j = 0; j < SP_BPT; ++j) {
            const uint32_t b = SP_BPT * tid + j;
            hi[j] = low[j] = n[j];
            if (!by_count && n[j]) {
                const uint32_t top = khi - (b << sh), bot = top - klo > span ? top - span : klo;
                hi[j] *= sc.weight(key_logit<TL>(top));
                low[j] = sh ? low[j] * sc.weight(key_logit<TL>(bot)) : hi[j];
            }
            hown += hi[j];
            lown += low[j];
            if (n[j]) atomicMax(&sm.last, static_cast<int>(b));
        }
        block_starts(sm, hown, lown, hs, ls);
        hs += A;
        ls += A;
        const double from = ls;   // the running sum at this thread's first bin
        uint32_t f0 = SP_BINS, f1 = SP_BINS;
#pragma unroll
        for (int j = 0; j < SP_BPT; ++j) {
            hs += hi[j];
            ls += low[j];
            if (hs * (1.0 + 1e-12) >= target) f0 = min(f0, static_cast<uint32_t>(SP_BPT * tid + j));
            if (ls >= target) f1 = min(f1, static_cast<uint32_t>(SP_BPT * tid + j));
        }
        f0 = __reduce_min_sync(0xffffffffu, f0);
        f1 = __reduce_min_sync(0xffffffffu, f1);
        if (lane == 0) {
            atomicMin(&sm.nb0, f0);
            atomicMin(&sm.nb1, f1);
        }
        __syncthreads();
        const uint32_t b1 = min(sm.nb1, static_cast<uint32_t>(sm.last));
        const uint32_t b0 = sh == 0 || by_count ? b1 : min(sm.nb0, b1);
        if (sh == 0 || by_count) {
            ls = from;
#pragma unroll
            for (int j = 0; j < SP_BPT; ++j) {
                if (b1 == static_cast<uint32_t>(SP_BPT * tid + j)) {
                    sm.sel_before = ls;
                    sm.sel_cnt = n[j];
                    sm.sel_w = n[j] ? low[j] / n[j] : 1.0;
                }
                ls += low[j];
            }
            __syncthreads();
            if (sh == 0) {
                const uint32_t ties = sm.sel_cnt;
                const double need = ceil((target - sm.sel_before) / sm.sel_w);
                const uint32_t keep = need < 1.0 ? 1u : need >= static_cast<double>(ties) ? ties : static_cast<uint32_t>(need);
                const float tau = key_logit<TL>(khi - b1);
                dropped = keep < ties ? ties - keep : 0u;
                return composite(tau, dropped ? tie_index<TL>(sm, ck, rank, C, w, tau, keep) : -1);
            }
            A = sm.sel_before;
            khi -= b1 << sh;
            klo = khi - klo > span ? khi - span : klo;
            cluster_sync_warp0();   // the counts have been read
            continue;
        }
        // the sums before range b0, and of it
        const uint32_t top = khi - (b0 << sh), bot = top - klo > span ? top - span : klo;
        double before = 0.0, of = 0.0;
        each_in<TL>(sm, ck, w, [&](float l) {
            const uint32_t key = order_key(l) >> KSH;
            if (key < bot || key > khi) return;
            const double x = sc.weight(l);
            if (key > top) before += x;
            else of += x;
        });
        share_two(sm.rsum, before, sm.wsum, of, rank, C);
        before = table_sum(sm.rsum, C, lane);
        of = table_sum(sm.wsum, C, lane);
        A += before;
        if (A + of >= target || bot == klo || b0 == b1) {
            khi = top;
            klo = bot;
        } else {
            A += of;
            const uint32_t end = khi - (b1 << sh);
            khi = bot - 1;
            klo = end - klo > span ? end - span : klo;
        }
        // (every CTA has read the counts before share_two()'s barrier, and reads the tables before the next one)
        if constexpr (KSH == 0) {   // (a bf16 window has few values)
            if (!w.listed) continue;
            if (tid == 0) sm.nfew = 0;
            __syncthreads();
            for (uint32_t i = tid; i < w.mine; i += SP_THREADS) {
                const unsigned long long k = sm.loc[i];
                const uint32_t key = static_cast<uint32_t>(k >> 32) >> KSH;
                if (key < klo || key > khi) continue;
                const uint32_t at = atomicAdd(&sm.nfew, 1u);
                if (at < 32) sm.few[at] = k;
            }
            cluster_sync_warp0();
            uint32_t all = 0, cta = 0, slot = 0;   // where this lane's token is
            for (uint32_t c = 0; c < C; ++c) {
                uint32_t x;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(sp_mapa(&sm.nfew, c)) : "memory");
                if (static_cast<uint32_t>(lane) >= all) {
                    cta = c;
                    slot = lane - all;
                }
                all += x;
            }
            if (all == 0 || all > 32) continue;
            // the few in order (all different), their running weight on top of A
            const bool has = static_cast<uint32_t>(lane) < all;
            if (tid < 32) {
                unsigned long long k = 0;
                if (has) asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(sp_mapa(&sm.few[slot], cta)) : "memory");
                uint32_t before = 0;
    #pragma unroll
                for (int i = 0; i < 32; ++i) before += __shfl_sync(0xffffffffu, k, i) > k ? 1u : 0u;
                if (has) sm.lst[before] = k;
            }
            __syncthreads();
            const unsigned long long k = has ? sm.lst[lane] : 0ull;
            const double run = A + warp_scan(has ? sc.weight(composite_value(k)) : 0.0, lane);
            const unsigned reach = __ballot_sync(0xffffffffu, has && run >= target);
            const int end = reach ? __ffs(reach) - 1 : static_cast<int>(all) - 1;
            const unsigned long long cut = __shfl_sync(0xffffffffu, k, end);
            dropped = __popc(__ballot_sync(0xffffffffu, has && lane > end && k >> 32 == cut >> 32));
            return dropped ? cut : cut & 0xffffffff00000000ull;
        }
    }
}

// Index of the keep-th of this CTA's elements equal to tau.
template <typename TL>
__device__ int own_tie(SampleSmem& sm, const SpChunk<TL>& ck, float tau, uint32_t keep) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    auto ties_at = [&](int i) { return i < q1 ? tie_mask<TL>(ck, i, tau) : 0u; };
    uint32_t n = 0;
    for (int i = q0 + lane; i < q1; i += 32) n += __popc(ties_at(i));
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sm.wcnt[warp] = n;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += sm.wcnt[w];
    if (keep > before && keep <= before + n) {
        uint32_t left = keep - before;
        for (int i0 = q0; i0 < q1; i0 += 32) {
            uint32_t mask = ties_at(i0 + lane), t;
            const uint32_t mine = __popc(mask), ex = lanes_before(mine, lane, t);
            if (ex + mine >= left && ex < left) {
                for (uint32_t skip = left - ex - 1; skip; --skip) mask &= mask - 1;
                sm.last = ck.index(i0 + lane, __ffs(mask) - 1);
            }
            if (t >= left) break;
            left -= t;
        }
    }
    __syncthreads();
    return sm.last;
}

// The count table of every CTA to zero (one cluster barrier).
__device__ void clear_counts(SampleSmem& sm) {
    for (int i = threadIdx.x; i < SP_BINS; i += SP_THREADS) sm.cnt[i] = 0;
    cluster_sync_warp0();
}

// Masks this CTA's elements equal to tau behind index icut.
template <typename TL>
__device__ void mask_ties(const SpChunk<TL>& ck, float tau, int icut) {
    constexpr int VEC = SpElem<TL>::VEC;
    for (int q = max(0, icut + 1 - ck.begin + ck.mis) / VEC + threadIdx.x; q < ck.nvec; q += SP_THREADS) {
        if (!SpElem<TL>::any_eq(reinterpret_cast<const uint4*>(ck.buf)[q], tau)) continue;
        for (int e = 0; e < VEC; ++e)
            if (ck.index(q, e) > icut && static_cast<float>(ck.buf[q * VEC + e]) == tau) ck.buf[q * VEC + e] = SpElem<TL>::ninf();
    }
}

// This thread's sum of the weights at or above lo in intervals before b0.
template <typename TL>
__device__ double above_part(const SpChunk<TL>& ck, float lo, const SpBins& bins, uint32_t b0, const SpScale& sc) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    double s = 0.0;
    if (b0 > 0) {
        const float floor = bins.lower(b0 - 1, lo);
        const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(floor);
        for (int v0 = q0; v0 < q1; v0 += 32) {
            const uint4 raw = ck.raw_to(v0 + lane, q1);
            if (!__any_sync(0xffffffffu, SpElem<TL>::any_ge(raw, tb))) continue;
            float v[VEC];
            SpElem<TL>::unpack(raw, v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const bool in = v[e] >= floor && bins.of(v[e]) < b0;
                if (!__any_sync(0xffffffffu, in)) continue;
                const double w = sc.weight(v[e]);
                if (in) s += w;
            }
        }
    }
    return s;
}

// The same for the window's weights that are kept, after masking those of its
// ties at tau that are not.
template <typename TL>
__device__ double border_part(const SampleSmem& sm, const SpChunk<TL>& ck, const SpWindow& win, unsigned long long cut,
                              const SpScale& sc) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float tau = composite_value(cut);
    if (win.listed) {
        double s = 0.0;
        for (uint32_t i = win.start + lane; i < win.start + win.count; i += 32) {
            const unsigned long long k = sm.loc[i];
            if (k >= cut) s += sc.weight(composite_value(k));
            else if (k >> 32 == cut >> 32) ck.mask(composite_index(k));
        }
        return s;
    }
    if (static_cast<uint32_t>(cut) != 0) mask_ties<TL>(ck, tau, composite_index(cut));
    __syncthreads();
    const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(tau);
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    double s = 0.0;
    for (int v0 = q0; v0 < q1; v0 += 32) {
        const uint4 raw = ck.raw_to(v0 + lane, q1);
        if (!__any_sync(0xffffffffu, SpElem<TL>::any_ge(raw, tb))) continue;
        float v[VEC];
        SpElem<TL>::unpack(raw, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (v[e] >= tau && v[e] <= win.top && win.bins.of(v[e]) >= win.b0) s += sc.weight(v[e]);
    }
    return s;
}

// The row's part of probs: w / S in fp32, 0 below tau.
template <typename TL>
__device__ void write_probs(float* out, const SpChunk<TL>& ck, float tau, const SpScale& sc, const double* tab) {
    constexpr int VEC = SpElem<TL>::VEC;
    const typename SpElem<TL>::Bound tb = SpElem<TL>::bound(tau);
    const bool wide = ck.mis == 0 && (reinterpret_cast<uintptr_t>(out + ck.begin) & 15u) == 0;
    const int lane = threadIdx.x & 31;
    for (int v0 = (threadIdx.x >> 5) * 32; v0 < ck.nvec; v0 += SP_THREADS) {
        const int vq = v0 + lane;
        float p[VEC];
        const uint4 raw = ck.raw_to(vq, ck.nvec);
        if (__all_sync(0xffffffffu, SpElem<TL>::all_ge(raw, tb))) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) p[e] = static_cast<float>(sc.weight(SpElem<TL>::scaled(raw, e), tab));
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) p[e] = 0.f;
            if (__any_sync(0xffffffffu, SpElem<TL>::any_ge(raw, tb))) {
                float v[VEC];
                SpElem<TL>::unpack(raw, v);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (v[e] >= tau) p[e] = static_cast<float>(sc.weight(SpElem<TL>::scaled(raw, e), tab));
            }
        }
        const int i0 = vq * VEC - ck.mis;   // position in the part
        if (vq >= ck.nvec) continue;
        if (wide && i0 + VEC <= ck.n) {
#pragma unroll
            for (int e = 0; e < VEC; e += 4)
                *reinterpret_cast<float4*>(out + ck.begin + i0 + e) = make_float4(p[e], p[e + 1], p[e + 2], p[e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (i0 + e >= 0 && i0 + e < ck.n) out[ck.begin + i0 + e] = p[e];
        }
    }
}

// One cluster per row.  512 threads and half of an SM's shared memory per CTA:
// two of them overlap one row's barriers with the other's passes (CTAs of 256
// threads took 51 us against 45 then, on 64 rows with probs).  Copying the part
// once beats re-reading it from L2 in every pass: clusters of 1 or 2 that do so
// took 315 and 206 us on the 512 mixed rows, against 148 then.
template <typename TL, bool VERIFY>
__global__ void __launch_bounds__(SP_THREADS, 1024 / SP_THREADS) sample_kernel(const SampleArgs a) {
    constexpr int VEC = SpElem<TL>::VEC;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ SampleSmem sm;
    const uint32_t rank = cluster_rank(), C = a.cluster;
    const int row = blockIdx.x / a.cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 16) sm.tab[tid] = __hiloint2double(__double2hiint(exp2(tid / 16.0)) - (tid << 16), __double2loint(exp2(tid / 16.0)));
    for (int i = tid; i < SP_BINS; i += SP_THREADS) sm.cnt[i] = 0;
    cluster_arrive();   // waited for before the first store to another CTA: all have started then
    grid_dep_wait();
    grid_dep_launch();

    // ---- the row's parameters
    const int seq = VERIFY ? row / a.per : row, pj = VERIFY ? row % a.per : 0;
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
    r.us = fmax(fmin(r.us, 1.0 - 0x1p-24), 0.0);   // (NaN: the largest)

    // ---- the row's part into shared memory, and its maximum
    SpChunk<TL> ck;
    ck.buf = reinterpret_cast<TL*>(dyn);
    ck.begin = static_cast<int>(rank) * a.chunk;
    ck.n = max(0, min(a.chunk, a.V - ck.begin));
    const TL* rowp = static_cast<const TL*>(a.logits) + static_cast<size_t>(row) * a.V;
    const TL* g = rowp + ck.begin;
    ck.mis = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(TL));
    ck.nvec = ck.n > 0 ? (ck.mis + ck.n + VEC - 1) / VEC : 0;
    typename SpElem<TL>::Max tmax;
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
            tmax.add(r[j]);   // NaN operands are ignored
        }
    }
    const float mine = tmax.get();
    float m = mine, low = mine > -INFINITY ? mine : INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    if (lane == 0) {
        sm.wmax[warp] = m;
        sm.wmin[warp] = low;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < SP_WARPS; ++w) {
        m = fmaxf(m, sm.wmax[w]);
        low = fminf(low, sm.wmin[w]);
    }
    cluster_wait();
    if (tid < static_cast<int>(C)) {
        st_cluster_f32(&sm.cmax[rank], tid, m);
        st_cluster_f32(&sm.cmin[rank], tid, low);
    }
    cluster_sync_warp0();
    m = -INFINITY;
    low = INFINITY;
    for (uint32_t i = 0; i < C; ++i) {
        m = fmaxf(m, sm.cmax[i]);
        low = fminf(low, sm.cmin[i]);
    }
    T = fmin(fmax(T, 1e-30), static_cast<double>(FLT_MAX));
    const double c = 1.4426950408889634 / T;
    const SpScale sc{m, scaled_f64(m), c * 0x1p896, c, sm.tab};
    double dmin = -44.361419555836498 * T;   // 64 ln 2
    if (mp > 0.0) dmin = fmax(dmin, T * log(fmin(mp, 1.0)));
    float lcut = fmaxf(__double2float_ru(static_cast<double>(m) + dmin), -FLT_MAX);

    if (m == -INFINITY) {   // nothing can be drawn
        if (rank == 0 && tid == 0) a.token[row] = -1;
        if (!VERIFY && a.probs)
            for (int i = tid; i < ck.n; i += SP_THREADS) a.probs[static_cast<size_t>(row) * a.V + ck.begin + i] = 0.f;
        return;
    }

    // ---- few candidates: a list of them, finished by the leader
    uint32_t n = 0xffffffffu;
    uint32_t* ccnt = sm.ccnt[0];
    double S_all = -1.0;
    if (mp > 0.0) n = gather<TL>(sm, ccnt = sm.ccnt[0], ck, rank, C, lcut, [](float) { return true; });
    if (n > SP_CAP && r.by_k && r.k <= SP_CAP) {
        const float lo = kth_bound(sm, C, lcut, low, m, mine, static_cast<uint32_t>(r.k));
        n = gather<TL>(sm, ccnt = sm.ccnt[1], ck, rank, C, lo, [](float) { return true; });
    }
    SpNucleus nu{};
    if (n > SP_CAP && r.by_p && !r.by_k) {
        nu = nucleus<TL>(sm, ck, sc, rank, C, a.V, lcut, r.p, 0.0);
        S_all = nu.S;
        if (nu.n <= SP_CAP) {
            const SpBins bins = first_bins<TL>(sc, lcut);
            n = gather<TL>(sm, ccnt = sm.ccnt[1], ck, rank, C, bins.lower(nu.b1, lcut), [&](float l) { return bins.of(l) <= nu.b1; });
        }
    }
    bool counted = false;   // bf16: the border is known from counts
    SpKeys keys{};
    SpBorder kb{};
    if constexpr (SpElem<TL>::KSH == 16) {
        if (n > SP_CAP && (r.by_k || r.by_p)) {
            const float lo = r.by_k ? lcut : first_bins<TL>(sc, lcut).lower(nu.b1, lcut);
            keys = make_keys(m, __bfloat162float(__float2bfloat16_ru(lo)));
            // (not with a cut or a certain draft among the collapsed values)
            bool can = !keys.mixed(keys.n - 1);
            if (VERIFY && r.x >= 0 && !r.q) can = can && !keys.mixed(keys.rank(static_cast<float>(rowp[r.x])));
            if (can) kb = key_border(sm, ck, sc, keys, rank, C, lo, r.by_k ? static_cast<uint32_t>(r.k) : 0u, r.p, nu.S);
            counted = can && kb.ok;
            if (counted) {   // what is left is to keep the first tokens down to the border
                lcut = keys.value(kb.r);
                r.by_p = false;
                r.by_k = kb.keep < kb.ties;
                r.k = static_cast<int>(kb.above + kb.keep);
                if (kb.above + kb.ties <= SP_CAP)
                    n = gather<TL>(sm, ccnt = sm.ccnt[2], ck, rank, C, lcut, [](float) { return true; });
            }
        }
    }
    if (n <= SP_CAP) {
        if (rank == 0) {
            pull_list(sm, ccnt, static_cast<int>(n));
        }
        cluster_sync_warp0();   // the other CTAs' lists have been read
        if (rank == 0)
            draw_from_list<VERIFY>(sm, static_cast<int>(n), SpElem<TL>::KSH, lcut, sc, r, S_all, a.token + row);
        if (VERIFY || !a.probs) return;
        if (rank == 0) {
            __syncthreads();
            if (tid < static_cast<int>(C)) {
                st_cluster_u64(&sm.list_cut, tid, sm.list_cut);
                st_cluster_f64(&sm.list_sum, tid, sm.list_sum);
            }
        }
        cluster_sync_warp0();
    }

    // ---- many: the border of the kept set by selection over the whole row, then sums and the draw
    float tau = lcut;              // kept: logits at or above tau; ties that are not are masked
    double S = 0.0;
    if (n <= SP_CAP) {
        S = sm.list_sum;
        tau = composite_value(sm.list_cut);
        if (static_cast<uint32_t>(sm.list_cut) != 0) {   // else all ties are kept
            mask_ties<TL>(ck, tau, composite_index(sm.list_cut));
            __syncthreads();
        }
    } else {
        bool summed = false;           // wsum holds the kept weights' sums
        uint32_t kept = 0;             // counted: the border's ties that this CTA keeps,
        uint32_t rx = 0xffffffffu;     // and the value of the certain draft, where it has that
        if (counted) {
            const uint32_t* hist = reinterpret_cast<const uint32_t*>(sm.lst);
            kept = hist[kb.r];
            if (r.by_k) {   // the first ones in index order
                uint32_t before = 0;
                for (uint32_t j = 0; j < rank; ++j) {
                    uint32_t x;
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(sp_mapa(&hist[kb.r], j)) : "memory");
                    before += x;
                }
                const uint32_t own = kept;
                kept = min(own, kb.keep - min(kb.keep, before));
                if (kept < own) {
                    mask_ties<TL>(ck, tau, kept > 0 ? own_tie<TL>(sm, ck, tau, kept) : ck.begin - 1);
                    __syncthreads();
                }
            }
        } else if (r.by_k || r.by_p) {
            unsigned long long cut = 0;
            uint32_t dropped = 0;   // ties of the k-th token that top-k leaves behind
            if (r.by_k) {
                clear_counts(sm);
                const SpKth kt = kth_interval<TL>(sm, ck, sc, C, lcut, static_cast<uint32_t>(r.k));
                const SpBins bins = first_bins<TL>(sc, lcut);
                const SpWindow win = make_window<TL>(sm, sm.ccnt[2], ck, rank, C, lcut, bins, kt.b, kt.b);
                cut = composite(lcut, -1);   // (fewer than k)
                if (win.all) {
                    cut = refine<TL>(sm, ck, sc, rank, C, win, true, static_cast<double>(kt.above), static_cast<double>(r.k), dropped);
                }
            }
            if (r.by_p) {
                const float kth = r.by_k ? composite_value(cut) : lcut;
                if (r.by_k) {
                    if (!dropped) cluster_sync_warp0();   // the other CTAs have read refine()'s counts (tie_index() waits too)
                    clear_counts(sm);
                    nu = nucleus<TL>(sm, ck, sc, rank, C, a.V, kth, r.p, static_cast<double>(dropped) * sc.weight(kth));
                }
                // the border lies in intervals b0..b1: the sum above them, then token by token
                const double target = fmax(r.p * nu.S, 1e-9);
                const SpBins bins = first_bins<TL>(sc, kth);
                const double mine_above = above_part<TL>(ck, kth, bins, nu.b0, sc);
                share_sums(sm.rsum, mine_above, rank, C);
                const double A = table_sum(sm.rsum, C, lane);
                const SpWindow win = make_window<TL>(sm, sm.ccnt[3], ck, rank, C, kth, bins, nu.b0, nu.b1);
                uint32_t behind;
                cut = max(cut, refine<TL>(sm, ck, sc, rank, C, win, false, A, target, behind));
                tau = composite_value(cut);
                const double mine_border = border_part<TL>(sm, ck, win, cut, sc);
                share_sums(sm.wsum, mine_above + mine_border, rank, C);
                summed = true;
            } else {
                tau = composite_value(cut);
                if (static_cast<uint32_t>(cut) != 0) mask_ties<TL>(ck, tau, composite_index(cut));
                __syncthreads();
            }
        }
        double wx = 0.0;
        if (r.x >= 0) {
            // the draft's weight, where it is kept, from the one CTA that holds it; a certain draft leaves the others
            const int i = r.x - ck.begin;
            if (i >= 0 && i < ck.n) {
                const float l = static_cast<float>(ck.buf[ck.mis + i]);
                const double w = l >= tau ? sc.weight(l) : 0.0;
                if (counted && !r.q && w > 0.0) rx = keys.rank(l);
                __syncthreads();
                if (tid == 0) {
                    for (uint32_t j = 0; j < C; ++j) st_cluster_f64(&sm.wx, j, w);
                    if (!r.q) ck.mask(r.x);
                }
            }
            if (summed) cluster_sync_warp0();
            else __syncthreads();
        }
        if (counted) share_sums(sm.wsum, key_sum(sm, sc, keys, kb, kept, rx), rank, C);
        else if (!summed) share_sums(sm.wsum, segment_part<TL>(ck, tau, sc), rank, C);
        if (r.x >= 0) wx = sm.wx;
        if (summed && wx > 0.0 && !r.q) {
            // the draft's segment without it
            const int c = r.x / a.chunk, first = c * a.chunk;
            const TL* part = rowp + first;
            const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(part) & 15u) / sizeof(TL));
            const int vecs = (mis + min(a.chunk, a.V - first) + VEC - 1) / VEC, per = ((vecs + SP_WARPS - 1) / SP_WARPS + 31) & ~31;
            const int seg = c * SP_WARPS + (mis + r.x - first) / VEC / per;
            __syncthreads();
            if (tid == 0) sm.wsum[seg] = fmax(0.0, sm.wsum[seg] - wx);
            __syncthreads();
        }
        const double rest = table_sum(sm.wsum, C, lane);
        S = r.has_draft && !r.q ? rest + wx : rest;
        if (r.has_draft) {
            const double qx = r.q ? (r.x >= 0 ? static_cast<double>(__ldg(r.q + r.x)) : 0.0) : 1.0;
            if (wx > 0.0 && r.ua * qx * S < wx) {
                if (rank == 0 && tid == 0) a.token[row] = SP_ACCEPTED;
                return;
            }
        }
        int tok = -1;
        const double* sums = sm.wsum;
        int nseg = static_cast<int>(C) * SP_WARPS, own_seg = static_cast<int>(rank) * SP_WARPS + warp;
        double target = r.us * rest;
        const float* q = nullptr;
        if (r.q) {
            residual_sums<TL>(sm.rsum, ck, rank, C, tau, sc, r.q, S * 0x1p896);
            const double left = table_sum(sm.rsum, C, lane);
            if (left > 0.0) {
                sums = sm.rsum;
                target = r.us * left;
                q = r.q;
            }
        }
        if (counted && !q && rest > 0.0) {
            // the table has sums per CTA only: the one that the draw falls to sums its segments
            double base = 0.0, first = 0.0, end = 0.0;
            int owner = -1;
            for (uint32_t j = 0; j < C; ++j) {
                const double x = warp_sum_f64(lane < SP_WARPS ? sm.wsum[j * SP_WARPS + lane] : 0.0);
                if (x > 0.0 && (owner < 0 || end <= target)) {
                    owner = static_cast<int>(j);
                    first = base;
                    end = base + x;
                }
                base += x;
            }
            own_seg = -2;   // (no segment of the others)
            if (owner == static_cast<int>(rank)) {
                double* own = sm.rsum + rank * SP_WARPS;
                __syncthreads();
                const double x = warp_sum_f64(segment_part<TL>(ck, tau, sc));
                if (lane == 0) own[warp] = x;
                __syncthreads();
                sums = own;
                nseg = SP_WARPS;
                own_seg = warp;
                target -= first;
            }
        }
        if (q || rest > 0.0) {
            if (own_seg >= 0) tok = draw_token<TL>(sums, nseg, own_seg, ck, tau, sc, q, S * 0x1p896, target);
        } else if (rank == 0 && warp == 0) {
            tok = r.x;   // the draft is the only token kept
        }
        if (tok >= 0 && lane == 0) a.token[row] = tok;
    }
    if (!VERIFY && a.probs) {
        // 2^(j/16) / S: sums of high words stay within the exponent's range, as probabilities are normal numbers
        if (tid < 16) {
            const double x = exp2(tid / 16.0) / S;
            sm.ptab[tid] = __hiloint2double(__double2hiint(x) - (tid << 16), __double2loint(x));
        }
        __syncthreads();
        write_probs<TL>(a.probs + static_cast<size_t>(row) * a.V, ck, tau, sc, sm.ptab);
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
    // The smallest cluster whose parts leave room for two CTAs per SM, then
    // wider while all rows still run at once.  At V = 129,280 one bf16 row takes
    // 8.5 us on 4 CTAs and 7.7 on 8, 512 rows 131 us on 4 and 193 on 8; 42 fp32 rows
    // of 32,003 take 35 us on 2, 24 on 4 and 29 on 8.
    const int eb = dt == MS_BF16 ? 2 : 4;
    int C = 1;
    while (C < SP_MAXC && (static_cast<long>(a.V) * eb > 66L * 1024 * C || a.V > SP_MAX_CHUNK * C)) C *= 2;
    while (C < SP_MAXC && a.V > 1024 * C && 2L * C * a.rows <= 2L * num_sms()) C *= 2;
    a.cluster = C;
    a.chunk = ((a.V + C - 1) / C + 7) / 8 * 8;
    if (dt == MS_BF16)
        return verify ? sample_launch_t<__nv_bfloat16, true>(a, s) : sample_launch_t<__nv_bfloat16, false>(a, s);
    return verify ? sample_launch_t<float, true>(a, s) : sample_launch_t<float, false>(a, s);
}

// Rows and vocabulary that one launch can take.
static bool sample_size_ok(long rows, int V) { return V <= SP_MAX_V && rows <= (1L << 24); }

// Every pointer of a call at a multiple of its element (a load elsewhere would fault).
static bool sample_aligned(const SampleArgs& a, ms_dtype dt) {
    return element_aligned(a.logits, dt) && words_aligned(a.temperature, a.top_p, a.min_p, a.u, a.top_k, a.draft, a.q,
                                                          a.token, a.probs);
}

}  // namespace ms

extern "C" ms_status spec_sample(const void* logits, ms_dtype logits_dtype, int T, int V, const float* temperature,
                                 const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                                 int32_t* token, float* probs, void* stream) {
    if (!logits || !u || !token) return MS_ERR_INVALID_ARG;
    if (T <= 0 || V <= 0) return MS_ERR_INVALID_ARG;
    if (logits_dtype != MS_F32 && logits_dtype != MS_BF16) return MS_ERR_INVALID_ARG;
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
    if (!ms::sample_aligned(a, logits_dtype)) return MS_ERR_INVALID_ARG;
    if (!ms::sample_size_ok(T, V)) return MS_ERR_UNSUPPORTED;
    return ms::sample_launch(a, logits_dtype, false, static_cast<cudaStream_t>(stream));
}

extern "C" ms_status spec_verify_sample(const void* logits, ms_dtype logits_dtype, const int32_t* draft,
                                        const float* draft_probs, const float* temperature, const int32_t* top_k,
                                        const float* top_p, const float* min_p, const float* u, int B, int K, int V,
                                        int32_t* committed, int32_t* n_committed, void* stream) {
    if (!logits || (K > 0 && !draft) || !u || !committed || !n_committed) return MS_ERR_INVALID_ARG;
    if (B <= 0 || V <= 0 || K < 0) return MS_ERR_INVALID_ARG;
    if (logits_dtype != MS_F32 && logits_dtype != MS_BF16) return MS_ERR_INVALID_ARG;
    ms::SampleArgs a{};
    a.logits = logits;
    a.V = V;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.draft = draft;
    a.q = K > 0 ? draft_probs : nullptr;
    a.token = committed;
    if (!ms::sample_aligned(a, logits_dtype) || !ms::words_aligned(n_committed)) return MS_ERR_INVALID_ARG;
    if (K > 8 || !ms::sample_size_ok(static_cast<long>(B) * (K + 1), V)) return MS_ERR_UNSUPPORTED;
    a.rows = B * (K + 1);
    a.per = K + 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const ms_status st = ms::sample_launch(a, logits_dtype, true, s);
    if (st != MS_OK) return st;
    return ms::launch(ms::K_SAMPLE_COMMIT, ms::sample_commit_kernel, dim3((B + 127) / 128), dim3(128), 0, s,
                      draft, B, K, committed, n_committed);
}
