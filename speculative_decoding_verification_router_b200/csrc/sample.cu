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
#include <math.h>

#include "ms_common.cuh"

namespace ms {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_MAXC = 8;              // CTAs of a row's cluster
constexpr int SP_MAX_CHUNK = 32768;     // elements of a row per CTA (bounds the histogram limbs)
constexpr int SP_BINS = 1024;
constexpr int SP_MAX_V = SP_MAXC * SP_MAX_CHUNK;
constexpr int SP_FIX = 45;              // fixed point of histogram masses: 2^18 weights of 1 fit 63 bits
constexpr int SP_LIMB = 15;             // 3 limbs; 2^15 elements x 2^15 fit a 32-bit counter
static_assert(SP_BINS == 2 * SP_THREADS, "the bin scan gives every thread two bins");

struct SampleArgs {
    const void* logits;         // [rows, V]
    int V, rows, chunk, cluster;
    int per;                    // rows that share one entry of the parameters (K + 1; 1 for plain sampling)
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    const int32_t* draft;       // verify: [rows / per, per - 1]
    const float* q;             // verify: [rows / per, per - 1, V] or NULL (the draft is certain)
    int32_t* token;             // [rows]
    int32_t* accepted;          // verify: [rows]
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

struct SampleSmem {
    double tab[16];
    double wsum[SP_MAXC * SP_WARPS];          // every warp's sum, of every CTA of the cluster
    double rsum[SP_MAXC * SP_WARPS];          // the same for the residual pass
    unsigned long long mass[SP_BINS];         // leader: masses pushed by the other CTAs
    unsigned long long scan[SP_WARPS];
    unsigned long long sel_above;             // broadcast results of a selection round
    uint32_t cnt[SP_BINS];
    uint32_t limb[3][SP_BINS];
    float cmax[SP_MAXC];
    uint32_t tie[SP_MAXC];
    uint32_t wcnt[SP_WARPS];
    uint32_t sel_bin, sel_cnt;
    uint32_t cut_idx;                         // broadcast: index of the last tied token kept
    int last;
};

// Where a CTA's part of the row sits: element i (row index begin + i) is
// buf[mis + i]; positions outside [mis, mis + n) hold -inf.
template <typename TL>
struct SpChunk {
    TL* buf;
    int mis, n, nvec, begin;
};

// A selected set: logits >= lcut whose composite key (order, lower index first)
// is at least `cut`.
struct SpCut {
    float lcut;
    unsigned long long cut;
};
__device__ __forceinline__ unsigned long long composite(uint32_t key, int idx) {
    return (static_cast<unsigned long long>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(idx));
}

// One selection round trip: histogram of the cluster's elements with keys in
// [klo, khi] over up to SP_BINS equal key intervals, counts always and masses
// (fixed point) when MASS; the leader finds the first interval, from the
// largest keys down, where `above` + the running total reaches the target.
// Repeats on that interval until it is a single key.  Every thread of every
// CTA of the cluster calls this with the same arguments.
template <typename TL, bool MASS>
__device__ void radix_select(SampleSmem& sm, const SpChunk<TL>& ck, uint32_t rank, uint32_t C, uint32_t klo,
                             uint32_t khi, float lcut, double md, double c, double target, uint32_t& key_out,
                             unsigned long long& above_out, uint32_t& cnt_out) {
    constexpr int VEC = SpElem<TL>::VEC, KSH = SpElem<TL>::KSH;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned long long above = 0;
    const uint4* bv = reinterpret_cast<const uint4*>(ck.buf);
    while (true) {
        int sh = 0;
        while (((khi - klo) >> sh) >= SP_BINS) ++sh;
        for (int i = tid; i < SP_BINS; i += SP_THREADS) {
            sm.cnt[i] = 0;
            if (MASS) {
                sm.limb[0][i] = sm.limb[1][i] = sm.limb[2][i] = 0;
                sm.mass[i] = 0;
            }
        }
        if (tid == 0) sm.last = 0;
        cluster_sync_all();   // the leader's tables are clear before anyone adds to them
        for (int q = tid; q < ck.nvec; q += SP_THREADS) {
            float v[VEC];
            SpElem<TL>::unpack(bv[q], v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (!(v[e] >= lcut)) continue;
                const uint32_t key = order_key(v[e]) >> KSH;
                if (key < klo || key > khi) continue;
                const uint32_t bin = (khi - key) >> sh;
                atomicAdd(&sm.cnt[bin], 1u);
                if (MASS) {
                    const double w = exp2_64((bits_to_f64(__float_as_uint(v[e])) - md) * c, sm.tab);
                    const unsigned long long W = __double2ull_rn(w * static_cast<double>(1ull << SP_FIX));
                    atomicAdd(&sm.limb[0][bin], static_cast<uint32_t>(W) & ((1u << SP_LIMB) - 1));
                    atomicAdd(&sm.limb[1][bin], static_cast<uint32_t>(W >> SP_LIMB) & ((1u << SP_LIMB) - 1));
                    atomicAdd(&sm.limb[2][bin], static_cast<uint32_t>(W >> (2 * SP_LIMB)));
                }
            }
        }
        __syncthreads();
        if (rank != 0) {
            for (int i = tid; i < SP_BINS; i += SP_THREADS) {
                if (sm.cnt[i] == 0) continue;
                if (MASS)
                    red_cluster_u64(&sm.mass[i], 0,
                                    sm.limb[0][i] + (static_cast<unsigned long long>(sm.limb[1][i]) << SP_LIMB) +
                                        (static_cast<unsigned long long>(sm.limb[2][i]) << (2 * SP_LIMB)));
                red_cluster_u32(&sm.cnt[i], 0, sm.cnt[i]);
            }
        }
        cluster_sync_all();
        if (rank == 0) {
            unsigned long long v[2];
            uint32_t n[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = 2 * tid + j;
                n[j] = sm.cnt[i];
                v[j] = n[j];
                if (MASS)
                    v[j] = sm.mass[i] + sm.limb[0][i] + (static_cast<unsigned long long>(sm.limb[1][i]) << SP_LIMB) +
                           (static_cast<unsigned long long>(sm.limb[2][i]) << (2 * SP_LIMB));
                if (n[j]) atomicMax(&sm.last, i);
            }
            const unsigned long long own = v[0] + v[1];
            const unsigned long long inc = warp_scan(own, lane);
            if (lane == 31) sm.scan[warp] = inc;
            __syncthreads();
            unsigned long long ex = above + inc - own;
            for (int w = 0; w < warp; ++w) ex += sm.scan[w];
            unsigned long long tot = above;
            for (int w = 0; w < SP_WARPS; ++w) tot += sm.scan[w];
            // the last occupied interval where rounding left the target above the total
            const bool never = static_cast<double>(tot) < target;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool hit = never ? 2 * tid + j == sm.last
                                       : n[j] && static_cast<double>(ex) < target &&
                                             static_cast<double>(ex + v[j]) >= target;
                if (hit)
                    for (uint32_t r = 0; r < C; ++r) {
                        st_cluster_s32(&sm.sel_bin, r, 2 * tid + j);
                        st_cluster_s32(&sm.sel_cnt, r, static_cast<int>(n[j]));
                        st_cluster_u64(&sm.sel_above, r, ex);
                    }
                ex += v[j];
            }
        }
        cluster_sync_all();
        above = sm.sel_above;
        khi -= sm.sel_bin << sh;
        const uint32_t span = (1u << sh) - 1;
        klo = khi - klo > span ? khi - span : klo;
        if (sh == 0) {
            key_out = khi;
            above_out = above;
            cnt_out = sm.sel_cnt;
            return;
        }
    }
}

// Index range of a warp's part of the chunk, in 16-byte vectors: contiguous,
// so that (warp, step, lane, element) runs in index order.
__device__ __forceinline__ void warp_segment(int nvec, int warp, int& q0, int& q1) {
    const int per = ((nvec + SP_WARPS - 1) / SP_WARPS + 31) & ~31;
    q0 = min(nvec, warp * per);
    q1 = min(nvec, q0 + per);
}

// The weight of one element under a cut, and of the residual max(w - q S, 0)
// where the row's draft probabilities are given.
template <typename TL>
__device__ __forceinline__ double kept_weight(float l, int idx, const SpCut& cut, double md, double c, int skip,
                                              const float* q, double S, const double* tab) {
    if (!(l >= cut.lcut) || idx == skip) return 0.0;
    if (composite(order_key(l) >> SpElem<TL>::KSH, idx) < cut.cut) return 0.0;
    const double w = exp2_64((bits_to_f64(__float_as_uint(l)) - md) * c, tab);
    if (!q) return w;
    const double r = w - static_cast<double>(__ldg(q + idx)) * S;
    return r > 0.0 ? r : 0.0;
}

// Sum of every warp's kept weights into sums[cta][warp] of every CTA (one
// cluster barrier).
template <typename TL>
__device__ void segment_sums(SampleSmem& sm, double* sums, const SpChunk<TL>& ck, uint32_t rank, uint32_t C,
                             const SpCut& cut, double md, double c, int skip, const float* q, double S) {
    constexpr int VEC = SpElem<TL>::VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint4* bv = reinterpret_cast<const uint4*>(ck.buf);
    int q0, q1;
    warp_segment(ck.nvec, warp, q0, q1);
    double s = 0.0;
    for (int v0 = q0 + lane; v0 < q1; v0 += 32) {
        float v[VEC];
        SpElem<TL>::unpack(bv[v0], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            s += kept_weight<TL>(v[e], ck.begin + v0 * VEC + e - ck.mis, cut, md, c, skip, q, S, sm.tab);
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

// The draw: the first index whose cumulative weight exceeds u times the total.
// Returns the token in lane 0 of the warp that owns it, -1 elsewhere.
template <typename TL>
__device__ int draw_token(SampleSmem& sm, const double* sums, const SpChunk<TL>& ck, uint32_t rank, uint32_t C,
                          const SpCut& cut, double md, double c, int skip, const float* q, double S, double u) {
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
    const uint4* bv = reinterpret_cast<const uint4*>(ck.buf);
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
            SpElem<TL>::unpack(bv[vq], v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                w[e] = kept_weight<TL>(v[e], ck.begin + vq * VEC + e - ck.mis, cut, md, c, skip, q, S, sm.tab);
                s += w[e];
                if (w[e] > 0.0) mine = ck.begin + vq * VEC + e - ck.mis;
            }
        }
        const double in = warp_scan(s, lane);
        const unsigned pass = __ballot_sync(0xffffffffu, s > 0.0 && base + in > target);
        if (pass) {
            int tok = mine;
            double acc = base + in - s;
#pragma unroll
            for (int e = VEC - 1; e >= 0; --e) {
                // from the back: the lowest element whose running sum exceeds the target stays
                double before = acc;
#pragma unroll
                for (int f = 0; f < e; ++f) before += w[f];
                if (w[e] > 0.0 && before + w[e] > target) tok = ck.begin + vq * VEC + e - ck.mis;
            }
            return __shfl_sync(0xffffffffu, tok, __ffs(pass) - 1);
        }
        const unsigned have = __ballot_sync(0xffffffffu, mine >= 0);
        if (have) last = __shfl_sync(0xffffffffu, mine, 31 - __clz(have));
        base += __shfl_sync(0xffffffffu, in, 31);
    }
    return last;
}

template <typename TL, bool VERIFY>
__global__ void __launch_bounds__(SP_THREADS) sample_kernel(const SampleArgs a) {
    constexpr int VEC = SpElem<TL>::VEC, KSH = SpElem<TL>::KSH;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ SampleSmem sm;
    const uint32_t rank = cluster_rank(), C = a.cluster;
    const int row = blockIdx.x / a.cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 16) sm.tab[tid] = exp2(static_cast<double>(tid) / 16.0);
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
    float m = -INFINITY;
    for (int q = tid; q < ck.nvec; q += SP_THREADS) {
        const int s0 = q * VEC;
        uint4 r;
        if (s0 >= ck.mis && s0 + VEC <= ck.mis + ck.n) {
            r = __ldg(reinterpret_cast<const uint4*>(g + (s0 - ck.mis)));
        } else {
            TL t[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                t[e] = s0 + e >= ck.mis && s0 + e < ck.mis + ck.n ? g[s0 + e - ck.mis] : SpElem<TL>::ninf();
            memcpy(&r, t, 16);
        }
        reinterpret_cast<uint4*>(ck.buf)[q] = r;
        float v[VEC];
        SpElem<TL>::unpack(r, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) m = fmaxf(m, v[e]);   // a NaN operand is ignored
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sm.wsum[warp] = m;
    __syncthreads();
    if (warp == 0) {
        m = lane < SP_WARPS ? static_cast<float>(sm.wsum[lane]) : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane < static_cast<int>(C)) st_cluster_f32(&sm.cmax[rank], lane, m);
    }
    cluster_sync_all();
    m = -INFINITY;
    for (uint32_t r = 0; r < C; ++r) m = fmaxf(m, sm.cmax[r]);

    // ---- the row's parameters
    const int pr = row / a.per, pj = row % a.per;
    double T = a.temperature ? static_cast<double>(__ldg(a.temperature + pr)) : 1.0;
    int k = a.top_k ? __ldg(a.top_k + pr) : 0;
    double p = a.top_p ? static_cast<double>(__ldg(a.top_p + pr)) : 2.0;
    double mp = a.min_p ? static_cast<double>(__ldg(a.min_p + pr)) : 0.0;
    if (!(T > 0.0)) {   // greedy
        T = 1.0;
        k = 1;
        p = 2.0;
        mp = 0.0;
    }
    const bool by_k = k > 0 && k < a.V;
    const bool by_p = p < 1.0;
    const double c = 1.4426950408889634 / T;
    const double md = bits_to_f64(__float_as_uint(m));
    double dmin = -44.361419555836498 * T;   // 64 ln 2
    if (mp > 0.0) dmin = fmax(dmin, T * log(fmin(mp, 1.0)));
    SpCut cut;
    cut.lcut = fmaxf(__double2float_ru(static_cast<double>(m) + dmin), -FLT_MAX);
    cut.cut = 0;

    const bool has_draft = VERIFY && pj < a.per - 1;
    if (m == -INFINITY) {   // nothing can be drawn
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (VERIFY) a.accepted[row] = 0;
        }
        if (!VERIFY && a.probs)
            for (int i = tid; i < ck.n; i += SP_THREADS) a.probs[static_cast<size_t>(row) * a.V + ck.begin + i] = 0.f;
        return;
    }

    // ---- top-k and top-p: the composite key of the last token kept
    if (by_k || by_p) {
        const uint32_t klo = order_key(cut.lcut) >> KSH, khi = order_key(m) >> KSH;
        uint32_t key = 0, ties = 0;   // the border key, and how many tokens have it
        unsigned long long keep = 0;  // how many of those are kept
        unsigned long long above = 0;
        uint32_t lo = klo;
        double S = 0.0;
        bool cutting = false;
        if (by_k) {
            radix_select<TL, false>(sm, ck, rank, C, klo, khi, cut.lcut, md, c, static_cast<double>(k), key, above,
                                    ties);
            const unsigned long long want = static_cast<unsigned long long>(k) - min(above, static_cast<unsigned long long>(k));
            keep = min(want, static_cast<unsigned long long>(ties));
            lo = key;
            cutting = true;
        }
        if (by_p) {
            // the sum over the top-k tokens: everything above the border key, and its kept ties
            SpCut all = cut;
            if (by_k) all.cut = (static_cast<unsigned long long>(key) + 1) << 32;
            segment_sums<TL>(sm, sm.wsum, ck, rank, C, all, md, c, -1, nullptr, 0.0);
            S = table_sum(sm.wsum, C, lane);
            if (by_k) {
                const float lk = key_value(KSH ? (key << KSH) | ((key >> 15) ? 0u : 0xffffu) : key);
                S += static_cast<double>(keep) * exp2_64((bits_to_f64(__float_as_uint(lk)) - md) * c, sm.tab);
            }
            const double target = fmax(p * S, 1e-9);
            const uint32_t kkey = key;
            const unsigned long long kkeep = keep;
            radix_select<TL, true>(sm, ck, rank, C, lo, khi, cut.lcut, md, c,
                                   target * static_cast<double>(1ull << SP_FIX), key, above, ties);
            const float lp = key_value(KSH ? (key << KSH) | ((key >> 15) ? 0u : 0xffffu) : key);
            const double wp = exp2_64((bits_to_f64(__float_as_uint(lp)) - md) * c, sm.tab);
            const double need = ceil((target - static_cast<double>(above) / static_cast<double>(1ull << SP_FIX)) / wp);
            keep = need < 1.0 ? 1 : need >= static_cast<double>(ties) ? ties : static_cast<unsigned long long>(need);
            if (by_k && key == kkey) keep = min(keep, kkeep);
            cutting = true;
        }
        if (cutting) {
            cut.cut = static_cast<unsigned long long>(key) << 32;
            if (keep < ties) {
                // the index of the keep-th token with the border key, in index order
                int q0, q1;
                warp_segment(ck.nvec, warp, q0, q1);
                const uint4* bv = reinterpret_cast<const uint4*>(ck.buf);
                uint32_t n = 0;
                for (int v0 = q0 + lane; v0 < q1; v0 += 32) {
                    float v[VEC];
                    SpElem<TL>::unpack(bv[v0], v);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) n += v[e] >= cut.lcut && (order_key(v[e]) >> KSH) == key;
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
                    uint32_t left = static_cast<uint32_t>(keep) - before;   // 1-based
                    for (int v0 = q0; v0 < q1; v0 += 32) {
                        uint32_t mask = 0;
                        if (v0 + lane < q1) {
                            float v[VEC];
                            SpElem<TL>::unpack(bv[v0 + lane], v);
#pragma unroll
                            for (int e = 0; e < VEC; ++e)
                                mask |= (v[e] >= cut.lcut && (order_key(v[e]) >> KSH) == key ? 1u : 0u) << e;
                        }
                        const uint32_t mine = __popc(mask);
                        const uint32_t in = warp_scan(mine, lane);
                        if (in >= left && in - mine < left) {
                            uint32_t skip = left - (in - mine) - 1;
                            while (skip--) mask &= mask - 1;
                            const int idx = ck.begin + (v0 + lane) * VEC + (__ffs(mask) - 1) - ck.mis;
                            for (uint32_t r = 0; r < C; ++r) st_cluster_s32(&sm.cut_idx, r, idx);
                        }
                        const uint32_t t = __shfl_sync(0xffffffffu, in, 31);
                        if (t >= left) break;
                        left -= t;
                    }
                }
                cluster_sync_all();
                cut.cut = composite(key, static_cast<int>(sm.cut_idx));
            }
        }
    }

    // ---- sums, acceptance of the draft, the draw
    const int seq = row / a.per;
    int x = -1;
    double wx = 0.0;
    const float* q = nullptr;
    if (has_draft) {
        x = __ldg(a.draft + static_cast<size_t>(seq) * (a.per - 1) + pj);
        if (x < 0 || x >= a.V) x = -1;
        if (a.q) q = a.q + (static_cast<size_t>(seq) * (a.per - 1) + pj) * a.V;
        if (x >= 0)
            wx = kept_weight<TL>(SpElem<TL>::load(rowp + x), x, cut, md, c, -1, nullptr, 0.0, sm.tab);
    }
    const int skip = has_draft && !q ? x : -1;   // a certain draft leaves the others
    segment_sums<TL>(sm, sm.wsum, ck, rank, C, cut, md, c, skip, nullptr, 0.0);
    const double rest = table_sum(sm.wsum, C, lane);
    const double S = skip >= 0 ? rest + wx : rest;
    if (has_draft) {
        const double ua = static_cast<double>(__ldg(a.u + static_cast<size_t>(seq) * a.per + pj));
        const double qx = q ? (x >= 0 ? static_cast<double>(__ldg(q + x)) : 0.0) : 1.0;
        if (x >= 0 && ua * qx * S < wx) {
            if (rank == 0 && tid == 0) {
                a.token[row] = x;
                a.accepted[row] = 1;
            }
            cluster_sync_all();
            return;
        }
    }
    const double us = static_cast<double>(VERIFY ? __ldg(a.u + static_cast<size_t>(seq) * a.per + a.per - 1) : __ldg(a.u + row));
    int tok = -1;
    if (q) {
        segment_sums<TL>(sm, sm.rsum, ck, rank, C, cut, md, c, -1, q, S);
        const bool left = table_sum(sm.rsum, C, lane) > 0.0;
        if (left) tok = draw_token<TL>(sm, sm.rsum, ck, rank, C, cut, md, c, -1, q, S, us);
        else tok = draw_token<TL>(sm, sm.wsum, ck, rank, C, cut, md, c, -1, nullptr, 0.0, us);
    } else if (rest > 0.0) {
        tok = draw_token<TL>(sm, sm.wsum, ck, rank, C, cut, md, c, skip, nullptr, 0.0, us);
    } else if (rank == 0 && warp == 0) {
        tok = x;   // the draft is the only token kept
    }
    if (tok >= 0 && lane == 0) {
        a.token[row] = tok;
        if (VERIFY) a.accepted[row] = 0;
    }
    if (!VERIFY && a.probs) {
        float* out = a.probs + static_cast<size_t>(row) * a.V + ck.begin;
        const double inv = 1.0 / S;
        for (int i = tid; i < ck.n; i += SP_THREADS) {
            const float l = static_cast<float>(ck.buf[ck.mis + i]);
            out[i] = static_cast<float>(kept_weight<TL>(l, ck.begin + i, cut, md, c, -1, nullptr, 0.0, sm.tab) * inv);
        }
    }
    cluster_sync_all();   // no CTA leaves while another may still write to its shared memory
}

// The verification's last step, one thread per sequence: accepted drafts up to
// the first rejection, then the token drawn at that position.
__global__ void __launch_bounds__(128) sample_commit_kernel(const int32_t* __restrict__ token,
                                                            const int32_t* __restrict__ accepted, int B, int K,
                                                            int32_t* __restrict__ committed,
                                                            int32_t* __restrict__ n_committed) {
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= B) return;
    const size_t base = static_cast<size_t>(b) * (K + 1);
    int n = 0;
    while (n < K && accepted[base + n]) ++n;
    for (int j = 0; j <= K; ++j) committed[base + j] = j <= n ? token[base + j] : -1;
    n_committed[b] = n + (token[base + n] >= 0 ? 1 : 0);
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

static size_t verify_sample_ws_bytes(int B, int K) {
    return 2 * align_up(static_cast<size_t>(B) * (K + 1) * sizeof(int32_t), 256);
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

extern "C" size_t spec_verify_sample_workspace_size(int B, int K, int V) {
    if (B <= 0 || K < 0 || V <= 0) return 0;
    return ms::verify_sample_ws_bytes(B, K);
}

extern "C" ms_status spec_verify_sample(const void* logits, ms_dtype logits_dtype, const int32_t* draft,
                                        const float* draft_probs, const float* temperature, const int32_t* top_k,
                                        const float* top_p, const float* min_p, const float* u, int B, int K, int V,
                                        int32_t* committed, int32_t* n_committed, void* ws, size_t ws_bytes,
                                        void* stream) {
    if (!logits || (K > 0 && !draft) || !u || !committed || !n_committed) return MS_ERR_INVALID_ARG;
    if (B <= 0 || V <= 0 || K < 0) return MS_ERR_INVALID_ARG;
    if (logits_dtype != MS_F32 && logits_dtype != MS_BF16) return MS_ERR_INVALID_ARG;
    if (!ms::element_aligned(logits, logits_dtype)) return MS_ERR_INVALID_ARG;
    if (K > 8 || !ms::sample_size_ok(static_cast<long>(B) * (K + 1), V)) return MS_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < ms::verify_sample_ws_bytes(B, K)) return MS_ERR_WORKSPACE;
    if (!ms::aligned16(ws)) return MS_ERR_INVALID_ARG;
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
    a.token = static_cast<int32_t*>(ws);
    a.accepted = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + ms::verify_sample_ws_bytes(B, K) / 2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const ms_status st = ms::sample_launch(a, logits_dtype, true, s);
    if (st != MS_OK) return st;
    return ms::launch(ms::K_SAMPLE_COMMIT, ms::sample_commit_kernel, dim3((B + 127) / 128), dim3(128), 0, s,
                      static_cast<const int32_t*>(a.token), static_cast<const int32_t*>(a.accepted), B, K, committed,
                      n_committed);
}
