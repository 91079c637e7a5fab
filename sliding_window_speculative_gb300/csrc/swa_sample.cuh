// Sampled verification of a draft block: one token per verify row from a
// given random number, under temperature, top-k, top-p and min-p.
//
// The definition (include/swa.h) orders a row's columns by falling logit, then
// rising column, keeps a prefix of that order and draws from it by the inverse
// of the cumulative weights.  Logits are bf16, so a row of V columns holds few
// distinct values, and columns of one value share one weight: how often each
// value occurs is all the order and the weights depend on.  So a row is read
// once into registers and counted into a histogram of its values; every
// cut-off is then a prefix sum over bins, and the chosen token is the r-th
// column, in column order, whose value is the chosen bin's.
//
// One cluster of C CTAs works on one row, each CTA on a contiguous part of
// its columns.  The CTAs agree on the row's maximum, count their columns into
// their own histograms, sum the histograms over the cluster (each CTA a slice
// of the bins, through distributed shared memory) and agree on the cut-offs
// slice by slice.  What bounds it: the one read of the logits, and one shared
// memory increment per column that can still be kept.
//
// Weights and masses are integers, so sums do not depend on any order and
// comparisons are exact: w = 2^-((max - x) log2(e) / T) in units of 2^-62 (the
// exponent in fixed point to 2^-50, the power from a table of 2^(-j/256) and a
// quartic; relative error below 2^-44), masses as 128-bit sums of count * w.
//
// Bins: for each sign 4096 values downwards from the row's largest magnitude
// of that sign, i.e. 32 octaves; what is smaller still shares the last bin and
// weighs like 0 (kept columns lie within 50 T of the maximum, so that is
// within 50 2^-32 of their weight), and its order is resolved by value when
// the draw lands in it.
#pragma once

#include <cooperative_groups.h>

#include "swa_common.cuh"

namespace swa {

constexpr int kSampThreads = 512;
constexpr int kSampWarps = kSampThreads / 32;
constexpr int kSampHalf = 4096;            // bins per sign
constexpr int kSampBins = 2 * kSampHalf;
constexpr int kSampVpt = 8;                // 16-byte vectors a thread holds in registers
constexpr int kSampMaxCluster = 8;
constexpr float kSampCut = 50.f;           // columns 50 T below the maximum weigh under 2^-72

struct SampleParams {
    const uint16_t *logits;    // bf16 bits [rows, V]
    const int32_t *keep;       // [V] or null
    const float *uniforms;     // [rows]
    const float *temperature;  // [B]
    const int32_t *top_k;      // [B] or null
    const float *top_p;        // [B] or null
    const float *min_p;        // [B] or null
    int32_t *tokens;           // [rows]
    float *logprobs;           // [rows] or null
    int32_t *accepted;         // [B]
    int q_len, V;
};

struct SampTable {
    uint64_t v[256];
};

// 2^(-j/256) in units of 2^-63, by the exponential series (53 bits).
constexpr SampTable samp_table() {
    SampTable t{};
    for (int j = 0; j < 256; ++j) {
        const double x = -0.69314718055994530942 * j / 256.0;
        double term = 1.0, sum = 0.0;
        for (int n = 30; n > 0; --n) {  // smallest terms first
            term = 1.0;
            for (int i = 1; i <= n; ++i) term *= x / i;
            sum += term;
        }
        t.v[j] = (uint64_t)((1.0 + sum) * 9223372036854775808.0);
    }
    return t;
}
__device__ constexpr SampTable kSampTable = samp_table();

using u128 = unsigned __int128;

__device__ __forceinline__ u128 shfl_up128(u128 x, int d) {
    const uint64_t lo = __shfl_up_sync(0xffffffffu, (uint64_t)x, d);
    const uint64_t hi = __shfl_up_sync(0xffffffffu, (uint64_t)(x >> 64), d);
    return ((u128)hi << 64) | lo;
}

// floor(x * f) for f in [0, 1) of 24 significant bits, x < 2^104
__device__ __forceinline__ u128 scale_down(u128 x, float f, bool up) {
    const uint32_t u = __float_as_uint(f);
    int e = (int)(u >> 23);
    const uint32_t m = (u & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);
    const int sh = 150 - (e > 0 ? e : 1);  // f = m 2^-sh
    const u128 p = x * m;
    if (sh >= 128) return up && p != 0 ? 1 : 0;
    return (p >> sh) + (up && (p & (((u128)1 << sh) - 1)) != 0 ? 1 : 0);
}

__device__ __forceinline__ double to_double(u128 x) {
    return (double)(uint64_t)(x >> 64) * 18446744073709551616.0 + (double)(uint64_t)x;
}

// floor(x / w) where the quotient is below 2^32
__device__ __forceinline__ uint32_t small_quotient(u128 x, uint64_t w) {
    uint64_t q = (uint64_t)(to_double(x) / (double)w);
    while ((u128)q * w > x) --q;
    while ((u128)(q + 1) * w <= x) ++q;
    return (uint32_t)q;
}

// log2(e) / T as C 2^e, C < 2^56.
struct SampScale {
    uint64_t c;
    int e;
};

__device__ __forceinline__ SampScale samp_scale(float T) {
    const double c = 1.4426950408889634 / (double)T;
    const uint64_t u = (uint64_t)__double_as_longlong(c);
    SampScale s;
    s.c = c > 0.0 ? ((u & 0xfffffffffffffull) | 0x10000000000000ull) << 3 : 0;
    s.e = (int)(u >> 52) - 1078;
    return s;
}

// |x| log2(e) / T of the bf16 magnitude `mk` in units of 2^-50, modulo 2^64
// (differences of kept columns are below 2^7).
__device__ __forceinline__ uint64_t samp_exponent(const SampScale &s, int mk) {
    const int e = mk >> 7;
    const uint64_t p = s.c * (uint64_t)((mk & 127) | (e > 0 ? 128 : 0));
    const int sh = (e > 0 ? e : 1) - 134 + s.e + 50;
    return sh >= 64 ? 0 : sh >= 0 ? p << sh : sh > -64 ? p >> -sh : 0;
}

// 2^(-y 2^-50) in units of 2^-62.
__device__ __forceinline__ uint64_t samp_weight(uint64_t y) {
    const uint32_t n = (uint32_t)(y >> 50);
    if (n >= 62) return 0;
    const uint64_t t = kSampTable.v[(y >> 42) & 255];
    const uint64_t z = __umul64hi((y & 0x3ffffffffffull) << 14, 12786308645202655660ull);  // ln 2
    const uint64_t z2 = __umul64hi(z, z), z3 = __umul64hi(z2, z), z4 = __umul64hi(z2, z2);
    const uint64_t s = z - (z2 >> 1) + z3 / 6 - z4 / 24;
    return (t - __umul64hi(t, s)) >> (n + 1);
}

// What one row's columns are counted by.
struct SampRow {
    float cut;     // columns below are left out (also NaN and -inf)
    int pt, nt;    // largest magnitude (bf16 bits) of the positive, negative columns
};

__device__ __forceinline__ bool samp_kept(const SampRow &r, uint32_t bits) {
    return __uint_as_float(bits << 16) >= r.cut;
}

__device__ __forceinline__ int samp_bin(const SampRow &r, uint32_t bits) {
    const int mk = (int)(bits & 0x7fffu);
    const bool pos = bits < 0x8000u && mk != 0;
    return pos ? min(r.pt - mk, kSampHalf - 1) : max(kSampBins - 1 - r.nt + mk, kSampHalf);
}

// Largest magnitude a bin's columns can have: their only one, but in the two
// shared bins.
__device__ __forceinline__ int samp_bin_mk(const SampRow &r, int bin) {
    return max(0, bin < kSampHalf ? r.pt - bin : r.nt - (kSampBins - 1 - bin));
}

__device__ __forceinline__ bool samp_shared_bin(int bin) {
    return bin == kSampHalf - 1 || bin == kSampHalf;
}

// Shared memory of a CTA besides the histogram.  The members written by other
// CTAs of the cluster are written once per row, between two cluster barriers.
struct SampShared {
    float max_[kSampMaxCluster], min_[kSampMaxCluster];
    uint32_t bound[kSampMaxCluster];                     // float bits
    uint32_t cnt[kSampMaxCluster], cnt_mp[kSampMaxCluster];
    uint64_t mass[kSampMaxCluster][2];
    uint64_t cut_mass[3][2];                             // after top-k, min-p, top-p
    uint32_t bin, rank;
    float lp;
    uint32_t refine[16][kSampMaxCluster];
    // this CTA's own
    float red[2][kSampWarps];
    uint32_t wcnt[kSampWarps], wmp[kSampWarps];
    uint64_t wmass[kSampWarps][2];
    uint32_t found[2][kSampWarps];
    SampScale scale;
};

template <int C, bool REG>
__global__ void __launch_bounds__(kSampThreads, 2) swa_sample_kernel(const SampleParams A) {
    namespace cg = cooperative_groups;
    constexpr int BPT = kSampBins / (C * kSampThreads);  // bins a thread sums over the cluster
    const float INF = __int_as_float(0x7f800000);
    __shared__ __align__(16) uint32_t hist[kSampBins];
    __shared__ SampShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;
    const long long row = C > 1 ? blockIdx.x / C : blockIdx.x;
    auto cluster_sync = [&]() {
        if constexpr (C > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    };
    auto at = [&](auto *p, int r) {
        if constexpr (C > 1)
            return cg::this_cluster().map_shared_rank(p, r);
        else
            return p;
    };
    // one thread's value to every CTA of the cluster
    auto publish = [&](auto *slot, auto value) {
#pragma unroll
        for (int r = 0; r < C; ++r) *at(slot, r) = value;
    };

    grid_dep_wait();
    grid_dep_trigger();

    // ---- this CTA's columns: 16-byte vectors [g0, g1) of the row, counted
    // from the 16-byte boundary at or below its first column
    const uint16_t *rp = A.logits + row * A.V;
    const int off = (int)((reinterpret_cast<uintptr_t>(rp) & 15) >> 1);
    const long long nvec = ((long long)A.V + off + 7) >> 3;
    const long long cv = (nvec + C - 1) / C;
    const long long g0 = rank * cv, g1 = min(nvec, g0 + cv);
    const int steps = REG ? kSampVpt : (int)((cv + kSampThreads - 1) / kSampThreads);
    auto load = [&](int v) -> uint4 {
        const long long g = g0 + (long long)v * kSampThreads + tid;
        uint4 w = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // NaN: no column
        if (g >= g1) return w;
        const long long j = 8 * g - off;
        if (j >= 0 && j + 8 <= A.V) return __ldg(reinterpret_cast<const uint4 *>(rp + j));
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long long a = j + 2 * e;
            const uint32_t lo = a >= 0 && a < A.V ? rp[a] : 0x7fffu;
            const uint32_t hi = a + 1 >= 0 && a + 1 < A.V ? rp[a + 1] : 0x7fffu;
            h[e] = lo | (hi << 16);
        }
        return make_uint4(h[0], h[1], h[2], h[3]);
    };
    uint4 reg[REG ? kSampVpt : 1];
    if constexpr (REG) {
#pragma unroll
        for (int v = 0; v < kSampVpt; ++v) reg[v] = load(v);
    }
    // f(step, vector) over this thread's vectors
    auto each = [&](auto f) {
        if constexpr (REG) {
#pragma unroll
            for (int v = 0; v < kSampVpt; ++v) f(v, reg[v]);
        } else {
            for (int v = 0; v < steps; ++v) f(v, load(v));
        }
    };

    // ---- the request's settings
    const int b = (int)(row / A.q_len);
    float T = A.temperature[b];
    long long k = A.top_k != nullptr ? A.top_k[b] : 0;
    if (k <= 0) k = A.V;
    if (!(T > 0.f)) {  // greedy: the first of the largest
        T = 1.f;
        k = 1;
    }
    const float tp = A.top_p != nullptr ? A.top_p[b] : 1.f;
    const bool has_p = tp < 1.f;
    float mp = A.min_p != nullptr ? A.min_p[b] : 0.f;
    if (!(mp > 0.f)) mp = 0.f;
    if (mp > 1.f) mp = 1.f;
    if (tid == 0) {
        sh.scale = samp_scale(T);
        sh.bin = sh.rank = 0;
        sh.lp = 0.f;
    }
    for (int i = tid; i < kSampBins / 4; i += kSampThreads)
        reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);

    // ---- the row's largest and smallest logit
    float mx, mn;
    {
        __nv_bfloat162 hi2 = __floats2bfloat162_rn(-INF, -INF), lo2 = __floats2bfloat162_rn(INF, INF);
        each([&](int, const uint4 &w) {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&u[e]);
                hi2 = __hmax2(hi2, x);  // (the other operand of a NaN)
                lo2 = __hmin2(lo2, x);
            }
        });
        mx = fmaxf(__low2float(hi2), __high2float(hi2));
        mn = fminf(__low2float(lo2), __high2float(lo2));
    }
    const float own_max = mx;  // this thread's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if (lane == 0) {
        sh.red[0][warp] = mx;
        sh.red[1][warp] = mn;
    }
    // top-k: of the threads' maxima the k-th largest is a bound that at least
    // k of this CTA's columns reach; bisected on ordered 16-bit keys
    float bound = -INF;
    if (k <= kSampThreads / 2) {
        const uint32_t u = __float_as_uint(own_max) >> 16;
        const uint32_t key = u & 0x8000u ? 0xffffu - u : u | 0x8000u;
        uint32_t lo = 0;
        for (uint32_t bit = 0x8000u; bit > 0; bit >>= 1)
            if (__syncthreads_count(key >= (lo | bit)) >= (int)k) lo |= bit;
        bound = __uint_as_float((lo & 0x8000u ? lo & 0x7fffu : 0xffffu - lo) << 16);
        if (!(bound > -INF)) bound = -INF;
    }
    __syncthreads();
    if (warp == 0) {
        mx = lane < kSampWarps ? sh.red[0][lane] : -INF;
        mn = lane < kSampWarps ? sh.red[1][lane] : INF;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        }
        if (lane < C) {
            *at(&sh.max_[rank], lane) = mx;
            *at(&sh.min_[rank], lane) = mn;
            *at(&sh.bound[rank], lane) = __float_as_uint(bound);
        }
    }
    cluster_sync();
    mx = -INF;
    mn = INF;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        mx = fmaxf(mx, sh.max_[r]);
        mn = fminf(mn, sh.min_[r]);
        bound = fmaxf(bound, __uint_as_float(sh.bound[r]));
    }
    if (mx == -INF) {
        // nothing to choose from: column 0
        if (rank == 0 && tid == 0) {
            A.tokens[row] = A.keep != nullptr ? A.keep[0] : 0;
            if (A.logprobs != nullptr) A.logprobs[row] = 0.f;
            if (A.q_len == 1) A.accepted[b] = 0;
        }
        return;
    }
    SampRow R;
    R.cut = fmaxf(mx - kSampCut * T, -3.4028234e38f);
    if (mx == INF) R.cut = INF;
    R.pt = mx > 0.f ? (int)(__float_as_uint(mx) >> 16) : 0;
    R.nt = (int)((__float_as_uint(fminf(fabsf(fminf(mn, 0.f)), fabsf(fminf(R.cut, 0.f)))) >> 16) &
                 0x7fffu);
    // columns that the filters cannot keep need no count: those below the
    // top-k bound, and without top-p those below the min-p line
    if (bound > R.cut) R.cut = bound;
    if (mp > 0.f && !has_p) {
        // (a little below the line: the weights themselves decide)
        const float line = mx + T * (__logf(mp) * 1.0001f - 1e-5f) - fabsf(mx) * 1e-6f;
        if (line > R.cut) R.cut = line;
    }

    // ---- count
    each([&](int, const uint4 &w) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = u[e] & 0xffffu, hi = u[e] >> 16;
            if (samp_kept(R, lo)) atomicAdd(&hist[samp_bin(R, lo)], 1u);
            if (samp_kept(R, hi)) atomicAdd(&hist[samp_bin(R, hi)], 1u);
        }
    });
    cluster_sync();

    // ---- sum this CTA's slice of the bins over the cluster; weights
    const int bin0 = rank * (kSampBins / C) + tid * BPT;
    uint32_t cnt[BPT];
#pragma unroll
    for (int i = 0; i < BPT; ++i) cnt[i] = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const uint32_t *h = at(hist, r) + bin0;
        if constexpr (BPT >= 4) {
#pragma unroll
            for (int i = 0; i < BPT; i += 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(h + i);
                cnt[i] += x.x; cnt[i + 1] += x.y; cnt[i + 2] += x.z; cnt[i + 3] += x.w;
            }
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(h);
            cnt[0] += x.x; cnt[1] += x.y;
        }
    }
    const SampScale sc = sh.scale;
    const uint64_t ymax = mx > 0.f ? samp_exponent(sc, R.pt)
                                   : 0 - samp_exponent(sc, (__float_as_uint(mx) >> 16) & 0x7fffu);
    // min-p as a weight
    const uint64_t mp_w = (uint64_t)scale_down((u128)1 << 63, 0.5f * mp, true);
    uint64_t wt[BPT];
    uint32_t c_sum = 0, c_mp = 0;
    u128 m_sum = 0;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
        wt[i] = 0;
        if (cnt[i] == 0) continue;
        const int bin = bin0 + i;
        const uint64_t y = samp_shared_bin(bin) ? 0 : samp_exponent(sc, samp_bin_mk(R, bin));
        wt[i] = samp_weight(bin < kSampHalf ? ymax - y : ymax + y);
        c_sum += cnt[i];
        if (wt[i] >= mp_w) c_mp += cnt[i];
        m_sum += (u128)wt[i] * cnt[i];
    }
    // exclusive prefix (count, mass) over the CTA's threads
    uint32_t c_pre = c_sum;
    u128 m_pre = m_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t c = __shfl_up_sync(0xffffffffu, c_pre, o);
        const u128 m = shfl_up128(m_pre, o);
        if (lane >= o) {
            c_pre += c;
            m_pre += m;
        }
    }
    c_mp = __reduce_add_sync(0xffffffffu, c_mp);
    if (lane == 31) {
        sh.wcnt[warp] = c_pre;
        sh.wmp[warp] = c_mp;
        sh.wmass[warp][0] = (uint64_t)m_pre;
        sh.wmass[warp][1] = (uint64_t)(m_pre >> 64);
    }
    __syncthreads();
    c_pre -= c_sum;
    m_pre -= m_sum;
    {
        uint32_t c_all = 0, mp_all = 0;
        u128 m_all = 0;
        for (int w = 0; w < kSampWarps; ++w) {
            const u128 m = ((u128)sh.wmass[w][1] << 64) | sh.wmass[w][0];
            if (w < warp) {
                c_pre += sh.wcnt[w];
                m_pre += m;
            }
            c_all += sh.wcnt[w];
            mp_all += sh.wmp[w];
            m_all += m;
        }
        if (tid < C) {
            *at(&sh.cnt[rank], tid) = c_all;
            *at(&sh.cnt_mp[rank], tid) = mp_all;
            *at(&sh.mass[rank][0], tid) = (uint64_t)m_all;
            *at(&sh.mass[rank][1], tid) = (uint64_t)(m_all >> 64);
        }
    }
    cluster_sync();
    uint32_t n_all = 0, n_mp = 0;
    u128 S = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const u128 m = ((u128)sh.mass[r][1] << 64) | sh.mass[r][0];
        if (r < rank) {
            c_pre += sh.cnt[r];
            m_pre += m;
        }
        n_all += sh.cnt[r];
        n_mp += sh.cnt_mp[r];
        S += m;
    }
    // the mass of the first n columns, published by the thread that holds the n-th
    auto publish_mass_of = [&](uint32_t n, int slot) {
        uint32_t c = c_pre;
        u128 m = m_pre;
#pragma unroll
        for (int i = 0; i < BPT; ++i) {
            if (c < n && n <= c + cnt[i]) {
                const u128 s = m + (u128)wt[i] * (n - c);
                publish(&sh.cut_mass[slot][0], (uint64_t)s);
                publish(&sh.cut_mass[slot][1], (uint64_t)(s >> 64));
            }
            c += cnt[i];
            m += (u128)wt[i] * cnt[i];
        }
    };
    auto cut_mass = [&](int slot) { return ((u128)sh.cut_mass[slot][1] << 64) | sh.cut_mass[slot][0]; };
    const uint32_t n_k = k < (long long)n_all ? (uint32_t)k : n_all;
    if (n_mp == 0) n_mp = 1;
    if (n_k < n_all || n_mp < n_all) {
        publish_mass_of(n_k, 0);
        publish_mass_of(n_mp, 1);
        cluster_sync();
        S = cut_mass(0);
    }
    if (has_p) {
        // columns kept by top-p: those with less than p S before them
        u128 X = tp > 0.f ? scale_down(S, tp, true) : 1;
        if (X == 0) X = 1;
        u128 m = m_pre;
#pragma unroll
        for (int i = 0; i < BPT; ++i) {
            const u128 e = m + (u128)wt[i] * cnt[i];
            if (m < X && X <= e) {
                const uint32_t n = small_quotient(X - m - 1, wt[i]) + 1;
                const u128 s = m + (u128)wt[i] * n;
                publish(&sh.cut_mass[2][0], (uint64_t)s);
                publish(&sh.cut_mass[2][1], (uint64_t)(s >> 64));
            }
            m = e;
        }
        cluster_sync();
        const u128 s = cut_mass(2);
        if (s < S) S = s;
    }
    if (n_mp < n_all) {
        const u128 s = cut_mass(1);
        if (s < S) S = s;
    }
    // ---- the draw: the column whose weights end first above u S
    {
        float u = A.uniforms[row];
        if (!(u > 0.f)) u = 0.f;
        if (u >= 1.f) u = 0.99999994f;
        const u128 target = scale_down(S, u, false);
        u128 m = m_pre;
#pragma unroll
        for (int i = 0; i < BPT; ++i) {
            const u128 e = m + (u128)wt[i] * cnt[i];
            if (m <= target && target < e) {
                publish(&sh.bin, (uint32_t)(bin0 + i));
                publish(&sh.rank, small_quotient(target - m, wt[i]));
                // ln(w / S), by the rest's share where w is most of S
                const float sf = (float)to_double(S);
                const float lp = 2 * (u128)wt[i] > S ? log1pf(-((float)to_double(S - wt[i]) / sf))
                                                    : logf((float)wt[i] / sf);
                publish(&sh.lp, lp);
            }
            m = e;
        }
    }
    cluster_sync();
    const int bin = (int)sh.bin;
    uint32_t r = sh.rank;

    // ---- its place: the r-th column, in column order, of the bin's value
    int mk = samp_bin_mk(R, bin);
    const bool pos = bin < kSampHalf;
    auto same_sign = [&](uint32_t bits) {
        return samp_kept(R, bits) && (bits < 0x8000u && (bits & 0x7fffu) != 0) == pos;
    };
    uint32_t before = 0, here;
    if (samp_shared_bin(bin)) {
        // a bin of several values: the value first, by bisection of its 15
        // bits (positive values fall with the magnitude, others rise)
        auto count = [&](auto pred, int slot) {
            uint32_t n = 0;
            each([&](int, const uint4 &w) {
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    n += pred(u[e] & 0xffffu) ? 1 : 0;
                    n += pred(u[e] >> 16) ? 1 : 0;
                }
            });
            n = __reduce_add_sync(0xffffffffu, n);
            __syncthreads();
            if (lane == 0) sh.found[0][warp] = n;
            __syncthreads();
            if (tid < C) {
                uint32_t s = 0;
                for (int w = 0; w < kSampWarps; ++w) s += sh.found[0][w];
                *at(&sh.refine[slot][rank], tid) = s;
            }
            cluster_sync();
        };
        const int top = mk;  // no column of the bin has a larger magnitude
        int v = 0;  // the value's magnitude: largest (smallest) with at most r columns before it
        uint32_t skipped = 0;
        for (int bit = 14; bit >= 0; --bit) {
            // columns of the bin in front of magnitude v | bit
            const int t = v | (1 << bit);
            count([&](uint32_t x) {
                const int xm = (int)(x & 0x7fffu);
                return same_sign(x) && xm <= top && (pos ? top - xm < t : xm < t);
            }, bit);
            uint32_t n = 0;
#pragma unroll
            for (int q = 0; q < C; ++q) n += sh.refine[bit][q];
            if (n <= r) {
                v = t;
                skipped = n;
            }
        }
        mk = pos ? top - v : v;
        r -= skipped;
        count([&](uint32_t x) { return same_sign(x) && (int)(x & 0x7fffu) == mk; }, 15);
#pragma unroll
        for (int q = 0; q < C; ++q)
            if (q < rank) before += sh.refine[15][q];
        here = sh.refine[15][rank];
    } else {
#pragma unroll
        for (int q = 0; q < C; ++q)
            if (q < rank) before += at(hist, q)[bin];
        here = hist[bin];
    }
    if (r >= before && r < before + here) {
        r -= before;
        bool done = false;
        each([&](int v, const uint4 &w) {
            if (done) return;
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t m8 = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = u[e] & 0xffffu, hi = u[e] >> 16;
                m8 |= (same_sign(lo) && (int)(lo & 0x7fffu) == mk ? 1u : 0u) << (2 * e);
                m8 |= (same_sign(hi) && (int)(hi & 0x7fffu) == mk ? 1u : 0u) << (2 * e + 1);
            }
            const uint32_t n = __popc(m8);
            uint32_t pre = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, pre, o);
                if (lane >= o) pre += x;
            }
            uint32_t *f = sh.found[v & 1];
            if (lane == 31) f[warp] = pre;
            __syncthreads();
            uint32_t total = 0, first = pre - n;
            for (int q = 0; q < kSampWarps; ++q) {
                if (q < warp) first += f[q];
                total += f[q];
            }
            if (r >= total) {
                r -= total;
                return;
            }
            done = true;
            if (r >= first && r < first + n) {
                uint32_t left = r - first;
                while (left-- > 0) m8 &= m8 - 1;
                const long long j =
                    8 * (g0 + (long long)v * kSampThreads + tid) - off + (__ffs(m8) - 1);
                A.tokens[row] = A.keep != nullptr ? A.keep[j] : (int32_t)j;
                if (A.logprobs != nullptr) A.logprobs[row] = sh.lp;
                if (A.q_len == 1) A.accepted[b] = 0;
            }
        });
    }
    if constexpr (C > 1) cluster_sync();  // no CTA leaves while its shared memory is read
}

// The accepted prefix of every sequence: the drafted tokens that equal the
// sampled ones, up to the first that does not.  One warp per sequence.
constexpr int kPrefixThreads = 128;

__global__ void __launch_bounds__(kPrefixThreads)
    swa_prefix_kernel(const int32_t *tokens, const int32_t *draft, int32_t *accepted, int B,
                      int q_len) {
    grid_dep_wait();
    grid_dep_trigger();
    const int b = blockIdx.x * (kPrefixThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (b >= B) return;
    const int n = q_len - 1;
    int hit = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const bool same = i < n && tokens[(long long)b * q_len + i] == draft[(long long)b * n + i];
        const uint32_t miss = ~__ballot_sync(0xffffffffu, same);
        if (miss != 0) {
            hit += __ffs(miss) - 1;
            break;
        }
        hit += 32;
    }
    if (lane == 0) accepted[b] = hit;
}

}  // namespace swa
