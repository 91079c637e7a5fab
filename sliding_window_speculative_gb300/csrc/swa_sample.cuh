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
// One cluster of C CTAs works on one row, each CTA on a contiguous part of its
// columns, by one of two ways.
//
// List: where a bound is known below which nothing can be kept (small top-k:
// at least k of the first chunk's columns reach it; min-p alone), the columns
// that reach it go to a list in the first CTA's shared memory, which sorts
// them and finishes the row by itself.  Almost every 16-byte vector of the row
// is dismissed by one packed maximum, so this way runs at the speed of the
// read.
//
// Histogram: else (or when the list overflows) every CTA counts its columns by
// value into its own histogram; the CTAs sum the histograms over the cluster
// (each a slice of the bins, through distributed shared memory), agree on the
// cut-offs slice by slice, and the CTA that holds the r-th column of the
// chosen value finds it in a second look at its part.  One shared memory
// increment per column bounds this way.
//
// Weights and masses are integers, so sums do not depend on any order and
// comparisons are exact: w = 2^-((max - x) log2(e) / T) in units of 2^-62 (the
// exponent in fixed point to 2^-50, the power from a table of 2^(-j/256) and a
// quartic; relative error below 2^-44), masses as 128-bit sums of count * w.
//
// Bins: for each sign 4096 values downwards from a top magnitude, i.e. 32
// octaves; the top is a few octaves above the first chunk's largest, and a row
// that exceeds it is counted again.  What is smaller still shares the last bin
// and weighs like 0 (kept columns lie within 50 T of the maximum, so that is
// within 2^-22 of their weight), and its order is resolved by value when the
// draw lands in it.
#pragma once

#include <cooperative_groups.h>

#include "swa_common.cuh"

namespace swa {

constexpr int kSampThreads = 512;
constexpr int kSampWarps = kSampThreads / 32;
constexpr int kSampHalf = 4096;            // bins per sign
constexpr int kSampBins = 2 * kSampHalf;
constexpr int kSampChunk = 8 * kSampThreads;  // 16-byte vectors of a CTA's first chunk
constexpr int kSampList = kSampBins / 2;   // columns the list holds
constexpr int kSampListK = kSampThreads / 2;  // largest top-k taken by list
constexpr int kSampMaxCluster = 8;
constexpr int kSampRoom = 4 << 7;          // four octaves above the first chunk's largest
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
__device__ __forceinline__ u128 shfl128(u128 x, int src) {
    const uint64_t lo = __shfl_sync(0xffffffffu, (uint64_t)x, src);
    const uint64_t hi = __shfl_sync(0xffffffffu, (uint64_t)(x >> 64), src);
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

// x to fp32 (24 bits, truncated).
__device__ __forceinline__ float to_float(u128 x) {
    const uint64_t hi = (uint64_t)(x >> 64);
    if (hi == 0) return __ull2float_rz((uint64_t)x);
    const int z = __clzll((long long)hi);
    return ldexpf(__ull2float_rz((uint64_t)(x >> (64 - z))), 64 - z);
}

// floor(x / w) where the quotient is below 2^32: an estimate to 2^-21, then
// Newton's correction by the remainder.
__device__ __forceinline__ uint32_t small_quotient(u128 x, uint64_t w) {
    const float wf = __ull2float_rz(w);
    uint64_t q = 0;
    for (int i = 0; i < 4; ++i) {  // what is left shrinks by 2^-20 each time
        const u128 left = x - (u128)q * w;
        const uint64_t d = (uint64_t)(to_float(left) / wf * 0.999999f);
        if (d == 0) break;
        q += d;
    }
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

// 2^(-y 2^-50) in units of 2^-62, with the table in shared memory.
__device__ __forceinline__ uint64_t samp_weight(uint64_t y, const uint64_t *table) {
    const uint32_t n = (uint32_t)(y >> 50);
    if (n >= 62) return 0;
    const uint64_t t = table[(y >> 42) & 255];
    const uint64_t z = __umul64hi((y & 0x3ffffffffffull) << 14, 12786308645202655660ull);  // ln 2
    const uint64_t z2 = __umul64hi(z, z), z3 = __umul64hi(z2, z), z4 = __umul64hi(z2, z2);
    const uint64_t s = z - (z2 >> 1) + z3 / 6 - z4 / 24;
    return (t - __umul64hi(t, s)) >> (n + 1);
}

// What one row's columns are counted by.
struct SampRow {
    float cut;     // columns below are left out (also NaN and -inf)
    int pt, nt;    // top magnitudes (bf16 bits) of the columns >= 0 and < 0
};

// A logit as fp32, -0 as 0.
__device__ __forceinline__ float samp_value(uint32_t bits) {
    return __uint_as_float(bits << 16) + 0.f;
}

// The bin of a kept value; outside [0, kSampBins) above a top magnitude.
__device__ __forceinline__ int samp_bin(const SampRow &r, float x) {
    const int m = (int)(__float_as_uint(x) >> 16);
    return m < 0x8000 ? min(r.pt - m, kSampHalf - 1)
                      : max(kSampBins - 1 - r.nt + (m - 0x8000), kSampHalf);
}

// Largest magnitude a bin's columns can have: their only one, but in the two
// shared bins.
__device__ __forceinline__ int samp_bin_mk(const SampRow &r, int bin) {
    return max(0, bin < kSampHalf ? r.pt - bin : r.nt - (kSampBins - 1 - bin));
}

__device__ __forceinline__ bool samp_shared_bin(int bin) {
    return bin == kSampHalf - 1 || bin == kSampHalf;
}

// A list entry: larger is earlier in the row's order (value, then column).
__device__ __forceinline__ uint64_t samp_entry(float x, uint32_t column) {
    const uint32_t u = __float_as_uint(x) >> 16;
    const uint32_t key = u & 0x8000u ? 0xffffu - u : u | 0x8000u;
    return ((uint64_t)key << 32) | (0xffffffffu - column);
}

// Shared memory of a CTA.  The members marked * are written by other CTAs of
// the cluster, each between two cluster barriers that separate it from its
// reads.
struct SampShared {
    union {
        uint32_t hist[kSampBins];
        uint64_t list[kSampList];                        // * (first CTA)
    };
    uint32_t merged[kSampBins / 2];                      // this CTA's slice (C > 1)
    uint64_t table[256];
    float max_[kSampMaxCluster], min_[kSampMaxCluster];  // *
    uint32_t bound[kSampMaxCluster];                     // * float bits
    uint32_t list_n;                                     // * (first CTA)
    float max2[2][kSampMaxCluster], min2[2][kSampMaxCluster];  // *
    uint32_t cnt[kSampMaxCluster], cnt_mp[kSampMaxCluster];  // *
    uint64_t mass[kSampMaxCluster][2];                   // *
    uint64_t cut_mass[3][2];                             // * after top-k, min-p, top-p
    uint32_t bin, rank;                                  // *
    float lp;                                            // *
    uint32_t refine[17][kSampMaxCluster];                // *
    float red[2][kSampWarps];
    uint32_t wcnt[kSampWarps], wmp[kSampWarps];
    uint64_t wmass[kSampWarps][2];
    uint32_t found[2][kSampWarps];
    uint64_t cut64;
    SampScale scale;
};

// The largest and smallest of eight bf16 logits (NaN left out), folded in.
__device__ __forceinline__ void samp_minmax(const uint4 &w, __nv_bfloat162 &hi, __nv_bfloat162 &lo) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&u[e]);
        hi = __hmax2(hi, x);  // (the other operand of a NaN)
        lo = __hmin2(lo, x);
    }
}

template <int C>
__global__ void __launch_bounds__(kSampThreads, 2) swa_sample_kernel(const SampleParams A) {
    namespace cg = cooperative_groups;
    constexpr int BPT = kSampBins / (C * kSampThreads);  // bins a thread sums over the cluster
    const float INF = __int_as_float(0x7f800000);
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SampShared &sh = *reinterpret_cast<SampShared *>(smem_raw);
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
    auto cluster_arrive = [&]() {
        if constexpr (C > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    };
    auto cluster_wait = [&]() {
        if constexpr (C > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    };
    // one thread's value to every CTA of the cluster
    auto publish = [&](auto *slot, auto value) {
#pragma unroll
        for (int r = 0; r < C; ++r) *at(slot, r) = value;
    };
    if (tid < 256) sh.table[tid] = kSampTable.v[tid];
    if (tid == 0) {
        sh.list_n = sh.bin = sh.rank = 0;
        sh.lp = 0.f;
    }
    for (int i = tid; i < kSampBins / 4; i += kSampThreads)
        reinterpret_cast<uint4 *>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
    cluster_arrive();  // (every CTA runs before another writes to its shared memory)

    grid_dep_wait();
    grid_dep_trigger();

    // ---- this CTA's columns: 16-byte vectors [g0, g1) of the row, counted
    // from the 16-byte boundary at or below its first column
    const uint16_t *rp = A.logits + row * A.V;
    const int off = (int)((reinterpret_cast<uintptr_t>(rp) & 15) >> 1);
    const int nvec = (int)(((long long)A.V + off + 7) >> 3);
    const int cv = (nvec + C - 1) / C;
    const int g0 = min(nvec, rank * cv), g1 = min(nvec, g0 + cv);
    auto load = [&](int g) -> uint4 {
        uint4 w = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // NaN: no column
        if (g >= g1) return w;
        const long long j = 8LL * g - off;
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
    // f(vector number, vector) over this thread's vectors of [g0, end), four
    // loads at a time; every thread of the CTA takes the same number of steps
    auto each = [&](int end, auto f) {
        for (int g = g0 + tid; g - tid < end; g += 4 * kSampThreads) {
            uint4 w[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) w[v] = load(g + v * kSampThreads);
#pragma unroll
            for (int v = 0; v < 4; ++v) f(g + v * kSampThreads, w[v]);
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
    float u = A.uniforms[row];
    if (!(u > 0.f)) u = 0.f;
    if (u >= 1.f) u = 0.99999994f;
    if (tid == kSampThreads - 1) sh.scale = samp_scale(T);
    auto finish = [&](long long column, float lp) {
        A.tokens[row] = A.keep != nullptr ? A.keep[column] : (int32_t)column;
        if (A.logprobs != nullptr) A.logprobs[row] = lp;
        if (A.q_len == 1) A.accepted[b] = 0;
    };

    // ---- the largest and smallest logit of the first chunk
    const bool rest = cv > kSampChunk;  // there are columns behind it
    float mx, mn;
    {
        __nv_bfloat162 hi2 = __floats2bfloat162_rn(-INF, -INF), lo2 = __floats2bfloat162_rn(INF, INF);
        each(min(g1, g0 + kSampChunk), [&](int, const uint4 &w) { samp_minmax(w, hi2, lo2); });
        mx = fmaxf(__low2float(hi2), __high2float(hi2));
        mn = fminf(__low2float(lo2), __high2float(lo2));
    }
    const float own_max = mx;  // this thread's
    auto block_minmax = [&](float &hi, float &lo) {  // in warp 0 afterwards
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        }
        if (lane == 0) {
            sh.red[0][warp] = hi;
            sh.red[1][warp] = lo;
        }
        __syncthreads();
        if (warp == 0) {
            hi = lane < kSampWarps ? sh.red[0][lane] : -INF;
            lo = lane < kSampWarps ? sh.red[1][lane] : INF;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            }
        }
    };
    // top-k: of the threads' maxima the k-th largest is a bound that at least
    // k of this CTA's columns reach; bisected on ordered 16-bit keys
    float bound = -INF;
    if (k <= kSampListK) {
        const uint32_t key = (uint32_t)(samp_entry(own_max, 0) >> 32);
        uint32_t lo = 0;
        for (uint32_t bit = 0x8000u; bit > 0; bit >>= 1)
            if (__syncthreads_count(key >= (lo | bit)) >= (int)k) lo |= bit;
        bound = __uint_as_float((lo & 0x8000u ? lo & 0x7fffu : 0xffffu - lo) << 16);
        if (!(bound > -INF)) bound = -INF;
    }
    block_minmax(mx, mn);
    cluster_wait();
    if (tid < C) {
        *at(&sh.max_[rank], tid) = mx;
        *at(&sh.min_[rank], tid) = mn;
        *at(&sh.bound[rank], tid) = __float_as_uint(bound);
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
    if (mx == -INF && !rest) {
        // nothing to choose from: column 0
        if (rank == 0 && tid == 0) finish(0, 0.f);
        return;
    }
    const SampScale sc = sh.scale;
    // the exponent of a value of magnitude mk, as it grows towards smaller weights
    auto falling = [&](bool neg, int mk) {
        const uint64_t y = samp_exponent(sc, mk);
        return neg ? y : 0 - y;
    };
    auto falling_of = [&](float x) {
        const uint32_t m = __float_as_uint(x) >> 16;
        return falling(m >= 0x8000u, (int)(m & 0x7fffu));
    };
    // min-p's line in logits, a little below: the weights themselves decide
    auto min_p_line = [&](float top) {
        return top + T * (__logf(mp) * 1.0001f - 1e-5f) - fabsf(top) * 1e-6f;
    };
    // columns that the filters cannot keep need no look: those far below the
    // maximum, those below the top-k bound, and without top-p those below
    // min-p's line (the first chunk's maximum stands in for the row's: lower)
    auto cut_of = [&](float top) {
        float cut = top == INF ? INF : fmaxf(top - kSampCut * T, -3.4028234e38f);
        cut = fmaxf(cut, bound);
        if (mp > 0.f && !has_p) cut = fmaxf(cut, min_p_line(top));
        return cut;
    };
    SampRow R;
    R.cut = cut_of(mx);

    if (mx > -INF && (bound > -INF || (mp > 0.f && !has_p))) {
        // ================================================= by list
        each(g1, [&](int g, const uint4 &w) {
            __nv_bfloat162 hi2 = __floats2bfloat162_rn(-INF, -INF), lo2 = hi2;
            samp_minmax(w, hi2, lo2);
            if (!(fmaxf(__low2float(hi2), __high2float(hi2)) >= R.cut)) return;
            const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = samp_value(e & 1 ? h[e >> 1] >> 16 : h[e >> 1] & 0xffffu);
                if (x >= R.cut) {
                    const uint32_t n = atomicAdd(at(&sh.list_n, 0), 1u);
                    if (n < kSampList)
                        *at(&sh.list[n], 0) = samp_entry(x, (uint32_t)(8LL * g - off + e));
                }
            }
        });
        cluster_sync();
        uint32_t n = *at(&sh.list_n, 0);
        if (n <= kSampList) {
            // (the first CTA stays until every CTA has read the count)
            cluster_arrive();
            if (rank != 0) return;
            if (n > 160 && k < (long long)n) {
                // more than top-k's: those that reach the k-th largest value
                uint32_t lo = 0;
                for (uint32_t bit = 0x8000u; bit > 0; bit >>= 1) {
                    int c = 0;
                    for (uint32_t i = tid; i < n; i += kSampThreads)
                        c += (uint32_t)(sh.list[i] >> 32) >= (lo | bit);
                    c = __reduce_add_sync(0xffffffffu, c);
                    __syncthreads();
                    if (lane == 0) sh.wcnt[warp] = c;
                    __syncthreads();
                    uint32_t all = 0;
#pragma unroll
                    for (int w = 0; w < kSampWarps; ++w) all += sh.wcnt[w];
                    if (all >= (uint32_t)k) lo |= bit;
                }
                // (each thread's entries first, then all of them packed anew)
                uint64_t mine[kSampList / kSampThreads];
                int c = 0;
#pragma unroll
                for (int i = 0; i < kSampList / kSampThreads; ++i) {
                    const uint32_t at_i = tid + i * kSampThreads;
                    mine[i] = at_i < n ? sh.list[at_i] : 0;
                    if ((uint32_t)(mine[i] >> 32) < lo) mine[i] = 0;
                    c += mine[i] != 0;
                }
                __syncthreads();
                if (tid == 0) sh.list_n = 0;
                __syncthreads();
                uint32_t to = c > 0 ? atomicAdd(&sh.list_n, (uint32_t)c) : 0;
#pragma unroll
                for (int i = 0; i < kSampList / kSampThreads; ++i)
                    if (mine[i] != 0) sh.list[to++] = mine[i];
                __syncthreads();
                n = sh.list_n;
            }
            if (n <= kSampThreads) {
                // every entry's place is the number of larger ones
                const uint64_t e = (uint32_t)tid < n ? sh.list[tid] : 0;
                uint32_t place = 0;
                if ((uint32_t)(tid & ~31) < n)
                    for (uint32_t i = 0; i < n; ++i) place += sh.list[i] > e;
                __syncthreads();
                if ((uint32_t)tid < n) sh.list[place] = e;
            } else {
                // many equal values: a bitonic network over the list
                uint32_t size = kSampThreads;
                while (size < n) size *= 2;
                for (uint32_t i = n + tid; i < size; i += kSampThreads) sh.list[i] = 0;
                __syncthreads();
                for (uint32_t span = 2; span <= size; span *= 2)
                    for (uint32_t d = span / 2; d > 0; d /= 2) {
                        for (uint32_t i = tid; i < size / 2; i += kSampThreads) {
                            const uint32_t x = 2 * i - (i & (d - 1)), y = x + d;
                            const uint64_t p = sh.list[x], q = sh.list[y];
                            if ((p < q) == ((x & span) == 0)) {
                                sh.list[x] = q;
                                sh.list[y] = p;
                            }
                        }
                        __syncthreads();
                    }
            }
            __syncthreads();
            // ---- in order: weights in units of 2^-50, running sums; eight
            // consecutive places per thread where there are many
            const uint32_t kept = k < (long long)n ? (uint32_t)k : n;
            const int per = kept <= kSampThreads ? 1 : kSampList / kSampThreads;
            auto value_of = [&](uint64_t e) {
                const uint32_t key = (uint32_t)(e >> 32);
                return __uint_as_float((key & 0x8000u ? key & 0x7fffu : 0xffffu - key) << 16);
            };
            const float top = value_of(sh.list[0]);
            const float cut = fmaxf(R.cut, cut_of(top));  // (the row's own, now)
            const uint64_t ymax = falling_of(top);
            auto weight_at = [&](uint32_t i) -> uint64_t {
                const float x = i < kept ? value_of(sh.list[i]) : -INF;
                return x >= cut ? samp_weight(falling_of(x) - ymax, sh.table) >> 12 : 0;
            };
            uint64_t sum = 0;
            for (int i = 0; i < per; ++i) sum += weight_at(tid * per + i);
            uint64_t pre = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t x = __shfl_up_sync(0xffffffffu, pre, o);
                if (lane >= o) pre += x;
            }
            if (lane == 31) sh.wmass[warp][0] = pre;
            if (tid == 0) sh.cut64 = ~0ull;
            __syncthreads();
            pre -= sum;
            uint64_t S = 0;
#pragma unroll
            for (int w = 0; w < kSampWarps; ++w) {
                if (w < warp) pre += sh.wmass[w][0];
                S += sh.wmass[w][0];
            }
            if (has_p || mp > 0.f) {
                const uint64_t mp_w = (uint64_t)scale_down((u128)1 << 51, 0.5f * mp, true);
                uint64_t X = tp > 0.f && has_p ? (uint64_t)scale_down(S, tp, true) : has_p ? 1 : S;
                if (X == 0) X = 1;
                uint64_t m = pre;
                for (int i = 0; i < per; ++i) {
                    const uint64_t w = weight_at(tid * per + i);
                    // where the running weight reaches p's share, and the last
                    // column on min-p's line
                    if (m < X && X <= m + w) atomicMin((unsigned long long *)&sh.cut64, m + w);
                    if (w >= mp_w && w != 0 && weight_at(tid * per + i + 1) < mp_w)
                        atomicMin((unsigned long long *)&sh.cut64, m + w);
                    m += w;
                }
                __syncthreads();
                if (sh.cut64 < S) S = sh.cut64;
            }
            const uint64_t target = (uint64_t)scale_down(S, u, false);
            if (pre <= target && target < pre + sum) {
                uint64_t m = pre;
                for (int i = 0; i < per; ++i) {
                    const uint64_t w = weight_at(tid * per + i);
                    if (m <= target && target < m + w) {
                        // ln(w / S), by the rest's share where w is most of S
                        const float sf = __ull2float_rn(S);
                        finish(0xffffffffu - (uint32_t)sh.list[tid * per + i],
                               2 * w > S ? log1pf(-(__ull2float_rn(S - w) / sf))
                                         : logf(__ull2float_rn(w) / sf));
                    }
                    m += w;
                }
            }
            cluster_wait();
            return;
        }
        // too many: count them (the first CTA's list gives way to its histogram)
        cluster_sync();
        for (int i = tid; i < kSampBins / 4; i += kSampThreads)
            reinterpret_cast<uint4 *>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }

    // ===================================================== by histogram
    {
        const float top = mx > 0.f ? mx : 0.f;
        R.pt = top == INF ? 0x7f80
                          : min((int)(__float_as_uint(fmaxf(top, T)) >> 16) + kSampRoom, 0x7f7f);
        const float low = fminf(fabsf(fminf(mn, 0.f)), 3.4028234e38f);
        R.nt = min((int)(__float_as_uint(fmaxf(low, T)) >> 16) + kSampRoom,
                   (int)(__float_as_uint(fabsf(fminf(fmaxf(R.cut, -3.4028234e38f), 0.f))) >> 16));
    }
    float full_max;
    for (int round = 0;; ++round) {
        // count; a column above its top magnitude shows in the largest logit or
        // the lowest kept one
        __nv_bfloat162 hi2 = __floats2bfloat162_rn(-INF, -INF);
        float lowest = 0.f;
        each(g1, [&](int, const uint4 &w) {
            const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                hi2 = __hmax2(hi2, *reinterpret_cast<const __nv_bfloat162 *>(&h[e]));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = samp_value(e & 1 ? h[e >> 1] >> 16 : h[e >> 1] & 0xffffu);
                if (x >= R.cut) {
                    const int bin = samp_bin(R, x);
                    if ((unsigned)bin < (unsigned)kSampBins)
                        atomicAdd(&sh.hist[bin], 1u);
                    else
                        lowest = fminf(lowest, x);  // (the positive ones leave it 0)
                }
            }
        });
        float hi = fmaxf(__low2float(hi2), __high2float(hi2));
        block_minmax(hi, lowest);
        if (tid < C) {
            *at(&sh.max2[round & 1][rank], tid) = hi;
            *at(&sh.min2[round & 1][rank], tid) = lowest;
        }
        cluster_sync();
        full_max = -INF;
        lowest = 0.f;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            full_max = fmaxf(full_max, sh.max2[round & 1][r]);
            lowest = fminf(lowest, sh.min2[round & 1][r]);
        }
        const bool over = lowest < 0.f || (full_max > 0.f &&
                                           (int)(__float_as_uint(full_max) >> 16) > R.pt);
        if (!over || round > 0) break;
        // a column above its top magnitude: once more, with tops that hold all
        mx = full_max;
        R.cut = cut_of(mx);
        R.pt = mx > 0.f ? (int)(__float_as_uint(mx) >> 16) : 0;
        R.nt = (int)(__float_as_uint(fabsf(fminf(fmaxf(R.cut, -3.4028234e38f), 0.f))) >> 16);
        cluster_sync();
        for (int i = tid; i < kSampBins / 4; i += kSampThreads)
            reinterpret_cast<uint4 *>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    const uint64_t ymax = falling_of(full_max + 0.f);
    const float cut = fmaxf(R.cut, cut_of(full_max));  // (the row's own, now)

    // ---- sum this CTA's slice of the bins over the cluster; weights
    const int bin0 = rank * (kSampBins / C) + tid * BPT;
    uint32_t *slice = C > 1 ? sh.merged + tid * BPT : sh.hist + tid * BPT;
    if constexpr (C > 1) {
        uint32_t cnt[BPT];
#pragma unroll
        for (int i = 0; i < BPT; ++i) cnt[i] = 0;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const uint32_t *h = at(sh.hist, r) + bin0;
#pragma unroll
            for (int i = 0; i < BPT; i += 2) {
                const uint2 x = *reinterpret_cast<const uint2 *>(h + i);
                cnt[i] += x.x;
                cnt[i + 1] += x.y;
            }
        }
#pragma unroll
        for (int i = 0; i < BPT; ++i) slice[i] = cnt[i];
    }
    auto bin_weight = [&](int bin) {
        const int mk = samp_shared_bin(bin) ? 0 : samp_bin_mk(R, bin);
        const float x = __uint_as_float((uint32_t)mk << 16);
        if (!((bin >= kSampHalf ? -x : x) >= cut)) return (uint64_t)0;
        return samp_weight(falling(bin >= kSampHalf, mk) - ymax, sh.table);
    };
    // min-p as a weight
    const uint64_t mp_w = (uint64_t)scale_down((u128)1 << 63, 0.5f * mp, true);
    uint32_t c_sum = 0, c_mp = 0;
    u128 m_sum = 0;
    for (int i = 0; i < BPT; ++i) {
        const uint32_t c = slice[i];
        if (c == 0) continue;
        const uint64_t w = bin_weight(bin0 + i);
        c_sum += c;
        if (w >= mp_w) c_mp += c;
        m_sum += (u128)w * c;
    }
    // exclusive prefix (count, mass) over the CTA's threads, then the cluster
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
    uint32_t n_all = 0, n_mp = 0;
    u128 S = 0;
#pragma unroll
    for (int w = 0; w < kSampWarps; ++w) {
        const u128 m = ((u128)sh.wmass[w][1] << 64) | sh.wmass[w][0];
        if (w < warp) {
            c_pre += sh.wcnt[w];
            m_pre += m;
        }
        n_all += sh.wcnt[w];
        n_mp += sh.wmp[w];
        S += m;
    }
    if constexpr (C > 1) {
        if (tid < C) {
            *at(&sh.cnt[rank], tid) = n_all;
            *at(&sh.cnt_mp[rank], tid) = n_mp;
            *at(&sh.mass[rank][0], tid) = (uint64_t)S;
            *at(&sh.mass[rank][1], tid) = (uint64_t)(S >> 64);
        }
        cluster_sync();
        n_all = n_mp = 0;
        S = 0;
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
    }
    if (n_all == 0) {
        if (rank == 0 && tid == 0) finish(0, 0.f);
        if constexpr (C > 1) cluster_sync();
        return;
    }
    // f(bin, count, weight, columns before, mass before) for the bins of the
    // one thread of the cluster that `mine` names, a lane per bin
    auto expand = [&](bool mine, auto f) {
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        if (who == 0) return;
        const int src = __ffs(who) - 1;
        const int bin = __shfl_sync(0xffffffffu, bin0, src) + lane;
        const uint32_t c = lane < BPT ? (slice - (lane - src) * BPT)[lane] : 0;
        const uint64_t w = c > 0 ? bin_weight(bin) : 0;
        const u128 m = (u128)w * c;
        uint32_t cp = c;
        u128 mpre = m;
#pragma unroll
        for (int o = 1; o < BPT; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, cp, o);
            const u128 y = shfl_up128(mpre, o);
            if (lane >= o) {
                cp += x;
                mpre += y;
            }
        }
        cp += __shfl_sync(0xffffffffu, c_pre, src) - c;
        mpre += shfl128(m_pre, src) - m;
        if (c > 0) f(bin, c, w, cp, mpre);
    };
    auto publish_cut = [&](int slot, u128 s) {
        publish(&sh.cut_mass[slot][0], (uint64_t)s);
        publish(&sh.cut_mass[slot][1], (uint64_t)(s >> 64));
    };
    auto cut_mass = [&](int slot) { return ((u128)sh.cut_mass[slot][1] << 64) | sh.cut_mass[slot][0]; };
    // the mass of the first n columns
    auto mass_of = [&](uint32_t n, int slot) {
        expand(c_pre < n && n <= c_pre + c_sum,
               [&](int, uint32_t c, uint64_t w, uint32_t c0, u128 m0) {
                   if (c0 < n && n <= c0 + c) publish_cut(slot, m0 + (u128)w * (n - c0));
               });
    };
    const uint32_t n_k = k < (long long)n_all ? (uint32_t)k : n_all;
    if (n_mp == 0) n_mp = 1;
    if (n_k < n_all || n_mp < n_all) {
        mass_of(n_k, 0);
        mass_of(n_mp, 1);
        cluster_sync();
        S = cut_mass(0);
    }
    if (has_p) {
        // columns kept by top-p: those with less than p S before them
        u128 X = tp > 0.f ? scale_down(S, tp, true) : 1;
        if (X == 0) X = 1;
        expand(m_pre < X && X <= m_pre + m_sum,
               [&](int, uint32_t c, uint64_t w, uint32_t, u128 m0) {
                   if (m0 < X && X <= m0 + (u128)w * c)
                       publish_cut(2, m0 + (u128)w * (small_quotient(X - m0 - 1, w) + 1));
               });
        cluster_sync();
        const u128 s = cut_mass(2);
        if (s < S) S = s;
    }
    if (n_mp < n_all) {
        const u128 s = cut_mass(1);
        if (s < S) S = s;
    }
    // ---- the draw: the column whose weights end first above u S
    const u128 target = scale_down(S, u, false);
    expand(m_pre <= target && target < m_pre + m_sum,
           [&](int bin, uint32_t c, uint64_t w, uint32_t, u128 m0) {
               if (m0 <= target && target < m0 + (u128)w * c) {
                   publish(&sh.bin, (uint32_t)bin);
                   publish(&sh.rank, small_quotient(target - m0, w));
                   // ln(w / S), by the rest's share where w is most of S
                   const float sf = to_float(S);
                   publish(&sh.lp, 2 * (u128)w > S ? log1pf(-(to_float(S - w) / sf))
                                                   : logf(__ull2float_rn(w) / sf));
               }
           });
    cluster_sync();
    const int bin = (int)sh.bin;
    uint32_t r = sh.rank;

    // ---- its place: the r-th column, in column order, of the bin's value
    int mk = samp_bin_mk(R, bin);
    const bool neg = bin >= kSampHalf;
    // (the magnitude of) a kept column of the bin's sign, else -1
    auto magnitude = [&](uint32_t bits) {
        const float x = samp_value(bits);
        const int m = (int)(__float_as_uint(x) >> 16);
        return x >= R.cut && (m >= 0x8000) == neg ? m & 0x7fff : -1;
    };
    uint32_t before = 0, here;
    if (samp_shared_bin(bin)) {
        // a bin of several values: the value first, by bisection of its 15
        // bits (values >= 0 fall with the magnitude, others rise)
        const int top = mk;  // no column of the bin has a larger magnitude
        auto count = [&](auto pred, int slot) {
            uint32_t n = 0;
            each(g1, [&](int, const uint4 &w) {
                const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    n += pred(magnitude(h[e] & 0xffffu)) ? 1 : 0;
                    n += pred(magnitude(h[e] >> 16)) ? 1 : 0;
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
        int v = 0;  // the value: magnitudes from the bin's first one with at most r columns before
        uint32_t skipped = 0;
        for (int bit = 14; bit >= 0; --bit) {
            const int t = v | (1 << bit);
            count([&](int m) { return m >= 0 && m <= top && (neg ? m < t : top - m < t); }, bit);
            uint32_t n = 0;
#pragma unroll
            for (int q = 0; q < C; ++q) n += sh.refine[bit][q];
            if (n <= r) {
                v = t;
                skipped = n;
            }
        }
        mk = neg ? v : top - v;
        r -= skipped;
        count([&](int m) { return m == mk; }, 15);
#pragma unroll
        for (int q = 0; q < C; ++q)
            if (q < rank) before += sh.refine[15][q];
        here = sh.refine[15][rank];
    } else {
#pragma unroll
        for (int q = 0; q < C; ++q)
            if (q < rank) before += at(sh.hist, q)[bin];
        here = sh.hist[bin];
    }
    cluster_arrive();  // no CTA leaves while its shared memory is read
    if (r >= before && r < before + here) {
        r -= before;
        // vectors in column order: one step of the CTA after the other
        for (int g = g0 + tid, step = 0; g - tid < g1; g += kSampThreads, ++step) {
            const uint4 w = load(g);
            const uint32_t h[4] = {w.x, w.y, w.z, w.w};
            uint32_t m8 = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                m8 |= (magnitude(e & 1 ? h[e >> 1] >> 16 : h[e >> 1] & 0xffffu) == mk ? 1u : 0u) << e;
            const uint32_t n = __popc(m8);
            uint32_t *f = sh.found[step & 1];
            const uint32_t all = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) f[warp] = all;
            __syncthreads();
            uint32_t total = 0, first = 0;
#pragma unroll
            for (int q = 0; q < kSampWarps; ++q) {
                if (q < warp) first += f[q];
                total += f[q];
            }
            if (r >= total) {
                r -= total;
                continue;
            }
            if (r >= first && r < first + all) {
                uint32_t pre = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, pre, o);
                    if (lane >= o) pre += x;
                }
                uint32_t left = r - first - (pre - n);
                if (left < n) {
                    while (left-- > 0) m8 &= m8 - 1;
                    finish(8LL * g - off + (__ffs(m8) - 1), sh.lp);
                }
            }
            break;
        }
    }
    cluster_wait();
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
