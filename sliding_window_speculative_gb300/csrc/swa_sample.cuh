// Sampled verification of a draft block: one token per verify row from a
// given random number, under temperature, top-k, top-p and min-p.
//
// The definition (include/swa.h) orders a row's columns by falling logit, then
// rising column, keeps a prefix of that order and draws from it by the inverse
// of the cumulative weights.  Logits are bf16, so a row of V columns holds few
// distinct values, and columns of one value share one weight: how often each
// value occurs is all the order and the weights depend on.  Counted into a
// histogram of its values, a row's every cut-off is a prefix sum over bins, and
// the chosen token is the r-th column, in column order, whose value is the
// chosen bin's.
//
// One cluster of C CTAs works on one row, each CTA on a contiguous part of its
// columns, by one of two ways.  What the columns must be compared with is not
// known before they are read, so the first chunk (8 vectors per thread) is read
// twice, the second time from L1 or L2 (or held in registers); the rest once.
//
// List: where a bound is known below which nothing can be kept (small top-k:
// at least k of the first chunk's columns reach it; min-p alone), and for rows
// short enough to be sorted whole, the columns that reach it go to a list in
// the first CTA's shared memory, which sorts them and finishes the row by
// itself.  Almost every 16-byte vector of the row is dismissed by one packed
// maximum: 512 rows of 262,144 under top-k 50 take 63 us (4.3 TB/s; the first
// chunk's and the list's latencies and the fourth row of some SMs are the
// rest), 8 rows 8.7 us, all latency (two cluster barriers, the list).
//
// Histogram: else (or when the list overflows) every CTA counts its columns by
// value into its own histogram; the CTAs weigh and sum the histograms over the
// cluster in blocks of 32 bins (each CTA a slice of the blocks, through
// distributed shared memory) and tell each other the blocks' sums.  From these
// every CTA finds the cut-offs and the draw for itself, looking into a block
// only where one falls, and the CTA that holds the r-th column of the chosen
// value finds it in a second look at its part, from the nearer end.  One shared
// memory increment per column bounds this way, 3.4 to 4.5 cycles per 32 of them
// with random bank conflicts (on average a quarter of a row is read again
// besides): 512 rows of 262,144 unfiltered take 121 us (2.2 TB/s), 64 rows 27.6,
// 8 rows 16.3, and 3.4, 1.7 and 1.8 us more under top-p 0.9; the blocks' weights
// are a fifth of that.  The 64 registers that four rows on an SM leave (128 for
// eight CTAs that hold a chunk) cost each instance 108 to 148 bytes of spills.
//
// Weights and masses are integers, so sums do not depend on any order and
// comparisons are exact: w = 2^-((max - x) log2(e) / T) in units of 2^-62 (the
// exponent in fixed point to 2^-50, the power from a table of 2^(-j/256) and a
// quartic; relative error below 2^-39), masses as 128-bit sums of count * w.
//
// Bins: for each sign 4096 values downwards from a top magnitude, i.e. 32
// octaves.  The top of the positive values is four octaves above the larger of
// the first chunk's largest and T, and a row that exceeds it is counted again;
// that of the negative ones is the lowest value that can weigh anything.  What
// is smaller still shares the last bin and weighs like 0 or, where that is one
// of them, like the maximum.  A column that is kept lies within 50 T of the
// maximum, so a shared one lies within 2^-22 T of 0 (positive: 2^-28 of at most
// 50 T; negative: 2^-32 of at most 200 T, or the row is counted again) and its
// weight is off by 2^-22.  Its order is resolved by value when the draw lands
// in it, by a bisection of 16 passes over the row and two to place it, a
// cluster barrier each: rows whose every logit is that near to 0 (a temperature
// far above them, a row of zeros) pay these 18 passes.  The first bin of each
// sign takes what does not count: NaN, and everything below the line.
#pragma once

#include <cooperative_groups.h>

#include "swa_common.cuh"

namespace swa {

constexpr int kSampMaxWarps = 16;
constexpr int kSampHalf = 4096;            // bins per sign
constexpr int kSampBins = 2 * kSampHalf;
constexpr int kSampVpt = 8;                // 16-byte vectors of the first chunk per thread
constexpr int kSampBlocks = kSampBins / 32;  // of 32 bins
constexpr int kSampList = kSampBins / 2;   // columns the list holds
constexpr int kSampSort = 1024;            // longer lists are counted instead
constexpr int kSampSmall = kSampSort;      // rows up to here are always taken by list
constexpr int kSampKeys = 512;             // maxima the top-k bound is taken from
// Largest top-k taken by list.  Measured on rows of 262144, us, top-k 256 listed /
// 257 counted: 8 rows 13.6 / 17.5, 64 rows 27.4 / 29.1, 512 rows 134 / 129; 48 rows
// of 12001 13.5 / 19.8, 512 rows of 4000 24.7 / 31.6.
constexpr int kSampListK = kSampKeys / 2;
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
// Sum over the warp of x < 2^104: its 26-bit pieces by one reduction each.
__device__ __forceinline__ u128 sum128(u128 x) {
    constexpr uint32_t kLow = (1u << 26) - 1;
    u128 sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum += (u128)__reduce_add_sync(0xffffffffu, (uint32_t)(x >> (26 * i)) & kLow) << (26 * i);
    return sum;
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
    // 1 - e^-z = z - z^2 / 2 + z^3 / 6 - z^4 / 24, z < 2^-8.5, from 32-bit
    // pieces: z in units of 2^-64 (ln 2 to 32 bits), a = z in units of 2^-40,
    // b = z^2 in units of 2^-48
    const uint64_t z = ((uint64_t)(uint32_t)(y >> 10) * 2977044472u) >> 8;
    const uint32_t a = (uint32_t)(z >> 24);
    const uint64_t z2 = ((uint64_t)a * a) >> 16;
    const uint32_t b = (uint32_t)(z2 >> 16);
    const uint64_t s = z - (z2 >> 1) + (((uint64_t)a * __umulhi(b, 715827883u)) >> 24) -
                       (((uint64_t)b * __umulhi(b, 178956971u)) >> 32);
    // t s, s in units of 2^-40
    const uint32_t s40 = (uint32_t)(s >> 24);
    const uint64_t ts = ((uint64_t)(uint32_t)(t >> 32) * s40 + (((uint64_t)(uint32_t)t * s40) >> 32)) >> 8;
    return (t - ts) >> (n + 1);
}

// What one row's columns are counted by.
struct SampRow {
    float cut;     // columns below are left out (also NaN and -inf)
    int pt, nt;    // top magnitudes (bf16 bits) of the columns >= 0 and < 0, exclusive
};

// A logit as fp32, -0 as 0.
__device__ __forceinline__ float samp_value(uint32_t bits) {
    return __uint_as_float(bits << 16) + 0.f;
}

// Byte offsets into the histogram of the bins of two packed logits, by packed
// 16-bit arithmetic: d = top - (the magnitude clamped to 4096 values below the
// top of its sign), bin d for positive values and 8191 - d = d ^ 8191 for
// negative ones.
struct SampBins {
    uint32_t pt, plo, nt, nlo;  // tops and lowest magnitudes, in both halves
};
__device__ __forceinline__ SampBins samp_bins(const SampRow &r) {
    auto both = [](int x) { return (uint32_t)x * 0x10001u; };
    return SampBins{both(r.pt), both(max(r.pt - kSampHalf + 1, 0)), both(r.nt),
                    both(max(r.nt - kSampHalf + 1, 0))};
}
__device__ __forceinline__ uint32_t samp_offsets(const SampBins &b, uint32_t w) {
    uint32_t neg, x = w & 0x7fff7fffu;
    asm("prmt.b32 %0, %1, %1, 0xbb99;" : "=r"(neg) : "r"(w));  // sign of each half, spread
    const uint32_t top = (b.pt & ~neg) | (b.nt & neg), low = (b.plo & ~neg) | (b.nlo & neg);
    asm("max.u16x2 %0, %0, %1;" : "+r"(x) : "r"(low));
    asm("min.u16x2 %0, %0, %1;" : "+r"(x) : "r"(top));
    return ((top - x) ^ (neg & 0x1fff1fffu)) << 2;
}

// The magnitude a bin stands for: its only one, but in the two shared bins
// their largest.
__device__ __forceinline__ int samp_bin_mk(const SampRow &r, int bin) {
    return max(0, bin < kSampHalf ? r.pt - bin : r.nt - (kSampBins - 1 - bin));
}

__device__ __forceinline__ bool samp_shared_bin(int bin) {
    return bin == kSampHalf - 1 || bin == kSampHalf;
}

// A value's place in the order, larger first (its bits, made monotone).
__device__ __forceinline__ uint32_t samp_key(float x) {
    const uint32_t u = __float_as_uint(x) >> 16;
    return u & 0x8000u ? 0xffffu - u : u | 0x8000u;
}

// A list entry: larger is earlier in the row's order (value, then column).
__device__ __forceinline__ uint64_t samp_entry(float x, uint32_t column) {
    return ((uint64_t)samp_key(x) << 32) | (0xffffffffu - column);
}

// Shared memory of a CTA.  The members marked * are written by the CTAs of the
// cluster, each between two cluster barriers that separate it from its reads.
struct SampShared {
    union {
        uint32_t hist[kSampBins];
        uint64_t list[kSampList];                        // * (first CTA's)
    };
    uint64_t table[256];
    uint32_t blk_cnt[kSampBlocks], blk_mp[kSampBlocks];  // *
    uint64_t blk_mass[kSampBlocks][2];                   // *
    float max_[kSampMaxCluster];                         // *
    uint32_t bound[2][kSampMaxCluster];                  // * float bits
    uint32_t list_n[kSampMaxCluster];                    // *
    float max2[2][kSampMaxCluster];                      // *
    uint32_t refine[18][kSampMaxCluster];                // *
    float red[kSampMaxWarps];
    uint32_t wcnt[kSampMaxWarps], wmp[kSampMaxWarps];
    uint64_t wmass[kSampMaxWarps][2];
    uint64_t cut_mass[3][2];                             // after top-k, min-p, top-p
    uint32_t found[2][kSampMaxWarps];
    uint32_t keys[kSampKeys];
    uint64_t cut64;
    uint32_t listed, most, bin, rank;
    float lp;
    SampScale scale;
};

// The largest of eight bf16 logits (NaN left out), folded into both halves of hi.
__device__ __forceinline__ void samp_max(const uint4 &w, __nv_bfloat162 &hi) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)  // (the other operand of a NaN)
        hi = __hmax2(hi, *reinterpret_cast<const __nv_bfloat162 *>(&u[e]));
}

// C CTAs of NT threads per row; HOLD: the first chunk stays in registers.
template <int C, int NT, bool HOLD>
__global__ void __launch_bounds__(NT, HOLD ? 1 : 1024 / NT) swa_sample_kernel(const SampleParams A) {
    namespace cg = cooperative_groups;
    constexpr int kWarps = NT / 32;
    constexpr int kChunk = kSampVpt * NT;      // vectors of the first chunk
    constexpr uint32_t kPart = kSampList / C;  // list entries of one CTA
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
    if (tid < 256) sh.table[tid] = kSampTable.v[tid];
    if (tid == 0) {
        sh.listed = sh.most = sh.bin = sh.rank = 0;
        sh.lp = 0.f;
    }
    for (int i = tid; i < kSampBins / 4; i += NT)
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
    // (those of the first and last column may reach over the row's ends)
    const uint4 *vp = reinterpret_cast<const uint4 *>(rp - off);
    const int in0 = off > 0 ? 1 : 0, in1 = (int)(((long long)A.V + off) >> 3);
    auto load = [&](int g) -> uint4 {
        if (g >= in0 && g < min(g1, in1)) return __ldg(vp + g);
        uint32_t h[4] = {0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu};  // NaN: no column
        if (g < g1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const long long a = 8LL * g - off + e;
                if (a >= 0 && a < A.V)
                    h[e >> 1] = e & 1 ? (h[e >> 1] & 0xffffu) | ((uint32_t)rp[a] << 16)
                                      : (h[e >> 1] & 0xffff0000u) | rp[a];
            }
        }
        return make_uint4(h[0], h[1], h[2], h[3]);
    };
    uint4 held[HOLD ? kSampVpt : 1];
    if constexpr (HOLD) {
#pragma unroll
        for (int v = 0; v < kSampVpt; ++v) held[v] = load(g0 + tid + v * NT);
    }
    // f(vector number, vector) over this thread's vectors of [g0, end), eight
    // loads at a time; every thread of the CTA takes the same number of steps,
    // and more(step) says after each whether to go on
    auto each = [&](int end, auto f, auto more) {
        if constexpr (HOLD) {
#pragma unroll
            for (int v = 0; v < kSampVpt; ++v) f(g0 + tid + v * NT, held[v]);
            if (!more(0)) return;
        }
        constexpr int U = kSampVpt;
        for (int s = g0 + (HOLD ? kChunk : 0); s < end; s += U * NT) {
            const int g = s + tid;
            uint4 w[U];
            if (s >= in0 && s + U * NT <= min(g1, in1)) {
#pragma unroll
                for (int v = 0; v < U; ++v) w[v] = __ldg(vp + g + v * NT);
            } else {
#pragma unroll
                for (int v = 0; v < U; ++v) w[v] = load(g + v * NT);
            }
#pragma unroll
            for (int v = 0; v < U; ++v) f(g + v * NT, w[v]);
            if (!more((s - g0) / kChunk)) return;
        }
    };
    auto always = [](int) { return true; };

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
    if (tid == NT - 1) sh.scale = samp_scale(T);
    auto finish = [&](long long column, float lp) {
        A.tokens[row] = A.keep != nullptr ? A.keep[column] : (int32_t)column;
        if (A.logprobs != nullptr) A.logprobs[row] = lp;
        if (A.q_len == 1) A.accepted[b] = 0;
    };

    // ---- the largest logit of the first chunk
    const bool rest = cv > kChunk;  // there are columns behind it
    float mx = -INF;
    {
        // (a thread's maxima of several parts of the chunk, as many as there
        // are keys)
        constexpr int kParts = kSampKeys / NT;
        static_assert(kParts == 1 || kParts == 2, "one or two maxima per thread");
        const __nv_bfloat162 none = __floats2bfloat162_rn(-INF, -INF);
        __nv_bfloat162 hi2[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) hi2[i] = none;
        each(min(g1, g0 + kChunk), [&](int g, const uint4 &w) {
            if constexpr (kParts == 1) {
                samp_max(w, hi2[0]);
            } else {
                __nv_bfloat162 x = none;
                samp_max(w, x);
                const bool second = g - g0 >= kChunk / 2;
                hi2[0] = __hmax2(hi2[0], second ? none : x);
                hi2[kParts - 1] = __hmax2(hi2[kParts - 1], second ? x : none);
            }
        }, always);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const float x = fmaxf(__low2float(hi2[i]), __high2float(hi2[i]));
            sh.keys[i * NT + tid] = samp_key(x);
            mx = fmaxf(mx, x);
        }
    }
    auto block_max = [&](float hi) {  // in warp 0 afterwards
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        if (lane == 0) sh.red[warp] = hi;
        __syncthreads();
        if (warp == 0) {
            hi = sh.red[lane % kWarps];
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1)
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        return hi;
    };
    mx = block_max(mx);
    cluster_wait();
    if (tid < C) *at(&sh.max_[rank], tid) = mx;
    // top-k: of the chunk's part maxima the k-th largest is a bound that at
    // least k of this CTA's columns reach, and where every CTA has a k/C-th
    // largest, k of the cluster's reach the smallest of those; a warp for each
    // bisects 16-bit keys
    if (warp == 1 || (C > 1 && warp == 2)) {
        float x = -INF;
        if (k <= kSampListK) {
            const int n = warp == 1 ? (int)k : (int)((k + C - 1) / C);
            uint32_t key[kSampKeys / 32], lo = 0;
#pragma unroll
            for (int i = 0; i < kSampKeys / 32; ++i) key[i] = sh.keys[i * 32 + lane];
            for (uint32_t bit = 0x8000u; bit > 0; bit >>= 1) {
                int c = 0;
#pragma unroll
                for (int i = 0; i < kSampKeys / 32; ++i) c += key[i] >= (lo | bit);
                if (__reduce_add_sync(0xffffffffu, c) >= n) lo |= bit;
            }
            x = __uint_as_float((lo & 0x8000u ? lo & 0x7fffu : 0xffffu - lo) << 16);
            if (!(x > -INF)) x = -INF;
        }
        if (lane < C) *at(&sh.bound[warp - 1][rank], lane) = __float_as_uint(x);
    }
    cluster_sync();
    float bound = -INF, share = INF;
    mx = -INF;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        mx = fmaxf(mx, sh.max_[r]);
        bound = fmaxf(bound, __uint_as_float(sh.bound[0][r]));
        if (C > 1) share = fminf(share, __uint_as_float(sh.bound[1][r]));
    }
    if (C > 1) bound = fmaxf(bound, share);
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
    // columns that weigh nothing lie far below the maximum
    auto line_of = [&](float top) {
        return top == INF ? INF : fmaxf(top - kSampCut * T, -3.4028234e38f);
    };
    // and those that the filters cannot keep below the top-k bound, or without
    // top-p below min-p's line (the first chunk's maximum stands in for the
    // row's: lower)
    auto cut_of = [&](float top) {
        float cut = fmaxf(line_of(top), bound);
        if (mp > 0.f && !has_p) cut = fmaxf(cut, min_p_line(top));
        return cut;
    };
    SampRow R;
    R.cut = cut_of(mx);  // (by list)

    if (mx > -INF && (bound > -INF || (mp > 0.f && !has_p) || A.V <= kSampSmall)) {
        // ================================================= by list
        const __nv_bfloat162 line = __bfloat162bfloat162(__float2bfloat16_ru(R.cut));
        each(g1, [&](int g, const uint4 &w) {
            __nv_bfloat162 hi2 = *reinterpret_cast<const __nv_bfloat162 *>(&w.x);
            hi2 = __hmax2(hi2, *reinterpret_cast<const __nv_bfloat162 *>(&w.y));
            hi2 = __hmax2(hi2, *reinterpret_cast<const __nv_bfloat162 *>(&w.z));
            hi2 = __hmax2(hi2, *reinterpret_cast<const __nv_bfloat162 *>(&w.w));
            if (__hge2_mask(hi2, line) == 0) return;  // (false for NaN)
            const uint32_t h[4] = {w.x, w.y, w.z, w.w};
            uint32_t hit = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                hit |= (samp_value(e & 1 ? h[e >> 1] >> 16 : h[e >> 1] & 0xffffu) >= R.cut ? 1u : 0u)
                       << e;
            uint32_t n = atomicAdd(&sh.listed, (uint32_t)__popc(hit));
            for (; hit != 0; hit &= hit - 1, ++n) {
                const int e = __ffs(hit) - 1;
                const uint32_t pair = e < 4 ? (e < 2 ? h[0] : h[1]) : (e < 6 ? h[2] : h[3]);
                if (n < kPart)
                    *at(&sh.list[rank * kPart + n], 0) =
                        samp_entry(samp_value(e & 1 ? pair >> 16 : pair & 0xffffu),
                                   (uint32_t)(8LL * g - off + e));
            }
        }, [&](int step) {
            // (a list that the first chunk shows to overflow is given up at once:
            // 512 rows of 262144, min-p 0.05 alone, 201 -> 130 us)
            const uint32_t listed = *(volatile uint32_t *)&sh.listed;
            if (step > 0 || !rest) return listed <= kPart;
            __syncthreads();
            const bool on = (uint64_t)sh.listed * (uint32_t)cv <= (uint64_t)kPart * kChunk;
            __syncthreads();
            if (!on && tid == 0) sh.listed = kPart + 1;
            return on;
        });
        __syncthreads();
        if (tid < C) *at(&sh.list_n[rank], tid) = sh.listed;
        cluster_sync();
        uint32_t n = 0;
        bool fits = true;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            n += sh.list_n[r];
            fits = fits && sh.list_n[r] <= kPart;
        }
        // (long lists cost more to sort than the histogram does; top-k's are cut
        // to k first, one CTA's by the row's own line.  Rows of 262144 with 2000
        // to 4000 columns on min-p's line, us, sorted / counted: 8 rows 57 / 23,
        // 64 rows 98 / 41; with 600 to 2300 listed by 2 CTAs each 128 rows
        // 58 / 68, by 4 each 64 rows 62 / 54)
        const bool by_line = mp > 0.f && !has_p, by_count = k < (long long)n;
        if (C > 1 && !by_count && n > kSampSort) fits = false;
        if (fits) {
            if (rank != 0) return;
            if constexpr (C > 1) {
                // the CTAs' parts moved together
                uint64_t mine[kSampList / NT];
#pragma unroll
                for (int i = 0; i < kSampList / NT; ++i) {
                    if ((uint32_t)(i * NT) >= n) break;
                    uint32_t from = tid + i * NT, part = 0;
#pragma unroll
                    for (int r = 0; r < C - 1; ++r)
                        if (part == (uint32_t)r && from >= sh.list_n[r]) {
                            from -= sh.list_n[r];
                            ++part;
                        }
                    mine[i] = tid + i * NT < n ? sh.list[part * kPart + from] : 0;
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kSampList / NT; ++i)
                    if (tid + i * NT < n) sh.list[tid + i * NT] = mine[i];
                __syncthreads();
            }
            auto value_of = [&](uint32_t key) {
                return __uint_as_float((key & 0x8000u ? key & 0x7fffu : 0xffffu - key) << 16);
            };
            if (n > 160 && (by_line || by_count)) {
                // (from 1 / 161 / 513 on, rows of 262144, us: 8 rows top-k 50
                // 10.1 / 8.8 / 8.8, 64 rows top-k 50 18.3 / 18.2 / 21.6, 512 rows
                // min-p 0.3 55.5 / 55.2 / 70.8; 48 rows of 12001 top-k 10
                // 10.0 / 8.2 / 8.2)
                // fewer to sort: those on min-p's line of the row's own maximum
                float low = R.cut;
                if (by_line) {
                    uint32_t most = 0;
                    for (uint32_t i = tid; i < n; i += NT)
                        most = max(most, (uint32_t)(sh.list[i] >> 32));
                    most = __reduce_max_sync(0xffffffffu, most);
                    if (lane == 0) atomicMax(&sh.most, most);
                    __syncthreads();
                    low = fmaxf(low, cut_of(value_of(sh.most)));
                }
                // and those that reach the k-th largest value, found by counting the
                // keys' upper, then their lower bytes
                uint32_t lo = 0, left = (uint32_t)k;  // left: still to find
                for (int half = 1; by_count && half >= 0; --half) {
                    if (tid < 256) sh.blk_cnt[tid] = 0;
                    __syncthreads();
                    for (uint32_t i = tid; i < n; i += NT) {
                        const uint32_t key = (uint32_t)(sh.list[i] >> 32);
                        if (half == 1 || (key >> 8) == (lo >> 8))
                            atomicAdd(&sh.blk_cnt[half == 1 ? key >> 8 : key & 255u], 1u);
                    }
                    __syncthreads();
                    // thread t: digit 255 - t, and the larger ones
                    const uint32_t c = tid < 256 ? sh.blk_cnt[255 - tid] : 0;
                    uint32_t upto = c;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += x;
                    }
                    if (lane == 31) sh.wcnt[warp] = upto;
                    __syncthreads();
                    for (int w = 0; w < warp; ++w) upto += sh.wcnt[w];
                    if (tid < 256 && upto - c < left && left <= upto) {
                        sh.found[0][0] = 255 - tid;
                        sh.found[0][1] = left - (upto - c);
                    }
                    __syncthreads();
                    lo |= sh.found[0][0] << (8 * half);
                    left = sh.found[0][1];
                }
                // (each thread's entries first, then all of them packed anew)
                uint64_t mine[kSampList / NT];
                int c = 0;
#pragma unroll
                for (int i = 0; i < kSampList / NT; ++i) {
                    const uint32_t at_i = tid + i * NT;
                    mine[i] = at_i < n ? sh.list[at_i] : 0;
                    const uint32_t key = (uint32_t)(mine[i] >> 32);
                    if (key < lo || !(value_of(key) >= low)) mine[i] = 0;
                    c += mine[i] != 0;
                }
                if (tid == 0) sh.listed = 0;
                __syncthreads();
                uint32_t to = c > 0 ? atomicAdd(&sh.listed, (uint32_t)c) : 0;
#pragma unroll
                for (int i = 0; i < kSampList / NT; ++i)
                    if (mine[i] != 0) sh.list[to++] = mine[i];
                __syncthreads();
                n = sh.listed;
            }
            if (C > 1 || n <= kSampSort) {
                if (n <= NT / 4) {
                    // every entry's place is the number of larger ones: four
                    // threads count for one
                    const uint32_t who = tid >> 2;
                    const uint64_t e = who < n ? sh.list[who] : 0;
                    uint32_t place = 0;
#pragma unroll 4
                    for (uint32_t i = tid & 3; i < n; i += 4) place += sh.list[i] > e;
                    place += __shfl_xor_sync(0xffffffffu, place, 1);
                    place += __shfl_xor_sync(0xffffffffu, place, 2);
                    __syncthreads();
                    if (who < n && (tid & 3) == 0) sh.list[place] = e;
                } else if (n <= NT) {
                    const uint64_t e = (uint32_t)tid < n ? sh.list[tid] : 0;
                    uint32_t place = 0;
                    if ((uint32_t)(tid & ~31) < n)
#pragma unroll 4
                        for (uint32_t i = 0; i < n; ++i) place += sh.list[i] > e;
                    __syncthreads();
                    if ((uint32_t)tid < n) sh.list[place] = e;
                } else {
                    // many equal values: a bitonic network over the list
                    uint32_t size = NT;
                    while (size < n) size *= 2;
                    for (uint32_t i = n + tid; i < size; i += NT) sh.list[i] = 0;
                    __syncthreads();
                    for (uint32_t span = 2; span <= size; span *= 2)
                        for (uint32_t d = span / 2; d > 0; d /= 2) {
                            for (uint32_t i = tid; i < size / 2; i += NT) {
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
                const int per = kept <= NT ? 1 : kSampList / NT;
                const float top = value_of((uint32_t)(sh.list[0] >> 32));
                const float cut = fmaxf(R.cut, cut_of(top));  // (the row's own, now)
                const uint64_t ymax = falling_of(top);
                auto weight_at = [&](uint32_t i) -> uint64_t {
                    const float x = i < kept ? value_of((uint32_t)(sh.list[i] >> 32)) : -INF;
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
                for (int w = 0; w < kWarps; ++w) {
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
                return;
            }
        }
        // too many: count them (the first CTA's list gives way to its histogram)
        __syncthreads();
        for (int i = tid; i < kSampBins / 4; i += NT)
            reinterpret_cast<uint4 *>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }

    // ===================================================== by histogram
    R.cut = line_of(mx);
    auto top_key = [](float x) { return (int)(__float_as_uint(fmaxf(x, 0.f)) >> 16); };
    // (never so low that 0 and -0 fall outside the shared bins)
    auto at_least = [](int top) { return max(top, kSampHalf); };
    R.pt = at_least(min(top_key(fmaxf(mx, T)) + kSampRoom, 0x7f81));
    float full_max;
    for (int round = 0;; ++round) {
        R.nt = at_least(top_key(-fmaxf(R.cut, -3.4028234e38f)) + 1);
        const SampBins bins = samp_bins(R);
        __nv_bfloat162 hi2 = __floats2bfloat162_rn(-INF, -INF);
        each(g1, [&](int, const uint4 &w) {
            samp_max(w, hi2);
            const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t o = samp_offsets(bins, h[e]);
                uint8_t *base = reinterpret_cast<uint8_t *>(sh.hist);
                atomicAdd(reinterpret_cast<uint32_t *>(base + (o & 0xffffu)), 1u);
                atomicAdd(reinterpret_cast<uint32_t *>(base + (o >> 16)), 1u);
            }
        }, always);
        const float hi = block_max(fmaxf(__low2float(hi2), __high2float(hi2)));
        if (tid < C) *at(&sh.max2[round][rank], tid) = hi;
        cluster_sync();
        full_max = -INF;
#pragma unroll
        for (int r = 0; r < C; ++r) full_max = fmaxf(full_max, sh.max2[round][r]);
        if (round > 0) break;
        // the first chunk may mislead: a column above the positive top, or a
        // line so far below the row's own that values a weight apart share
        // the negative values' last bin.  Then once more, from the row's own
        // maximum
        const float own = line_of(full_max);
        const float shared = __uint_as_float((uint32_t)max(R.nt - kSampHalf + 1, 0) << 16);
        const bool coarse = own < 0.f && 2.f * own > R.cut && shared > T * 2.3841858e-7f;  // 2^-22
        if (top_key(full_max) < R.pt && !coarse) break;
        R.cut = own;
        R.pt = at_least(top_key(full_max) + 1);
        cluster_sync();
        for (int i = tid; i < kSampBins / 4; i += NT)
            reinterpret_cast<uint4 *>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    const uint64_t ymax = falling_of(full_max + 0.f);
    const float cut = line_of(full_max);  // (the row's own, now)

    // ---- this CTA's slice of the blocks: counts over the cluster, weights
    const float shared_max = __uint_as_float((uint32_t)max(R.pt - kSampHalf + 1, 0) << 16);
    auto bin_weight = [&](int bin) {
        // (the shared bins' values as 0, or as the maximum if that is one of them)
        const bool shared = samp_shared_bin(bin);
        const int mk = shared ? 0 : samp_bin_mk(R, bin);
        const float x = __uint_as_float((uint32_t)mk << 16);
        const bool none = bin == 0 || bin == kSampBins - 1 ||
                          !(bin == kSampHalf - 1 ? cut <= shared_max
                            : shared             ? cut <= 0.f
                                                 : (bin >= kSampHalf ? -x : x) >= cut);
        const uint64_t y =
            shared && full_max <= shared_max ? 0 : falling(bin >= kSampHalf, mk) - ymax;
        const uint64_t w = samp_weight(y, sh.table);
        return none ? (uint64_t)0 : w;
    };
    auto bin_count = [&](int bin) {
        uint32_t c = 0;
        if (bin == 0) return c;  // no columns
#pragma unroll
        for (int r = 0; r < C; ++r) c += at(sh.hist, r)[bin];
        return c;
    };
    // min-p as a weight
    const uint64_t mp_w = (uint64_t)scale_down((u128)1 << 63, 0.5f * mp, true);
    {
        constexpr int kMine = kSampBlocks / C / kWarps;  // blocks of this warp
        static_assert(kMine * kWarps * C == kSampBlocks, "whole warps of blocks");
        auto block_of = [&](int i) { return rank * (kSampBlocks / C) + warp + i * kWarps; };
        auto tell = [&](int blk, uint32_t c, uint32_t c_mp, u128 m) {
            if (lane < C) {
                *at(&sh.blk_cnt[blk], lane) = c;
                *at(&sh.blk_mp[blk], lane) = c_mp;
                *at(&sh.blk_mass[blk][0], lane) = (uint64_t)m;
                *at(&sh.blk_mass[blk][1], lane) = (uint64_t)(m >> 64);
            }
        };
        // several blocks at a time: a weight is a long chain of multiplications
        auto weigh = [&](const auto &blk, auto &c) {
            constexpr int n = sizeof(c) / sizeof(c[0]);
            uint32_t c_mp[n];
            u128 m[n];
#pragma unroll
            for (int v = 0; v < n; ++v) {
                const uint64_t w = bin_weight(blk[v] * 32 + lane);
                c_mp[v] = w >= mp_w ? c[v] : 0;
                m[v] = (u128)w * c[v];
            }
#pragma unroll
            for (int v = 0; v < n; ++v) {
                c[v] = __reduce_add_sync(0xffffffffu, c[v]);
                c_mp[v] = __reduce_add_sync(0xffffffffu, c_mp[v]);
                m[v] = sum128(m[v]);
                tell(blk[v], c[v], c_mp[v], m[v]);
            }
        };
        if constexpr (C > 1) {
            // (the counts come from afar: read once)
            uint32_t c[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) c[i] = bin_count(block_of(i) * 32 + lane);
            constexpr int n = kMine < 4 ? kMine : 4;
            static_assert(kMine % n == 0, "whole groups of blocks");
#pragma unroll
            for (int i = 0; i < kMine; i += n) {
                int blk[n];
                uint32_t some[n], any = 0;
#pragma unroll
                for (int v = 0; v < n; ++v) {
                    blk[v] = block_of(i + v);
                    some[v] = c[i + v];
                    any |= some[v];
                }
                if (__any_sync(0xffffffffu, any != 0)) {
                    weigh(blk, some);
                } else {
#pragma unroll
                    for (int v = 0; v < n; ++v) tell(blk[v], 0, 0, 0);
                }
            }
        } else {
            static_assert(kMine <= 32, "a bit per block of a warp");
            uint32_t full = 0;  // those with columns
#pragma unroll 8
            for (int i = 0; i < kMine; ++i)
                if (__any_sync(0xffffffffu, bin_count(block_of(i) * 32 + lane) > 0))
                    full |= 1u << i;
                else
                    tell(block_of(i), 0, 0, 0);
            while (full != 0) {
                constexpr int n = 4;  // (the last of them over again where fewer are left)
                int blk[n];
                uint32_t c[n];
                int i = 0;
#pragma unroll
                for (int v = 0; v < n; ++v) {
                    if (full != 0) i = __ffs(full) - 1;
                    full &= full - 1;
                    blk[v] = block_of(i);
                    c[v] = bin_count(blk[v] * 32 + lane);
                }
                weigh(blk, c);
            }
        }
    }
    cluster_sync();
    // ---- one thread per block: its sums, and those of the blocks before it
    const bool holds = tid < kSampBlocks;
    const uint32_t c_sum = holds ? sh.blk_cnt[tid] : 0;
    const u128 m_sum = holds ? ((u128)sh.blk_mass[tid][1] << 64) | sh.blk_mass[tid][0] : 0;
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
    const uint32_t w_mp = __reduce_add_sync(0xffffffffu, holds ? sh.blk_mp[tid] : 0);
    if (lane == 31) {
        sh.wcnt[warp] = c_pre;
        sh.wmp[warp] = w_mp;
        sh.wmass[warp][0] = (uint64_t)m_pre;
        sh.wmass[warp][1] = (uint64_t)(m_pre >> 64);
    }
    __syncthreads();
    c_pre -= c_sum;
    m_pre -= m_sum;
    uint32_t n_all = 0, n_mp = 0;
    u128 S = 0;
#pragma unroll
    for (int w = 0; w < kSampBlocks / 32; ++w) {
        const u128 m = ((u128)sh.wmass[w][1] << 64) | sh.wmass[w][0];
        if (w < warp) {
            c_pre += sh.wcnt[w];
            m_pre += m;
        }
        n_all += sh.wcnt[w];
        n_mp += sh.wmp[w];
        S += m;
    }
    if (full_max == -INF) {
        if (rank == 0 && tid == 0) finish(0, 0.f);
        return;
    }
    // f(bin, count, weight, columns before, mass before), a lane per bin, for
    // the block of the one thread that `mine` names
    auto expand = [&](bool mine, auto f) {
        const uint32_t who = __ballot_sync(0xffffffffu, holds && mine);
        if (who == 0) return;
        const int src = __ffs(who) - 1;
        const int bin = 32 * (tid - lane + src) + lane;
        const uint32_t c = bin_count(bin);
        const uint64_t w = c > 0 ? bin_weight(bin) : 0;
        const u128 m = (u128)w * c;
        uint32_t cp = c;
        u128 mpre = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
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
    auto put_cut = [&](int slot, u128 s) {
        sh.cut_mass[slot][0] = (uint64_t)s;
        sh.cut_mass[slot][1] = (uint64_t)(s >> 64);
    };
    auto cut_mass = [&](int slot) { return ((u128)sh.cut_mass[slot][1] << 64) | sh.cut_mass[slot][0]; };
    // the mass of the first n columns
    auto mass_of = [&](uint32_t n, int slot) {
        expand(c_pre < n && n <= c_pre + c_sum,
               [&](int, uint32_t c, uint64_t w, uint32_t c0, u128 m0) {
                   if (c0 < n && n <= c0 + c) put_cut(slot, m0 + (u128)w * (n - c0));
               });
    };
    const uint32_t n_k = k < (long long)n_all ? (uint32_t)k : n_all;
    if (n_mp == 0) n_mp = 1;
    if (n_k < n_all || n_mp < n_all) {
        mass_of(n_k, 0);
        mass_of(n_mp, 1);
        __syncthreads();
        S = cut_mass(0);
    }
    if (has_p) {
        // columns kept by top-p: those with less than p S before them
        u128 X = tp > 0.f ? scale_down(S, tp, true) : 1;
        if (X == 0) X = 1;
        expand(m_pre < X && X <= m_pre + m_sum,
               [&](int, uint32_t c, uint64_t w, uint32_t, u128 m0) {
                   if (m0 < X && X <= m0 + (u128)w * c)
                       put_cut(2, m0 + (u128)w * (small_quotient(X - m0 - 1, w) + 1));
               });
        __syncthreads();
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
                   sh.bin = (uint32_t)bin;
                   sh.rank = small_quotient(target - m0, w);
                   // ln(w / S), by the rest's share where w is most of S
                   const float sf = to_float(S);
                   sh.lp = 2 * (u128)w > S ? log1pf(-(to_float(S - w) / sf))
                                           : logf(__ull2float_rn(w) / sf);
               }
           });
    __syncthreads();
    const int bin = (int)sh.bin;
    uint32_t r = sh.rank;

    // ---- its place: the r-th column, in column order, of the bin's value
    uint32_t value = (uint32_t)samp_bin_mk(R, bin) | (bin >= kSampHalf ? 0x8000u : 0u);
    uint32_t before = 0, here;
    if (samp_shared_bin(bin)) {
        // the two bins of many values, in order one after the other: the value
        // first, by bisection of its 16 bits
        if (bin == kSampHalf) r += bin_count(kSampHalf - 1);
        const float plo = __uint_as_float((uint32_t)max(R.pt - kSampHalf + 1, 0) << 16);
        const float nlo = __uint_as_float((uint32_t)max(R.nt - kSampHalf + 1, 0) << 16);
        auto count = [&](auto pred, int slot) {
            uint32_t n = 0;
            each(g1, [&](int, const uint4 &w) {
                const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = samp_value(e & 1 ? h[e >> 1] >> 16 : h[e >> 1] & 0xffffu);
                    n += x <= plo && x >= -nlo && pred(samp_key(x)) ? 1 : 0;
                }
            }, always);
            n = __reduce_add_sync(0xffffffffu, n);
            __syncthreads();
            if (lane == 0) sh.found[0][warp] = n;
            __syncthreads();
            if (tid < C) {
                uint32_t all = 0;
                for (int w = 0; w < kWarps; ++w) all += sh.found[0][w];
                *at(&sh.refine[slot][rank], tid) = all;
            }
            cluster_sync();
            n = 0;
#pragma unroll
            for (int q = 0; q < C; ++q) n += sh.refine[slot][q];
            return n;
        };
        uint32_t key = 0;  // the largest that more than r columns reach
        for (int bit = 15; bit >= 0; --bit) {
            const uint32_t t = key | (1u << bit);
            if (count([&](uint32_t x) { return x >= t; }, bit) > r) key = t;
        }
        r -= count([&](uint32_t x) { return x > key; }, 16);
        count([&](uint32_t x) { return x == key; }, 17);
#pragma unroll
        for (int q = 0; q < C; ++q)
            if (q < rank) before += sh.refine[17][q];
        here = sh.refine[17][rank];
        value = key & 0x8000u ? key & 0x7fffu : 0xffffu - key;
    } else {
#pragma unroll
        for (int q = 0; q < C; ++q)
            if (q < rank) before += at(sh.hist, q)[bin];
        here = sh.hist[bin];
    }
    cluster_arrive();  // no CTA leaves while its shared memory is read
    if (r >= before && r < before + here) {
        r -= before;
        // vectors in column order (compared as numbers: 0 equals -0), eight of
        // a thread's per step; from whichever end the column is nearer to,
        // counted in columns of the value
        const uint32_t both = value * 0x10001u;
        const __nv_bfloat162 want = *reinterpret_cast<const __nv_bfloat162 *>(&both);
        constexpr int U = 8;
        const int steps = (g1 - g0 + U * NT - 1) / (U * NT);
        const bool back = r >= here - here / 2;
        if (back) r = here - 1 - r;
        uint4 w[U];
        auto fetch = [&](int i) {
            const int first = g0 + (back ? steps - 1 - i : i) * (U * NT), g = first + tid;
            if (first >= in0 && first + U * NT <= min(g1, in1)) {
#pragma unroll
                for (int v = 0; v < U; ++v) w[v] = __ldg(vp + g + v * NT);
            } else {
#pragma unroll
                for (int v = 0; v < U; ++v) w[v] = load(g + v * NT);
            }
            return g;
        };
        int next = fetch(0);
        for (int step = 0; step < steps; ++step) {
            const int g = next;
            uint32_t hit[U];  // bit 2 e (2 e + 1): the lower (upper) half of word e
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const uint32_t h[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
                hit[v] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t m =
                        __heq2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&h[e]), want);
                    hit[v] |= ((m & 1u) | ((m >> 15) & 2u)) << (2 * e);
                }
            }
            if (step + 1 < steps) next = fetch(step + 1);
            auto block_sum = [&](uint32_t n, uint32_t *f, uint32_t &first) {
                n = __reduce_add_sync(0xffffffffu, n);
                if (lane == 0) f[warp] = n;
                __syncthreads();
                uint32_t total = 0;
                first = 0;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) {
                    if (q < warp) first += f[q];
                    total += f[q];
                }
                return total;
            };
            uint32_t n = 0, first;
#pragma unroll
            for (int v = 0; v < U; ++v) n += __popc(hit[v]);
            const uint32_t total = block_sum(n, sh.found[step & 1], first);
            if (r >= total) {
                r -= total;
                continue;
            }
            if (back) r = total - 1 - r;
            // in this step: its vectors one after the other
            bool done = false;
#pragma unroll
            for (int v = 0; v < U; ++v) {
                if (done) continue;
                __syncthreads();
                const uint32_t c = __popc(hit[v]);
                const uint32_t all = block_sum(c, sh.found[v & 1], first);
                if (r >= all) {
                    r -= all;
                    continue;
                }
                done = true;
                uint32_t upto = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += x;
                }
                uint32_t skip = r - first - (upto - c);
                if (r >= first && skip < c) {
                    uint32_t m = hit[v];
                    while (skip-- > 0) m &= m - 1;
                    finish(8LL * (g + v * NT) - off + (__ffs(m) - 1), sh.lp);
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
