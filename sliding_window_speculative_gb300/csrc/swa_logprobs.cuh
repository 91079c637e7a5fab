// Log probabilities of given tokens, entropies and the likeliest tokens.
//
// One pass over a row of logits keeps, with M the largest logit so far,
//   s = sum 2^(c (x - M)),   w = sum 2^(c (x - M)) (x - M),   c = log2(e) / T,
// so that ln p_j = ln2 (c (x_j - M) - log2 s) and the entropy is
// ln2 (log2 s - c w / s); counts what comes before the given token in the order;
// and stores the largest logit of every block of columns: of a vector of 8 in
// rows of up to 2048 vectors per CTA, else of a warp's 32 vectors.
//
// The top n columns of the order lie in the n blocks that come first by falling
// largest logit, equal ones by rising place: a column in another block has n
// blocks before its own, each with a column before it in the order.  So
// whatever the logits are, n blocks are read a second time (from L2), and of
// their columns those at least as large as the last block's largest are ranked
// by counting.
//
// What bounds it is the one read of the logits: 5.6 instructions and one
// exponential per logit, pairs in packed arithmetic.  A cluster of CTAs shares a
// row where there are few rows.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "swa_tc_ptx.cuh"

namespace swa {

constexpr int kLogpMaxTop = 32;
constexpr int kLogpMaxCluster = 8;
constexpr int kLogpBlocks = 2048;   // blocks per CTA at most
constexpr int kLogpPerBlock = 32;   // candidates taken of one block at most
constexpr int kLogpList = 256;      // blocks ranked by counting at most

// Smaller logits count as -2^100 in the sums: a difference of two is then finite.
constexpr float kLogpLow = -1.2676506e30f;

struct LogpParams {
    const uint16_t *logits;
    const int32_t *keep, *tokens;
    const float *temperature;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *ranks, *top_tokens;
    int q_len, V, top;
};

struct LogpStats {
    float m, s, w;
    int before;
};

struct LogpSums {
    LogpStats warp[16];
    LogpStats cta;                    // read by the cluster's first CTA
    int col, infs, n_cand, n_list;
    uint32_t least, kth[16];
};

struct LogpShared : LogpSums {
    uint32_t block[kLogpBlocks];      // a block's largest logit as a rising key
    union {
        struct {
            alignas(16) uint32_t list[kLogpBlocks - 512];  // the CTA's blocks that may be first
            uint32_t lane[512];                // per thread its first block of the CTA
        };
        unsigned long long cand[kLogpMaxTop * kLogpPerBlock];
    };
    uint32_t best[kLogpMaxCluster * kLogpMaxTop];
    uint32_t first[kLogpMaxTop];      // the CTA's first blocks, in order
    uint32_t pick[kLogpMaxTop];       // the row's
};

// Rising with the value; -0 counts as 0.
__device__ __forceinline__ uint32_t logp_key16(float x) {
    const uint32_t b = __float_as_uint(x + 0.f) >> 16;
    return b & 0x8000u ? (~b & 0xffffu) : (b | 0x8000u);
}
__device__ __forceinline__ float logp_of_key16(uint32_t k) {
    return __uint_as_float((k & 0x8000u ? k & 0x7fffu : ~k & 0xffffu) << 16);
}

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));  // (a NaN is ignored)
    return r;
}
// 1 in each half where a > b
__device__ __forceinline__ uint32_t bf16x2_gt(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float logp_warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The running sums moved from reference m to n >= m.
__device__ __forceinline__ void logp_move(float c, float m, float n, float &s, float &w) {
    const float d = m - n, a = fast_exp2(d * c);
    w = a * fmaf(d, s, w);
    s *= a;
}

// A row's columns in vectors of 8 at 16-byte addresses: column of element e of
// vector v is 8 v + e - shift.  Elements outside the row are -inf.
struct LogpRow {
    const uint16_t *x;  // the row
    int V, shift;
    __device__ __forceinline__ uint4 load(long long v) const {
        const long long c0 = 8 * v - shift;
        if (c0 >= 0 && c0 + 8 <= V) return __ldcs(reinterpret_cast<const uint4 *>(x + c0));
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long long c = c0 + 2 * e;
            const uint32_t lo = c >= 0 && c < V ? x[c] : 0xff80u;
            const uint32_t hi = c + 1 >= 0 && c + 1 < V ? x[c + 1] : 0xff80u;
            r[e] = lo | (hi << 16);
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
};

// C CTAs of NT threads (a cluster) per row; with TOP the likeliest tokens too.
template <int NT, bool TOP>
__global__ void __launch_bounds__(NT, NT == 128 && TOP ? 7 : 1024 / NT)
    swa_logprobs_kernel(const LogpParams A, const int log_c) {
    namespace cg = cooperative_groups;
    using namespace tc;
    constexpr int NW = NT / 32, U = 4;
    const float INF = __int_as_float(0x7f800000);
    constexpr uint32_t kNegInf2 = 0xff80ff80u, kLow2 = 0xf180f180u;  // -2^100
    __shared__ std::conditional_t<TOP, LogpShared, LogpSums> S;
    cg::cluster_group cluster = cg::this_cluster();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int C = 1 << log_c;
    const int rank = (int)blockIdx.x & (C - 1);
    grid_dep_wait();
    grid_dep_trigger();
    const long long row = blockIdx.x >> log_c;
    LogpRow R;
    R.x = A.logits + row * A.V;
    R.V = A.V;
    R.shift = (int)((reinterpret_cast<uintptr_t>(R.x) >> 1) & 7);
    const long long nvec = ((long long)R.shift + A.V + 7) / 8;
    const long long units = (nvec + 31) / 32;        // of 32 vectors
    // blocks of 2^bshift vectors: one, or units and powers of two of them
    int bshift = 0;
    if (((units + C - 1) >> log_c) * 32 > kLogpBlocks) {
        bshift = 5;
        while ((((units + C - 1) >> log_c) >> (bshift - 5)) + 2 > kLogpBlocks) ++bshift;
    }
    const bool fine = bshift == 0;
    const int ushift = fine ? 0 : bshift - 5;        // a CTA has whole blocks and units
    const long long groups_of = ((units - 1) >> ushift) + 1;
    const long long u0 = ((groups_of * rank) >> log_c) << ushift;
    const long long u1 = min(((groups_of * (rank + 1)) >> log_c) << ushift, units);
    const long long b0 = (u0 * 32) >> bshift;        // this CTA's first block
    const int n_blocks =
        u1 > u0 ? (int)(((min(u1 * 32, nvec) - 1) >> bshift) + 1 - b0) : 0;
    const long long blocks = ((nvec - 1) >> bshift) + 1;  // the row's

    float T = A.temperature ? A.temperature[(uint32_t)row / (uint32_t)A.q_len] : 1.f;
    T = T > 0.f ? fminf(T, 3.0e38f) : 1.f;
    const float inv_t = fminf(1.f / T, 3.0e38f), c = fminf(kLog2e / T, 3.0e38f);

    // the given token's column and logit
    const int tok = A.tokens[row];
    int col = A.keep || tok < 0 || tok >= A.V ? -1 : tok;
    if (t == 0) {
        S.col = 0x7fffffff;
        S.infs = S.n_cand = S.n_list = 0;
        S.least = 0;
    }
    if constexpr (TOP)
        if (!fine)
            for (int i = t; i < n_blocks; i += NT) S.block[i] = 0;
    __syncthreads();
    if (A.keep && tok >= 0) {
        const int j0 = (int)(((long long)A.V * rank) >> log_c);
        const int j1 = (int)(((long long)A.V * (rank + 1)) >> log_c);
        for (int j = j0 + t; j < j1; j += NT)
            if (A.keep[j] == tok) atomicMin(&S.col, j);
        if (C > 1) cluster.sync();
        else __syncthreads();
        int first = 0x7fffffff;
        for (int r = 0; r < C; ++r)
            first = min(first, C > 1 ? *cluster.map_shared_rank(&S.col, r) : S.col);
        if (first < A.V) col = first;
    }
    // a column before the token's counts if its logit is at least the token's:
    // above the next number below that; behind it if it is larger
    float xt = 0.f;
    uint32_t thr_before = 0x7f807f80u, thr_behind = 0x7f807f80u;
    long long tv = 0;
    int tpos = 0;
    if (col >= 0) {
        uint32_t b = R.x[col];
        if ((b & 0x7fffu) > 0x7f80u) b = 0xff80u;   // NaN
        if (b == 0x8000u) b = 0;
        xt = __uint_as_float(b << 16);
        const uint32_t below = b == 0 ? 0x8001u : (b & 0x8000u ? b + 1 : b - 1);
        // (a token of -inf: the columns before it all come before it, counted below)
        if (b != 0xff80u) thr_before = below | (below << 16);
        thr_behind = b | (b << 16);
        tv = ((long long)col + R.shift) >> 3;
        tpos = (col + R.shift) & 7;
    }

    // ---------------------------------------------------------------- the pass
    float m = kLogpLow;
    uint64_t s2 = 0, w2 = 0;   // pairs of partial sums
    int before = 0;
    const uint64_t c2 = f2_pack(c, c);
    // K units u, u + NW, ... whose vectors are in x; `exact`: one of them may hold
    // the given token's column
    auto take = [&](auto K, const uint4 *x, long long u, bool exact) {
        constexpr int N = decltype(K)::value;
        uint32_t count = 0;  // bf16 pairs, at most 4 N in each half
        float n = m, mine = -INF;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&x[k]);
            const uint32_t a = bf16x2_max(
                bf16x2_max(bf16x2_max(y[0], y[1]), bf16x2_max(y[2], y[3])), kNegInf2);
            const float own = fmaxf(bf16lo(a), bf16hi(a));
            const float mu = logp_warp_max(own);
            n = fmaxf(n, mu);
            if (lane == k) mine = mu;
            if constexpr (TOP) {
                if (fine) {
                    const long long b = (u + NW * k) * 32 + lane - b0;
                    if (b < n_blocks) S.block[b] = logp_key16(own);
                }
            }
            uint32_t thr = u + NW * k < (tv >> 5) ? thr_before : thr_behind;
            if (exact) {
                const long long v = (u + NW * k) * 32 + lane;
                thr = v < tv ? thr_before : thr_behind;
                if (v == tv && col >= 0) {
                    const bool none = thr_before == 0x7f807f80u;
                    for (int e = 0; e < tpos; ++e) {
                        const uint32_t z2 = bf16x2_max(y[e >> 1], kNegInf2);
                        const float z = e & 1 ? bf16hi(z2) : bf16lo(z2);
                        before += none ? -(z > xt) : (z == xt);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) count = bf16x2_add(count, bf16x2_gt(y[e], thr));
        }
        before += (int)(bf16lo(count) + bf16hi(count));
        if constexpr (TOP)
            if (!fine && lane < N)
                atomicMax(&S.block[(int)(((u + NW * lane) >> (bshift - 5)) - b0)], logp_key16(mine));
        if (n > m) {  // (the warp's)
            float sa, sb, wa, wb;
            f2_unpack(s2, sa, sb);
            f2_unpack(w2, wa, wb);
            logp_move(c, m, n, sa, wa);
            logp_move(c, m, n, sb, wb);
            s2 = f2_pack(sa, sb);
            w2 = f2_pack(wa, wb);
            m = n;
        }
        const uint64_t m2 = f2_pack(m, m);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&x[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t z = bf16x2_max(y[e], kLow2);
                const uint64_t d2 = f2_sub(f2_pack(bf16lo(z), bf16hi(z)), m2);
                float a, b;
                f2_unpack(f2_mul(d2, c2), a, b);
                const uint64_t e2 = f2_pack(fast_exp2(a), fast_exp2(b));
                s2 = f2_add(s2, e2);
                w2 = f2_fma(e2, d2, w2);
            }
        }
    };
    // the units that lie wholly inside the row, U at a time, then the others
    const long long i0 = max(u0, R.shift > 0 ? 1LL : 0LL);
    const long long i1 = min(u1, ((long long)R.shift + A.V) / 256);
    const long long groups = i1 > i0 ? (i1 - i0) / (NW * U) : 0;
    const uint4 *p = reinterpret_cast<const uint4 *>(R.x - R.shift) + (i0 + warp) * 32 + lane;
    long long u = i0 + warp;
    for (long long g = 0; g < groups; ++g, u += NW * U, p += NW * U * 32) {
        uint4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) x[k] = __ldcs(p + NW * 32 * k);
        const long long at = (tv >> 5) - u;
        take(std::integral_constant<int, U>{}, x, u, at >= 0 && at < NW * U && at % NW == 0);
    }
    for (long long q = warp; q < (u1 - u0) - groups * (NW * U); q += NW) {
        // (those before i0, then those behind the groups)
        const long long un = u0 + q < i0 ? u0 + q : u0 + q + groups * (NW * U);
        const long long v = un * 32 + lane;
        const uint4 x = v < nvec ? R.load(v) : make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
        take(std::integral_constant<int, 1>{}, &x, un, true);
    }
    // ---------------------------------------------- sums of the warp, CTA, row
    float s, w;
    {
        float sb, wb;
        f2_unpack(s2, s, sb);
        f2_unpack(w2, w, wb);
        s += sb;
        w += wb;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, off);
        w += __shfl_xor_sync(0xffffffffu, w, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    if (lane == 0) S.warp[warp] = LogpStats{m, s, w, before};
    __syncthreads();
    const int top = A.top;
    if constexpr (TOP) {
        // This CTA's first blocks.  A key holds a block's logit and, equal logits
        // falling, its place: all differ.  Threads' own largest keys bound the
        // top-th largest key from below: `per` of them in each warp are at least the
        // warps' smallest per-th largest.
        constexpr int PER = kLogpBlocks / NT;
        uint32_t key[PER], mine = 0;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int b = q * NT + t;
            key[q] = b < n_blocks ? (S.block[b] << 16) | (0xffffu - (uint32_t)(b0 + b)) : 0u;
            mine = max(mine, key[q]);
        }
        const int per = (top + NW - 1) / NW;
        uint32_t left = mine, kth = 0;
        for (int i = 0; i < per; ++i) {
            kth = __reduce_max_sync(0xffffffffu, left);
            if (left == kth) left = 0;
        }
        if (lane == 0) S.kth[warp] = kth;
        if (t < top) S.first[t] = 0;
        __syncthreads();
        uint32_t least = S.kth[0];
        for (int i = 1; i < NW; ++i) least = min(least, S.kth[i]);
        int above = 0;
#pragma unroll
        for (int q = 0; q < PER; ++q) above += key[q] != 0 && key[q] >= least;
        int at = above > 0 ? atomicAdd(&S.n_list, above) : 0;
        __syncthreads();
        int n_list = S.n_list;
        if (n_list > kLogpList) {
            // too loose (large logits crowd in few warps): the top-th largest of all
            // threads' own largest, which leaves at most top * PER
            S.lane[t] = mine;
            __syncthreads();
            if (t == 0) S.n_list = 0;
            int r = 0;
            const uint4 *all = reinterpret_cast<const uint4 *>(S.lane);
            for (int i = 0; i < NT / 4; ++i) {
                const uint4 k = all[i];
                r += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
            }
            if (mine != 0 && r == top - 1) S.least = mine;
            __syncthreads();
            least = S.least;
            above = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q) above += key[q] != 0 && key[q] >= least;
            at = above > 0 ? atomicAdd(&S.n_list, above) : 0;
            __syncthreads();
            n_list = S.n_list;
        }
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (key[q] != 0 && key[q] >= least) S.list[at++] = key[q];
        __syncthreads();
        for (int i = t; i < n_list; i += NT) {
            const uint32_t k = S.list[i];
            int r = 0;
            for (int q = 0; q < n_list; ++q) r += S.list[q] > k;
            if (r < top) S.first[r] = k;
        }
    }
    auto join = [&](LogpStats &a, const LogpStats &b) {
        const float n = fmaxf(a.m, b.m);
        float bs = b.s, bw = b.w;
        logp_move(c, a.m, n, a.s, a.w);
        logp_move(c, b.m, n, bs, bw);
        a = LogpStats{n, a.s + bs, a.w + bw, a.before + b.before};
    };
    if (t == 0) {
        LogpStats a = S.warp[0];
        for (int i = 1; i < NW; ++i) join(a, S.warp[i]);
        S.cta = a;
    }
    if (C > 1) cluster.sync();
    else __syncthreads();
    LogpStats a = C > 1 ? *cluster.map_shared_rank(&S.cta, 0) : S.cta;
    for (int r = 1; r < C; ++r) join(a, *cluster.map_shared_rank(&S.cta, r));
    if (a.m == INF) {
        // the columns of +inf share the row
        int n = 0;
        for (long long v = u0 * 32 + t; v < min(u1 * 32, nvec); v += NT) {
            const uint4 x = R.load(v);
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&x);
            for (int e = 0; e < 4; ++e) n += (bf16lo(y[e]) == INF) + (bf16hi(y[e]) == INF);
        }
        if (n) atomicAdd(&S.infs, n);
        if (C > 1) cluster.sync();
        else __syncthreads();
        n = 0;
        for (int r = 0; r < C; ++r) n += C > 1 ? *cluster.map_shared_rank(&S.infs, r) : S.infs;
        a.s = (float)n;
        a.w = 0.f;
    }
    bool none = false;
    if (a.m < INF && (a.m <= kLogpLow || T > 1.0e25f)) {
        // no logit above what the sums tell apart, or a temperature at which even
        // -2^100 has weight: the row again, from its own largest logit and
        // without those of -inf (every CTA all of it)
        float n = -INF;
        for (long long v = t; v < nvec; v += NT) {
            const uint4 x = R.load(v);
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&x);
            for (int e = 0; e < 4; ++e) n = fmax3(n, bf16lo(y[e]), bf16hi(y[e]));
        }
        n = logp_warp_max(n);
        __syncthreads();
        if (lane == 0) S.warp[warp].m = n;
        __syncthreads();
        for (int i = 0; i < NW; ++i) n = fmaxf(n, S.warp[i].m);
        none = n == -INF;
        s = w = 0.f;
        for (long long v = t; v < nvec && !none; v += NT) {
            const uint4 x = R.load(v);
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&x);
            for (int e = 0; e < 8; ++e) {
                const float z = e & 1 ? bf16hi(y[e >> 1]) : bf16lo(y[e >> 1]);
                if (!(z > -INF)) continue;
                const float f = fast_exp2((z - n) * c);
                s += f;
                w = fmaf(f, z - n, w);
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, off);
            w += __shfl_xor_sync(0xffffffffu, w, off);
        }
        if (lane == 0) {
            S.warp[warp].s = s;
            S.warp[warp].w = w;
        }
        __syncthreads();
        a.m = n;
        a.s = a.w = 0.f;
        for (int i = 0; i < NW; ++i) {
            a.s += S.warp[i].s;
            a.w += S.warp[i].w;
        }
    }
    const float ls = log2f(a.s);
    auto logprob = [&](float x) {
        if (none || x == -INF) return -INF;
        const float d = x == a.m ? 0.f : x - a.m;
        return d * inv_t - ls * kLn2;
    };
    if (rank == 0 && t == 0) {
        A.logprobs[row] = col >= 0 ? logprob(xt) : -INF;
        if (A.ranks)
            A.ranks[row] = col < 0 ? 0 : a.before + 1 + (xt == -INF ? col : 0);
        if (A.entropy) A.entropy[row] = none ? 0.f : kLn2 * (ls - c * (a.w / a.s));
    }

    // -------------------------------------------------------- the first n columns
    if constexpr (TOP)
    if (rank == 0) {
        // the row's first blocks among the CTAs' by counting
        for (int i = t; i < C * top; i += NT)
            S.best[i] = C > 1 ? *cluster.map_shared_rank(&S.first[i % top], i / top) : S.first[i];
        __syncthreads();
        for (int i = t; i < C * top; i += NT) {
            const uint32_t k = S.best[i];
            int r = 0;
            for (int q = 0; q < C * top; ++q) r += S.best[q] > k;
            if (k != 0 && r < top) S.pick[r] = k;
        }
        __syncthreads();
        // their columns at least as large as the last one's largest; a lane's first
        // vector of each of the warp's blocks at once (the only one unless rows are
        // longer than kLogpBlocks blocks of 256)
        const int nb = (int)min((long long)top, blocks);
        const float least = nb < top ? -INF : logp_of_key16(S.pick[nb - 1] >> 16);
        if (fine) {
            // a thread per element
            for (int i = t; i < 8 * nb; i += NT) {
                const long long j =
                    8 * (0xffffLL - (S.pick[i >> 3] & 0xffffu)) + (i & 7) - R.shift;
                if (j < 0 || j >= A.V) continue;
                uint32_t b = R.x[j];
                if ((b & 0x7fffu) > 0x7f80u) b = 0xff80u;
                const float f = __uint_as_float(b << 16);
                if (f >= least)
                    S.cand[atomicAdd(&S.n_cand, 1)] =
                        ((unsigned long long)logp_key16(f) << 32) | (uint32_t)~(uint32_t)j;
            }
        }
        constexpr int BW = (kLogpMaxTop + NW - 1) / NW;  // blocks per warp
        uint4 x0[BW];
        const int nw = fine ? 0 : nb;
#pragma unroll
        for (int h = 0; h < BW; ++h) {
            const int i = warp + NW * h;
            x0[h] = make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
            if (i < nw) {
                const long long v = ((0xffffLL - (S.pick[i] & 0xffffu)) << bshift) + lane;
                if (v < nvec) x0[h] = R.load(v);
            }
        }
#pragma unroll
        for (int h = 0; h < BW; ++h) {
            const int i = warp + NW * h;
            if (i >= nw) break;
            const long long b = 0xffffLL - (S.pick[i] & 0xffffu);
            const long long v0 = b << bshift, v1 = min((b + 1) << bshift, nvec);
            auto vec = [&](long long v) { return v < v0 + 32 ? x0[h] : R.load(v); };
            // elements of a vector that are candidates, and the key of one
            auto mask_of = [&](const uint4 &x, long long v) -> uint32_t {
                const uint32_t *y = reinterpret_cast<const uint32_t *>(&x);
                uint32_t m8 = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t z = bf16x2_max(y[e >> 1], kNegInf2);
                    m8 |= (uint32_t)((e & 1 ? bf16hi(z) : bf16lo(z)) >= least) << e;
                }
                if (least == -INF)
                    for (int e = 0; e < 8; ++e) {
                        const long long j = 8 * v + e - R.shift;
                        if (j < 0 || j >= A.V) m8 &= ~(1u << e);
                    }
                return m8;
            };
            auto key_of = [&](const uint4 &x, int e, long long v) -> unsigned long long {
                const uint32_t y = e < 4 ? (e < 2 ? x.x : x.y) : (e < 6 ? x.z : x.w);
                const uint32_t z = bf16x2_max(y, kNegInf2);
                return ((unsigned long long)logp_key16(e & 1 ? bf16hi(z) : bf16lo(z)) << 32) |
                       (uint32_t)~(uint32_t)(8 * v + e - R.shift);
            };
            int n = 0;
            for (long long v = v0 + lane; v < v1; v += 32) n += __popc(mask_of(vec(v), v));
            const int sum = __reduce_add_sync(0xffffffffu, n);
            if (sum <= kLogpPerBlock) {
                if (n == 0) continue;
                int at = atomicAdd(&S.n_cand, n);
                for (long long v = v0 + lane; v < v1; v += 32) {
                    const uint4 x = vec(v);
                    for (uint32_t m8 = mask_of(x, v); m8 != 0; m8 &= m8 - 1)
                        S.cand[at++] = key_of(x, __ffs(m8) - 1, v);
                }
            } else {
                // many equal ones: the block's first kLogpPerBlock, one after another
                unsigned long long last = ~0ull;
                int at = 0;
                if (lane == 0) at = atomicAdd(&S.n_cand, kLogpPerBlock);
                for (int q = 0; q < kLogpPerBlock; ++q) {
                    unsigned long long k = 0;
                    for (long long v = v0 + lane; v < v1; v += 32) {
                        const uint4 x = vec(v);
                        for (uint32_t m8 = mask_of(x, v); m8 != 0; m8 &= m8 - 1) {
                            const unsigned long long z = key_of(x, __ffs(m8) - 1, v);
                            if (z < last && z > k) k = z;
                        }
                    }
                    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
                    const uint32_t lo = __reduce_max_sync(
                        0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
                    last = ((unsigned long long)hi << 32) | lo;
                    if (lane == 0) S.cand[at + q] = last;
                }
            }
        }
        __syncthreads();
        const int n = S.n_cand;
        for (int i = t; i < n; i += NT) {
            const unsigned long long k = S.cand[i];
            int r = 0;
            for (int q = 0; q < n; ++q) r += S.cand[q] > k;
            if (r < top) {
                const int j = (int)~(uint32_t)k;
                A.top_tokens[row * top + r] = A.keep ? A.keep[j] : j;
                A.top_logprobs[row * top + r] = logprob(logp_of_key16((uint32_t)(k >> 32)));
            }
        }
    }
    // the other CTAs' shared memory is read above
    if (C > 1) cluster.sync();
}

}  // namespace swa
