// RMS norm of every query and key head and the position rotation in one pass
// over a verify block's projected rows, the key and value rows going to fresh
// tensors or straight into the (contiguous or paged) cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w                       (heads of q and k)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = (q_pos + i) * f_n
//
// for the n-th pair (a, b) of the first rot dims: dims (n, n + rot/2), or
// (2n, 2n + 1) when interleaved.  All in fp32, rounded to bf16 once.
//
// D / 16 lanes hold one head row, 16 dims each: the 8 dims [8l, 8l + 8) and those
// rot/2 further, so a lane owns both members of its pairs in either layout and
// no value crosses lanes but the sum of squares.  (Two pieces next to each
// other instead make every load and store touch half sectors.)  A
// warp works on one token (or a part of its heads): the angles depend on the
// token alone, so cosine and sine are computed once and used for all heads.
//
// What bounds it is the one read and one write of the rows: 512 x 64 tokens of
// 12 heads (403 MB) take 72.5 us, 82% of the measured copy bandwidth, with the
// next batch's loads in flight while one is worked on, whole 32-byte sectors
// per thread pair and paired fp32 arithmetic (85.0 us without the three).  A
// block of 8 rows takes 3.5 us, a launch and one memory latency.
//
// Angles of far positions: f / 2 pi is held as a 64-bit binary fraction of a
// turn, and (q_pos + i) times it modulo 2^64 is the angle modulo one turn
// (exact but for f's own rounding, 2^-61 of it per position), where a product
// in fp32 would have lost the fraction.
#pragma once

#include "swa_simt.cuh"
#include "swa_tc_ptx.cuh"

namespace swa {

constexpr int kRopeThreads = 128;
constexpr int kRopeBlocksPerSm = 4;

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    long long q_row, k_row, v_row;  // elements between consecutive tokens
    const float *q_weight, *k_weight, *inv_freq;
    const int32_t *q_pos;
    __nv_bfloat16 *q_out, *k_out, *v_out;  // k_out / v_out: the caches, with to_cache
    AttnParams cache;  // q_len; with to_cache also seq_lens, the block table, Hkv, L
    int to_cache;
    int tokens, Hq, Hkv, rot, interleaved, parts;
    float eps;
};

// f / 2 pi as a fraction of a turn in units of 2^-64, modulo a turn:
// f = m 2^e with a 24-bit m (f finite), and K = round(2^64 / 2 pi).
__device__ __forceinline__ uint64_t rope_turns(float f) {
    constexpr uint64_t K = 2935890503282001226ull;
    const uint32_t u = __float_as_uint(f);
    int e = (int)((u >> 23) & 255u);
    const uint64_t m = (u & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);
    e = (e > 0 ? e : 1) - 150;
    const uint64_t lo = m * K, hi = __umul64hi(m, K);
    uint64_t t;
    if (e >= 0)
        t = e < 64 ? lo << e : 0;
    else if (e > -64)
        t = (lo >> -e) | (hi << (64 + e));
    else
        t = e > -128 ? hi >> (-64 - e) : 0;
    return (u >> 31) ? 0 - t : t;
}

// An infinite or NaN frequency has no angle: its pairs become NaN.
__device__ __forceinline__ bool rope_finite(float f) {
    return (__float_as_uint(f) & 0x7f800000u) != 0x7f800000u;
}

// Cosine and sine of t 2^-32 turns: the nearest quarter turn q and the rest r
// (in half turns, |r| <= 1/4) by the Taylor polynomials of degree 9 and 8 in
// pi r (remainders below 2^-25), then turned by q quarters.
__device__ __forceinline__ void rope_cos_sin(uint32_t t, float &c, float &s) {
    const uint32_t q = (t + 0x20000000u) >> 30;
    const float r = (float)(int32_t)(t - (q << 30)) * 4.656612873077393e-10f;  // 2^-31
    const float r2 = r * r;
    float sp = fmaf(r2, 0.082145887f, -0.59926453f);  // pi^9 / 9!, -pi^7 / 7!
    sp = fmaf(r2, sp, 2.5501640f);                    // pi^5 / 5!
    sp = fmaf(r2, sp, -5.1677128f);                   // -pi^3 / 3!
    sp = r * fmaf(r2, sp, 3.1415927f);
    float cp = fmaf(r2, 0.23533063f, -1.3352628f);    // pi^8 / 8!, -pi^6 / 6!
    cp = fmaf(r2, cp, 4.0587121f);                    // pi^4 / 4!
    cp = fmaf(r2, cp, -4.9348022f);                   // -pi^2 / 2!
    cp = fmaf(r2, cp, 1.f);
    const bool odd = q & 1;
    c = __uint_as_float(__float_as_uint(odd ? sp : cp) ^ (((q + 1) & 2u) << 30));
    s = __uint_as_float(__float_as_uint(odd ? cp : sp) ^ ((q & 2u) << 30));
}

// Eight fp32 weights, as pairs, from (16-byte aligned) shared memory.
__device__ __forceinline__ void rope_weights(const float *w, uint64_t (&o)[4]) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(w);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(w + 4);
    o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) swa_rope_kernel(const RopeParams R) {
    using namespace tc;
    constexpr int LPR = D / 16;        // lanes per head row
    constexpr int RPW = 32 / LPR;      // head rows per warp and step
    constexpr int U = 3;               // steps whose loads are in flight together
    __shared__ __align__(16) float w_s[2][D];
    __shared__ uint64_t turn_s[D / 2];
    __shared__ volatile int odd_s;  // some frequency is not finite
    const int tid = threadIdx.x, lane = tid & 31;
    const int l = lane % LPR, slot = lane / LPR;
    const int heads = R.Hq + 2 * R.Hkv;
    const int q_len = R.cache.q_len;
    const float kNan = __int_as_float(0x7fffffff);
    grid_dep_wait();
    grid_dep_trigger();
    const bool turns = l < R.rot / 16;  // this lane's dims are rotated
    // first dims of the lane's two 8-dim pieces, half of the rotated (or of the
    // other) dims apart: neighbouring lanes' pieces are neighbours in memory
    const int span0 = turns ? 0 : R.rot, span = turns ? R.rot : D - R.rot;
    const int da = span0 + 8 * (l - span0 / 16), db = da + span / 2;
    // first pair of each piece's four (interleaved) or the first piece's eight
    const int pair0 = R.interleaved ? 4 * l : 8 * l;
    const int pair1 = R.interleaved ? R.rot / 4 + 4 * l : 8 * l + 4;
    const long long n_work = (long long)R.tokens * R.parts;
    const int warps = gridDim.x * (kRopeThreads / 32);
    const int step = R.parts * RPW;
    // the heads [h0, h0 + U steps) of token work / parts
    struct Batch {
        long long work;
        int h0;
    };
    auto token_of = [&](const Batch &a) { return (int)(a.work / R.parts); };
    auto fetch = [&](const Batch &a, uint4 (&fa)[U], uint4 (&fb)[U]) {
        if (a.work >= n_work) return;
        // bases that a head's index h leads from, whatever it is a head of
        const long long tok = token_of(a);
        const __nv_bfloat16 *q_src = R.q + tok * R.q_row + da;
        const __nv_bfloat16 *k_src = R.k + tok * R.k_row + da - R.Hq * D;
        const __nv_bfloat16 *v_src = R.v + tok * R.v_row + da - (R.Hq + R.Hkv) * D;
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const int h = a.h0 + v * step + slot;
            if (h >= heads) continue;
            const __nv_bfloat16 *src =
                (h < R.Hq ? q_src : h < R.Hq + R.Hkv ? k_src : v_src) + h * D;
            fa[v] = __ldg(reinterpret_cast<const uint4 *>(src));
            fb[v] = __ldg(reinterpret_cast<const uint4 *>(src + (db - da)));
        }
    };
    // one batch is worked on while the next one's loads are in flight
    uint4 wa[U], wb[U], na[U], nb[U];
    Batch cur{blockIdx.x * (kRopeThreads / 32) + (tid >> 5), 0};
    cur.h0 = (int)(cur.work % R.parts) * RPW;
    fetch(cur, wa, wb);
    // (the tables' loads go out behind the first batch's)
    for (int i = tid; i < D; i += kRopeThreads) {
        w_s[0][i] = R.q_weight != nullptr ? R.q_weight[i] : 0.f;
        w_s[1][i] = R.k_weight != nullptr ? R.k_weight[i] : 0.f;
    }
    bool odd = false;
    for (int i = tid; i < R.rot / 2; i += kRopeThreads) {
        const float f = R.inv_freq[i];
        turn_s[i] = rope_turns(f);
        odd = odd || !rope_finite(f);
    }
    odd = __syncthreads_or(odd);
    if (tid == 0) odd_s = odd;
    __syncthreads();
    while (cur.work < n_work) {
        const int tok = token_of(cur);
        const int b = tok / q_len, i = tok - b * q_len;
        const long long pos = (long long)R.q_pos[b] + i;
        bool kv_live = true;            // the token's key and value rows are stored
        long long kv_step = D, row = 0;  // elements between heads' rows; the first one's
        if (R.to_cache) {
            const AttnParams &P = R.cache;
            kv_live = pos >= 0 && pos < P.L && pos < P.seq_lens[b];
            if (kv_live) {
                bool bad = false;
                row = cache_row(P, b, 0, (int)pos, &bad) * D;
                kv_live = !bad;
            }
            kv_step = (long long)(P.block_table != nullptr ? P.page_size : P.L) * D;
        } else {
            row = (long long)tok * R.Hkv * D;
        }
        __nv_bfloat16 *q_dst = R.q_out + (long long)tok * R.Hq * D + da;
        __nv_bfloat16 *k_dst = R.k_out + row + da - R.Hq * kv_step;
        __nv_bfloat16 *v_dst = R.v_out + row + da - (R.Hq + R.Hkv) * kv_step;
        // cosines and sines of the lane's pairs, two to a register pair
        uint64_t cs[4], sn[4];
        if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float c[2], s[2];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int n = (e < 2 ? pair0 : pair1) + 2 * (e & 1) + o;
                    rope_cos_sin((uint32_t)((turn_s[n] * (uint64_t)pos) >> 32), c[o], s[o]);
                }
                cs[e] = f2_pack(c[0], c[1]);
                sn[e] = f2_pack(s[0], s[1]);
            }
            // (looked up for every token: held in a register 72.9 us)
            if (odd_s) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = (e < 2 ? pair0 : pair1) + 2 * (e & 1);
                    const uint64_t none = f2_pack(rope_finite(R.inv_freq[n]) ? 0.f : kNan,
                                                  rope_finite(R.inv_freq[n + 1]) ? 0.f : kNan);
                    cs[e] = f2_add(cs[e], none);
                    sn[e] = f2_add(sn[e], none);
                }
            }
        }
        for (bool same = true; same;) {
            const int h0 = cur.h0;
            Batch nxt{cur.work, cur.h0 + U * step};
            same = nxt.h0 < heads;
            if (!same) {
                nxt.work += warps;
                nxt.h0 = (int)(nxt.work % R.parts) * RPW;
            }
            fetch(nxt, na, nb);
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const int h = h0 + v * step + slot;
                if (h0 + v * step >= heads) break;
                const bool live = h < heads;
                const int kind = h < R.Hq ? 0 : (h < R.Hq + R.Hkv ? 1 : 2);
                // the lane's 16 dims, as pairs of neighbours
                uint64_t x[8];
                {
                    const uint32_t w[8] = {wa[v].x, wa[v].y, wa[v].z, wa[v].w,
                                           wb[v].x, wb[v].y, wb[v].z, wb[v].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = f2_pack(bf16lo(w[e]), bf16hi(w[e]));
                }
                uint4 oa = wa[v], ob = wb[v];
                if (kind == 0 ? R.q_weight != nullptr : R.k_weight != nullptr) {
                    uint64_t s2 = f2_mul(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 8; ++e) s2 = f2_fma(x[e], x[e], s2);
                    float s0, s1;
                    f2_unpack(s2, s0, s1);
                    // (the lanes of a row hold the same kind of head)
                    const uint32_t row_lanes =
                        (LPR == 32 ? 0xffffffffu : (1u << LPR) - 1u) << (slot * LPR);
                    float ss = s0 + s1;
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1)
                        ss += __shfl_xor_sync(row_lanes, ss, off);
                    if (kind != 2) {
                        const float inv = rsqrtf(ss * (1.f / D) + R.eps);
                        const uint64_t inv2 = f2_pack(inv, inv);
                        uint64_t w[4];
                        rope_weights(w_s[kind] + da, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = f2_mul(f2_mul(x[e], inv2), w[e]);
                        rope_weights(w_s[kind] + db, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[4 + e] = f2_mul(f2_mul(x[4 + e], inv2), w[e]);
                    }
                }
                if (kind != 2) {
                    if (turns) {
                        if (R.interleaved) {
                            // pair e: both its members in x[e]
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float a, c, ct[2], st[2];
                                f2_unpack(x[e], a, c);
                                f2_unpack(cs[e >> 1], ct[0], ct[1]);
                                f2_unpack(sn[e >> 1], st[0], st[1]);
                                x[e] = f2_pack(a * ct[e & 1] - c * st[e & 1],
                                               c * ct[e & 1] + a * st[e & 1]);
                            }
                        } else {
                            // pairs 2 e and 2 e + 1: their members in x[e] and x[4 + e]
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint64_t a = x[e], c = x[4 + e];
                                x[e] = f2_sub(f2_mul(a, cs[e]), f2_mul(c, sn[e]));
                                x[4 + e] = f2_fma(c, cs[e], f2_mul(a, sn[e]));
                            }
                        }
                    }
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float a, c;
                        f2_unpack(x[e], a, c);
                        o[e] = pack_bf16x2(a, c);
                    }
                    oa = make_uint4(o[0], o[1], o[2], o[3]);
                    ob = make_uint4(o[4], o[5], o[6], o[7]);
                }
                if (live && (kind == 0 || kv_live)) {
                    __nv_bfloat16 *dst = (kind == 0 ? q_dst : kind == 1 ? k_dst : v_dst) +
                                         h * (kind == 0 ? (long long)D : kv_step);
                    *reinterpret_cast<uint4 *>(dst) = oa;
                    *reinterpret_cast<uint4 *>(dst + (db - da)) = ob;
                }
            }
#pragma unroll
            for (int v = 0; v < U; ++v) {
                wa[v] = na[v];
                wb[v] = nb[v];
            }
            cur = nxt;
        }
    }
}

}  // namespace swa
