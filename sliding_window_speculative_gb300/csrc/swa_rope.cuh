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
// D / 16 lanes hold one head row, 16 dims each: with the halves layout the 8
// dims [8l, 8l + 8) and their partners rot/2 further, so a lane owns both
// members of its pairs and no value crosses lanes but the sum of squares.  A
// warp works on one token (or a part of its heads): the angles depend on the
// token alone, so cosine and sine are computed once and used for all heads.
//
// Angles of far positions: f / 2 pi is held as a 64-bit binary fraction of a
// turn, and (q_pos + i) times it modulo 2^64 is the angle modulo one turn
// (exact but for f's own rounding, 2^-61 of it per position), where a product
// in fp32 would have lost the fraction.
#pragma once

#include "swa_simt.cuh"

namespace swa {

constexpr int kRopeThreads = 128;

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    long long q_row, k_row, v_row;  // elements between consecutive tokens
    const float *q_weight, *k_weight, *inv_freq;
    const int32_t *q_pos;
    __nv_bfloat16 *q_out, *k_out, *v_out;  // k_out / v_out unused with a cache
    AttnParams cache;  // k, v, seq_lens, block table, B, q_len, Hkv, L (cache form)
    int to_cache;
    int tokens, Hq, Hkv, rot, interleaved, parts;
    float eps;
};

// f / 2 pi as a fraction of a turn in units of 2^-64, modulo a turn:
// f = m 2^e with a 24-bit m, and K = round(2^64 / 2 pi).
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

template <int D>
__global__ void __launch_bounds__(kRopeThreads) swa_rope_kernel(const RopeParams R) {
    constexpr int LPR = D / 16;        // lanes per head row
    constexpr int RPW = 32 / LPR;      // head rows per warp and step
    __shared__ __align__(16) float w_s[2][D];
    __shared__ uint64_t turn_s[D / 2];
    const int tid = threadIdx.x, lane = tid & 31;
    const int l = lane % LPR, slot = lane / LPR;
    const int heads = R.Hq + 2 * R.Hkv;
    const int q_len = R.cache.q_len;
    grid_dep_wait();
    grid_dep_trigger();
    for (int i = tid; i < D; i += kRopeThreads) {
        w_s[0][i] = R.q_weight != nullptr ? R.q_weight[i] : 0.f;
        w_s[1][i] = R.k_weight != nullptr ? R.k_weight[i] : 0.f;
    }
    for (int i = tid; i < R.rot / 2; i += kRopeThreads) turn_s[i] = rope_turns(R.inv_freq[i]);
    __syncthreads();

    const bool turns = l < R.rot / 16;  // this lane's dims are rotated
    // first dims of the lane's two 8-dim pieces
    int da = 16 * l, db = 16 * l + 8;
    if (!R.interleaved && turns) {
        da = 8 * l;
        db = R.rot / 2 + 8 * l;
    }
    const long long n_work = (long long)R.tokens * R.parts;
    const int warps = gridDim.x * (kRopeThreads / 32);
    for (long long work = blockIdx.x * (kRopeThreads / 32) + (tid >> 5); work < n_work;
         work += warps) {
        const int tok = (int)(work / R.parts), part = (int)(work % R.parts);
        const int b = tok / q_len, i = tok - b * q_len;
        const int pos = R.q_pos[b] + i;
        long long row = -1;  // cache row of head 0 (cache form), -1: not stored
        long long head_rows = 0;
        if (R.to_cache) {
            const AttnParams &P = R.cache;
            if (pos >= 0 && pos < P.L && pos < P.seq_lens[b]) {
                bool bad = false;
                row = cache_row(P, b, 0, pos, &bad);
                if (bad) row = -1;
            }
            head_rows = P.block_table != nullptr ? P.page_size : P.L;
        }
        float cs[8], sn[8];
        if (turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t t = turn_s[8 * l + e] * (uint64_t)(int64_t)pos;
                // signed fraction of a turn, 32 bits of it: half turns for sincospi
                const float half = (float)(int32_t)(t >> 32) * 4.656612873077393e-10f;
                sincospif(half, &sn[e], &cs[e]);
            }
        }
        for (int h0 = part * RPW; h0 < heads; h0 += R.parts * RPW) {
            const int h = h0 + slot;
            const bool live = h < heads;
            const int kind = h < R.Hq ? 0 : (h < R.Hq + R.Hkv ? 1 : 2);
            const int hk = kind == 0 ? h : (kind == 1 ? h - R.Hq : h - R.Hq - R.Hkv);
            const __nv_bfloat16 *src =
                kind == 0   ? R.q + tok * R.q_row + (long long)hk * D
                : kind == 1 ? R.k + tok * R.k_row + (long long)hk * D
                            : R.v + tok * R.v_row + (long long)hk * D;
            uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
            if (live) {
                wa = __ldg(reinterpret_cast<const uint4 *>(src + da));
                wb = __ldg(reinterpret_cast<const uint4 *>(src + db));
            }
            float x[16];
            x[0] = bf16lo(wa.x); x[1] = bf16hi(wa.x); x[2] = bf16lo(wa.y); x[3] = bf16hi(wa.y);
            x[4] = bf16lo(wa.z); x[5] = bf16hi(wa.z); x[6] = bf16lo(wa.w); x[7] = bf16hi(wa.w);
            x[8] = bf16lo(wb.x); x[9] = bf16hi(wb.x); x[10] = bf16lo(wb.y); x[11] = bf16hi(wb.y);
            x[12] = bf16lo(wb.z); x[13] = bf16hi(wb.z); x[14] = bf16lo(wb.w); x[15] = bf16hi(wb.w);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            if (kind != 2) {
                if (kind == 0 ? R.q_weight != nullptr : R.k_weight != nullptr) {
                    const float inv = rsqrtf(ss * (1.f / D) + R.eps);
                    const float *w = w_s[kind];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] *= inv * w[da + e];
                        x[8 + e] *= inv * w[db + e];
                    }
                }
                if (turns) {
                    if (R.interleaved) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float a = x[2 * e], c = x[2 * e + 1];
                            x[2 * e] = a * cs[e] - c * sn[e];
                            x[2 * e + 1] = c * cs[e] + a * sn[e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float a = x[e], c = x[8 + e];
                            x[e] = a * cs[e] - c * sn[e];
                            x[8 + e] = c * cs[e] + a * sn[e];
                        }
                    }
                }
                wa = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
                wb = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]),
                                pack_bf16x2(x[12], x[13]), pack_bf16x2(x[14], x[15]));
            }
            __nv_bfloat16 *dst;
            bool store = live;
            if (kind == 0) {
                dst = R.q_out + ((long long)tok * R.Hq + hk) * D;
            } else if (R.to_cache) {
                store = live && row >= 0;
                dst = const_cast<__nv_bfloat16 *>(kind == 1 ? R.cache.k : R.cache.v) +
                      (row + hk * head_rows) * D;
            } else {
                dst = (kind == 1 ? R.k_out : R.v_out) + ((long long)tok * R.Hkv + hk) * D;
            }
            if (store) {
                *reinterpret_cast<uint4 *>(dst + da) = wa;
                *reinterpret_cast<uint4 *>(dst + db) = wb;
            }
        }
    }
}

}  // namespace swa
