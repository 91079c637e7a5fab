// Windowed verify attention over the 8-bit cache on the fp8 tensor cores
// (tcgen05 kind::f8f6f4), the e4m3 rows fed to them as they lie in the cache.
//
// The structure is that of the bf16 key-major kernel: persistent CTAs, keys as
// the MMA's M dimension, K and V tiles of 128 keys by TMA into a ring,
//
//   S^T[128 keys x 2N] = K8_tile[128 x D] . [Q_hi; Q_lo][2N x D]^T
//   O^T[D x 2N]       += V8_tile^T[D x 128] . [P_hi; P_lo][2N x 128]^T
//
// What is not 8-bit by nature is carried in two e4m3 numbers of four
// significant bits each:
//   q = 2^eq (q_hi + q_lo / 16), eq per query row.  A bf16 number has eight
//     significant bits, so this is exact down to 2^-14 of the row's largest
//     element and off by at most 2^-22 of it below.
//   P = p_hi + p_lo / 56: within 2^-9 of P, or within 2^-21 of the row's largest
//     P where that is more.  (56 is the largest 2^i m, m odd and at most 7,
//     that keeps the rest of a P up to 256 within 448; a P is first an fp16
//     number, whose rest times 7 is still exact.)
// Products of e4m3 numbers are exact and summed in fp32 (measured: within 2^-21
// of the summed magnitudes).
//
// The rows' exponents: a key's belong to one thread, which owns that key's
// column of scores.  k's scales its scores.  v's becomes part of the weight: the
// softmax runs on u = s + e_v (log2 units), so that P = 2^(u - ref) multiplies
// the bare v8, and the row sum adds P 2^-e_v.  The reference follows the largest
// u: weights are resolved relative to what they contribute to the result, so a
// heavy key of small values does not push the others below the format's range.
//
// Warp roles (384 threads): 0 TMA producer, 1 TMEM owner and MMA issuer, 2..9
// softmax (two warpgroups that split the rows), 10..11 the operands that are not
// copied as they are: query rows split into their two numbers, and the keys'
// exponents with the query rows' scales (a ring of tables, a few tiles ahead).
#pragma once

#include "swa_q8.cuh"
#include "swa_tc.cuh"

namespace swa {

constexpr int kQ8TcThreads = 384;
constexpr int kQ8Tabs = 4;          // tables of key and row scales
// The reference maximum of a row sits this far below the largest u of the tile
// that set it: P = 2^5.2 there, and a later tile may exceed it by 2^2.8 before
// the references are raised (P at most 2^8).  A lower one would cost the small
// weights' resolution (2^-10 / 56 / 2^5.2 = 2^-21 of the largest).
constexpr float kQ8RefBelow = 5.2f;
constexpr float kQ8RaiseAt = 8.f;
constexpr float kQ8PLo = 56.f;      // P_lo's scale
constexpr float kQ8QLo = 16.f;      // Q_lo's

struct Q8TcParams {
    TcParams T;
    const int8_t *k_exp, *v_exp;
};

// A tile's table: per key the factor of its scores (log2 units) and v's
// exponent, per packed row its query scale.
template <int N>
struct Q8Tab {
    float2 key[kTcTileKeys];
    float row[N];
};

template <int D, int N, int NT, int QB, int PB, int OB>
struct Q8Cfg {
    static constexpr int SLABS = D / 128;
    static constexpr int ATOM_BYTES = SLABS * 1024;  // 8 keys x D
    static constexpr int TILE_BYTES = (kTcTileKeys / 8) * ATOM_BYTES;
    static constexpr int Q_SLAB = 2 * N * 128;       // N hi + N lo rows of 128 elements
    static constexpr int Q_BUF = SLABS * Q_SLAB;
    // P: blocks of 32 columns, [block][key][32 bytes] with 32-byte swizzle;
    // columns: N hi, then N lo
    static constexpr int P_BLOCK = kTcTileKeys * 32;
    static constexpr int P_BUF = (2 * N / 32) * P_BLOCK;
    static constexpr int RING_OFF = 0;
    static constexpr int Q_OFF = RING_OFF + NT * TILE_BYTES;
    static constexpr int P_OFF = Q_OFF + QB * Q_BUF;
    static constexpr int TAB_OFF = P_OFF + PB * P_BUF;               // Q8Tab<N> [kQ8Tabs]
    static constexpr int RED_OFF = TAB_OFF + kQ8Tabs * (int)sizeof(Q8Tab<N>);  // float [2][4][N]
    static constexpr int LINV_OFF = RED_OFF + 2 * 4 * N * 4;         // float [N]
    static constexpr int ALPHA_OFF = LINV_OFF + N * 4;               // float [N]
    static constexpr int ROW_OFF = ALPHA_OFF + N * 4;                // uint32 [N] output rows
    static constexpr int META_OFF = ROW_OFF + N * 4;                 // TcItem [kTcMetaItems]
    static constexpr int FTAB_OFF = META_OFF + kTcMetaItems * (int)sizeof(TcItem);
    static constexpr int BAR_OFF = (FTAB_OFF + kFillTab * 4 + 7) / 8 * 8;
    static constexpr int B_FULL = 0, B_EMPTY = NT, B_QFULL = 2 * NT, B_QEMPTY = B_QFULL + QB,
                         B_SFULL = B_QEMPTY + QB, B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2,
                         B_PVDONE = B_PFULL + PB, B_OFREE = B_PVDONE + PB, B_DRAIN = B_OFREE + 2,
                         B_TFULL = B_DRAIN + 1, B_TEMPTY = B_TFULL + kQ8Tabs,
                         NBARS = B_TEMPTY + kQ8Tabs;
    static constexpr int B_MIX = 0;  // (the producer's fused appends: none here)
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
    static constexpr int END = MISC_OFF + 16;
    static constexpr int SMEM_BYTES = END + 1024;
    static constexpr int O_COLS = (D / 128) * 2 * N;  // one O^T buffer: hi and lo halves
    static constexpr int S_COLS = 2 * N;              // one S^T buffer: hi and lo halves
    static constexpr int O_COL = 2 * S_COLS;
    static constexpr int TMEM_USED = O_COL + OB * O_COLS;
    static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
    static_assert(N == 16 || N == 32 || N == 64, "rows per tile");
    static_assert(NT >= 2 && NT <= 16, "ring slots");
    static_assert(TMEM_USED <= 512, "TMEM");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(Q_OFF % 1024 == 0 && P_OFF % 1024 == 0, "operand alignment");
    static_assert(RED_OFF % 16 == 0 && META_OFF % 8 == 0, "alignment");
};

namespace tc {

// As smem_desc_sw128 with the 32-byte swizzle: of an MN-major operand, blocks of
// 32 bytes along MN lbo apart, groups of 8 along K sbo apart.
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr, uint32_t lbo_bytes,
                                                   uint32_t sbo_bytes) {
    return (smem_desc_sw128(saddr, lbo_bytes, sbo_bytes) & ~((uint64_t)7 << 61)) |
           ((uint64_t)6 << 61);
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T, K = 32, single issuing thread.
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

}  // namespace tc

// 2^e for any int8 e, kept finite and normal.
__device__ __forceinline__ float q8_pow2(int e) { return pow2f(e < -126 ? -126 : e); }

// Two floats in [0, 448] as fp16, then as e4m3 hi and lo = e4m3((fp16 - hi) 56):
// bytes of the first in the low halves.
__device__ __forceinline__ void split_p(float p0, float p1, uint16_t &hi, uint16_t &lo) {
    const __half2 p = __floats2half2_rn(p0, p1);
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
        : "=h"(hi)
        : "r"(*reinterpret_cast<const uint32_t *>(&p)));
    const uint32_t hb = e4m3x2_to_f16x2(hi);
    const __half2 r = __hmul2(__hsub2(p, *reinterpret_cast<const __half2 *>(&hb)),
                              __floats2half2_rn(kQ8PLo, kQ8PLo));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
        : "=h"(lo)
        : "r"(*reinterpret_cast<const uint32_t *>(&r)));
}

// Warps 10 and 11: the query rows of every item as two e4m3 numbers each, and
// per tile the table of key and row scales.  Warp w of the two takes rows w,
// w + 2, ..., (RP at a time), the lane i keeping the scale of its i-th row, and
// keys 64 w ...
template <class C, int D, int N, int QB>
__device__ __forceinline__ void q8_operands(const Q8TcParams &A, const TcItem *meta, uint8_t *qs,
                                            Q8Tab<N> *tabs, uint64_t *bars, int w) {
    using namespace tc;
    const TcParams &T = A.T;
    const AttnParams &P = T.a;
    constexpr int LPR = D / 8, RP = 32 / LPR;  // lanes per row, rows per pass
    constexpr int U = 4;                       // passes in flight
    const int lane = (int)(threadIdx.x & 31);
    const int sub = lane / LPR, l = lane % LPR;
    uint32_t g = 0, k = 0;
    const int n_items = cta_items(T);
    for (int j = 0; j < n_items; ++j) {
        const TcItem it = tc_decode<false>(T, cta_item(T, j), j, meta);
        if (it.n_tiles == 0) continue;
        const uint32_t qb = k % QB, quse = k / QB;
        ++k;
        uint8_t *q = qs + qb * C::Q_BUF;
        float scale = 1.f;  // of row w + 2 * lane
        bool waited = false;
        const int mine = (it.rows - w + 1) / 2;  // rows w, w + 2, ... of this warp
        for (int i0 = 0; i0 < mine; i0 += RP * U) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = w + 2 * (i0 + u * RP + sub);
                x[u] = make_uint4(0, 0, 0, 0);
                if (r < it.rows) {
                    const int rg = it.row0 + r, i = rg / P.G, gg = rg - i * P.G;
                    const size_t row = ((size_t)it.b * P.q_len + i) * P.Hq + (size_t)it.h * P.G + gg;
                    x[u] = __ldg(reinterpret_cast<const uint4 *>(P.q + row * D) + l);
                }
            }
            if (!waited) {
                // the buffer's previous rows are done with
                if (!mbar_wait_bounded(&bars[C::B_QEMPTY + qb], (quse & 1) ^ 1, P.fault,
                                       kFaultCopyTimeout, P.wait_limit))
                    return;
                waited = true;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t b[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                float f[8], a = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = bf16lo(b[e]);
                    f[2 * e + 1] = bf16hi(b[e]);
                    a = fmaxf(a, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
                }
#pragma unroll
                for (int off = LPR / 2; off >= 1; off >>= 1)
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                // the smallest exponent that holds the row, as for the cache
                const uint32_t ab = __float_as_uint(a);
                int e = (int)(ab >> 23) - 135 + ((ab & 0x7fffffu) > 0x600000u ? 1 : 0);
                e = e < -126 ? -126 : (e > 126 ? 126 : e);
                const float sc = pow2f(-e);
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float y0 = f[2 * p] * sc, y1 = f[2 * p + 1] * sc;
                    const uint16_t h = e4m3x2(y0, y1);
                    const uint32_t hb = e4m3x2_to_f16x2(h);
                    const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hb));
                    const uint16_t r = e4m3x2((y0 - hf.x) * kQ8QLo, (y1 - hf.y) * kQ8QLo);
                    if (p & 1) {
                        hi[p >> 1] |= (uint32_t)h << 16;
                        lo[p >> 1] |= (uint32_t)r << 16;
                    } else {
                        hi[p >> 1] = h;
                        lo[p >> 1] = r;
                    }
                }
                const int i = i0 + u * RP + sub, r = w + 2 * i;
#pragma unroll
                for (int s = 0; s < RP; ++s) {
                    const float v = __shfl_sync(0xffffffffu, pow2f(e), s * LPR);
                    if (lane == i0 + u * RP + s) scale = v;
                }
                if (r < it.rows) {
                    // 8 bytes at element 8 l: 16-byte chunk (l / 2) % 8 of slab l / 16
                    const uint32_t ch = (uint32_t)(l >> 1) & 7;
                    const uint32_t at = (uint32_t)(l >> 4) * C::Q_SLAB + (uint32_t)(l & 1) * 8;
                    // (N is a multiple of 8: both rows have the same swizzle phase)
                    const uint32_t sw = (ch ^ (uint32_t)(r & 7)) << 4;
                    *reinterpret_cast<uint2 *>(q + at + r * 128 + sw) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(q + at + (N + r) * 128 + sw) =
                        make_uint2(lo[0], lo[1]);
                }
            }
        }
        if (!waited &&
            !mbar_wait_bounded(&bars[C::B_QEMPTY + qb], (quse & 1) ^ 1, P.fault, kFaultCopyTimeout,
                               P.wait_limit))
            return;
        fence_proxy_async_smem();
        mbar_arrive(&bars[C::B_QFULL + qb]);

        for (int t = 0; t < it.n_tiles; ++t, ++g) {
            float2 key[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int jk = it.t0 + kTcTileKeys * t + 64 * w + 32 * c + lane;
                int ke = 0, ve = 0;
                if (jk >= it.cr.c_lo && jk < it.cr.c_hi) {
                    const long long row = cache_row(P, it.b, it.h, jk);
                    ke = A.k_exp[row];
                    ve = A.v_exp[row];
                }
                key[c] = make_float2(P.qk_scale * q8_pow2(ke), (float)ve);
            }
            const uint32_t slot = g % kQ8Tabs;
            if (!mbar_wait_bounded(&bars[C::B_TEMPTY + slot], ((g / kQ8Tabs) & 1) ^ 1, P.fault,
                                   kFaultCopyTimeout, P.wait_limit))
                return;
            tabs[slot].key[64 * w + lane] = key[0];
            tabs[slot].key[64 * w + 32 + lane] = key[1];
            if (lane < N / 2) tabs[slot].row[w + 2 * lane] = scale;
            mbar_arrive(&bars[C::B_TFULL + slot]);
        }
    }
}

template <int D, int N, int NT, int QB, int PB, int OB>
__global__ void __launch_bounds__(kQ8TcThreads, 1)
    swa_q8_tc_kernel(const __grid_constant__ Q8TcParams A, const __grid_constant__ TcMaps M) {
    using C = Q8Cfg<D, N, NT, QB, PB, OB>;
    using namespace tc;
    constexpr int MH = D / 128;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const TcParams &T = A.T;
    const AttnParams &P = T.a;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    uint8_t *ring = sm + C::RING_OFF;
    uint8_t *qs = sm + C::Q_OFF;
    uint8_t *ps = sm + C::P_OFF;
    Q8Tab<N> *tabs = reinterpret_cast<Q8Tab<N> *>(sm + C::TAB_OFF);
    float *red = reinterpret_cast<float *>(sm + C::RED_OFF);
    float *linv = reinterpret_cast<float *>(sm + C::LINV_OFF);
    float *alpha_sm = reinterpret_cast<float *>(sm + C::ALPHA_OFF);
    uint32_t *rowidx = reinterpret_cast<uint32_t *>(sm + C::ROW_OFF);
    TcItem *meta = reinterpret_cast<TcItem *>(sm + C::META_OFF);
    volatile uint32_t *ftab = reinterpret_cast<volatile uint32_t *>(sm + C::FTAB_OFF);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::BAR_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC_OFF);

    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;

    // ---------------------------------------------------------------- setup
    if (warp == 0 && lane < 10) {
        const CUtensorMap *mp = lane < 4    ? &M.k_atoms[lane]
                                : lane < 8  ? &M.v_atoms[lane - 4]
                                : lane == 8 ? &M.k_atom
                                            : &M.v_atom;
        prefetch_tmap(mp);
    }
    if (tid == 0) {
        for (int i = 0; i < NT; ++i) {
            mbar_init(&bars[C::B_FULL + i], 1);
            mbar_init(&bars[C::B_EMPTY + i], 1);
        }
        for (int i = 0; i < QB; ++i) {
            mbar_init(&bars[C::B_QFULL + i], 64);
            mbar_init(&bars[C::B_QEMPTY + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[C::B_SFULL + i], 1);
            mbar_init(&bars[C::B_SFREE + i], 256);
            mbar_init(&bars[C::B_OFREE + i], 256);
        }
        for (int i = 0; i < PB; ++i) {
            mbar_init(&bars[C::B_PFULL + i], 256);
            mbar_init(&bars[C::B_PVDONE + i], 1);
        }
        for (int i = 0; i < kQ8Tabs; ++i) {
            mbar_init(&bars[C::B_TFULL + i], 64);
            mbar_init(&bars[C::B_TEMPTY + i], 256);
        }
        mbar_init(&bars[C::B_DRAIN], 1);
        fence_barrier_init();
    }
    // query rows past an item's stay what they are here: zero, or another
    // item's (their columns are never looked at, but should not raise the
    // references either)
    for (int i = tid; i < QB * C::Q_BUF / 16; i += kQ8TcThreads)
        reinterpret_cast<uint4 *>(qs)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    for (int i = tid; i < kFillTab; i += kQ8TcThreads) ftab[i] = 0xffffffffu;
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_trigger();
    if (lane == 0) issue_early_fills<C, NT, false, false, false>(T, M, ftab, ring, qs, bars, warp);
    for (int j = tid; j < kTcMetaItems; j += kQ8TcThreads)
        if (j < cta_items(T)) meta[j] = tc_decode_global<false>(T, cta_item(T, j));
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ======================================================= producer
        tile_producer<C, NT, QB, false, false, false>(T, M, meta, ftab, ring, qs, bars, true);
    } else if (warp == 1) {
        // ============================================================ MMA
        // The event loop of the bf16 key-major kernel: S of the next tile and
        // PV of the oldest tile whose P is ready, each as soon as its operands
        // have landed.
        const bool leader = lane == 0;
        constexpr uint32_t ID_QK = idesc_e4m3_f32(128, 2 * N, 0, 0);
        constexpr uint32_t ID_PV = idesc_e4m3_f32(128, 2 * N, 1, 1);
        const uint32_t ring_a = smem_u32(ring);
        const uint32_t qs_a = smem_u32(qs);
        const uint32_t ps_a = smem_u32(ps);
        struct Cursor {
            int j, t, n_tiles;
            int last_keys;  // keys of the item's last tile
            int head;       // key rows before the chunk in its first tile (paged cache)
            uint32_t k, g;
            bool valid;
            int slot;       // this cursor's fill: slot, parity (-1: not yet looked up)
            uint32_t par;
        };
        auto lookup = [&](Cursor &c, uint32_t fill) -> bool {
            if (c.slot >= 0) return true;
            const uint32_t e = ftab[fill % kFillTab];
            if ((e >> 8) != (fill & 0xffffffu)) return false;
            c.slot = (int)(e & 15u);
            c.par = (e >> 4) & 1u;
            return true;
        };
        const int n_items = cta_items(T);
        auto seek = [&](Cursor &c) {
            for (; c.j < n_items; ++c.j) {
                const TcItem it = tc_decode<false>(T, cta_item(T, c.j), c.j, meta);
                if (it.n_tiles > 0) {
                    c.n_tiles = it.n_tiles;
                    c.last_keys = it.cr.c_hi - it.t0 - kTcTileKeys * (it.n_tiles - 1);
                    c.head = it.cr.c_lo - it.t0;
                    c.t = 0;
                    c.valid = true;
                    return;
                }
            }
            c.valid = false;
        };
        auto advance = [&](Cursor &c) {
            ++c.g;
            c.slot = -1;
            if (++c.t < c.n_tiles) return;
            ++c.k;
            ++c.j;
            seek(c);
        };
        Cursor qc{0, 0, 0, 0, 0, 0u, 0u, false, -1, 0u};
        seek(qc);
        Cursor pc = qc;
        long long idle_since = clock64();
        while (pc.valid) {
            bool progressed = false;
            // ---- PV of tile pc.g (its S was issued before)
            if (pc.g < qc.g || !qc.valid) {
                const uint32_t pb = pc.g % PB;
                bool ready = mbar_test(&bars[C::B_PFULL + pb], (pc.g / PB) & 1);
                if (ready && pc.t == 0)
                    ready = mbar_test(&bars[C::B_OFREE + pc.k % OB], ((pc.k / OB) & 1) ^ 1);
                ready = ready && lookup(pc, 2 * pc.g + 1) &&
                        mbar_test(&bars[C::B_FULL + pc.slot], pc.par);
                const uint32_t vslot = (uint32_t)pc.slot;
                if (ready) {
                    fence_after_sync();
                    // only the 32-key steps that hold valid keys are multiplied; the
                    // rows of the last step past the chunk's end, and those before
                    // the chunk in a paged cache's first tile, are zeroed first, so
                    // that 0 * (whatever the slot holds there) cannot reach O
                    const int nv = pc.t == pc.n_tiles - 1 ? pc.last_keys : kTcTileKeys;
                    const int steps = (nv + 31) >> 5;
                    uint8_t *vt = ring + vslot * C::TILE_BYTES;
                    const int z = pc.t == 0 ? pc.head : 0;
                    if ((nv & 31) || z > 0) {
                        zero_v_rows<C>(vt, nv, 32 * steps, lane);
                        zero_v_rows<C>(vt, 0, z, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (leader) {
                        // A = V^T, MN-major: a slab holds 128 dims, 8-key groups one
                        // atom apart; B = [P_hi; P_lo], MN-major, 2N columns
                        const uint64_t bbase =
                            smem_desc_sw32(ps_a + pb * C::P_BUF, C::P_BLOCK, 256);
                        const uint64_t abase = smem_desc_sw128(ring_a + vslot * C::TILE_BYTES, 16,
                                                               C::ATOM_BYTES);
                        const uint32_t ob = pc.k % OB;
                        const uint32_t acc0 = pc.t > 0 ? 1u : 0u;
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            if (k4 >= steps) break;
#pragma unroll
                            for (int mh = 0; mh < MH; ++mh)
                                mma_e4m3_ss(tmem + C::O_COL + ob * C::O_COLS + mh * 2 * N,
                                            abase + (uint64_t)((mh * 1024 + k4 * 4 * C::ATOM_BYTES) >> 4),
                                            bbase + (uint64_t)(k4 * 1024 >> 4), ID_PV,
                                            (acc0 | (uint32_t)k4) != 0);
                        }
                        mma_commit(&bars[C::B_EMPTY + vslot]);
                        mma_commit(&bars[C::B_PVDONE + pb]);
                    }
                    __syncwarp();
                    advance(pc);
                    progressed = true;
                }
            }
            // ---- S of tile qc.g, at most one tile ahead of the PV cursor
            if (qc.valid && qc.g <= pc.g + 1) {
                const uint32_t sb = qc.g & 1;
                const bool ready = mbar_test(&bars[C::B_SFREE + sb], ((qc.g >> 1) & 1) ^ 1) &&
                                   mbar_test(&bars[C::B_QFULL + qc.k % QB], (qc.k / QB) & 1) &&
                                   lookup(qc, 2 * qc.g) &&
                                   mbar_test(&bars[C::B_FULL + qc.slot], qc.par);
                const uint32_t kslot = (uint32_t)qc.slot;
                if (ready) {
                    fence_after_sync();
                    if (leader) {
                        const uint64_t qbase =
                            smem_desc_sw128(qs_a + (qc.k % QB) * C::Q_BUF, 16, 1024);
                        const uint64_t abase =
                            smem_desc_sw128(ring_a + kslot * C::TILE_BYTES, 16, C::ATOM_BYTES);
#pragma unroll
                        for (int s = 0; s < C::SLABS; ++s)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_e4m3_ss(tmem + sb * C::S_COLS,
                                            abase + (uint64_t)(s * 64 + kk * 2),
                                            qbase + (uint64_t)(s * (C::Q_SLAB >> 4) + kk * 2), ID_QK,
                                            (s | kk) != 0);
                        mma_commit(&bars[C::B_EMPTY + kslot]);
                        mma_commit(&bars[C::B_SFULL + sb]);
                        if (qc.t == qc.n_tiles - 1) mma_commit(&bars[C::B_QEMPTY + qc.k % QB]);
                    }
                    __syncwarp();
                    advance(qc);
                    progressed = true;
                }
            }
            if (progressed) {
                idle_since = clock64();
            } else if (clock64() - idle_since > P.wait_limit) {
                atomicOr(P.fault, kFaultCopyTimeout);
                break;
            }
        }
        // all issued MMAs complete before TMEM is released
        if (leader) {
            mma_commit(&bars[C::B_DRAIN]);
            mbar_wait_bounded(&bars[C::B_DRAIN], 0, P.fault, kFaultCopyTimeout, P.wait_limit);
        }
        __syncwarp();
    } else if (warp < 10) {
        // ===================================================== softmax
        constexpr int HN = N / 2;                // rows per softmax warpgroup
        constexpr int OW = HN >= 16 ? 16 : 8;    // TMEM columns per O or S load
        constexpr int NCH = HN / OW;
        const int wg = (warp - 2) >> 2;          // softmax warpgroup
        const int sw = (warp - 2) & 3;           // warp within the group
        const int quad = warp & 3;               // TMEM lane quadrant of this warp
        const int lk = quad * 32 + lane;         // TMEM lane: key of S^T, dim row of O^T
        const int gtid = sw * 32 + lane;         // 0..127 within the group
        const int r0 = wg * HN;                  // first packed row of this group
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t flip = (uint32_t)(lk >> 2) & 1;  // 32-byte swizzle phase of key lk
        uint32_t g = 0, k = 0;
        bool ok = true;
        const int n_items = cta_items(T);
        for (int j = 0; j < n_items && ok; ++j) {
            const TcItem it = tc_decode<false>(T, cta_item(T, j), j, meta);
            const size_t bh = (size_t)it.b * P.Hkv + it.h;
            const int my_rows = min(HN, it.rows - r0);  // rows of this group in the item
            if (it.n_tiles == 0) {
                // no key in this chunk: empty result for every row
                for (int idx = gtid; idx < my_rows * D; idx += 128) {
                    const int r = it.row0 + r0 + idx / D, d = idx % D;
                    const int i = r / P.G, gg = r - i * P.G;
                    const size_t orow =
                        ((size_t)it.b * P.q_len + i) * P.Hq + (size_t)it.h * P.G + gg;
                    if (P.splits == 1) {
                        P.out[orow * D + d] = __float2bfloat16_rn(0.f);
                        if (d == 0 && P.lse != nullptr) P.lse[orow] = NEG_INF;
                    } else {
                        const size_t prow = (bh * P.splits + it.split) * P.R + r;
                        P.part_acc[prow * D + d] = 0.f;
                        if (d == 0) {
                            P.part_ml[prow * 2] = NEG_INF;
                            P.part_ml[prow * 2 + 1] = 0.f;
                        }
                    }
                }
                continue;
            }
            const uint32_t ob = k % OB;
            const uint32_t ocol0 = tl + C::O_COL + ob * C::O_COLS;  // this lane's O^T row
            float mref[HN], lrow[HN];
#pragma unroll
            for (int r = 0; r < HN; ++r) {
                mref[r] = kNoRef;
                lrow[r] = 0.f;
            }

            const int qp_i0 = it.cr.qp + it.i0;  // position of the item's first draft row
            for (int t = 0; t < it.n_tiles; ++t, ++g) {
                const uint32_t sb = g & 1, slot = g % kQ8Tabs;
                const int j0 = it.t0 + kTcTileKeys * t;
                const int jk = j0 + lk;
                // packed rows [ra, rb) of this group whose window holds key jk
                int ra = 0, rb = 0;
                if (jk >= it.cr.c_lo && jk < it.cr.c_hi) {
                    const long long lo_i = (long long)jk - qp_i0;
                    const long long hi_i = (long long)jk + P.window - qp_i0;
                    const long long a = lo_i < 0 ? 0 : lo_i * P.G;
                    long long bnd = hi_i < 0 ? 0 : hi_i * P.G;
                    if (bnd > it.rows) bnd = it.rows;
                    ra = (int)(a < it.rows ? a : it.rows) - r0;
                    rb = (int)bnd - r0;
                }
                bool got = mbar_wait_bounded(&bars[C::B_TFULL + slot], (g / kQ8Tabs) & 1, P.fault,
                                             kFaultCopyTimeout, P.wait_limit);
                const float2 key = tabs[slot].key[lk];
                got = got && mbar_wait_bounded(&bars[C::B_SFULL + sb], (g >> 1) & 1, P.fault,
                                               kFaultCopyTimeout, P.wait_limit);
                fence_after_sync();
                // u = (S_hi + S_lo / 16) * row scale * key factor + e_v
                float v[HN];
                {
                    const uint64_t lo2 = f2_pack(1.f / kQ8QLo, 1.f / kQ8QLo);
                    const uint64_t ks2 = f2_pack(key.x, key.x), ve2 = f2_pack(key.y, key.y);
                    const bool all = ra <= 0 && rb >= HN;
                    uint32_t hi[HN], lo[HN];
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        tmem_load<OW>(tl + sb * C::S_COLS + r0 + c * OW, hi + c * OW);
                        tmem_load<OW>(tl + sb * C::S_COLS + N + r0 + c * OW, lo + c * OW);
                    }
                    tmem_wait_ld();
                    fence_before_sync();
                    mbar_arrive(&bars[C::B_SFREE + sb]);
#pragma unroll
                    for (int r4 = 0; r4 < HN; r4 += 4) {
                        const float4 rs = *reinterpret_cast<const float4 *>(&tabs[slot].row[r0 + r4]);
                        const uint64_t rs2[2] = {f2_pack(rs.x, rs.y), f2_pack(rs.z, rs.w)};
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const int r = r4 + 2 * p;
                            const uint64_t s2 =
                                f2_fma(f2_pack(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1])),
                                       lo2,
                                       f2_pack(__uint_as_float(hi[r]), __uint_as_float(hi[r + 1])));
                            f2_unpack(f2_fma(f2_mul(s2, rs2[p]), ks2, ve2), v[r], v[r + 1]);
                        }
                    }
                    mbar_arrive(&bars[C::B_TEMPTY + slot]);
                    if (!all) {
#pragma unroll
                        for (int r = 0; r < HN; ++r)
                            if (r < ra || r >= rb) v[r] = NEG_INF;
                    }
                }

                bool flag = false;
#pragma unroll
                for (int r = 0; r < HN; ++r) flag |= v[r] > mref[r] + kQ8RaiseAt;
                const bool raise = group_any(wg, flag || !got);
                if (raise) {
                    ok = !group_any(wg, !got);
                    if (!ok) break;
                    // exact tile maximum per row; raise the references
                    float *rd = red + (g & 1) * 4 * N + r0;
                    constexpr int CW = HN >= 32 ? 32 : HN;
#pragma unroll
                    for (int c = 0; c < HN / CW; ++c) {
                        float tmp[CW];
#pragma unroll
                        for (int e = 0; e < CW; ++e) tmp[e] = v[c * CW + e];
                        const float m = lane_reduce<CW, true>(tmp);
                        if (lane < CW) rd[sw * N + c * CW + lane] = m;
                    }
                    group_sync(wg);
                    const bool rescale = t > 0;
                    float my_alpha = 1.f;
#pragma unroll
                    for (int r4 = 0; r4 < HN; r4 += 4) {
                        const float4 a0 = *reinterpret_cast<const float4 *>(rd + r4);
                        const float4 a1 = *reinterpret_cast<const float4 *>(rd + N + r4);
                        const float4 a2 = *reinterpret_cast<const float4 *>(rd + 2 * N + r4);
                        const float4 a3 = *reinterpret_cast<const float4 *>(rd + 3 * N + r4);
                        const float tm[4] = {fmaxf(fmaxf(a0.x, a1.x), fmaxf(a2.x, a3.x)),
                                             fmaxf(fmaxf(a0.y, a1.y), fmaxf(a2.y, a3.y)),
                                             fmaxf(fmaxf(a0.z, a1.z), fmaxf(a2.z, a3.z)),
                                             fmaxf(fmaxf(a0.w, a1.w), fmaxf(a2.w, a3.w))};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = r4 + e;
                            const float mo = mref[r];
                            const float mn = fmaxf(mo, tm[e] - kQ8RefBelow);
                            if (rescale) {
                                const float al = mn == mo ? 1.f : fast_exp2(mo - mn);
                                if (gtid == r) my_alpha = al;
                                lrow[r] *= al;
                            }
                            mref[r] = mn;
                        }
                    }
                    if (rescale) {
                        if (gtid < HN) alpha_sm[r0 + gtid] = my_alpha;
                        // every PV of this item so far has completed before O is scaled
                        const uint32_t gp = g - 1;
                        ok = !group_any(wg, !mbar_wait_bounded(&bars[C::B_PVDONE + gp % PB],
                                                               (gp / PB) & 1, P.fault,
                                                               kFaultCopyTimeout, P.wait_limit));
                        if (!ok) break;
                        fence_after_sync();  // (the vote also published alpha_sm)
#pragma unroll 1
                        for (int mh = 0; mh < 2 * MH; ++mh) {  // hi and lo halves of each
#pragma unroll 1
                            for (int c0 = 0; c0 < HN; c0 += OW) {
                                uint32_t o[OW];
                                const uint32_t ocol = ocol0 + mh * N + r0 + c0;
                                tmem_load<OW>(ocol, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < OW; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) *
                                                           alpha_sm[r0 + c0 + e]);
                                tmem_store<OW>(ocol, o);
                            }
                        }
                        tmem_wait_st();
                    }
                }
                // P buffer free: its previous PV has completed
                const uint32_t pb = g % PB;
                if (g >= (uint32_t)PB) {
                    const uint32_t gp = g - PB;
                    ok = !group_any(wg, !mbar_wait_bounded(&bars[C::B_PVDONE + pb], (gp / PB) & 1,
                                                           P.fault, kFaultCopyTimeout,
                                                           P.wait_limit));
                    if (!ok) break;
                }
                // P = 2^(u - ref) as two e4m3 numbers; the row sum adds P 2^-e_v
                const float ive = pow2f(-(int)key.y < -126 ? -126 : (int)-key.y > 127 ? 127 : (int)-key.y);
                const uint64_t iv2 = f2_pack(ive, ive);
                uint32_t ph[HN / 4], pl[HN / 4];
#pragma unroll
                for (int r = 0; r < HN; r += 2) {
                    float d0, d1;
                    f2_unpack(f2_sub(f2_pack(v[r], v[r + 1]), f2_pack(mref[r], mref[r + 1])), d0, d1);
                    const float p0 = fast_exp2(d0), p1 = fast_exp2(d1);
                    f2_unpack(f2_fma(f2_pack(p0, p1), iv2, f2_pack(lrow[r], lrow[r + 1])), lrow[r],
                              lrow[r + 1]);
                    uint16_t h, l;
                    split_p(p0, p1, h, l);
                    if (r & 2) {
                        ph[r / 4] |= (uint32_t)h << 16;
                        pl[r / 4] |= (uint32_t)l << 16;
                    } else {
                        ph[r / 4] = h;
                        pl[r / 4] = l;
                    }
                }
                // columns r0 .. of hi and N + r0 .. of lo, key lk's 32-byte rows
                uint8_t *pt = ps + pb * C::P_BUF + lk * 32;
                if constexpr (HN == 8) {
                    *reinterpret_cast<uint2 *>(pt + (flip << 4) + wg * 8) = make_uint2(ph[0], ph[1]);
                    *reinterpret_cast<uint2 *>(pt + ((flip ^ 1) << 4) + wg * 8) =
                        make_uint2(pl[0], pl[1]);
                } else if constexpr (HN == 16) {
                    const uint32_t ch = ((uint32_t)wg ^ flip) << 4;
                    *reinterpret_cast<uint4 *>(pt + ch) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                    *reinterpret_cast<uint4 *>(pt + C::P_BLOCK + ch) =
                        make_uint4(pl[0], pl[1], pl[2], pl[3]);
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t ch = ((uint32_t)c ^ flip) << 4;
                        *reinterpret_cast<uint4 *>(pt + wg * C::P_BLOCK + ch) =
                            make_uint4(ph[4 * c], ph[4 * c + 1], ph[4 * c + 2], ph[4 * c + 3]);
                        *reinterpret_cast<uint4 *>(pt + (2 + wg) * C::P_BLOCK + ch) =
                            make_uint4(pl[4 * c], pl[4 * c + 1], pl[4 * c + 2], pl[4 * c + 3]);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars[C::B_PFULL + pb]);
            }
            if (!ok) break;

            // -------------------------------------------------- epilogue
            // row sums (they do not depend on the last PV): lanes, then the
            // group's four warps
            float *rl = red + (g & 1) * 4 * N + r0;
            {
                constexpr int CW = HN >= 32 ? 32 : HN;
#pragma unroll
                for (int c = 0; c < HN / CW; ++c) {
                    float tmp[CW];
#pragma unroll
                    for (int e = 0; e < CW; ++e) tmp[e] = lrow[c * CW + e];
                    const float s = lane_reduce<CW, false>(tmp);
                    if (lane < CW) rl[sw * N + c * CW + lane] = s;
                }
            }
            group_sync(wg);
            if (gtid < my_rows) {
                const int r = gtid;
                const float l = (rl[r] + rl[N + r]) + (rl[2 * N + r] + rl[3 * N + r]);
                float m = NEG_INF;
#pragma unroll
                for (int q = 0; q < HN; ++q)
                    if (q == r) m = mref[q];
                const bool any = !(l <= 0.f);  // (a NaN stays one)
                linv[r0 + r] = any ? __frcp_rn(l) : 0.f;
                const int rg = it.row0 + r0 + r;
                if (P.splits == 1) {
                    const int i = rg / P.G, gg = rg - i * P.G;
                    const uint32_t orow =
                        (uint32_t)(((size_t)it.b * P.q_len + i) * P.Hq + (size_t)it.h * P.G + gg);
                    rowidx[r0 + r] = orow;
                    if (P.lse != nullptr) P.lse[orow] = any ? (m + __log2f(l)) * kLn2 : NEG_INF;
                } else {
                    const size_t prow = (bh * P.splits + it.split) * P.R + rg;
                    P.part_ml[prow * 2] = any ? m : NEG_INF;
                    P.part_ml[prow * 2 + 1] = l;
                }
            }
            const uint32_t gl = g - 1;  // the item's last tile
            ok = !group_any(wg, !mbar_wait_bounded(&bars[C::B_PVDONE + gl % PB], (gl / PB) & 1,
                                                   P.fault, kFaultCopyTimeout, P.wait_limit));
            if (!ok) break;
            fence_after_sync();  // (the vote also published linv and rowidx)
            const size_t prow0 = (bh * P.splits + it.split) * P.R + it.row0 + r0;
#pragma unroll
            for (int mh = 0; mh < MH; ++mh) {
                const int d = mh * 128 + lk;
#pragma unroll
                for (int c0 = 0; c0 < HN; c0 += OW) {
                    uint32_t o[OW], ol[OW];
                    tmem_load<OW>(ocol0 + mh * 2 * N + r0 + c0, o);
                    tmem_load<OW>(ocol0 + mh * 2 * N + N + r0 + c0, ol);
                    tmem_wait_ld();
                    if (mh == MH - 1 && c0 == HN - OW) {
                        fence_before_sync();
                        mbar_arrive(&bars[C::B_OFREE + ob]);  // O buffer may be reused
                    }
                    float x[OW];
#pragma unroll
                    for (int e = 0; e < OW; ++e)
                        x[e] = fmaf(__uint_as_float(ol[e]), 1.f / kQ8PLo, __uint_as_float(o[e]));
                    if (P.splits == 1) {
                        // neighbouring lanes hold neighbouring dims: each pair swaps
                        // halves of two rows, so a lane stores two dims of one row
#pragma unroll
                        for (int e = 0; e < OW; e += 2) {
                            const float a = x[e] * linv[r0 + c0 + e], b = x[e + 1] * linv[r0 + c0 + e + 1];
                            const bool odd = lane & 1;
                            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                            const int r = c0 + e + (odd ? 1 : 0);
                            const uint32_t w = odd ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
                            if (r < my_rows)
                                *reinterpret_cast<uint32_t *>(P.out + (size_t)rowidx[r0 + r] * D +
                                                              (d & ~1)) = w;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < OW; ++e)
                            if (c0 + e < my_rows) P.part_acc[(prow0 + c0 + e) * D + d] = x[e];
                    }
                }
            }
            ++k;
        }
    } else {
        // ============================================== the other operands
        q8_operands<C, D, N, QB>(A, meta, qs, tabs, bars, warp - 10);
    }

    // ---------------------------------------------------------- teardown
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace swa
