// Windowed verify attention over the 8-bit cache on the fp8 tensor cores
// (tcgen05 kind::f8f6f4), the e4m3 rows fed to them as they lie in the cache.
//
// As in the bf16 key-major kernel keys are the MMA's M dimension; per tile of 128
// keys
//
//   S^T[128 keys x 2N] = K8_tile[128 x D] . [Q_hi; Q_lo][2N x D]^T
//   O^T[D x 3N]       += V8_tile^T[D x 128] . [P_0; P_1; P_2][3N x 128]^T
//
// What is not 8-bit by nature is carried in e4m3 numbers of four significant
// bits each:
//   q = 2^eq (q_hi + q_lo / 16), eq per query row.  A bf16 number has eight
//     significant bits, so this is exact down to 2^-14 of the row's largest
//     element and off by at most 2^-22 of it below.
//   P = P_0 + (P_1 + P_2 / 16) / 56: that holds an fp16 number's eleven bits, so P
//     is within 2^-11, or within 2^-21 of the row's largest P where that is more.
//     (56 is the largest 2^i m, m odd and at most 7, that keeps what P_0 leaves of
//     a P up to 256 within 448; times 7 that is still exact in fp16.)  An M = 128
//     MMA takes 45 cycles with 32 columns, 49 with 64, 57 with 96 (measured), so
//     neither the second half of Q nor the second and third of P cost much.
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
// A CTA runs two pipelines, each taking every other of the CTA's items on its own
// from the first copy to the output, so that what one waits for (a tile, the
// tensor core, its own epilogue) is the other's time.  Per pipeline:
//   loader     one warp: K and V tiles by TMA
//   issuer     one warp: the MMAs
//   softmax    four warps, a thread per key, all N rows of the item each: query rows
//              into their two numbers, softmax, epilogue
// (384 threads.)  Measured, 512 sequences of 8 rows, windows 188 / 1024: one
// pipeline whose rows were split between two warpgroups took 52 / 125-131 us; waits
// on one another and instruction fetches were most of it.
//
// Every wait is bounded; one that gives up sets the fault word and a flag that
// ends all other waits of the CTA, whose roles then run through their loops.
#pragma once

#include "swa_q8.cuh"
#include "swa_tc.cuh"

namespace swa {

constexpr int kQ8TcThreads = 384;
constexpr int kQ8Meta = 16;         // items per CTA decoded once into shared memory
constexpr float kQ8QLo = 16.f;      // scale of Q_lo
constexpr float kQ8P1 = 56.f;       // scale of P_1, and of P_2 beside it
constexpr float kQ8P2 = 16.f;
// The reference maximum of a row sits this far (log2) below the largest u of the
// tile that set it, and P stays at most 2^8: a later tile may exceed that u by 2^6
// before the references are raised.  A lower one would cost the small weights'
// resolution: half a smallest step of P_2, 2^-10 / 56 / 16, is to be within 2^-21 of
// the largest weight.
constexpr float kQ8RefBelow = 2.f;
constexpr float kQ8RaiseAt = 8.f;

struct Q8TcParams {
    TcParams T;
    const int8_t *k_exp, *v_exp;
};

template <int D, int N, int NK>
struct Q8Cfg {
    static constexpr int SLABS = D / 128;
    static constexpr int ATOM_BYTES = SLABS * 1024;  // 8 keys x D
    static constexpr int TILE_BYTES = (kTcTileKeys / 8) * ATOM_BYTES;
    static constexpr int Q_SLAB = 2 * N * 128;       // N hi + N lo rows of 128 elements
    static constexpr int Q_BUF = SLABS * Q_SLAB;
    // P: blocks of 32 columns, [block][key][32 bytes] with 32-byte swizzle; the
    // N columns of P_0, then of P_1 and P_2
    static constexpr int P_BLOCK = kTcTileKeys * 32;
    static constexpr int P_BUF = ((3 * N + 31) / 32) * P_BLOCK;
    // one pipeline's part
    static constexpr int K_OFF = 0;                   // NK tiles
    static constexpr int V_OFF = K_OFF + NK * TILE_BYTES;
    static constexpr int Q_OFF = V_OFF + NK * TILE_BYTES;
    static constexpr int RAW_OFF = Q_OFF + Q_BUF;     // bf16 [N][D]: the next item's queries
    static constexpr int P_OFF = RAW_OFF + N * D * 2;
    static constexpr int RED_OFF = P_OFF + P_BUF;     // float [4][N]: per warp maxima, sums
    static constexpr int REF_OFF = RED_OFF + 4 * N * 4;   // float [N] references
    static constexpr int QSC_OFF = REF_OFF + N * 4;       // float [2][N] query scales
    static constexpr int ALPHA_OFF = QSC_OFF + 2 * N * 4; // float [N]: rescale factors, 1 / l
    static constexpr int ROW_OFF = ALPHA_OFF + N * 4;     // uint32 [N] output rows
    static constexpr int PIPE = (ROW_OFF + N * 4 + 1023) / 1024 * 1024;
    // the CTA's
    static constexpr int META_OFF = 2 * PIPE;         // TcItem [kQ8Meta]
    static constexpr int BAR_OFF = (META_OFF + kQ8Meta * (int)sizeof(TcItem) + 7) / 8 * 8;
    // per pipeline
    static constexpr int B_KFULL = 0, B_KEMPTY = NK, B_VFULL = 2 * NK, B_VEMPTY = 3 * NK,
                         B_QFULL = 4 * NK, B_SFULL = B_QFULL + 1, B_SFREE = B_SFULL + 1,
                         B_PFULL = B_SFREE + 1, B_PVDONE = B_PFULL + 1, B_DRAIN = B_PVDONE + 1,
                         NBARS = B_DRAIN + 1;
    static constexpr int MISC_OFF = BAR_OFF + 2 * NBARS * 8;  // tmem base, failed
    static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
    static constexpr int O_HALF = 3 * N;              // O^T columns of 128 dims
    static constexpr int O_COL = 2 * N;               // behind the S^T buffer
    static constexpr int PIPE_COLS = O_COL + (D / 128) * O_HALF;
    static constexpr int TMEM_COLS = 2 * PIPE_COLS <= 128   ? 128
                                     : 2 * PIPE_COLS <= 256 ? 256
                                                            : 512;
    static_assert(N == 16 || N == 32, "rows per item");
    static_assert(2 * PIPE_COLS <= 512, "TMEM");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(Q_OFF % 1024 == 0 && P_OFF % 1024 == 0 && RED_OFF % 16 == 0, "alignment");
};

// Output (and query) row of an item's packed row r: draft row r / G of head
// r % G.  (An item starts on a draft row; r < 64 and G <= 64, where the product
// with the rounded-up 2^16 / G is exact.)
__device__ __forceinline__ size_t q8_row(const AttnParams &P, const TcItem &it, uint32_t inv_g,
                                         int r) {
    const int i = (int)((uint32_t)r * inv_g >> 16), gg = r - i * P.G;
    return ((size_t)it.b * P.q_len + it.i0 + i) * P.Hq + (size_t)it.h * P.G + gg;
}
__device__ __forceinline__ uint32_t q8_inv_g(const AttnParams &P) {
    return 65536u / (uint32_t)P.G + 1u;
}

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

// The e4m3 pair nearest to an fp16 pair (at most 448), the fp16 pair becoming
// what is left times `scale`: exact if that has at most 11 bits.
__device__ __forceinline__ uint16_t take_e4m3(__half2 &p, float scale) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
        : "=h"(c)
        : "r"(*reinterpret_cast<const uint32_t *>(&p)));
    const uint32_t b = e4m3x2_to_f16x2(c);
    p = __hmul2(__hsub2(p, *reinterpret_cast<const __half2 *>(&b)), __floats2half2_rn(scale, scale));
    return c;
}
__device__ __forceinline__ uint16_t last_e4m3(__half2 p) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
        : "=h"(c)
        : "r"(*reinterpret_cast<const uint32_t *>(&p)));
    return c;
}

// The largest of the warp's values, in every lane (a NaN is ignored).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The hot code has to stay in the instruction caches beside that of 11 other warps
// (with everything inlined an earlier form was 187 KB, and warps waited 26% of
// their time for instructions): what is rare is a function of its own.
__device__ __noinline__ void q8_decode(const TcParams *T, int j, TcItem *it) {
    *it = tc_decode_global<false>(*T, cta_item(*T, j));
}

// One lane's copies of a K or V tile: `whole` atoms of consecutive cache rows
// from row y on, and `partial` one more.
template <class C>
__device__ __noinline__ void q8_copy(const CUtensorMap *m4, const CUtensorMap *m1, int y, int whole,
                                     bool partial, uint8_t *dst, uint64_t *bar, uint64_t policy) {
    atom_run<C::ATOM_BYTES>(m4, m1, y, whole, partial, dst, bar, policy);
}

// The warp's arrival once all its lanes are here (32 arrivals on one barrier would
// be served one after another).
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Lane 0 waits for phase `parity` of `bar`, or until some wait of the CTA gave up;
// the warp goes on together.
__device__ __forceinline__ void q8_wait(uint64_t *bar, uint32_t parity, const AttnParams &P,
                                        volatile uint32_t *failed) {
    if ((threadIdx.x & 31) == 0 && !mbar_try_wait(bar, parity)) {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity) && *failed == 0) {
            if (clock64() - t0 > P.wait_limit) {
                atomicOr(P.fault, kFaultCopyTimeout);
                *failed = 1;
            }
        }
    }
    __syncwarp();
}

// A polling loop's patience: false once it ran `limit` cycles without progress, or
// another wait gave up.
struct Q8Patience {
    long long since = 0;
    int idle = 0;
    __device__ __forceinline__ bool more(const AttnParams &P, volatile uint32_t *failed) {
        if ((++idle & 63) != 0) return true;
        const long long now = clock64();
        if (idle == 64) since = now;
        if (now - since > P.wait_limit) {
            atomicOr(P.fault, kFaultCopyTimeout);
            *failed = 1;
        }
        return __any_sync(0xffffffffu, *failed != 0) == 0;
    }
};

// A walk over the tiles of a pipeline's items: every second of the CTA's.
struct Q8Cursor {
    int j, t;
    uint32_t g;   // tiles so far
    TcItem it;
    bool valid;
    __device__ __forceinline__ void seek(const TcParams &T, const TcItem *meta, int n_items) {
        t = 0;
        for (valid = false; j < n_items; j += 2) {
            if (j < kQ8Meta && meta != nullptr) it = meta[j];
            else q8_decode(&T, j, &it);
            if (it.n_tiles > 0) {
                valid = true;
                return;
            }
        }
    }
    __device__ __forceinline__ void next(const TcParams &T, const TcItem *meta, int n_items) {
        ++g;
        if (++t < it.n_tiles) return;
        j += 2;
        seek(T, meta, n_items);
    }
};

// Loader of pipeline p: K and V tiles into their rings, each as soon as its slot is
// free.  A contiguous cache's tile is copied by lane 0; a paged one's runs of pages
// by a lane each, the page ids read a tile ahead.  begin() issues the first tiles,
// before the CTA's items are decoded for all roles; run() the rest, and waits for
// every copy.
template <class C, int NK>
struct Q8Loader {
    const TcParams &T;
    const TcMaps &M;
    uint8_t *pipe;
    uint64_t *bars;
    volatile uint32_t *failed;
    Q8Cursor c[2];  // K, V
    int page[2];
    int n_items, lane, p;

    __device__ __forceinline__ int first_atom(const TcItem &it, int t) const {
        const int ps = T.a.page_size, at = it.t0 + kTcTileKeys * t;
        return lane == 0 ? 0 : ((ps - at % ps) >> 3) + (lane - 1) * (ps >> 3);
    }
    __device__ __forceinline__ void prefetch(int kv) {
        const AttnParams &P = T.a;
        if (P.block_table == nullptr || !c[kv].valid) return;
        const TcItem &it = c[kv].it;
        const int at = it.t0 + kTcTileKeys * c[kv].t;
        if (8 * first_atom(it, c[kv].t) < min(kTcTileKeys, it.cr.c_hi - at))
            page[kv] = __ldg(P.block_table + (long long)it.b * P.max_blocks + at / P.page_size + lane);
    }
    __device__ __noinline__ void fill(int kv, const TcItem *meta) {
        using namespace tc;
        const AttnParams &P = T.a;
        const TcItem &it = c[kv].it;
        const int at = it.t0 + kTcTileKeys * c[kv].t;
        const int n = min(kTcTileKeys, it.cr.c_hi - at), natoms = (n + 7) >> 3;
        const uint32_t slot = c[kv].g % NK;
        uint64_t *bar = &bars[(kv ? C::B_VFULL : C::B_KFULL) + slot];
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)natoms * C::ATOM_BYTES);
        __syncwarp();
        int a = 0, run = lane == 0 ? natoms : 0, y;
        if (P.block_table != nullptr) {
            const int ps = P.page_size, in = at % ps;
            a = first_atom(it, c[kv].t);
            run = min(lane == 0 ? (ps - in) >> 3 : ps >> 3, natoms - a);
            y = (checked_page(P, page[kv], nullptr) * P.Hkv + it.h) * ps + (lane == 0 ? in : 0);
        } else {
            y = (int)(((long long)it.b * P.Hkv + it.h) * P.L + at);
        }
        // (tests of the bounded waits: this fill's copies are never issued)
        const bool withhold =
            P.withhold_fill == (int)(2 * c[kv].g) + kv && blockIdx.x == 0 && p == 0;
        if (run > 0 && !withhold) {
            const int whole = min(max((n >> 3) - a, 0), run);
            q8_copy<C>(kv ? M.v_atoms : M.k_atoms, kv ? &M.v_atom : &M.k_atom, y, whole,
                       run > whole,
                       pipe + (kv ? C::V_OFF : C::K_OFF) + slot * C::TILE_BYTES + a * C::ATOM_BYTES,
                       bar, P.row_tiles > 1 ? l2_policy_evict_normal() : l2_policy_evict_first());
        }
        c[kv].next(T, meta, n_items);
        prefetch(kv);
    }
    __device__ __forceinline__ void begin() {
        c[0].j = p;
        c[0].g = 0;
        c[0].seek(T, nullptr, n_items);
        c[1] = c[0];
        page[0] = page[1] = 0;
        prefetch(0);
        page[1] = page[0];
        if (c[0].valid) {
            fill(0, nullptr);
            fill(1, nullptr);
        }
    }
    __device__ __forceinline__ void run(const TcItem *meta) {
        const AttnParams &P = T.a;
        Q8Patience patience;
        while (c[0].valid || c[1].valid) {
            bool free = false;
            if (lane < 2 && c[lane].valid)
                free = mbar_test(&bars[(lane ? C::B_VEMPTY : C::B_KEMPTY) + c[lane].g % NK],
                                 ((c[lane].g / NK) & 1) ^ 1);
            const uint32_t f = __ballot_sync(0xffffffffu, free);
            if (f & 1u) fill(0, meta);
            if (f & 2u) fill(1, meta);
            if (f != 0) patience.idle = 0;
            else if (!patience.more(P, failed)) break;
            else if (patience.idle > 8) __nanosleep(32);
        }
        // every copy issued has landed before the CTA exits
        if (lane < 2 * NK) {
            const uint32_t kv = (uint32_t)lane / NK, slot = (uint32_t)lane % NK, g = c[kv].g;
            if (g > slot)
                mbar_wait_bounded(&bars[(kv ? C::B_VFULL : C::B_KFULL) + slot],
                                  ((g - 1 - slot) / NK) & 1, P.fault, kFaultCopyTimeout,
                                  P.wait_limit);
        }
        __syncwarp();
    }
};

// Issuer of pipeline p's MMAs: the next tile's scores and the oldest tile's PV, each
// as soon as its operands are there (one barrier per lane, tested by one
// instruction).
template <class C, int D, int N, int NK>
__device__ __forceinline__ void q8_issue(const TcParams &T, const TcItem *meta, uint8_t *pipe,
                                         uint64_t *bars, uint32_t tmem, int n_items, int p,
                                         volatile uint32_t *failed) {
    using namespace tc;
    constexpr int MH = D / 128;
    constexpr uint32_t ID_QK = idesc_e4m3_f32(128, 2 * N, 0, 0);
    constexpr uint32_t ID_PV = idesc_e4m3_f32(128, 3 * N, 1, 1);
    const AttnParams &P = T.a;
    const int lane = (int)(threadIdx.x & 31);
    const uint64_t k_d = smem_desc_sw128(smem_u32(pipe + C::K_OFF), 16, C::ATOM_BYTES);
    const uint64_t v_d = smem_desc_sw128(smem_u32(pipe + C::V_OFF), 16, C::ATOM_BYTES);
    const uint64_t q_d = smem_desc_sw128(smem_u32(pipe + C::Q_OFF), 16, 1024);
    const uint64_t p_d = smem_desc_sw32(smem_u32(pipe + C::P_OFF), C::P_BLOCK, 256);
    Q8Cursor s, o;  // the next scores, the next PV
    s.j = p;
    s.g = 0;
    s.seek(T, meta, n_items);
    o = s;
    uint32_t k = 0;  // items whose scores have begun
    Q8Patience patience;
    while (o.valid) {
        // 0: the K tile, 1: the S buffer, 2: an item's queries; 3: the V tile, 4: P
        const int which = lane == 0   ? C::B_KFULL + (int)(s.g % NK)
                          : lane == 1 ? C::B_SFREE
                          : lane == 2 ? C::B_QFULL
                          : lane == 3 ? C::B_VFULL + (int)(o.g % NK)
                                      : C::B_PFULL;
        const uint32_t par = lane == 0   ? s.g / NK
                             : lane == 1 ? s.g + 1
                             : lane == 2 ? k
                             : lane == 3 ? o.g / NK
                                         : o.g;
        bool there = false;
        if (lane < 5 && (lane > 2 ? o.g < s.g : s.valid))
            there = (lane == 2 && s.t > 0) || mbar_test(&bars[which], par & 1);
        const uint32_t r = __ballot_sync(0xffffffffu, there);
        if ((r & 7u) == 7u) {
            const bool last = s.t == s.it.n_tiles - 1;
            const uint32_t slot = s.g % NK;
            fence_after_sync();
            if (lane == 0) {
                const uint64_t a = k_d + (uint64_t)(slot * (C::TILE_BYTES >> 4));
#pragma unroll
                for (int sl = 0; sl < C::SLABS; ++sl)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_e4m3_ss(tmem, a + (uint64_t)(sl * 64 + kk * 2),
                                    q_d + (uint64_t)(sl * (C::Q_SLAB >> 4) + kk * 2), ID_QK,
                                    (sl | kk) != 0);
                mma_commit(&bars[C::B_SFULL]);
                mma_commit(&bars[C::B_KEMPTY + slot]);
            }
            __syncwarp();
            if (last) ++k;
            s.next(T, meta, n_items);
        }
        if ((r & 24u) == 24u) {
            const uint32_t slot = o.g % NK;
            const bool last = o.t == o.it.n_tiles - 1;
            fence_after_sync();
            // only the 32-key steps that hold valid keys are multiplied; the rows of
            // the last step past the chunk's end, and those before the chunk in a
            // paged cache's first tile, are zeroed first, so that 0 * (whatever the
            // slot holds there) cannot reach O
            const int nv = last ? o.it.cr.c_hi - o.it.t0 - kTcTileKeys * o.t : kTcTileKeys;
            const int steps = (nv + 31) >> 5;
            const int z = o.t == 0 ? o.it.cr.c_lo - o.it.t0 : 0;
            if ((nv & 31) || z > 0) {
                uint8_t *vt = pipe + C::V_OFF + slot * C::TILE_BYTES;
                zero_v_rows<C>(vt, nv, 32 * steps, lane);
                zero_v_rows<C>(vt, 0, z, lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) {
                // A = V^T, MN-major: a slab holds 128 dims, 8-key groups one atom
                // apart; B = the parts of P, MN-major
                const uint64_t a = v_d + (uint64_t)(slot * (C::TILE_BYTES >> 4));
                const uint32_t acc = o.t > 0 ? 1u : 0u;
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4) {
                    if (k4 >= steps) break;
#pragma unroll
                    for (int mh = 0; mh < MH; ++mh)
                        mma_e4m3_ss(tmem + C::O_COL + mh * C::O_HALF,
                                    a + (uint64_t)((mh * 1024 + k4 * 4 * C::ATOM_BYTES) >> 4),
                                    p_d + (uint64_t)(k4 * 1024 >> 4), ID_PV, k4 > 0 ? 1u : acc);
                }
                mma_commit(&bars[C::B_PVDONE]);
                mma_commit(&bars[C::B_VEMPTY + slot]);
            }
            __syncwarp();
            o.next(T, meta, n_items);
        }
        if ((r & 7u) == 7u || (r & 24u) == 24u) patience.idle = 0;
        else if (!patience.more(P, failed)) break;
    }
    // all issued MMAs complete before TMEM is released
    if (lane == 0 && s.g > 0) {
        mma_commit(&bars[C::B_DRAIN]);
        mbar_wait_bounded(&bars[C::B_DRAIN], 0, P.fault, kFaultCopyTimeout, P.wait_limit);
    }
    __syncwarp();
}

// Barriers of one pipeline's softmax warps, and a vote of theirs.
__device__ __forceinline__ void q8_sync(int p) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + p) : "memory");
}
__device__ __forceinline__ bool q8_any(int p, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(3 + p)
        : "memory");
    return r != 0;
}

// An item's query rows into the raw buffer, an item ahead of their use: a plain
// load takes microseconds while the tiles' copies keep the memory busy.  Warp w of
// the four has rows w, w + 4, ..., as q8_queries: a thread splits what it copied.
template <int D>
__device__ __forceinline__ void q8_fetch_queries(const AttnParams &P, const TcItem &it, uint8_t *raw,
                                                 int w, uint32_t inv_g) {
    constexpr int LPR = D / 8, RP = 32 / LPR;  // lanes per row, rows per pass
    const int lane = (int)(threadIdx.x & 31), l = lane % LPR;
#pragma unroll 1
    for (int r = w + 4 * (lane / LPR); r < it.rows; r += 4 * RP)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         smem_u32(raw + r * (D * 2) + l * 16)),
                     "l"(P.q + q8_row(P, it, inv_g, r) * D + l * 8)
                     : "memory");
}

// The rows from the raw buffer as two e4m3 numbers each, and their scales.
template <class C, int D, int N>
__device__ __forceinline__ void q8_queries(int rows, const uint8_t *raw, uint8_t *q, float *qsc,
                                           uint64_t *bars, int w) {
    constexpr int LPR = D / 8, RP = 32 / LPR;
    const int lane = (int)(threadIdx.x & 31);
    const int sub = lane / LPR, l = lane % LPR;
    // 8 bytes at element 8 l: 16-byte chunk (l / 2) % 8 of slab l / 16
    const uint32_t at = (uint32_t)(l >> 4) * C::Q_SLAB + (uint32_t)(l & 1) * 8;
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
    for (int r0 = w; r0 < rows; r0 += 4 * RP) {
        const int r = r0 + 4 * sub;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < rows) x = *reinterpret_cast<const uint4 *>(raw + r * (D * 2) + l * 16);
        const uint32_t b[4] = {x.x, x.y, x.z, x.w};
        // the smallest exponent that holds the row, as for the cache
        const uint32_t a = __reduce_max_sync(
            LPR == 32 ? 0xffffffffu : 0xffffu << (16 * sub),
            max_u16x2_half(max_u16x2(max_u16x2(b[0] & 0x7fff7fffu, b[1] & 0x7fff7fffu),
                                     max_u16x2(b[2] & 0x7fff7fffu, b[3] & 0x7fff7fffu))));
        int e = (int)(a >> 7) - 135 + ((a & 0x7fu) > 0x60u ? 1 : 0);
        e = e < -126 ? -126 : (e > 126 ? 126 : e);
        const float sc = pow2f(-e);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            // (exact in fp16 from 2^-17 on: eight bits above its 2^-24)
            __half2 y = __floats2half2_rn(bf16lo(b[p]) * sc, bf16hi(b[p]) * sc);
            const uint32_t h = take_e4m3(y, kQ8QLo), t = last_e4m3(y);
            hi[p >> 1] = p & 1 ? hi[p >> 1] | (h << 16) : h;
            lo[p >> 1] = p & 1 ? lo[p >> 1] | (t << 16) : t;
        }
        if (r < rows) {
            // (N is a multiple of 8: both rows have the same swizzle phase)
            const uint32_t sw = (((uint32_t)(l >> 1) & 7) ^ (uint32_t)(r & 7)) << 4;
            *reinterpret_cast<uint2 *>(q + at + r * 128 + sw) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(q + at + (N + r) * 128 + sw) = make_uint2(lo[0], lo[1]);
            if (l == 0) qsc[r] = pow2f(e);
        }
    }
    fence_proxy_async_smem();
    warp_arrive(&bars[C::B_QFULL]);
}

// The rows of an item without keys.
template <int D>
__device__ __noinline__ void q8_empty_item(const AttnParams *A, const TcItem *item, uint32_t inv_g,
                                           int t) {
    const AttnParams &P = *A;
    const TcItem &it = *item;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const size_t prow0 =
        (((size_t)it.b * P.Hkv + it.h) * P.splits + it.split) * P.R + it.row0;
    for (int idx = t; idx < it.rows * D; idx += 128) {
        const int r = idx / D, d = idx % D;
        if (P.splits == 1) {
            const size_t orow = q8_row(P, it, inv_g, r);
            P.out[orow * D + d] = __float2bfloat16_rn(0.f);
            if (d == 0 && P.lse != nullptr) P.lse[orow] = NEG_INF;
        } else {
            P.part_acc[(prow0 + r) * D + d] = 0.f;
            if (d == 0) {
                P.part_ml[(prow0 + r) * 2] = NEG_INF;
                P.part_ml[(prow0 + r) * 2 + 1] = 0.f;
            }
        }
    }
}

// The softmax warps of pipeline p: queries, softmax and epilogue of its items.
template <class C, int D, int N>
__device__ __forceinline__ void q8_softmax(const Q8TcParams &A, const TcItem *meta, uint8_t *pipe,
                                           uint64_t *bars, uint32_t tmem, int n_items, int p,
                                           volatile uint32_t *failed) {
    using namespace tc;
    constexpr int MH = D / 128;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const TcParams &T = A.T;
    const AttnParams &P = T.a;
    uint8_t *q = pipe + C::Q_OFF, *raw = pipe + C::RAW_OFF;
    float *red = reinterpret_cast<float *>(pipe + C::RED_OFF);
    float *ref = reinterpret_cast<float *>(pipe + C::REF_OFF);
    float *qsc = reinterpret_cast<float *>(pipe + C::QSC_OFF);
    float *alpha = reinterpret_cast<float *>(pipe + C::ALPHA_OFF);
    uint32_t *rowidx = reinterpret_cast<uint32_t *>(pipe + C::ROW_OFF);
    const int lane = (int)(threadIdx.x & 31), sw = (int)(threadIdx.x >> 5) & 3;
    const int lk = sw * 32 + lane;  // TMEM lane: key of S^T, dim row of O^T
    const uint32_t s_col = tmem + ((uint32_t)(sw * 32) << 16), o_col = s_col + C::O_COL;
    const uint32_t inv_g = q8_inv_g(P);
    uint8_t *pt = pipe + C::P_OFF + lk * 32;        // key lk's row of P
    const uint32_t flip = (uint32_t)(lk >> 2) & 1;  // its 32-byte swizzle phase

    auto item = [&](int j) {
        TcItem it;
        if (j < kQ8Meta) it = meta[j];
        else q8_decode(&T, j, &it);
        return it;
    };
    // the exponents of this thread's key in tile t of an item, k's and v's
    int8_t ke = 0, ve = 0;
    auto fetch_key = [&](const TcItem &it, int t) {
        const int jk = it.t0 + kTcTileKeys * t + lk;
        ke = ve = 0;
        if (jk >= it.cr.c_lo && jk < it.cr.c_hi) {
            const long long row = cache_row(P, it.b, it.h, jk);
            ke = A.k_exp[row];
            ve = A.v_exp[row];
        }
    };
    // the next item with keys: its queries are on their way, or split already
    int jn = p;
    TcItem nx;
    auto seek = [&]() {
        for (; jn < n_items; jn += 2) {
            nx = item(jn);
            if (nx.n_tiles > 0) return;
        }
    };
    seek();
    if (jn < n_items) {
        q8_fetch_queries<D>(P, nx, raw, sw, inv_g);
        fetch_key(nx, 0);
        q8_queries<C, D, N>(nx.rows, raw, q, qsc, bars, sw);
    }
    q8_sync(p);  // (the scales; later items' are behind the epilogue's)
    uint32_t g = 0, k = 0;
#pragma unroll 1
    for (int j = p; j < n_items; j += 2) {
        const TcItem it = item(j);
        if (it.n_tiles == 0) {
            q8_empty_item<D>(&P, &it, inv_g, lk);
            continue;
        }
        jn = j + 2;
        seek();
        if (jn < n_items) q8_fetch_queries<D>(P, nx, raw, sw, inv_g);
        const float *rs = qsc + (k & 1) * N;
        float lrow[N];
#pragma unroll
        for (int r = 0; r < N; ++r) lrow[r] = 0.f;
        const int qp_i0 = it.cr.qp + it.i0;  // position of the item's first draft row
        // first keys of the tiles that every row sees whole
        const int i_last = (int)((uint32_t)(it.rows - 1) * inv_g >> 16);
        const int inner_lo =
            (int)max((long long)qp_i0 + i_last - P.window + 1, (long long)it.cr.c_lo);
        const int inner_hi = min(qp_i0, it.cr.c_hi - 1) - (kTcTileKeys - 1);
#pragma unroll 1
        for (int t = 0; t < it.n_tiles; ++t, ++g) {
            // this key's factor (log2 units) and v's exponent; the next tile's are
            // on their way from here on
            const float kx = P.qk_scale * pow2f(ke < -126 ? -126 : ke), vx = (float)ve;
            const float ive = pow2f(ve > 126 ? -126 : (ve < -127 ? 127 : -ve));
            if (t + 1 < it.n_tiles) fetch_key(it, t + 1);
            else if (jn < n_items) fetch_key(nx, 0);
            // packed rows [ra, rb) whose window holds the key
            const int j0 = it.t0 + kTcTileKeys * t;
            int ra = 0, rb = N;
            if (j0 < inner_lo || j0 > inner_hi) {
                const int jk = j0 + lk;
                ra = rb = 0;
                if (jk >= it.cr.c_lo && jk < it.cr.c_hi) {
                    // (jk < q_pos + q_len: the first difference is below 512)
                    const int lo_i = jk - qp_i0;
                    const long long hi_i = (long long)lo_i + P.window;
                    ra = min(max(lo_i, 0) * P.G, (int)it.rows);
                    rb = hi_i >= it.rows ? (int)it.rows
                                         : min(max((int)hi_i, 0) * P.G, (int)it.rows);
                }
            }
            q8_wait(&bars[C::B_SFULL], g & 1, P, failed);
            fence_after_sync();
            // u = (S_hi + S_lo / 16) * row scale * key factor + e_v
            float v[N];
            {
                const uint64_t lo2 = f2_pack(1.f / kQ8QLo, 1.f / kQ8QLo);
                const uint64_t ks2 = f2_pack(kx, kx), ve2 = f2_pack(vx, vx);
#pragma unroll
                for (int c = 0; c < N; c += 16) {
                    uint32_t hi[16], lo[16];
                    tmem_load<16>(s_col + c, hi);
                    tmem_load<16>(s_col + N + c, lo);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 s4 = *reinterpret_cast<const float4 *>(rs + c + e);
                        const uint64_t rs2[2] = {f2_pack(s4.x, s4.y), f2_pack(s4.z, s4.w)};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = e + 2 * h;
                            const uint64_t s2 =
                                f2_fma(f2_pack(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1])),
                                       lo2,
                                       f2_pack(__uint_as_float(hi[r]), __uint_as_float(hi[r + 1])));
                            f2_unpack(f2_fma(f2_mul(s2, rs2[h]), ks2, ve2), v[c + r], v[c + r + 1]);
                        }
                    }
                }
                fence_before_sync();
                warp_arrive(&bars[C::B_SFREE]);
                if (ra > 0 || rb < N) {
#pragma unroll
                    for (int r = 0; r < N; ++r)
                        if (r < ra || r >= rb) v[r] = NEG_INF;
                }
            }
            bool raise = t == 0;  // an item's first tile sets the references
            if (t > 0) {
                float over = NEG_INF;
#pragma unroll
                for (int r = 0; r < N; r += 4) {
                    const float4 m4 = *reinterpret_cast<const float4 *>(ref + r);
                    over = fmax3(over, v[r] - m4.x, v[r + 1] - m4.y);
                    over = fmax3(over, v[r + 2] - m4.z, v[r + 3] - m4.w);
                }
                raise = q8_any(p, over > kQ8RaiseAt);
            }
            if (raise) {
                // exact tile maximum per row
                float mine = NEG_INF;
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    const float m = warp_max(v[r]);
                    if (lane == r) mine = m;
                }
                if (lane < N) red[sw * N + lane] = mine;
                q8_sync(p);
                if (lk < N) {
                    const float tm =
                        fmaxf(fmax3(red[lk], red[N + lk], red[2 * N + lk]), red[3 * N + lk]);
                    const float mo = t == 0 ? kNoRef : ref[lk];
                    const float mn = fmaxf(mo, tm - kQ8RefBelow);
                    ref[lk] = mn;
                    alpha[lk] = fast_exp2(mo - mn);
                }
                if (t > 0) {
                    // every PV of this item so far has completed before O is scaled
                    q8_wait(&bars[C::B_PVDONE], (g - 1) & 1, P, failed);
                    fence_after_sync();
                }
                q8_sync(p);
                if (t > 0) {
#pragma unroll
                    for (int r = 0; r < N; ++r) lrow[r] *= alpha[r];
#pragma unroll 1
                    for (int c = 0; c < MH * 3 * N; c += 16) {
                        uint32_t o[16];
                        tmem_load<16>(o_col + c, o);
                        tmem_wait_ld();
                        const float *a = alpha + c % N;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * a[e]);
                        tmem_store<16>(o_col + c, o);
                    }
                    tmem_wait_st();
                }
            }
            // the P buffer's previous PV has completed
            if (g > 0) q8_wait(&bars[C::B_PVDONE], (g - 1) & 1, P, failed);
            // P = 2^(u - ref) in e4m3 numbers; the row sum adds P 2^-e_v
            const uint64_t iv2 = f2_pack(ive, ive);
#pragma unroll
            for (int c = 0; c < N; c += 16) {
                uint32_t pk[3][4];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 m4 = *reinterpret_cast<const float4 *>(ref + c + e);
                    const uint64_t m2[2] = {f2_pack(m4.x, m4.y), f2_pack(m4.z, m4.w)};
                    uint32_t w[3][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = c + e + 2 * h;
                        float d0, d1;
                        f2_unpack(f2_sub(f2_pack(v[r], v[r + 1]), m2[h]), d0, d1);
                        const float p0 = fast_exp2(d0), p1 = fast_exp2(d1);
                        f2_unpack(f2_fma(f2_pack(p0, p1), iv2, f2_pack(lrow[r], lrow[r + 1])),
                                  lrow[r], lrow[r + 1]);
                        __half2 x = __floats2half2_rn(p0, p1);
                        w[0][h] = take_e4m3(x, kQ8P1);
                        w[1][h] = take_e4m3(x, kQ8P2);
                        w[2][h] = last_e4m3(x);
                    }
#pragma unroll
                    for (int i = 0; i < 3; ++i) pk[i][e / 4] = w[i][0] | (w[i][1] << 16);
                }
                // columns i N + c .. of part i
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int col = i * N + c;
                    *reinterpret_cast<uint4 *>(pt + (col >> 5) * C::P_BLOCK +
                                               (((uint32_t)(col >> 4) & 1u) ^ flip) * 16) =
                        make_uint4(pk[i][0], pk[i][1], pk[i][2], pk[i][3]);
                }
            }
            fence_proxy_async_smem();
            warp_arrive(&bars[C::B_PFULL]);
        }

        // ------------------------------------------------------ epilogue
        // (the last scores are complete, so the queries' buffer is free)
        if (jn < n_items) q8_queries<C, D, N>(nx.rows, raw, q, qsc + ((k + 1) & 1) * N, bars, sw);
        const float l1 = lane_reduce<N, false>(lrow);
        if (lane < N) red[sw * N + lane] = l1;
        q8_sync(p);
        const size_t prow0 =
            (((size_t)it.b * P.Hkv + it.h) * P.splits + it.split) * P.R + it.row0;
        if (lk < it.rows) {
            const float l = (red[lk] + red[N + lk]) + (red[2 * N + lk] + red[3 * N + lk]);
            const float m = ref[lk];
            const bool any = !(l <= 0.f);  // (a NaN stays one)
            const uint32_t orow = (uint32_t)q8_row(P, it, inv_g, lk);
            alpha[lk] = any ? __frcp_rn(l) : 0.f;
            rowidx[lk] = orow;  // (below 2^31 by the plan's size checks)
            if (P.splits > 1) {
                P.part_ml[(prow0 + lk) * 2] = any ? m : NEG_INF;
                P.part_ml[(prow0 + lk) * 2 + 1] = l;
            } else if (P.lse != nullptr) {
                P.lse[orow] = any ? (m + __log2f(l)) * kLn2 : NEG_INF;
            }
        }
        q8_wait(&bars[C::B_PVDONE], (g - 1) & 1, P, failed);
        fence_after_sync();
        q8_sync(p);
        const uint64_t s1 = f2_pack(1.f / kQ8P1, 1.f / kQ8P1);
        const uint64_t s2 = f2_pack(1.f / kQ8P2, 1.f / kQ8P2);
        // neighbouring lanes hold neighbouring dims: each pair swaps halves of two
        // rows, so that a lane stores two dims of one row
        const bool odd = lane & 1;
        __nv_bfloat16 *out = P.out + (lk & ~1);
#pragma unroll 1
        for (int c0 = 0; c0 < it.rows; c0 += 16) {
#pragma unroll 1
            for (int mh = 0; mh < MH; ++mh) {
                uint32_t o[3][16];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    tmem_load<16>(o_col + mh * C::O_HALF + i * N + c0, o[i]);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    auto pair = [&](int i) {
                        return f2_pack(__uint_as_float(o[i][e]), __uint_as_float(o[i][e + 1]));
                    };
                    const uint64_t x2 = f2_fma(f2_fma(pair(2), s2, pair(1)), s1, pair(0));
                    float a, b;
                    if (P.splits == 1) {
                        const float2 l2 = *reinterpret_cast<const float2 *>(alpha + c0 + e);
                        f2_unpack(f2_mul(x2, f2_pack(l2.x, l2.y)), a, b);
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                        const int r = c0 + e + (odd ? 1 : 0);
                        const uint32_t w = odd ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
                        if (r < it.rows)
                            *reinterpret_cast<uint32_t *>(out + (size_t)rowidx[r] * D + mh * 128) =
                                w;
                    } else {
                        f2_unpack(x2, a, b);
                        float *acc = P.part_acc + (prow0 + c0 + e) * D + mh * 128 + lk;
                        if (c0 + e < it.rows) acc[0] = a;
                        if (c0 + e + 1 < it.rows) acc[D] = b;
                    }
                }
            }
        }
        fence_before_sync();  // (O is read before the next item's first P is announced)
        ++k;
    }
}

template <int D, int N, int NK>
__global__ void __launch_bounds__(kQ8TcThreads, 1)
    swa_q8_tc_kernel(const __grid_constant__ Q8TcParams A, const __grid_constant__ TcMaps M) {
    using C = Q8Cfg<D, N, NK>;
    using namespace tc;
    const TcParams &T = A.T;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    TcItem *meta = reinterpret_cast<TcItem *>(sm + C::META_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC_OFF);
    volatile uint32_t *failed = tmem_slot + 1;
    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    // the pipeline of this warp: 0 and 3 load, 1 and 2 issue, 4..7 and 8..11 softmax
    const int p = warp < 4 ? warp >> 1 : (warp - 4) >> 2;
    uint8_t *pipe = sm + p * C::PIPE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::BAR_OFF) + p * C::NBARS;

    // ---------------------------------------------------------------- setup
    if (warp == 0 && lane < 10) {
        const CUtensorMap *mp = lane < 4    ? &M.k_atoms[lane]
                                : lane < 8  ? &M.v_atoms[lane - 4]
                                : lane == 8 ? &M.k_atom
                                            : &M.v_atom;
        prefetch_tmap(mp);
    }
    if ((warp == 0 || warp == 3) && lane < C::NBARS) {
        // arrivals: one (a commit, or a copy's bytes), or one per softmax warp
        mbar_init(&bars[lane], lane == C::B_QFULL || lane == C::B_SFREE || lane == C::B_PFULL ? 4 : 1);
        fence_barrier_init();
    }
    if (tid == 0) *failed = 0;
    // query rows past an item's stay what they are here: zero, or another item's
    // (their columns are never looked at, but should not raise the references
    // either)
    if (warp >= 4) {
        for (int i = tid & 127; i < C::Q_BUF / 16; i += 128)
            reinterpret_cast<uint4 *>(pipe + C::Q_OFF)[i] = make_uint4(0, 0, 0, 0);
        float *z = reinterpret_cast<float *>(pipe + C::RED_OFF);
        for (int i = tid & 127; i < (C::PIPE - C::RED_OFF) / 4; i += 128) z[i] = 0.f;
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_trigger();
    const int n_items = cta_items(T);
    if (warp == 0 || warp == 3) {
        Q8Loader<C, NK> load{T, M, pipe, bars, failed, {}, {}, n_items, lane, p};
        load.begin();
        __syncthreads();
        load.run(meta);
    } else {
        for (int j = tid - 128; j >= 0 && j < kQ8Meta; j += kQ8TcThreads)
            if (j < n_items) q8_decode(&T, j, &meta[j]);
        fence_before_sync();
        __syncthreads();
        fence_after_sync();
        const uint32_t tmem = *tmem_slot + p * C::PIPE_COLS;
        if (warp < 4) q8_issue<C, D, N, NK>(T, meta, pipe, bars, tmem, n_items, p, failed);
        else q8_softmax<C, D, N>(A, meta, pipe, bars, tmem, n_items, p, failed);
    }

    // ---------------------------------------------------------- teardown
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 1) tmem_dealloc(*tmem_slot, C::TMEM_COLS);
}

}  // namespace swa
