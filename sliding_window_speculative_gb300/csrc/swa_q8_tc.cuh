// Windowed verify attention over the 8-bit cache on the fp8 tensor cores
// (tcgen05 kind::f8f6f4), the e4m3 rows fed to them as they lie in the cache.
//
// The structure is that of the bf16 key-major kernel: persistent CTAs, keys as
// the MMA's M dimension, K and V tiles of 128 keys by TMA into a ring,
//
//   S^T[128 keys x 2N] = K8_tile[128 x D] . [Q_hi; Q_lo][2N x D]^T
//   O^T[D x 3N]       += V8_tile^T[D x 128] . [P_0; P_1; P_2][3N x 128]^T
//
// What is not 8-bit by nature is carried in e4m3 numbers of four significant
// bits each:
//   q = 2^eq (q_hi + q_lo / 16), eq per query row.  A bf16 number has eight
//     significant bits, so this is exact down to 2^-14 of the row's largest
//     element and off by at most 2^-21 of it below.
//   P = P_0 + (P_1 + P_2 / 32) / 32: what a number leaves is signed and at most half
//     a step of its four bits, so each further one adds five: P is within 2^-14 of
//     itself, or a smallest step of P_2 (2^-9 / 1024 = 2^-19) where that is more.  (P
//     is at most 256, of which P_0 leaves at most 8: 32 is the largest power of two
//     that keeps that within 448.)  The row's largest P is at least 2^2 (kQ8RefBelow),
//     so that step is 2^-21 of it.  Weights that small count by their number: alike
//     ones, rounded alike, would be off together.  So P_2 is rounded with an offset,
//     of up to half that step, that runs evenly through it from key to key (multiples
//     of the golden ratio): the offsets cancel, and n such weights are off by some
//     sqrt(n) 2^-22 of the largest.  That no choice of weights is off without limit, an
//     item takes at most kQ8ItemKeys.  An M = 128 MMA takes 45 cycles with 32 columns,
//     49 with 64, 57 with 96 (measured), so neither the second half of Q nor the second
//     and third of P cost much.
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
// Heads of 64 lie in tiles of 128 dims: the TMA fills what is past a row's end with
// zeros, and the kernel is that of 128.
//
// What bounds it beside the cache's bytes is the instruction caches: sixteen warps
// of five roles run different code, and a warp that runs straight through code that
// the nearest cache (some hundred instructions for four warps) does not hold waits
// for every line of it.  Unrolled, the kernel issued an instruction in 30% of its
// cycles and a single MMA took 100 cycles to issue; so the loops over rows stay
// rolled, eight rows a turn, and what is rare is out of line (512 sequences of 8
// rows, 4 heads of 256 to a KV head, window 1024: 125 us unrolled, 116 rolled, 103 with
// less code in the other roles too).  Tried and not kept: two tiles per softmax turn
// (125), two independent pipelines of half the ring each (145), a warpgroup to every
// other tile for up to 8 rows (103).
// Measured, of the bytes' time at 6.78 TB/s: those calls 82% (103 us), of one row 97%
// (82.6), window 188 48% and 46% (an item of two tiles costs 6 us from its queries to
// its output), 4 sequences of 32768 keys, heads of 128 in pages of 64: 50% (32.4 us: at
// their lengths 124 SMs have keys, up to 29 tiles each at 0.8 us, whose bytes take 0.7;
// the first and last steps, the merge).
//
// Warp roles (512 threads; the registers of the first and last warpgroup that
// they do not need go to the softmax):
//   warp 0       TMA producer
//   warp 1       TMEM owner, issuer of the scores' MMAs
//   warp 2       issuer of the MMAs into O
//   warp 3       the keys' factors: a ring of tables, a few tiles ahead
//   warps 4..11  softmax, two warpgroups that split the packed rows
//   warps 12..15 query rows split into their two numbers, one item ahead, and
//                the epilogue of the item before: O is double-buffered, so the
//                softmax goes on with the next item meanwhile
//
// Every wait is bounded; one that gives up sets the fault word and a flag that
// ends all other waits of the CTA, whose roles then run through their loops.
#pragma once

#include "swa_q8.cuh"
#include "swa_tc.cuh"

namespace swa {

constexpr int kQ8TcThreads = 512;
constexpr int kQ8Tabs = 4;          // tables of key factors
constexpr float kQ8QLo = 16.f;      // scale of Q_lo
constexpr float kQ8PStep = 32.f;    // scale of P_1 to P_0, and of P_2 to P_1
// The reference maximum of a row sits this far (log2) below the largest u of the
// tiles that set it, and P stays at most 2^8: a later tile may exceed that u by 2^6
// before the references are raised.  A lower one would cost the small weights'
// resolution, a higher one time (512 sequences of 8 rows, 8 heads of 256 on 2, window
// 1024: 2 103 us, 4 116, 5 125).
constexpr float kQ8RefBelow = 2.f;
constexpr float kQ8RaiseAt = 8.f;

struct Q8TcParams {
    TcParams T;
    const int8_t *k_exp, *v_exp;
};

template <int D, int N, int NT>
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
    static constexpr int RING_OFF = 0;
    static constexpr int Q_OFF = RING_OFF + NT * TILE_BYTES;
    static constexpr int P_OFF = Q_OFF + 2 * Q_BUF;
    static constexpr int TAB_OFF = P_OFF + 2 * P_BUF;                // float2 [kQ8Tabs][128]
    static constexpr int RED_OFF = TAB_OFF + kQ8Tabs * kTcTileKeys * 8;  // float [4][N]
    static constexpr int REF_OFF = RED_OFF + 4 * N * 4;              // float [N] references
    static constexpr int ALPHA_OFF = REF_OFF + N * 4;                // float [N]
    static constexpr int QSC_OFF = ALPHA_OFF + N * 4;                // float [2][N] query scales
    // float [4][5][N]: per item, a row's sums over each warp's keys, its reference
    static constexpr int SUM_OFF = QSC_OFF + 2 * N * 4;
    static constexpr int LINV_OFF = SUM_OFF + 4 * 5 * N * 4;         // float [2][N]
    static constexpr int ROW_OFF = LINV_OFF + 2 * N * 4;             // uint32 [2][N] output rows
    static constexpr int META_OFF = ROW_OFF + 2 * N * 4;             // TcItem [kTcMetaItems]
    static constexpr int FTAB_OFF = META_OFF + kTcMetaItems * (int)sizeof(TcItem);
    static constexpr int BAR_OFF = (FTAB_OFF + kFillTab * 4 + 7) / 8 * 8;
    static constexpr int B_FULL = 0, B_EMPTY = NT, B_QFULL = 2 * NT, B_QEMPTY = B_QFULL + 2,
                         B_SFULL = B_QEMPTY + 2, B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2,
                         B_PVDONE = B_PFULL + 2, B_OFULL = B_PVDONE + 2, B_OFREE = B_OFULL + 2,
                         B_LFULL = B_OFREE + 2, B_DRAIN = B_LFULL + 4, B_TFULL = B_DRAIN + 2,
                         B_TEMPTY = B_TFULL + kQ8Tabs, NBARS = B_TEMPTY + kQ8Tabs;
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;  // tmem base, failed
    static constexpr int END = MISC_OFF + 16;
    static constexpr int SMEM_BYTES = END + 1024;
    static constexpr int O_HALF = 3 * N;              // O^T columns of 128 dims
    static constexpr int O_COLS = (D / 128) * O_HALF;
    static constexpr int S_COLS = 2 * N;              // one tile's S^T: hi and lo halves
    static constexpr int O_COL = 2 * S_COLS;
    static constexpr int TMEM_USED = O_COL + 2 * O_COLS;
    static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
    // registers per thread: the launch's 128, shifted to the softmax
    static constexpr int SOFT_REGS = 160, OTHER_REGS = 256 - SOFT_REGS;
    static_assert(N == 16 || N == 32, "rows per item");
    // (K tiles are multiplied up to four ahead of the oldest V tile and their slots
    // refilled, while the table still has to hold that V tile's entry)
    static_assert(NT >= 2 && NT + 5 <= kFillTab, "ring slots");
    static_assert(TMEM_USED <= 512, "TMEM");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(Q_OFF % 1024 == 0 && P_OFF % 1024 == 0, "operand alignment");
    static_assert(RED_OFF % 16 == 0 && META_OFF % 8 == 0, "alignment");
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

// D[tmem] (+)= A[smem] * B[smem]^T, K = 32, issued by the lane whose `lead` is set.
// (All lanes come here: the operands are then uniform registers without a move for
// each.)
__device__ __forceinline__ void mma_e4m3_ss(bool lead, uint32_t d_tmem, uint64_t a_desc,
                                            uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void mma_commit_by(bool lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"((uint32_t)lead)
        : "memory");
}

}  // namespace tc

// 2^e for any int8 e, kept finite and normal.
__device__ __forceinline__ float q8_pow2(int e) { return pow2f(e < -126 ? -126 : e); }

// The e4m3 pair nearest to a pair of weights, the weights becoming what is left times
// kQ8PStep (exact: a difference of two numbers so near, and a power of two), plus `more`.
__device__ __forceinline__ uint16_t take_e4m3(uint64_t &p2, uint64_t more) {
    constexpr uint16_t MINUS_STEP = 0xd000;  // -kQ8PStep in fp16
    float a, b;
    tc::f2_unpack(p2, a, b);
    const uint16_t c = e4m3x2(a, b);
    const uint32_t h = e4m3x2_to_f16x2(c);
    tc::f2_unpack(tc::f2_fma(p2, tc::f2_pack(kQ8PStep, kQ8PStep), more), a, b);
    asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(a) : "h"((uint16_t)h), "h"(MINUS_STEP));
    asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(b) : "h"((uint16_t)(h >> 16)), "h"(MINUS_STEP));
    p2 = tc::f2_pack(a, b);
    return c;
}
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

// The kernel's hot code has to stay in the instruction caches beside that of 15
// other warps (with everything inlined it was 187 KB, and warps waited 26% of
// their time for instructions): what is rare, or run by several roles, is a
// function of its own.
__device__ __noinline__ void q8_wait_on(uint64_t *bar, uint32_t parity, const AttnParams *P,
                                        volatile uint32_t *failed) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*failed) return;
        if (clock64() - t0 > P->wait_limit) {
            atomicOr(P->fault, kFaultCopyTimeout);
            *failed = 1;
            return;
        }
    }
}

// Waits for phase `parity` of `bar`, or until some wait of the CTA gave up.
__device__ __forceinline__ void q8_wait(uint64_t *bar, uint32_t parity, const AttnParams &P,
                                        volatile uint32_t *failed) {
    if (!mbar_try_wait(bar, parity)) q8_wait_on(bar, parity, &P, failed);
}

// The same without a call, for the softmax: its registers are its rows.
__device__ __forceinline__ void q8_wait_here(uint64_t *bar, uint32_t parity, const AttnParams &P,
                                             volatile uint32_t *failed) {
    if (mbar_try_wait(bar, parity)) return;
    const uint32_t t0 = (uint32_t)(clock64() >> 10);
    while (!mbar_try_wait(bar, parity)) {
        if (*failed) return;
        if ((uint32_t)(clock64() >> 10) - t0 > (uint32_t)(P.wait_limit >> 10)) {
            atomicOr(P.fault, kFaultCopyTimeout);
            *failed = 1;
            return;
        }
    }
}

// The warp's arrival once all its lanes are here (32 arrivals on one barrier would
// be served one after another).
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The j-th item of this CTA: the first kTcMetaItems from shared memory.
__device__ __noinline__ void q8_decode(const TcParams *T, int j, TcItem *it) {
    *it = tc_decode_global<false>(*T, cta_item(*T, j));
}
__device__ __forceinline__ TcItem q8_item(const TcParams &T, int j, const TcItem *meta) {
    if (j < kTcMetaItems) return meta[j];
    TcItem it;
    q8_decode(&T, j, &it);
    return it;
}

// One lane's copies of a K or V tile: `whole` atoms of consecutive cache rows
// from row y on, and `partial` one more.
template <class C>
__device__ __noinline__ void q8_copy(const CUtensorMap *m4, const CUtensorMap *m1, int y, int whole,
                                     bool partial, uint8_t *dst, uint64_t *bar, uint64_t policy) {
    atom_run<C::ATOM_BYTES>(m4, m1, y, whole, partial, dst, bar, policy);
}

// Fills 0 .. early_fills - 1 of the CTA's first item, one from each of the first
// warps' lane 0, ahead of the producer (a contiguous cache; see swa_tc.cuh).
template <class C, int NT>
__device__ __forceinline__ void q8_early_fills(const TcParams &T, const TcMaps &M,
                                               volatile uint32_t *ftab, uint8_t *ring,
                                               uint64_t *bars, int warp) {
    const AttnParams &P = T.a;
    if (P.block_table != nullptr || warp >= NT || cta_items(T) < 1) return;
    TcItem it;
    q8_decode(&T, 0, &it);
    if (warp >= early_fills<NT, false>(T, it)) return;
    const int t = warp >> 1, kv = warp & 1;  // K, V, K, V, ...
    const int p = it.t0 + kTcTileKeys * t;
    const int n = min(kTcTileKeys, it.cr.c_hi - p);
    ftab[warp] = ((uint32_t)warp << 8) | (uint32_t)warp;  // fill w -> slot w, use parity 0
    mbar_arrive_expect_tx(&bars[C::B_FULL + warp], (uint32_t)((n + 7) >> 3) * C::ATOM_BYTES);
    if (P.withhold_fill == warp && blockIdx.x == 0) return;
    q8_copy<C>(kv ? M.v_atoms : M.k_atoms, kv ? &M.v_atom : &M.k_atom,
               (int)(((long long)it.b * P.Hkv + it.h) * P.L + p), n >> 3, (n & 7) != 0,
               ring + warp * C::TILE_BYTES, &bars[C::B_FULL + warp],
               P.row_tiles > 1 ? l2_policy_evict_normal() : l2_policy_evict_first());
}

// The TMA producer (warp 0): every item's K and V tiles in order into the first free
// ring slots.  Lane s looks after slot s, so that one test finds the free ones, and
// issues its slot's copy (a paged tile's runs of pages go to a lane each, the page
// ids read a tile ahead).  Waits for every copy it issued before returning.
//
// A turn takes some 1000 cycles.  With PAIRS a tile's K and V share one where two
// slots are free: for tiles of 128 dims (1350 cycles of bytes) and 16 rows, where the
// turns are what bounds.  Elsewhere it is the softmax or the bytes, and turns apart
// are better (one turn / two, us: 512 sequences, window 1024, heads of 128, 1 row 52.3
// / 57.6, of 256 84.5 / 82.6; 8 rows of 128 96.3 / 94.8, of 256 105.8 / 102.9; 4
// sequences of 32768 keys 32.3 / 35.1).
template <class C, int NT, bool PAIRS>
__device__ __forceinline__ void q8_producer(const TcParams &T, const TcMaps &M, const TcItem *meta,
                                            volatile uint32_t *ftab, uint8_t *ring, uint64_t *bars,
                                            volatile uint32_t *failed) {
    using namespace tc;
    const AttnParams &P = T.a;
    const int lane = (int)(threadIdx.x & 31);
    const bool paged = P.block_table != nullptr;
    const uint64_t policy = P.row_tiles > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    const int ps = paged ? P.page_size : 8, pa = ps >> 3;  // rows, atoms per page
    const int blks = kTcTileKeys / ps, rest = kTcTileKeys % ps;  // pages per tile
    const int n_items = cta_items(T);
    const int n_early = n_items > 0 ? early_fills<NT, false>(T, meta[0]) : 0;
    uint32_t uses = lane < n_early ? 1 : 0;  // fills handed to this lane's slot so far
    uint32_t f = (uint32_t)n_early;
#pragma unroll 1
    for (int j = 0; j < n_items; ++j) {
        const TcItem it = q8_item(T, j, meta);
        const int y0 = paged ? it.h * ps : (int)(((long long)it.b * P.Hkv + it.h) * P.L);
        int page = 0, next = 0;  // of this lane's run of a tile
        int blk = it.t0 / ps, in = it.t0 - blk * ps, in1 = in;  // where the next tile begins
#pragma unroll 1
        for (int t = paged ? -1 : 0; t < it.n_tiles; ++t) {
            // this lane's run of atoms: all of the tile, or (paged) a page's
            const int p = it.t0 + kTcTileKeys * t;
            const int n = min(kTcTileKeys, it.cr.c_hi - p);
            const int natoms = (n + 7) >> 3;
            int a = 0, run = natoms, y = y0 + p;
            if (paged) {
                // the next tile's page ids are on their way during this one's fills
                page = next;
                const int in0 = in1;
                in1 = in;
                if (t + 1 < it.n_tiles) {
                    const int a1 = lane == 0 ? 0 : ((ps - in) >> 3) + (lane - 1) * pa;
                    if (8 * a1 < min(kTcTileKeys, it.cr.c_hi - p - kTcTileKeys))
                        next = __ldg(P.block_table + (long long)it.b * P.max_blocks + blk + lane);
                    blk += blks;
                    in += rest;
                    if (in >= ps) {
                        in -= ps;
                        ++blk;
                    }
                }
                if (t < 0) continue;
                const int first = (ps - in0) >> 3;
                a = lane == 0 ? 0 : first + (lane - 1) * pa;
                run = min(lane == 0 ? first : pa, natoms - a);
                y = checked_page(P, page, nullptr) * P.Hkv * ps + y0 + (lane == 0 ? in0 : 0);
            }
            const int whole = min(max((n >> 3) - a, 0), run);
            // fills of the tile issued so far
            int done = j == 0 ? min(max(n_early - 2 * t, 0), 2) : 0;
#pragma unroll 1
            while (done < 2) {
                uint32_t free;
                int idle = 0;
                long long since = 0;
                for (;;) {
                    free = __ballot_sync(
                        0xffffffffu,
                        lane < NT && (uses == 0 ||
                                      mbar_test(&bars[C::B_EMPTY + lane], (uses - 1) & 1)));
                    if (free) break;
                    if ((++idle & 63) == 0) {
                        const long long now = clock64();
                        if (idle == 64) since = now;
                        const bool over = now - since > P.wait_limit;
                        if (over && lane == 0) {
                            atomicOr(P.fault, kFaultCopyTimeout);
                            *failed = 1;
                        }
                        if (__any_sync(0xffffffffu, over || *failed)) break;
                    }
                }
                if (!free) goto drain;
                const uint32_t rest = free & (free - 1);
                const bool both = PAIRS && done == 0 && rest != 0;
                const int s0 = __ffs((int)free) - 1, s1 = both ? __ffs((int)rest) - 1 : -1;
                const bool mine = lane == s0 || lane == s1;
                const uint32_t fill = lane == s1 ? f + 1 : f;
                if (mine) {
                    ftab[fill % kFillTab] = (fill << 8) | ((uses & 1) << 4) | (uint32_t)lane;
                    mbar_arrive_expect_tx(&bars[C::B_FULL + lane], (uint32_t)natoms * C::ATOM_BYTES);
                    ++uses;
                }
                __syncwarp();
                // (tests of the bounded waits: one fill's copies are never issued)
                const int held = blockIdx.x == 0 ? P.withhold_fill : -1;
                const int turns = paged && both ? 2 : 1;
#pragma unroll 1
                for (int x = 0; x < turns; ++x) {
                    const int slot = !paged ? lane : (x ? s1 : s0);
                    const int kv = !paged ? (lane == s1 ? 1 : done) : done + x;
                    if ((paged ? run > 0 : mine) && held != (int)(paged ? f + x : fill)) {
                        uint8_t *dst = ring + slot * C::TILE_BYTES + a * C::ATOM_BYTES;
                        const CUtensorMap *m4 = kv ? M.v_atoms : M.k_atoms;
                        // (16, 8, 4 or 2 whole atoms are one copy)
                        if (run == whole && whole > 1 && (whole & (whole - 1)) == 0)
                            tma_load_4d_hint(dst, m4 + (__clz(whole) - 27), 0, y, 0, 0,
                                             &bars[C::B_FULL + slot], policy);
                        else
                            q8_copy<C>(m4, kv ? &M.v_atom : &M.k_atom, y, whole, run > whole, dst,
                                       &bars[C::B_FULL + slot], policy);
                    }
                }
                f += both ? 2 : 1;
                done += both ? 2 : 1;
            }
        }
    }
drain:
    // every copy this CTA issued has landed before it exits
    if (uses > 0)
        mbar_wait_bounded(&bars[C::B_FULL + lane], (uses - 1) & 1, P.fault, kFaultCopyTimeout,
                          P.wait_limit);
    __syncwarp();
}

// Warp 3: per tile and key the factor of its scores (k's scale, in log2 units) and
// v's exponent.  A lane takes four keys of a tile (of one page, if paged: tiles
// then start on an 8-key boundary).  A load takes microseconds beside the tiles'
// copies, several tiles' time: the exponents of SLOTS tiles are on their way at
// once, and the page ids of SLOTS more.  (Each slot has registers of its own: to
// move a value on is to wait for it.)
template <class C>
__device__ __forceinline__ void q8_tables(const Q8TcParams &A, const TcItem *meta, float2 *tabs,
                                          uint64_t *bars, volatile uint32_t *failed) {
    const TcParams &T = A.T;
    const AttnParams &P = T.a;
    constexpr int SLOTS = 3;
    const int lane = (int)(threadIdx.x & 31);
    const int n_items = cta_items(T);
    const bool paged = P.block_table != nullptr;
    const int8_t *kx = A.k_exp, *vx = A.v_exp;
    int e[SLOTS][8], page[SLOTS], row[SLOTS];
    uint32_t masks = 0;  // per slot four bits: this lane's keys that exist
    // the tiles in order; in a paged cache where this lane's keys are
    int j = -1, t = 0, blk = 0, in = 0;
    const int ps = paged ? P.page_size : 8;
    const int blks = kTcTileKeys / ps, rest = kTcTileKeys % ps;  // pages per tile
    TcItem it;
    it.n_tiles = 0;
    // slot s: where the next tile's exponents are; false past the last
    auto locate = [&](int s) -> bool {
        while (t >= it.n_tiles) {
            if (++j >= n_items) return false;
            it = q8_item(T, j, meta);
            t = 0;
            if (paged) {
                blk = (it.t0 + 4 * lane) / ps;
                in = it.t0 + 4 * lane - blk * ps;
            }
        }
        const int jk = it.t0 + kTcTileKeys * t++ + 4 * lane;
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (jk + c >= it.cr.c_lo && jk + c < it.cr.c_hi) m |= 1u << c;
        masks = (masks & ~(0xfu << (4 * s))) | (m << (4 * s));
        // (rows are below 2^31, as the tensor maps' are)
        if (paged) {
            row[s] = it.h * ps + in;
            if (m) page[s] = __ldg(P.block_table + (long long)it.b * P.max_blocks + blk);
            blk += blks;
            in += rest;
            if (in >= ps) {
                in -= ps;
                ++blk;
            }
        } else {
            row[s] = (int)(((long long)it.b * P.Hkv + it.h) * P.L + jk);
        }
        return true;
    };
    int located = 0, f = -2 * SLOTS;  // tiles located, published
#pragma unroll 1
    for (;;) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s, ++f) {
            if (f >= 0) {
                if (f >= located) return;
                const uint32_t slot = f % kQ8Tabs;
                q8_wait(&bars[C::B_TEMPTY + slot], ((f / kQ8Tabs) & 1) ^ 1, P, failed);
                float4 *tab = reinterpret_cast<float4 *>(tabs + slot * kTcTileKeys + 4 * lane);
#pragma unroll
                for (int c = 0; c < 4; c += 2)
                    tab[c / 2] =
                        make_float4(P.qk_scale * q8_pow2(e[s][c]), (float)e[s][4 + c],
                                    P.qk_scale * q8_pow2(e[s][c + 1]), (float)e[s][5 + c]);
                warp_arrive(&bars[C::B_TFULL + slot]);
            }
            if (f + SLOTS >= 0 && f + SLOTS < located) {
                long long at = row[s];
                const uint32_t m = (masks >> (4 * s)) & 0xfu;
                if (paged && m)
                    at += (long long)checked_page(P, page[s], nullptr) * P.Hkv * ps;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    e[s][c] = e[s][4 + c] = 0;
                    if (m >> c & 1) {
                        e[s][c] = kx[at + c];
                        e[s][4 + c] = vx[at + c];
                    }
                }
            }
            if (locate(s)) ++located;
        }
    }
}

// Warps 12..15, first job: an item's query rows as two e4m3 numbers each, and
// their scales.  Warp w of the four takes rows w, w + 4, ..., RP at a time, a lane
// eight elements.  They are on their way an item ahead (a plain load takes
// microseconds while the tiles' copies keep the memory busy), to the very sixteen
// bytes that their two numbers take afterwards: eight at q8_query_at(r, l), eight
// at row N + r.
template <class C>
__device__ __forceinline__ uint32_t q8_query_at(int r, int l) {
    // elements 8 l ..: 16-byte chunk (l / 2) % 8 of slab l / 16
    return (uint32_t)(l >> 4) * C::Q_SLAB + r * 128 +
           ((((uint32_t)(l >> 1) & 7) ^ (uint32_t)(r & 7)) << 4) + (uint32_t)(l & 1) * 8;
}

// The k-th item with keys, once the buffer's previous rows are done with.
template <class C, int HD, int N>
__device__ __forceinline__ void q8_fetch_queries(const AttnParams &P, const TcItem &it, uint32_t k,
                                                 uint8_t *qs, uint64_t *bars,
                                                 volatile uint32_t *failed, int w,
                                                 uint32_t inv_g) {
    constexpr int LPR = HD / 8, RP = 32 / LPR;  // lanes per row, rows per pass
    const int lane = (int)(threadIdx.x & 31);
    const int l = lane % LPR;
    uint8_t *q = qs + (k & 1) * C::Q_BUF;
    q8_wait(&bars[C::B_QEMPTY + (k & 1)], ((k >> 1) & 1) ^ 1, P, failed);
#pragma unroll 1
    for (int r = w + 4 * (lane / LPR); r < it.rows; r += 4 * RP) {
        const __nv_bfloat16 *src = P.q + q8_row(P, it, inv_g, r) * HD + l * 8;
        const uint32_t dst = smem_u32(q + q8_query_at<C>(r, l));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + N * 128), "l"(src + 4)
                     : "memory");
    }
}

template <class C, int HD, int N>
__device__ __forceinline__ void q8_queries(const TcItem &it, uint32_t k, uint8_t *qs, float *qsc,
                                           uint64_t *bars, int w) {
    constexpr int LPR = HD / 8, RP = 32 / LPR;
    const int lane = (int)(threadIdx.x & 31);
    const int sub = lane / LPR, l = lane % LPR;
    uint8_t *q = qs + (k & 1) * C::Q_BUF;
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
    for (int r0 = w; r0 < it.rows; r0 += 4 * RP) {
        const int r = r0 + 4 * sub;
        // (N is a multiple of 8: both rows have the same swizzle phase)
        uint2 *at = reinterpret_cast<uint2 *>(q + q8_query_at<C>(r, l));
        uint32_t b[4] = {0, 0, 0, 0};
        if (r < it.rows) {
            const uint2 x = at[0], y = at[N * 16];
            b[0] = x.x, b[1] = x.y, b[2] = y.x, b[3] = y.y;
        }
        // the smallest exponent that holds the row, as for the cache
        const uint32_t a =
            row_max<LPR>(max_u16x2(max_u16x2(b[0] & 0x7fff7fffu, b[1] & 0x7fff7fffu),
                                   max_u16x2(b[2] & 0x7fff7fffu, b[3] & 0x7fff7fffu)));
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
        if (r < it.rows) {
            at[0] = make_uint2(hi[0], hi[1]);
            at[N * 16] = make_uint2(lo[0], lo[1]);
            // (a row with an infinity or a NaN has scores of NaN: its two numbers are
            // finite where the conversion bounds them)
            if (l == 0) qsc[(k & 1) * N + r] = a < 0x7f80u ? pow2f(e) : __int_as_float(0x7fffffff);
        }
    }
    fence_proxy_async_smem();
    warp_arrive(&bars[C::B_QFULL + (k & 1)]);
}

// Warps 12..15, second job: the k-th item's O through 1 / l to the output (or to
// the split partials), and the rows of an item without keys.
template <class C, int HD, int D, int N, int OB>
__device__ __forceinline__ void q8_epilogue(const AttnParams &P, const TcItem &it, uint32_t k,
                                            uint32_t tmem, const float *sums, float *linv,
                                            uint32_t *rowidx, uint64_t *bars,
                                            volatile uint32_t *failed, uint32_t inv_g) {
    using namespace tc;
    constexpr int MH = D / 128;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int t = (int)threadIdx.x - (kQ8TcThreads - 128);  // 0..127
    const int quad = t >> 5;
    const size_t bh = (size_t)it.b * P.Hkv + it.h;
    const size_t prow0 = (bh * P.splits + it.split) * P.R + it.row0;
    if (it.n_tiles == 0) {
        for (int idx = t; idx < it.rows * HD; idx += 128) {
            const int r = idx / HD, d = idx % HD;
            if (P.splits == 1) {
                const size_t orow = q8_row(P, it, inv_g, r);
                P.out[orow * HD + d] = __float2bfloat16_rn(0.f);
                if (d == 0 && P.lse != nullptr) P.lse[orow] = NEG_INF;
            } else {
                P.part_acc[(prow0 + r) * HD + d] = 0.f;
                if (d == 0) {
                    P.part_ml[(prow0 + r) * 2] = NEG_INF;
                    P.part_ml[(prow0 + r) * 2 + 1] = 0.f;
                }
            }
        }
        return;
    }
    // (below 2^31 by the plan's size checks)
    uint32_t *rows = rowidx + (k & 1) * N;
    float *li = linv + (k & 1) * N;
    const uint32_t ob = k % OB;
    const uint32_t orow = t < it.rows ? (uint32_t)q8_row(P, it, inv_g, t) : 0u;
    q8_wait(&bars[C::B_LFULL + (k & 3)], (k >> 2) & 1, P, failed);
    if (t < it.rows) {
        const float *sum = sums + (k & 3) * 5 * N + t;
        const float l = (sum[0] + sum[N]) + (sum[2 * N] + sum[3 * N]);
        const float m = sum[4 * N];
        const bool any = !(l <= 0.f);  // (a NaN stays one)
        rows[t] = orow;
        li[t] = any ? __frcp_rn(l) : 0.f;
        if (P.splits > 1) {
            P.part_ml[(prow0 + t) * 2] = any ? m : NEG_INF;
            P.part_ml[(prow0 + t) * 2 + 1] = l;
        } else if (P.lse != nullptr) {
            P.lse[orow] = any ? (m + __log2f(l)) * kLn2 : NEG_INF;
        }
    }
    asm volatile("bar.sync 5, 128;" ::: "memory");
    q8_wait(&bars[C::B_OFULL + ob], (k / OB) & 1, P, failed);
    fence_after_sync();
    const uint32_t o0 = tmem + ((uint32_t)(quad * 32) << 16) + C::O_COL + ob * C::O_COLS;
    const uint64_t sp = f2_pack(1.f / kQ8PStep, 1.f / kQ8PStep);
    // (a warp stores 64 bytes of a row at a time: whole sectors)
    __nv_bfloat16 *out = P.out + t;
#pragma unroll 1
    for (int c = 0; c < it.rows; c += 8) {
        uint32_t o[MH][3][8];
#pragma unroll
        for (int mh = 0; mh < MH; ++mh)
#pragma unroll
            for (int p = 0; p < 3; ++p) tmem_load<8>(o0 + mh * C::O_HALF + p * N + c, o[mh][p]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint2 row = *reinterpret_cast<const uint2 *>(rows + c + e);
            const float2 l2 = *reinterpret_cast<const float2 *>(li + c + e);
            const bool one = t < HD && c + e < it.rows, two = t < HD && c + e + 1 < it.rows;
#pragma unroll
            for (int mh = 0; mh < MH; ++mh) {
                auto part = [&](int p) {
                    return f2_pack(__uint_as_float(o[mh][p][e]), __uint_as_float(o[mh][p][e + 1]));
                };
                const uint64_t x2 = f2_fma(f2_fma(part(2), sp, part(1)), sp, part(0));
                float a, b;
                if (P.splits == 1) {
                    f2_unpack(f2_mul(x2, f2_pack(l2.x, l2.y)), a, b);
                    if (one) out[(size_t)row.x * HD + mh * 128] = __float2bfloat16_rn(a);
                    if (two) out[(size_t)row.y * HD + mh * 128] = __float2bfloat16_rn(b);
                } else {
                    f2_unpack(x2, a, b);
                    float *acc = P.part_acc + (prow0 + c + e) * HD + mh * 128 + t;
                    if (one) acc[0] = a;
                    if (two) acc[HD] = b;
                }
            }
        }
    }
    // O and the item's sums may be overwritten
    fence_before_sync();
    warp_arrive(&bars[C::B_OFREE + ob]);
}

// HD: head_dim.  Rows of 64 lie in tiles of D = 128 dims like rows of 128: the TMA
// fills what is past their end with zeros.
template <int HD, int N, int NT>
__global__ void __launch_bounds__(kQ8TcThreads, 1)
    swa_q8_tc_kernel(const __grid_constant__ Q8TcParams A, const __grid_constant__ TcMaps M) {
    constexpr int D = HD < 128 ? 128 : HD;
    using C = Q8Cfg<D, N, NT>;
    using namespace tc;
    constexpr int MH = D / 128, OB = 2;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const TcParams &T = A.T;
    const AttnParams &P = T.a;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    uint8_t *ring = sm + C::RING_OFF;
    uint8_t *qs = sm + C::Q_OFF;
    uint8_t *ps = sm + C::P_OFF;
    float2 *tabs = reinterpret_cast<float2 *>(sm + C::TAB_OFF);
    float *red = reinterpret_cast<float *>(sm + C::RED_OFF);
    float *refs = reinterpret_cast<float *>(sm + C::REF_OFF);
    float *alphas = reinterpret_cast<float *>(sm + C::ALPHA_OFF);
    float *qsc = reinterpret_cast<float *>(sm + C::QSC_OFF);
    float *sums = reinterpret_cast<float *>(sm + C::SUM_OFF);
    float *linv = reinterpret_cast<float *>(sm + C::LINV_OFF);
    uint32_t *rowidx = reinterpret_cast<uint32_t *>(sm + C::ROW_OFF);
    TcItem *meta = reinterpret_cast<TcItem *>(sm + C::META_OFF);
    volatile uint32_t *ftab = reinterpret_cast<volatile uint32_t *>(sm + C::FTAB_OFF);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::BAR_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC_OFF);
    volatile uint32_t *failed = tmem_slot + 1;

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    // ---------------------------------------------------------------- setup
    if (warp == 0 && lane < 10) {
        const CUtensorMap *mp = lane < 4    ? &M.k_atoms[lane]
                                : lane < 8  ? &M.v_atoms[lane - 4]
                                : lane == 8 ? &M.k_atom
                                            : &M.v_atom;
        prefetch_tmap(mp);
    }
    // arrivals on a barrier: one (a commit, a copy's bytes, one warp), or one from
    // each warp of a role
    for (int i = tid; i < C::NBARS; i += kQ8TcThreads) {
        const bool soft = (i >= C::B_SFREE && i < C::B_PVDONE) ||
                          (i >= C::B_LFULL && i < C::B_DRAIN) || i >= C::B_TEMPTY;
        const bool four = (i >= C::B_QFULL && i < C::B_QEMPTY) ||
                          (i >= C::B_OFREE && i < C::B_LFULL);
        mbar_init(&bars[i], soft ? 8 : four ? 4 : 1);
        fence_barrier_init();
    }
    if (tid == 0) *failed = 0;
    // query rows past an item's stay what they are here: zero, or another
    // item's (their columns are never looked at, but should not raise the
    // references either)
    for (int i = tid; i < 2 * C::Q_BUF / 16; i += kQ8TcThreads)
        reinterpret_cast<uint4 *>(qs)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < 2 * N; i += kQ8TcThreads) qsc[i] = 0.f;
    fence_proxy_async_smem();
    for (int i = tid; i < kFillTab; i += kQ8TcThreads) ftab[i] = 0xffffffffu;
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_trigger();
    if (lane == 0) q8_early_fills<C, NT>(T, M, ftab, ring, bars, warp);
    for (int j = tid; j < kTcMetaItems; j += kQ8TcThreads)
        if (j < cta_items(T)) q8_decode(&T, j, &meta[j]);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int n_items = cta_items(T);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    }
    if (warp == 0) {
        // ======================================================= producer
        q8_producer<C, NT, D == 128 && N == 16>(T, M, meta, ftab, ring, bars, failed);
    } else if (warp <= 2) {
        // ============================================================ MMA
        // Warp 1 issues S = K8 Q^T of every tile, warp 2 O += V8^T P^T, each as
        // soon as its operands have landed.  A step's conditions are one barrier
        // per lane, tested by one instruction.
        const bool pv = warp == 2;
        const bool leader = lane == 0;
        constexpr uint32_t ID_QK = idesc_e4m3_f32(128, 2 * N, 0, 0);
        constexpr uint32_t ID_PV = idesc_e4m3_f32(128, 3 * N, 1, 1);
        const uint64_t ring_d = smem_desc_sw128(smem_u32(ring), 16, C::ATOM_BYTES);
        const uint64_t q_d = smem_desc_sw128(smem_u32(qs), 16, 1024);
        const uint64_t p_d = smem_desc_sw32(smem_u32(ps), C::P_BLOCK, 256);
        // lane 0: the tile's fill; 1 and 2: barriers b1 and b2 (b < 0: none)
        auto ready = [&](uint32_t fill, int b1, uint32_t par1, int b2, uint32_t par2) -> int {
            uint32_t e = 0xffffffffu;
            int idle = 0;
            long long since = 0;
            const int b = lane == 1 ? b1 : b2;
            const uint32_t par = (lane == 1 ? par1 : par2) & 1;
            bool done = lane > 2 || (lane > 0 && b < 0);
            for (;;) {
                if (lane == 0) {
                    e = ftab[fill % kFillTab];
                    if ((e >> 8) == (fill & 0xffffffu))
                        done = mbar_test(&bars[C::B_FULL + (e & 15u)], (e >> 4) & 1u);
                } else if (!done) {
                    done = mbar_test(&bars[b], par);
                }
                if (__all_sync(0xffffffffu, done)) break;
                if ((++idle & 63) == 0) {
                    const long long now = clock64();
                    if (idle == 64) since = now;
                    const bool over = now - since > P.wait_limit;
                    if (over && lane == 0) {
                        atomicOr(P.fault, kFaultCopyTimeout);
                        *failed = 1;
                    }
                    if (__any_sync(0xffffffffu, over || *failed)) return -1;
                }
            }
            return (int)(__shfl_sync(0xffffffffu, e, 0) & 15u);
        };
        uint32_t g = 0, k = 0;  // tiles, items with keys so far
        bool ok = true;
#pragma unroll 1
        for (int j = 0; j < n_items && ok; ++j) {
            const TcItem it = q8_item(T, j, meta);
            const int n_tiles = __shfl_sync(0xffffffffu, it.n_tiles, 0);
            if (n_tiles == 0) continue;
            const int left0 = __shfl_sync(0xffffffffu, it.cr.c_hi - it.t0, 0);
            const int z0 = __shfl_sync(0xffffffffu, it.cr.c_lo - it.t0, 0);
#pragma unroll 1
            for (int t = 0; t < n_tiles; ++t, ++g) {
                const bool first = t == 0, last = t == n_tiles - 1;
                const uint32_t h = g & 1;
                if (!pv) {
                    const uint32_t qb = k & 1;
                    const int slot = ready(2 * g, C::B_SFREE + (int)h, (g >> 1) + 1,
                                           first ? C::B_QFULL + (int)qb : -1, k >> 1);
                    ok = slot >= 0;
                    if (!ok) break;
                    fence_after_sync();
                    const uint64_t qbase = q_d + (uint64_t)(qb * (C::Q_BUF >> 4));
                    const uint64_t abase = ring_d + (uint64_t)(slot * (C::TILE_BYTES >> 4));
                    const uint32_t d = tmem + h * C::S_COLS;
#pragma unroll
                    for (int s = 0; s < C::SLABS; ++s)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_e4m3_ss(leader, d, abase + (uint64_t)(s * 64 + kk * 2),
                                        qbase + (uint64_t)(s * (C::Q_SLAB >> 4) + kk * 2), ID_QK,
                                        (s | kk) != 0);
                    mma_commit_by(leader, &bars[C::B_SFULL + h]);
                    mma_commit_by(leader, &bars[C::B_EMPTY + slot]);
                    if (last) mma_commit_by(leader, &bars[C::B_QEMPTY + qb]);
                } else {
                    const uint32_t ob = k % OB;
                    const int slot = ready(2 * g + 1, C::B_PFULL + (int)h, g >> 1,
                                           first ? C::B_OFREE + (int)ob : -1, (k / OB) + 1);
                    ok = slot >= 0;
                    if (!ok) break;
                    fence_after_sync();
                    // only the 32-key steps that hold valid keys are multiplied; the
                    // rows of the last step past the chunk's end, and those before
                    // the chunk in a paged cache's first tile, are zeroed first, so
                    // that 0 * (whatever the slot holds there) cannot reach O
                    const int nv = last ? left0 - kTcTileKeys * t : kTcTileKeys;
                    const int steps = (nv + 31) >> 5;
                    const int z = first ? z0 : 0;
                    if ((nv & 31) || z > 0) {
                        uint8_t *vt = ring + slot * C::TILE_BYTES;
                        zero_v_rows<C>(vt, nv, 32 * steps, lane);
                        zero_v_rows<C>(vt, 0, z, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    // A = V^T, MN-major: a slab holds 128 dims, 8-key groups one
                    // atom apart; B = the parts of P, MN-major
                    const uint64_t bbase = p_d + (uint64_t)(h * (C::P_BUF >> 4));
                    const uint64_t abase = ring_d + (uint64_t)(slot * (C::TILE_BYTES >> 4));
                    const uint32_t d = tmem + C::O_COL + ob * C::O_COLS;
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        if (k4 >= steps) break;
#pragma unroll
                        for (int mh = 0; mh < MH; ++mh)
                            mma_e4m3_ss(leader, d + mh * C::O_HALF,
                                        abase + (uint64_t)((mh * 1024 + k4 * 4 * C::ATOM_BYTES) >> 4),
                                        bbase + (uint64_t)(k4 * 1024 >> 4), ID_PV,
                                        k4 > 0 || !first);
                    }
                    mma_commit_by(leader, &bars[C::B_PVDONE + h]);
                    mma_commit_by(leader, &bars[C::B_EMPTY + slot]);
                    if (last) mma_commit_by(leader, &bars[C::B_OFULL + ob]);
                }
                __syncwarp();
            }
            ++k;
        }
        // all issued MMAs complete before TMEM is released
        if (leader) {
            mma_commit(&bars[C::B_DRAIN + (pv ? 1 : 0)]);
            mbar_wait_bounded(&bars[C::B_DRAIN + (pv ? 1 : 0)], 0, P.fault, kFaultCopyTimeout,
                              P.wait_limit);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ===================================================== key factors
        q8_tables<C>(A, meta, tabs, bars, failed);
    } else if (warp < 12) {
        // ===================================================== softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFT_REGS));
        constexpr int HN = N / 2;                // rows per softmax warpgroup
        const int wg = (warp - 4) >> 2;          // softmax warpgroup
        const int sw = warp & 3;                 // warp within the group: TMEM lane quadrant
        const int lk = sw * 32 + lane;           // TMEM lane: key of S^T, dim row of O^T
        const int r0 = wg * HN;                  // first packed row of this group
        const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16);
        const uint32_t flip = (uint32_t)(lk >> 2) & 1;  // 32-byte swizzle phase of key lk
        float *rd = red + r0, *ref = refs + r0, *alpha = alphas + r0;
        constexpr int CH = HN / 8;               // chunks of eight rows
        constexpr uint32_t ALL = (1u << HN) - 1;
        // the loops over a thread's rows are rolled: the arrays turn by eight rows a
        // time instead
        auto turn = [](float(&x)[HN]) {
            if constexpr (HN == 16) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = x[e];
                    x[e] = x[8 + e];
                    x[8 + e] = y;
                }
            }
        };
        uint32_t g = 0, k = 0;                   // tiles, items with keys so far
#pragma unroll 1
        for (int j = 0; j < n_items; ++j) {
            const TcItem it = q8_item(T, j, meta);
            if (it.n_tiles == 0) continue;
            const float *rs = qsc + (k & 1) * N + r0;
            float lrow[HN];
#pragma unroll
            for (int r = 0; r < HN; ++r) lrow[r] = 0.f;
            const int qp_i0 = it.cr.qp + it.i0;  // position of the item's first draft row
            // first keys of the tiles that every row sees whole
            const int i_last = (it.rows - 1) / P.G;
            const int inner_lo =
                (int)max((long long)qp_i0 + i_last - P.window + 1, (long long)it.cr.c_lo);
            const int inner_hi = min(qp_i0, it.cr.c_hi - 1) - (kTcTileKeys - 1);
#pragma unroll 1
            for (int t = 0; t < it.n_tiles; ++t, ++g) {
                const uint32_t h = g & 1, slot = g % kQ8Tabs;
                const int j0 = it.t0 + kTcTileKeys * t;
                // bit r: this group's row r sees the key; all of them in a tile between
                // the item's last window start and its first row's position
                uint32_t sees = ALL;
                if (j0 < inner_lo || j0 > inner_hi) {
                    const int jk = j0 + lk;
                    sees = 0;
                    if (jk >= it.cr.c_lo && jk < it.cr.c_hi) {
                        // the draft rows [lo, lo + window) (jk < q_pos + q_len: lo < 512)
                        const int lo = jk - qp_i0;
                        const int ra = max(max(lo, 0) * P.G - r0, 0);
                        const int rb = (lo >= it.rows - P.window
                                            ? (int)it.rows
                                            : min(max(lo + P.window, 0) * P.G, (int)it.rows)) - r0;
                        if (ra < HN && rb > ra) sees = (ALL << ra) & (ALL >> max(HN - rb, 0));
                    }
                }
                // one barrier per lane, tested by one instruction: the tile's table
                // and scores, the previous PV of the tile's P buffer, an item's query
                // scales
                {
                    uint64_t *bar = &bars[lane == 0   ? C::B_TFULL + slot
                                          : lane == 1 ? C::B_SFULL + h
                                          : lane == 2 ? C::B_PVDONE + h
                                                      : C::B_QFULL + (k & 1)];
                    const uint32_t par = (lane == 0   ? g / kQ8Tabs
                                          : lane == 1 ? g >> 1
                                          : lane == 2 ? (g >> 1) + 1
                                                      : k >> 1) & 1;
                    if (lane < (t == 0 ? 4 : 3)) q8_wait_here(bar, par, P, failed);
                    __syncwarp();
                }
                if (r0 >= it.rows) {
                    // none of this group's rows exists (their columns are never
                    // looked at): only the barriers are kept going
                    if (lane < 3)
                        mbar_arrive(&bars[lane == 0   ? C::B_SFREE + h
                                          : lane == 1 ? C::B_TEMPTY + slot
                                                      : C::B_PFULL + h]);
                    continue;
                }
                const float2 key = tabs[slot * kTcTileKeys + lk];
                fence_after_sync();
                // u = (S_hi + S_lo / 16) * (row scale * key factor) + e_v
                float v[HN], over = NEG_INF;
                const uint64_t lo2 = f2_pack(1.f / kQ8QLo, 1.f / kQ8QLo);
                const uint64_t ks2 = f2_pack(key.x, key.x), ve2 = f2_pack(key.y, key.y);
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    uint32_t hi[8], lo[8];
                    tmem_load<8>(tl + h * C::S_COLS + r0 + 8 * c, hi);
                    tmem_load<8>(tl + h * C::S_COLS + N + r0 + 8 * c, lo);
                    tmem_wait_ld();
#pragma unroll
                    for (int r4 = 0; r4 < 8; r4 += 4) {
                        const float4 s4 = *reinterpret_cast<const float4 *>(rs + 8 * c + r4);
                        const uint64_t rs2[2] = {f2_pack(s4.x, s4.y), f2_pack(s4.z, s4.w)};
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const int r = r4 + 2 * p;
                            const uint64_t s2 =
                                f2_fma(f2_pack(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1])),
                                       lo2,
                                       f2_pack(__uint_as_float(hi[r]), __uint_as_float(hi[r + 1])));
                            // (the two scales first: a row's alone may take the score past
                            // the range, where the key's brings it back)
                            f2_unpack(f2_fma(s2, f2_mul(rs2[p], ks2), ve2), v[r], v[r + 1]);
                        }
                    }
                    if (sees != ALL) {
                        const uint32_t s8 = sees >> (8 * c);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            if (!(s8 & (1u << r))) v[r] = NEG_INF;
                    }
#pragma unroll
                    for (int r4 = 0; r4 < 8; r4 += 4) {
                        const float4 m4 = *reinterpret_cast<const float4 *>(ref + 8 * c + r4);
                        over = fmax3(over, v[r4] - m4.x, v[r4 + 1] - m4.y);
                        over = fmax3(over, v[r4 + 2] - m4.z, v[r4 + 3] - m4.w);
                    }
                    turn(v);
                }
                // the scores and the table are read
                fence_before_sync();
                __syncwarp();
                if (lane < 2)
                    mbar_arrive(&bars[lane == 0 ? C::B_SFREE + h : C::B_TEMPTY + slot]);

                // an item's first tile sets the references
                if (t == 0 || group_any(wg, over > kQ8RaiseAt)) {
                    // exact maximum per row over the tile's keys
#pragma unroll 1
                    for (int c = 0; c < CH; ++c) {
                        float m = NEG_INF;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float x = warp_max(v[e]);
                            if (lane == e) m = x;
                        }
                        if (lane < 8) rd[sw * N + 8 * c + lane] = m;
                        turn(v);
                    }
                    group_sync(wg);
                    if (lk < HN) {
                        const float tm =
                            fmaxf(fmax3(rd[lk], rd[N + lk], rd[2 * N + lk]), rd[3 * N + lk]);
                        const float mo = t == 0 ? kNoRef : ref[lk];
                        const float mn = fmaxf(mo, tm - kQ8RefBelow);
                        ref[lk] = mn;
                        alpha[lk] = fast_exp2(mo - mn);
                    }
                    // every PV of this item so far has completed before O is scaled
                    if (t > 0) {
                        q8_wait_here(&bars[C::B_PVDONE + (h ^ 1)], ((g - 1) >> 1) & 1, P, failed);
                        fence_after_sync();
                    }
                    group_sync(wg);
                    if (t > 0) {
                        const uint32_t o0 = tl + C::O_COL + (k % OB) * C::O_COLS + r0;
#pragma unroll 1
                        for (int c = 0; c < CH; ++c) {
                            const float *al = alpha + 8 * c;
#pragma unroll
                            for (int e = 0; e < 8; ++e) lrow[e] *= al[e];
                            turn(lrow);
#pragma unroll 1
                            for (int i = 0; i < MH * 3; ++i) {
                                uint32_t o[8];
                                tmem_load<8>(o0 + i * N + 8 * c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * al[e]);
                                tmem_store<8>(o0 + i * N + 8 * c, o);
                            }
                        }
                        tmem_wait_st();
                        fence_before_sync();  // (the arrival below orders it for the next PV)
                    }
                }
                // P = 2^(u - ref) in e4m3 numbers; the row sum adds P 2^-e_v
                const int ev = (int)key.y;
                const float ive = pow2f(ev > 126 ? -126 : (ev < -127 ? 127 : -ev));
                const uint64_t iv2 = f2_pack(ive, ive);
                // P_2's offset: the fraction of key * 0.618.., in [-2^-10, 2^-10)
                const float offset = (float)(int)((uint32_t)(j0 + lk) * 0x9e3779b9u) * 0x1p-41f;
                const uint64_t offset2 = f2_pack(offset, offset);
                uint8_t *pt = ps + h * C::P_BUF + lk * 32;
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    uint32_t pk[3][4];
#pragma unroll
                    for (int r4 = 0; r4 < 8; r4 += 4) {
                        const float4 m4 = *reinterpret_cast<const float4 *>(ref + 8 * c + r4);
                        const uint64_t m2[2] = {f2_pack(m4.x, m4.y), f2_pack(m4.z, m4.w)};
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int r = r4 + 2 * q;
                            float d0, d1;
                            f2_unpack(f2_sub(f2_pack(v[r], v[r + 1]), m2[q]), d0, d1);
                            const float p0 = fast_exp2(d0), p1 = fast_exp2(d1);
                            uint64_t p2 = f2_pack(p0, p1);
                            f2_unpack(f2_fma(p2, iv2, f2_pack(lrow[r], lrow[r + 1])), lrow[r],
                                      lrow[r + 1]);
                            pk[0][r / 2] = take_e4m3(p2, 0);
                            pk[1][r / 2] = take_e4m3(p2, offset2);
                            f2_unpack(p2, d0, d1);
                            pk[2][r / 2] = e4m3x2(d0, d1);
                        }
                    }
                    // columns i N + r0 + 8 c .. of part i, in key lk's 32-byte rows
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        const uint32_t at =
                            N == 16 ? (i >> 1) * C::P_BLOCK + (((uint32_t)(i & 1) ^ flip) << 4) + wg * 8
                                    : i * C::P_BLOCK + (((uint32_t)wg ^ flip) << 4) + 8 * c;
                        *reinterpret_cast<uint2 *>(pt + at) =
                            make_uint2(pk[i][0] | (pk[i][1] << 16), pk[i][2] | (pk[i][3] << 16));
                    }
                    turn(v);
                    turn(lrow);
                }
                fence_proxy_async_smem();
                warp_arrive(&bars[C::B_PFULL + h]);
            }

            // the warp's row sums and the references, for the epilogue
            const float l = lane_reduce<HN, false>(lrow);
            float *sum = sums + (k & 3) * 5 * N + r0 + lane;
            if (lane < HN) {
                sum[sw * N] = l;
                if (sw == 0) sum[4 * N] = ref[lane];
            }
            warp_arrive(&bars[C::B_LFULL + (k & 3)]);
            ++k;
        }
    } else {
        // ====================================== query rows and epilogues
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
        const uint32_t inv_g = q8_inv_g(P);
        const int w = warp - 12;
        uint32_t kq = 0, k = 0;  // items with keys whose queries are fetched, finished
        int jq = 0;
        TcItem next;             // the item whose queries are on their way
        auto fetch = [&]() {
            for (next.n_tiles = 0; jq < n_items && next.n_tiles == 0; ++jq) next = q8_item(T, jq, meta);
            if (next.n_tiles > 0)
                q8_fetch_queries<C, HD, N>(P, next, kq++, qs, bars, failed, w, inv_g);
        };
        fetch();
        // queries one item ahead of the epilogues
#pragma unroll 1
        for (int j = -1; j < n_items; ++j) {
            TcItem it;
            it.n_tiles = 1;
            if (j >= 0) it = q8_item(T, j, meta);
            if (it.n_tiles > 0 && next.n_tiles > 0) {
                q8_queries<C, HD, N>(next, kq - 1, qs, qsc, bars, w);
                fetch();
            }
            if (j < 0) continue;
            q8_epilogue<C, HD, D, N, OB>(P, it, k, tmem, sums, linv, rowidx, bars, failed, inv_g);
            if (it.n_tiles > 0) ++k;
        }
    }

    // ---------------------------------------------------------- teardown
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace swa
