// Entry points of the 8-bit KV cache: argument checks, launches, and the
// attention over it.
#include <cuda_runtime.h>

#include "../../include/swa.h"
#include "swa_host.h"
#include "swa_q8.cuh"
#include "swa_q8_host.h"
#include "swa_tc_host.h"

namespace {

using swa::aligned_to;
using swa::api_fail;

swa_status check_dims(const swa_dims *d, bool rows) {
    if (d == nullptr) return api_fail(SWA_ERR_INVALID_ARG, "dims is NULL");
    if (d->batch < 1 || d->batch > 65535)
        return api_fail(SWA_ERR_INVALID_ARG, "batch %d outside [1, 65535]", d->batch);
    if (rows && (d->q_len < 1 || d->q_len > swa::kMaxBlockLen))
        return api_fail(SWA_ERR_INVALID_ARG, "q_len %d outside [1, %d]", d->q_len,
                        swa::kMaxBlockLen);
    if (d->num_kv_heads < 1 || d->num_kv_heads > 65535)
        return api_fail(SWA_ERR_INVALID_ARG, "num_kv_heads %d outside [1, 65535]",
                        d->num_kv_heads);
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
        return api_fail(SWA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", d->head_dim);
    if (d->max_len < 1) return api_fail(SWA_ERR_INVALID_ARG, "max_len %d < 1", d->max_len);
    return SWA_OK;
}

swa_status check_cache(const swa_q8_cache *c, const swa_paged *paged, const swa_dims *d) {
    if (c == nullptr || !c->k || !c->v || !c->k_exp || !c->v_exp)
        return api_fail(SWA_ERR_INVALID_ARG, "the cache or one of its pointers is NULL");
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16))
        return api_fail(SWA_ERR_INVALID_ARG, "the K and V caches must be 16-byte aligned");
    return paged != nullptr ? swa::api_check_paged(paged, d) : SWA_OK;
}

// The fields that a cache row's place depends on.
void set_cache(swa::AttnParams &P, const swa_paged *paged, const swa_dims *d,
               const int32_t *seq_lens, uint32_t *fault) {
    P.fault = fault;
    P.B = d->batch;
    P.Hkv = d->num_kv_heads;
    P.L = d->max_len;
    P.seq_lens = seq_lens;
    if (paged != nullptr) {
        P.block_table = paged->block_table;
        P.page_size = paged->page_size;
        P.max_blocks = paged->max_blocks;
        P.num_pages = paged->num_pages;
    }
}

// CTAs of U rows per group of lanes: chunks of `rows` rows for each of `units`.
struct Shape {
    int unroll, chunks;
};
// Four rows at once, their loads all in flight, where a unit has that many rows for
// every group of lanes and every SM still gets two CTAs; otherwise one.  Measured, head
// dim 256, 2 heads, q tokens written and n read back per sequence, one row / four, us:
// 512 sequences, 64 and 64: 42.6 / 29.7; 64 of them 7.7 / 6.4; 512 of 8 and 8 (16 and
// 8 rows per unit) 7.5 / 8.5; 8 of 8 and 64 (64 CTAs) 3.0 / 3.5.
Shape shape_of(long long units, long long rows, int D, int sms) {
    Shape f;
    for (f.unroll = 4;; f.unroll = 1) {
        const int per = swa::kQ8Threads * 8 / D * f.unroll;
        f.chunks = (int)((rows + per - 1) / per);
        if (f.unroll == 1 || (rows >= per && units * f.chunks >= 2LL * sms)) return f;
    }
}

template <int D, int U>
cudaError_t append_as(const swa::Q8AppendParams &A, dim3 grid, cudaStream_t s) {
    return swa::launch_kernel(swa::swa_q8_append_kernel<D, U>, grid, dim3(swa::kQ8Threads), 0, s,
                              A);
}
template <int D, int U>
cudaError_t read_as(const swa::Q8ReadParams &A, dim3 grid, cudaStream_t s) {
    return swa::launch_kernel(swa::swa_q8_read_kernel<D, U>, grid, dim3(swa::kQ8Threads), 0, s, A);
}

uint32_t page_inv(const swa::AttnParams &P) {
    return P.page_size > 0 ? 0xffffffffu / (uint32_t)P.page_size : 0;
}

cudaError_t launch_append(swa::Q8AppendParams &A, int D, int sms, cudaStream_t s) {
    const Shape f = shape_of(2LL * A.cache.B, (long long)A.cache.q_len * A.cache.Hkv, D, sms);
    const dim3 grid(2u * (unsigned)f.chunks, (unsigned)A.cache.B);  // (at most 65535 sequences)
    const int groups = swa::kQ8Threads * 8 / D;
    A.step_tok = groups / A.cache.Hkv;
    A.step_h = groups % A.cache.Hkv;
    A.page_inv = page_inv(A.cache);
    if (f.unroll == 1)
        return D == 64    ? append_as<64, 1>(A, grid, s)
               : D == 128 ? append_as<128, 1>(A, grid, s)
                          : append_as<256, 1>(A, grid, s);
    return D == 64    ? append_as<64, 4>(A, grid, s)
           : D == 128 ? append_as<128, 4>(A, grid, s)
                      : append_as<256, 4>(A, grid, s);
}

cudaError_t launch_read(swa::Q8ReadParams &A, int D, int sms, cudaStream_t s) {
    const Shape f = shape_of(2LL * A.cache.B * A.cache.Hkv, A.n, D, sms);
    const unsigned z = 2u * (unsigned)A.cache.Hkv;
    const dim3 grid((unsigned)f.chunks, (unsigned)A.cache.B, z < 65535u ? z : 65535u);
    A.page_inv = page_inv(A.cache);
    if (f.unroll == 1)
        return D == 64    ? read_as<64, 1>(A, grid, s)
               : D == 128 ? read_as<128, 1>(A, grid, s)
                          : read_as<256, 1>(A, grid, s);
    return D == 64    ? read_as<64, 4>(A, grid, s)
           : D == 128 ? read_as<128, 4>(A, grid, s)
                      : read_as<256, 4>(A, grid, s);
}

// The bf16 rows of every sequence's windows, [B, Hkv, span, D] for K and for V,
// the lengths and positions counted from the first of them, and the split
// partials of the attention over them.
struct RowsLayout {
    int span;
    size_t v, shifted, parts;
};

RowsLayout rows_layout(const swa_dims *d, int32_t window) {
    RowsLayout l;
    const long long span = (long long)window + d->q_len - 1;
    l.span = (int)(span < d->max_len ? span : d->max_len);
    const size_t bytes = (size_t)d->batch * d->num_kv_heads * l.span * d->head_dim * 2;
    l.v = bytes;
    l.shifted = 2 * bytes;
    l.parts = l.shifted + ((size_t)d->batch * 8 + 15) / 16 * 16;
    return l;
}

// The fp8 tensor-core kernel's work of a call: items of `rows` packed rows and
// `splits` chunks of `chunk` keys per (sequence, KV head).
struct Plan {
    int rows, q_rows, row_tiles, n, splits, chunk, grid, early;
    long long items;
    size_t workspace;
};

constexpr int kTileKeys = 128;
constexpr int kMaxSplits = 64;

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Key tiles per item for `units` windows of `tiles` each: the fewest steps, of an SM's
// items one after another, where an item costs two tiles beside its own and a split
// six (its partials and the merge's launch) and a quarter for every part.  Measured,
// unsplit / split: 8 sequences of 8 rows, 8 heads of 256 on 2 (16 units), window 500
// 10.0 / 11.7 us, 1000 13.1 / 13.5, 2000 19.3 / 15.0.
long long split_tiles(long long units, long long tiles, int sms) {
    long long best = tiles, least = 0;
    for (long long n = 1; n <= kMaxSplits && n <= tiles; ++n) {
        const long long per = (tiles + n - 1) / n, parts = (tiles + per - 1) / per;
        if (parts < n) continue;  // (no fewer tiles than with fewer parts)
        const long long turns = (units * parts + sms - 1) / sms;
        const long long cost = 4 * turns * (per + 2) + (n > 1 ? 24 + n : 0);
        if (n == 1 || cost < least) least = cost, best = per;
    }
    return best;
}

// Splits that a call takes at least: an item's weights are resolved relative to the
// largest of them, and so many keys may share one (see swa_q8_tc.cuh).  Without rows
// that see more than that, any number will do.
int least_splits(long long span, long long item) {
    return item > swa::kQ8ItemKeys ? ceil_div(span, swa::kQ8ItemKeys) : 1;
}

// False where that kernel does not take the shape.
bool plan_direct(const swa_dims *d, int32_t window, int sms, Plan *out) {
    const int G = d->num_q_heads / d->num_kv_heads, D = d->head_dim;
    const int R = d->q_len * G;
    if (G > 32 ||
        (long long)d->batch * d->num_kv_heads * d->max_len >= (1LL << 31) ||
        (long long)d->batch * d->q_len * d->num_q_heads >= (1LL << 31) ||
        (long long)d->batch * d->num_kv_heads * d->q_len * kMaxSplits >= (1LL << 31))
        return false;
    Plan p;
    auto rows_of = [&](int r) {
        p.rows = r >= R ? R : (r < G ? G : r / G * G);
        p.q_rows = p.rows / G;
        p.row_tiles = ceil_div(d->q_len, p.q_rows);
    };
    rows_of(32);
    long long span = (long long)window + d->q_len - 1;
    if (span > d->max_len) span = d->max_len;
    long long item = (long long)window + p.q_rows - 1;  // keys of an item without a split
    if (item > span) item = span;
    const int least = least_splits(span, item);
    if (least > kMaxSplits) return false;
    const long long units = (long long)d->batch * d->num_kv_heads * p.row_tiles;
    long long chunk = span;
    if (d->num_splits > 0) {
        int n = d->num_splits < kMaxSplits ? d->num_splits : kMaxSplits;
        if (n < least) n = least;
        chunk = (span + n - 1) / n;
    } else {
        chunk = split_tiles(units, (item + kTileKeys - 1) / kTileKeys, sms) * kTileKeys;
        if (chunk >= item) chunk = span;
        if (least > 1 && chunk > swa::kQ8ItemKeys) chunk = swa::kQ8ItemKeys;
        if ((span + chunk - 1) / chunk > kMaxSplits) chunk = (span + kMaxSplits - 1) / kMaxSplits;
    }
    p.chunk = (int)chunk;
    p.splits = ceil_div(span, chunk);
    if (d->num_splits == 0) {
        // fewer rows per item while many SMs would stay idle: 8 while that gives up to
        // 2/5 of the SMs an item, 16 up to 3/5 (8 rows of 4 heads per KV head, head_dim
        // 256, window 188, 8 / 16 / 32 rows per item, us: 1 sequence 7.3 / 7.9 / 10.1, 6
        // 7.9 / 8.1 / 10.1, 12 10.1 / 8.2 / 10.3, 20 14.8 / 10.1 / 10.3, 48 16.2 / 13.2
        // / 12.3)
        const long long per_unit = (long long)d->batch * d->num_kv_heads * p.splits;
        for (int r : {8, 16}) {
            const int rows = r < G ? G : r / G * G;
            if (rows >= p.rows) break;
            const long long n = per_unit * ceil_div(d->q_len, rows / G);
            if (n * 5 <= (r == 8 ? 2LL : 3LL) * sms) {
                rows_of(r);
                break;
            }
        }
    }
    p.n = p.rows <= 16 ? 16 : 32;
    p.items = (long long)p.splits * d->batch * d->num_kv_heads * p.row_tiles;
    p.grid = (int)(p.items < sms ? p.items : sms);
    // (once every SM loads at once the first K tile should land first)
    p.early = p.grid * 2 >= sms ? 1 : 8;
    p.workspace = p.splits > 1 ? (size_t)d->batch * d->num_kv_heads * p.splits * R * (D + 2) * 4 : 0;
    *out = p;
    return true;
}

// Whether reading the windows in place is the faster way whatever the device.  An
// item's draft rows read their window for themselves; the other path reads and writes
// a sequence's window once, in bf16, whatever the number of rows, and its kernel takes
// more rows at a time.  So it is for one item per window, and for more of them where
// windows are long; heads of 64 always take it (the bf16 kernel for them has no tensor
// cores).  Measured, 8 query heads on 2, in place / over bf16 rows, us (in place with
// weights of 11 bits; of 14 it takes 1 to 3% more):
//   rows x sequences, items per window      window 188     600        1024      1900
//   8 x 512, 1        256                   41.5 / 107.5
//   16 x 512, 2       256                   89.6 / 118.7              230 / 481
//                     128                   82.4 / 76.8               211 / 280
//   24 x 64, 3        256                   21.4 / 19.4  32.5 / 42.3  47.8 / 70.6  71 / 121
//                     128                   20.4 / 15.0  31.2 / 24.0  44.0 / 37.8  66 / 70
//   32 x 48, 4        256                   21.3 / 18.7  33.9 / 33.9  47.0 / 59.7  70 / 103
//                     128                   20.4 / 15.1  31.4 / 22.6  44.4 / 33.5  65 / 61
//   64 x 24, 8        256                   21.5 / 18.5  33.0 / 28.2               70 / 78
//   128 x 12, 16      256                                33.0 / 26.5               69 / 61
//   32 x 64, 4        64                    24.5 / 106.6
bool in_place(const swa_dims *d, int32_t window, const Plan &p) {
    const long long all = (long long)window + d->q_len - 1;
    const long long span = all < d->max_len ? all : d->max_len;
    return d->head_dim == 64 ||
           span >= (d->head_dim == 256 ? 200LL : 800LL) * (p.row_tiles - 1);
}

// Whether a call runs on the fp8 tensor cores straight from the cache, unless a
// kernel is forced (2: that one; others: bf16 rows and that kernel over them).  While
// every SM has at most one item that is the faster way for any number of rows: one
// sequence of 512 rows, window 188, 256: 12.6 / 14.0, 128: 12.0 / 11.6; 8 of 64 rows
// 12.3 / 14.7, 12.2 / 12.6.
bool direct(const swa_dims *d, int32_t window, int sms, const swa_paged *paged, Plan *plan) {
    const int force = swa::api_forced_kernel();
    if (force != 0 && force != 2) return false;
    if (!plan_direct(d, window, sms, plan)) return false;
    // (rows of a cache tensor are counted in 32 bits there)
    if (paged != nullptr &&
        (long long)paged->num_pages * d->num_kv_heads * paged->page_size >= (1LL << 31))
        return false;
    return force == 2 || in_place(d, window, *plan) || plan->items <= sms;
}

swa_status attend_direct(const void *q, const swa_q8_cache *cache, const swa_paged *paged,
                         const int32_t *seq_lens, const int32_t *q_pos, int32_t window,
                         float scale, void *out, float *lse, const swa_dims *d,
                         const Plan &pl, int dev, uint32_t *fault, cudaStream_t s) {
    swa::Q8TcLaunch L{};
    swa::AttnParams &P = L.T.a;
    set_cache(P, paged, d, seq_lens, fault);
    P.q = static_cast<const __nv_bfloat16 *>(q);
    P.q_pos = q_pos;
    P.out = static_cast<__nv_bfloat16 *>(out);
    P.lse = lse;
    P.q_len = d->q_len;
    P.Hq = d->num_q_heads;
    P.G = d->num_q_heads / d->num_kv_heads;
    P.window = window;
    P.R = P.q_len * P.G;
    P.splits = pl.splits;
    P.chunk = pl.chunk;
    P.row_tiles = pl.row_tiles;
    P.rows_per_tile = pl.rows;
    P.qk_scale = scale * swa::kLog2e;
    P.wait_limit = swa::api_wait_limit();
    P.withhold_fill = swa::api_withhold_fill();
    if (pl.splits > 1) {
        void *ws = nullptr;
        const swa_status st = swa::api_workspace(dev, pl.workspace, s, &ws);
        if (st != SWA_OK) return st;
        P.part_acc = static_cast<float *>(ws);
        P.part_ml = P.part_acc + (size_t)P.B * P.Hkv * P.splits * P.R * d->head_dim;
    }
    L.T.rows_per_tile = pl.rows;
    L.T.q_rows_per_tile = pl.q_rows;
    L.T.items = (int)pl.items;
    L.T.items_per_cta = (int)(pl.items / pl.grid);
    L.T.items_extra = (int)(pl.items % pl.grid);
    L.T.early_max = pl.early;
    L.k_exp = cache->k_exp;
    L.v_exp = cache->v_exp;
    L.k = cache->k;
    L.v = cache->v;
    L.head_dim = d->head_dim;
    L.n = pl.n;
    L.grid = pl.grid;
    L.cache_rows = paged != nullptr
                       ? (long long)paged->num_pages * d->num_kv_heads * paged->page_size
                       : (long long)d->batch * d->num_kv_heads * d->max_len;
    char msg[256] = "";
    cudaError_t e = swa::q8_tc_launch(L, s, msg, sizeof msg);
    if (e != cudaSuccess)
        return msg[0] ? api_fail(SWA_ERR_CUDA, "%s", msg)
                      : swa::api_cuda_fail(e, "8-bit attention kernel launch");
    if (pl.splits > 1) {
        e = swa::api_merge(P, d->head_dim, /*nan_lse=*/true, s);
        if (e != cudaSuccess) return swa::api_cuda_fail(e, "merge kernel launch");
    }
    return swa::api_ok();
}

}  // namespace

extern "C" {

swa_status swa_q8_append(const void *k_new, const void *v_new, size_t k_row, size_t v_row,
                         const swa_q8_cache *cache, const swa_paged *paged,
                         const int32_t *seq_lens, const int32_t *q_pos, const swa_dims *dims,
                         swa_stream_t stream) {
    swa_status st = check_dims(dims, true);
    if (st != SWA_OK) return st;
    if (!k_new || !v_new || !seq_lens || !q_pos)
        return api_fail(SWA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned_to(k_new, 16) || !aligned_to(v_new, 16))
        return api_fail(SWA_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    if (!aligned_to(seq_lens, 4) || !aligned_to(q_pos, 4))
        return api_fail(SWA_ERR_INVALID_ARG, "seq_lens and q_pos must be 4-byte aligned");
    st = check_cache(cache, paged, dims);
    if (st != SWA_OK) return st;
    const size_t need = (size_t)dims->num_kv_heads * dims->head_dim;
    for (size_t row : {k_row, v_row})
        if (row < need || row % 8 != 0 || row > ((size_t)1 << 36))
            return api_fail(SWA_ERR_INVALID_ARG,
                            "token stride %zu elements is not a multiple of 8 of at least %zu", row,
                            need);
    int dev = 0;
    uint32_t *fault = nullptr;
    st = swa::api_device(&dev, &fault);
    if (st != SWA_OK) return st;
    swa::Q8AppendParams A{};
    A.src[0] = static_cast<const __nv_bfloat16 *>(k_new);
    A.src[1] = static_cast<const __nv_bfloat16 *>(v_new);
    A.row[0] = (long long)k_row;
    A.row[1] = (long long)v_row;
    A.dst[0] = static_cast<uint8_t *>(cache->k);
    A.dst[1] = static_cast<uint8_t *>(cache->v);
    A.exp[0] = cache->k_exp;
    A.exp[1] = cache->v_exp;
    set_cache(A.cache, paged, dims, seq_lens, fault);
    A.cache.q_pos = q_pos;
    A.cache.q_len = dims->q_len;
    const cudaError_t e = launch_append(A, dims->head_dim, swa::api_device_sms(dev),
                                        reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return swa::api_cuda_fail(e, "8-bit append kernel launch");
    return swa::api_ok();
}

swa_status swa_q8_read(const swa_q8_cache *cache, const swa_paged *paged, const int32_t *seq_lens,
                       const int32_t *start, int32_t n, void *k_out, void *v_out,
                       const swa_dims *dims, swa_stream_t stream) {
    swa_status st = check_dims(dims, false);
    if (st != SWA_OK) return st;
    if (n < 1) return api_fail(SWA_ERR_INVALID_ARG, "n %d < 1", n);
    if (!seq_lens || !start || !k_out || !v_out)
        return api_fail(SWA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned_to(k_out, 16) || !aligned_to(v_out, 16))
        return api_fail(SWA_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
    if (!aligned_to(seq_lens, 4) || !aligned_to(start, 4))
        return api_fail(SWA_ERR_INVALID_ARG, "seq_lens and start must be 4-byte aligned");
    st = check_cache(cache, paged, dims);
    if (st != SWA_OK) return st;
    int dev = 0;
    uint32_t *fault = nullptr;
    st = swa::api_device(&dev, &fault);
    if (st != SWA_OK) return st;
    swa::Q8ReadParams A{};
    A.src[0] = static_cast<const uint8_t *>(cache->k);
    A.src[1] = static_cast<const uint8_t *>(cache->v);
    A.exp[0] = cache->k_exp;
    A.exp[1] = cache->v_exp;
    A.dst[0] = static_cast<__nv_bfloat16 *>(k_out);
    A.dst[1] = static_cast<__nv_bfloat16 *>(v_out);
    set_cache(A.cache, paged, dims, seq_lens, fault);
    A.start = start;
    A.n = n;
    const cudaError_t e = launch_read(A, dims->head_dim, swa::api_device_sms(dev),
                                      reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return swa::api_cuda_fail(e, "8-bit read kernel launch");
    return swa::api_ok();
}

size_t swa_q8_workspace_bytes(const swa_dims *dims, int32_t window) {
    if (swa::api_check_dims(dims, window) != SWA_OK) return 0;
    Plan p;
    const bool can = plan_direct(dims, window, 1, &p);
    // (a plan may have more splits than were asked for)
    swa_dims d = *dims;
    if (can && d.num_splits > 0 && d.num_splits < p.splits) d.num_splits = p.splits;
    const size_t split = can ? swa_workspace_bytes(&d, window) : 0;
    if (can && in_place(dims, window, p)) return split;
    const RowsLayout l = rows_layout(dims, window);
    d = *dims;
    d.max_len = l.span;
    const size_t rows = l.parts + swa_workspace_bytes(&d, window);
    return rows > split ? rows : split;
}

swa_status swa_q8_verify_attn(const void *q, const swa_q8_cache *cache, const swa_paged *paged,
                              const int32_t *seq_lens, const int32_t *q_pos, int32_t window,
                              float scale, void *out, float *lse, const swa_dims *dims,
                              swa_stream_t stream) {
    swa_status st = swa::api_check_dims(dims, window);
    if (st != SWA_OK) return st;
    if (!q || !seq_lens || !q_pos || !out)
        return api_fail(SWA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned_to(q, 16) || !aligned_to(out, 16))
        return api_fail(SWA_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
    if (!aligned_to(seq_lens, 4) || !aligned_to(q_pos, 4) || !aligned_to(lse, 4))
        return api_fail(SWA_ERR_INVALID_ARG, "seq_lens, q_pos and lse must be 4-byte aligned");
    if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f)
        return api_fail(SWA_ERR_INVALID_ARG, "scale must be finite");
    st = check_cache(cache, paged, dims);
    if (st != SWA_OK) return st;
    int dev = 0;
    uint32_t *fault = nullptr;
    st = swa::api_device(&dev, &fault);
    if (st != SWA_OK) return st;

    Plan plan;
    if (direct(dims, window, swa::api_device_sms(dev), paged, &plan))
        return attend_direct(q, cache, paged, seq_lens, q_pos, window, scale, out, lse, dims, plan,
                             dev, fault, reinterpret_cast<cudaStream_t>(stream));

    const RowsLayout l = rows_layout(dims, window);
    swa_dims rd = *dims;
    rd.max_len = l.span;
    const size_t parts = swa::api_plan_bytes(&rd, window, dev);
    void *ws = nullptr;
    st = swa::api_workspace(dev, l.parts + parts, reinterpret_cast<cudaStream_t>(stream), &ws);
    if (st != SWA_OK) return st;
    uint8_t *w = static_cast<uint8_t *>(ws);
    swa::Q8ReadParams A{};
    A.src[0] = static_cast<const uint8_t *>(cache->k);
    A.src[1] = static_cast<const uint8_t *>(cache->v);
    A.exp[0] = cache->k_exp;
    A.exp[1] = cache->v_exp;
    A.dst[0] = reinterpret_cast<__nv_bfloat16 *>(w);
    A.dst[1] = reinterpret_cast<__nv_bfloat16 *>(w + l.v);
    set_cache(A.cache, paged, dims, seq_lens, fault);
    A.cache.q_pos = q_pos;
    A.cache.window = window;
    A.shifted = reinterpret_cast<int32_t *>(w + l.shifted);
    A.n = l.span;
    const cudaError_t e = launch_read(A, dims->head_dim, swa::api_device_sms(dev),
                                      reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return swa::api_cuda_fail(e, "8-bit window kernel launch");
    return swa::api_verify_rows(q, w, w + l.v, A.shifted, A.shifted + dims->batch, window, scale,
                                out, lse, &rd, w + l.parts, stream);
}

}  // extern "C"
