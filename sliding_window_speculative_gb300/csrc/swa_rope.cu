// Entry points of the head norm + rotation kernel: argument checks and launch.
#include <cuda_runtime.h>

#include "../../include/swa.h"
#include "swa_host.h"
#include "swa_rope.cuh"
#include "swa_tc_host.h"

namespace {

using swa::aligned_to;
using swa::api_fail;

swa_status check(const void *q, const void *k, const void *v, const swa_rope *r,
                 const int32_t *q_pos, const void *q_out, const swa_dims *d) {
    if (d == nullptr) return api_fail(SWA_ERR_INVALID_ARG, "dims is NULL");
    if (r == nullptr) return api_fail(SWA_ERR_INVALID_ARG, "rope is NULL");
    if (d->batch < 1 || d->batch > 65535)
        return api_fail(SWA_ERR_INVALID_ARG, "batch %d outside [1, 65535]", d->batch);
    if (d->q_len < 1 || d->q_len > swa::kMaxBlockLen)
        return api_fail(SWA_ERR_INVALID_ARG, "q_len %d outside [1, %d]", d->q_len,
                        swa::kMaxBlockLen);
    if (d->num_q_heads < 1 || d->num_kv_heads < 1 || d->num_q_heads % d->num_kv_heads != 0 ||
        d->num_q_heads > 65535)
        return api_fail(SWA_ERR_INVALID_ARG, "head counts Hq %d, Hkv %d: Hkv >= 1 must divide Hq "
                        "<= 65535", d->num_q_heads, d->num_kv_heads);
    const int D = d->head_dim;
    if (D != 64 && D != 128 && D != 256)
        return api_fail(SWA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", D);
    if (r->rot_dim < 0 || r->rot_dim > D || r->rot_dim % 16 != 0)
        return api_fail(SWA_ERR_INVALID_ARG, "rot_dim %d is not a multiple of 16 in [0, %d]",
                        r->rot_dim, D);
    if (r->interleaved != 0 && r->interleaved != 1)
        return api_fail(SWA_ERR_INVALID_ARG, "interleaved %d is not 0 or 1", r->interleaved);
    if (!q || !k || !v || !q_pos || !q_out || (r->rot_dim > 0 && !r->inv_freq))
        return api_fail(SWA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(q_out, 16) ||
        !aligned_to(r->q_weight, 16) || !aligned_to(r->k_weight, 16))
        return api_fail(SWA_ERR_INVALID_ARG, "q, k, v, q_out and the weights must be 16-byte "
                        "aligned");
    if (!aligned_to(q_pos, 4) || !aligned_to(r->inv_freq, 4))
        return api_fail(SWA_ERR_INVALID_ARG, "q_pos and inv_freq must be 4-byte aligned");
    if ((r->q_weight || r->k_weight) && !(r->eps > 0.f && r->eps < 3.0e38f))
        return api_fail(SWA_ERR_INVALID_ARG, "eps must be positive and finite");
    const int64_t rows[3] = {r->q_row, r->k_row, r->v_row};
    for (int t = 0; t < 3; ++t) {
        const int64_t need = (int64_t)(t == 0 ? d->num_q_heads : d->num_kv_heads) * D;
        if (rows[t] < need || rows[t] % 8 != 0 || rows[t] > ((int64_t)1 << 36))
            return api_fail(SWA_ERR_INVALID_ARG, "%s: token stride %lld elements is not a multiple "
                            "of 8 of at least %lld", t == 0 ? "q" : t == 1 ? "k" : "v",
                            (long long)rows[t], (long long)need);
    }
    return SWA_OK;
}

template <int D>
cudaError_t launch(swa::RopeParams &R, int sms, cudaStream_t s) {
    constexpr int kWarps = swa::kRopeThreads / 32;
    const int steps = (R.Hq + 2 * R.Hkv + 512 / D - 1) / (512 / D);  // warp steps per token
    // one warp per token; a token's heads go to several warps while the launch
    // would leave SMs with fewer than four (measured on GB300, 64 x 8 tokens
    // into pages, us, 2 / 4 / 8 / 16 warps: 6.2 / 6.0 / 6.2 / 7.7)
    const long long want = 4LL * sms;
    long long parts = R.tokens < want ? (want + R.tokens - 1) / R.tokens : 1;
    R.parts = (int)(parts < steps ? parts : steps);
    long long blocks = ((long long)R.tokens * R.parts + kWarps - 1) / kWarps;
    const long long cap = (long long)swa::kRopeBlocksPerSm * sms;
    if (blocks > cap) blocks = cap;
    return swa::launch_kernel(swa::swa_rope_kernel<D>, dim3((unsigned)blocks),
                              dim3(swa::kRopeThreads), 0, s, R);
}

swa_status run(const void *q, const void *k, const void *v, const swa_rope *r,
               const int32_t *q_pos, void *q_out, const swa_dims *d, swa::RopeParams &R,
               swa_stream_t stream) {
    int dev = 0;
    uint32_t *fault = nullptr;
    const swa_status st = swa::api_device(&dev, &fault);
    if (st != SWA_OK) return st;
    R.q = static_cast<const __nv_bfloat16 *>(q);
    R.k = static_cast<const __nv_bfloat16 *>(k);
    R.v = static_cast<const __nv_bfloat16 *>(v);
    R.q_row = r->q_row;
    R.k_row = r->k_row;
    R.v_row = r->v_row;
    R.q_weight = r->q_weight;
    R.k_weight = r->k_weight;
    R.inv_freq = r->inv_freq;
    R.q_pos = q_pos;
    R.q_out = static_cast<__nv_bfloat16 *>(q_out);
    R.cache.fault = fault;
    R.cache.B = d->batch;
    R.cache.q_len = d->q_len;
    R.cache.Hkv = d->num_kv_heads;
    R.tokens = d->batch * d->q_len;
    R.Hq = d->num_q_heads;
    R.Hkv = d->num_kv_heads;
    R.rot = r->rot_dim;
    R.interleaved = r->interleaved;
    R.eps = r->eps;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int sms = swa::api_device_sms(dev);
    const cudaError_t e = d->head_dim == 64    ? launch<64>(R, sms, s)
                          : d->head_dim == 128 ? launch<128>(R, sms, s)
                                               : launch<256>(R, sms, s);
    if (e != cudaSuccess) return swa::api_cuda_fail(e, "head norm and rotation kernel launch");
    return swa::api_ok();
}

}  // namespace

extern "C" {

swa_status swa_qk_norm_rope(const void *q, const void *k, const void *v, const swa_rope *rope,
                            const int32_t *q_pos, void *q_out, void *k_out, void *v_out,
                            const swa_dims *dims, swa_stream_t stream) {
    const swa_status st = check(q, k, v, rope, q_pos, q_out, dims);
    if (st != SWA_OK) return st;
    if (!k_out || !v_out) return api_fail(SWA_ERR_INVALID_ARG, "k_out and v_out must not be NULL");
    if (!aligned_to(k_out, 16) || !aligned_to(v_out, 16))
        return api_fail(SWA_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
    swa::RopeParams R{};
    R.k_out = static_cast<__nv_bfloat16 *>(k_out);
    R.v_out = static_cast<__nv_bfloat16 *>(v_out);
    return run(q, k, v, rope, q_pos, q_out, dims, R, stream);
}

swa_status swa_qk_norm_rope_append(const void *q, const void *k, const void *v,
                                   const swa_rope *rope, void *k_cache, void *v_cache,
                                   const swa_paged *paged, const int32_t *seq_lens,
                                   const int32_t *q_pos, void *q_out, const swa_dims *dims,
                                   swa_stream_t stream) {
    swa_status st = check(q, k, v, rope, q_pos, q_out, dims);
    if (st != SWA_OK) return st;
    if (dims->max_len < 1)
        return api_fail(SWA_ERR_INVALID_ARG, "max_len %d < 1", dims->max_len);
    if (!k_cache || !v_cache || !seq_lens)
        return api_fail(SWA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16))
        return api_fail(SWA_ERR_INVALID_ARG, "the K and V caches must be 16-byte aligned");
    if (!aligned_to(seq_lens, 4))
        return api_fail(SWA_ERR_INVALID_ARG, "seq_lens must be 4-byte aligned");
    swa::RopeParams R{};
    if (paged != nullptr) {
        st = swa::api_check_paged(paged, dims);
        if (st != SWA_OK) return st;
        R.cache.block_table = paged->block_table;
        R.cache.page_size = paged->page_size;
        R.cache.max_blocks = paged->max_blocks;
        R.cache.num_pages = paged->num_pages;
    }
    R.k_out = static_cast<__nv_bfloat16 *>(k_cache);
    R.v_out = static_cast<__nv_bfloat16 *>(v_cache);
    R.cache.seq_lens = seq_lens;
    R.cache.L = dims->max_len;
    R.to_cache = 1;
    return run(q, k, v, rope, q_pos, q_out, dims, R, stream);
}

}  // extern "C"
