// Entry point of the token log probabilities: argument checks and launch.
#include <cuda_runtime.h>

#include "../../include/swa.h"
#include "swa_host.h"
#include "swa_logprobs.cuh"
#include "swa_tc_host.h"

using swa::aligned_to;
using swa::api_fail;

namespace {

template <int NT>
cudaError_t launch(const swa::LogpParams &A, long long rows, int c, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * c));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = swa::pdl_enabled() ? 2 : 1;
    if (swa::launch_fault_due()) return cudaErrorLaunchOutOfResources;
    return cudaLaunchKernelEx(&cfg, swa::swa_logprobs_kernel<NT>, A, c);
}

cudaError_t launch_rows(const swa::LogpParams &A, long long rows, int sms, cudaStream_t s) {
    const long long nvec = ((long long)A.V + 14) / 8;
    int c = 1;
    while (c < swa::kLogpMaxCluster && rows * c * 2 <= 2LL * sms && nvec > 1024LL * c) c *= 2;
    return c >= 8 ? launch<512>(A, rows, c, s) : launch<256>(A, rows, c, s);
}

}  // namespace

extern "C" swa_status swa_token_logprobs(const void *logits, const int32_t *keep_ids,
                                         const int32_t *tokens, const float *temperature,
                                         int32_t top_n, float *logprobs, int32_t *ranks,
                                         float *entropy, int32_t *top_tokens, float *top_logprobs,
                                         int32_t batch, int32_t q_len, int32_t vocab,
                                         swa_stream_t stream) {
    if (batch < 1 || batch > 65535)
        return api_fail(SWA_ERR_INVALID_ARG, "batch %d outside [1, 65535]", batch);
    if (q_len < 1 || q_len > swa::kMaxBlockLen)
        return api_fail(SWA_ERR_INVALID_ARG, "q_len %d outside [1, %d]", q_len, swa::kMaxBlockLen);
    if (vocab < 1) return api_fail(SWA_ERR_INVALID_ARG, "vocab %d < 1", vocab);
    if (top_n < 0 || top_n > swa::kLogpMaxTop || top_n > vocab)
        return api_fail(SWA_ERR_INVALID_ARG, "top_n %d outside [0, %d] or above vocab %d", top_n,
                        swa::kLogpMaxTop, vocab);
    if (!logits || !tokens || !logprobs || (top_n > 0 && (!top_tokens || !top_logprobs)))
        return api_fail(SWA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned_to(logits, 2))
        return api_fail(SWA_ERR_INVALID_ARG, "logits must be 2-byte aligned");
    const void *words[] = {keep_ids, tokens, temperature, logprobs, ranks, entropy, top_tokens,
                           top_logprobs};
    for (const void *p : words)
        if (!aligned_to(p, 4))
            return api_fail(SWA_ERR_INVALID_ARG, "the int32 and fp32 arrays must be 4-byte aligned");
    int dev = 0;
    uint32_t *fault = nullptr;
    const swa_status st = swa::api_device(&dev, &fault);
    if (st != SWA_OK) return st;
    swa::LogpParams A{};
    A.logits = static_cast<const uint16_t *>(logits);
    A.keep = keep_ids;
    A.tokens = tokens;
    A.temperature = temperature;
    A.logprobs = logprobs;
    A.ranks = ranks;
    A.entropy = entropy;
    A.top_tokens = top_tokens;
    A.top_logprobs = top_logprobs;
    A.q_len = q_len;
    A.V = vocab;
    A.top = top_n;
    const cudaError_t e = launch_rows(A, (long long)batch * q_len, swa::api_device_sms(dev),
                                      reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return swa::api_cuda_fail(e, "log probability kernel launch");
    return swa::api_ok();
}
