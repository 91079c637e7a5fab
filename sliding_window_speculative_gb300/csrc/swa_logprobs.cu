// Entry point of the token log probabilities: argument checks and launch.
#include <cuda_runtime.h>

#include "../../include/swa.h"
#include "swa_host.h"
#include "swa_logprobs.cuh"
#include "swa_tc_host.h"

using swa::aligned_to;
using swa::api_fail;

namespace {

template <int NT, bool TOP>
cudaError_t launch_as(const swa::LogpParams &A, long long rows, int c, cudaStream_t s) {
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
    return cudaLaunchKernelEx(&cfg, swa::swa_logprobs_kernel<NT, TOP>, A,
                              c == 8 ? 3 : c >> 1);
}

template <int NT>
cudaError_t launch(const swa::LogpParams &A, long long rows, int c, cudaStream_t s) {
    return A.top > 0 ? launch_as<NT, true>(A, rows, c, s) : launch_as<NT, false>(A, rows, c, s);
}

cudaError_t launch_rows(const swa::LogpParams &A, long long rows, int sms, cudaStream_t s) {
    // One CTA per row, four to an SM; clusters of up to four share a row while that
    // leaves at most three CTAs to an SM and each CTA over 1024 vectors (four per
    // thread), of eight while that leaves at most three CTAs to two SMs.  The eight have
    // 512 threads where every thread has eight vectors and half the SMs stay without a
    // CTA: with fewer vectors a row's loads are no longer four at a time.  Many rows that
    // are not long get CTAs of 128 threads: the steps behind the pass are a larger share
    // of theirs.  Measured on GB300, calls behind one another in a replayed graph, us
    // (rows x columns, alternatives):
    //   64 x 262144, 5     4 of 256 13.9, 2 of 512 14.6, 8 of 256 17.2, 1 of 512 21.2
    //   200 x 262144, 5    4 of 256 34.9, 2 of 256 36.4, 1 of 512 35.0, 1 of 256 43.0
    //   512 x 262144, 20   1 of 256 65.7, 1 of 512 70.7, 2 of 128 70.9, 2 of 256 75.0
    //   512 x 50257, 5     1 of 128 19.3, 1 of 256 21.3, 1 of 512 26.7
    //   240 x 12001, 20    1 of 256 7.7, 1 of 128 9.4, 1 of 512 9.7
    //   100 x 32000, 5     2 of 256 9.2, 4 of 256 11.3, 1 of 256 10.2
    //   4000 x 1000, 5     1 of 128 24.3, 1 of 256 43.0
    //   40880 x 3120, 0    1 of 128 153, 1 of 256 232, 1 of 32 157
    //   20000 x 12001, 0   1 of 128 136, 1 of 256 177, 1 of 32 224
    //   400 x 1000, 0      1 of 128 2.6, 1 of 256 3.5
    // and with other logits from one call to the next, so that they come from memory:
    //   8 x 262144, 5      8 of 512 10.5, 8 of 256 11.3, 4 of 512 13.1, 2 of 512 15.8
    //   16 x 262144, 5     8 of 256 12.6, 8 of 512 13.0, 4 of 512 13.8, 4 of 256 14.7
    //   8 x 100352, 5      8 of 256 8.3, 8 of 512 9.2, 4 of 256 9.3, 2 of 512 11.0
    //   28 x 100352, 5     8 of 256 10.8, 4 of 256 10.9, 8 of 512 13.4, 2 of 512 12.4
    //   28 x 262144, 5     8 of 256 13.5, 4 of 512 14.2, 8 of 512 15.0, 4 of 256 15.0
    //   57 x 100352, 5     4 of 256 11.9, 2 of 512 12.8, 8 of 256 14.2, 8 of 512 24.4
    //   40 x 66000, 0      4 of 256 6.4, 2 of 512 6.8, 4 of 512 6.9, 8 of 512 14.2
    const long long nvec = ((long long)A.V + 14) / 8;
    int c = 1;
    while (c < swa::kLogpMaxCluster && rows * c * 2 <= (c == 4 ? 3LL * sms / 2 : 3LL * sms) &&
           nvec > 2048LL * c)
        c *= 2;
    if (c == swa::kLogpMaxCluster && rows * c * 2 <= sms && nvec >= 4096LL * c)
        return launch<512>(A, rows, c, s);
    if (c == 1 && rows > (A.top > 0 ? 3LL : 2LL) * sms && nvec <= 8192) return launch<128>(A, rows, c, s);
    return launch<256>(A, rows, c, s);
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
