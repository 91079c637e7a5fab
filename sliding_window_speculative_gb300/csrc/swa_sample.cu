// Entry point of the sampled verification: argument checks and launches.
#include <cuda_runtime.h>

#include "../../include/swa.h"
#include "swa_host.h"
#include "swa_sample.cuh"
#include "swa_tc_host.h"

namespace {

using swa::aligned_to;
using swa::api_fail;

constexpr int kMaxQLen = 64;  // SPLITKV_VERIFY_MAX_Q: draft rows of a verification

template <int C, int NT, bool HOLD>
cudaError_t launch(const swa::SampleParams &A, long long rows, cudaStream_t s) {
    static std::atomic<bool> attr_done[swa::kMaxDevices];
    const cudaError_t e = swa::raise_smem_limit(swa::swa_sample_kernel<C, NT, HOLD>,
                                                (int)sizeof(swa::SampShared), attr_done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.dynamicSmemBytes = sizeof(swa::SampShared);
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = swa::pdl_enabled() ? 2 : 1;
    if (swa::launch_fault_due()) return cudaErrorLaunchOutOfResources;
    return cudaLaunchKernelEx(&cfg, swa::swa_sample_kernel<C, NT, HOLD>, A);
}

cudaError_t launch_rows(const swa::SampleParams &A, long long rows, int sms, cudaStream_t s) {
    // One CTA per row, four to an SM; clusters share a row while SMs would be
    // left without two CTAs and each still has two vectors per thread.  Measured
    // on GB300, calls behind one another in a replayed graph, rows of 262144,
    // us, unfiltered / top-k 50:
    //   8 rows    8 CTAs of 512 threads, first chunk held in registers 16.3 / 8.7,
    //             read again 17.6 / 9.4, 8 of 256 17.7 / 11.9, 4 of 512 20.7 / 12.3
    //   64 rows   4 of 256 27.6 / 18.3, 4 of 512 30.6 / 17.7, 2 of 512 29.4 / 18.1,
    //             8 of 256 32.3 / 18.8
    //   128 rows  2 of 512 44.4 / 23.7, 2 of 256 43.7 / 27.0, 4 of 256 41.9 / 24.3,
    //             1 of 256 53.1 / 38.8
    //   512 rows  1 of 256 120.6 / 63.1, 1 of 512 122.9 / 64.6, 2 of 256
    //             124.7 / 69.3, 2 of 512 135.2 / 79.5; at most three CTAs of 256 to
    //             an SM 145.5 / 90.5
    // and shorter rows: 48 of 12001 2 of 512 18.6 / 8.5, 1 of 256 19.7 / 7.2, 4 of
    // 256 18.7 / 9.0; 100 of 12001 2 of 512 22.5 / 10.4, 1 of 256 20.1 / 7.2; 100
    // of 50257 2 of 512 26.8 / 12.3, 2 of 256 25.6 / 13.5, 1 of 256 29.3 / 15.6;
    // 30 of 32000 4 of 256 18.3 / 8.7, 8 of 512 20.3 / 10.9, 2 of 512 19.2 / 8.6.
    const long long nvec = ((long long)A.V + 14) / 8;
    int c = 1;
    while (c < swa::kSampMaxCluster && rows * c * 2 <= 2LL * sms && nvec > 1024LL * c) c *= 2;
    switch (c) {
        case 1: return launch<1, 256, false>(A, rows, s);
        case 2: return launch<2, 512, false>(A, rows, s);
        case 4: return launch<4, 256, false>(A, rows, s);
        default:
            return rows * c <= sms ? launch<8, 512, true>(A, rows, s)
                                   : launch<8, 512, false>(A, rows, s);
    }
}

}  // namespace

extern "C" swa_status swa_sample_accept(const void *logits, const int32_t *keep_ids,
                                        const int32_t *draft, const float *uniforms,
                                        const swa_sampling *sampling, int32_t *tokens,
                                        float *logprobs, int32_t *accepted, int32_t batch,
                                        int32_t q_len, int32_t vocab, swa_stream_t stream) {
    if (batch < 1 || batch > 65535)
        return api_fail(SWA_ERR_INVALID_ARG, "batch %d outside [1, 65535]", batch);
    if (q_len < 1 || q_len > kMaxQLen)
        return api_fail(SWA_ERR_INVALID_ARG, "q_len %d outside [1, %d]", q_len, kMaxQLen);
    if (vocab < 1) return api_fail(SWA_ERR_INVALID_ARG, "vocab %d < 1", vocab);
    if (!logits || !uniforms || !sampling || !sampling->temperature || !tokens || !accepted ||
        (q_len > 1 && !draft))
        return api_fail(SWA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned_to(logits, 2))
        return api_fail(SWA_ERR_INVALID_ARG, "logits must be 2-byte aligned");
    const void *words[] = {keep_ids, draft, uniforms, sampling->temperature, sampling->top_k,
                           sampling->top_p, sampling->min_p, tokens, logprobs, accepted};
    for (const void *p : words)
        if (!aligned_to(p, 4))
            return api_fail(SWA_ERR_INVALID_ARG, "the int32 and fp32 arrays must be 4-byte aligned");
    int dev = 0;
    uint32_t *fault = nullptr;
    const swa_status st = swa::api_device(&dev, &fault);
    if (st != SWA_OK) return st;
    swa::SampleParams A{};
    A.logits = static_cast<const uint16_t *>(logits);
    A.keep = keep_ids;
    A.uniforms = uniforms;
    A.temperature = sampling->temperature;
    A.top_k = sampling->top_k;
    A.top_p = sampling->top_p;
    A.min_p = sampling->min_p;
    A.tokens = tokens;
    A.logprobs = logprobs;
    A.accepted = accepted;
    A.q_len = q_len;
    A.V = vocab;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_rows(A, (long long)batch * q_len, swa::api_device_sms(dev), s);
    if (e != cudaSuccess) return swa::api_cuda_fail(e, "sampling kernel launch");
    if (q_len > 1) {
        constexpr int kSeqs = swa::kPrefixThreads / 32;
        e = swa::launch_kernel(swa::swa_prefix_kernel, dim3((unsigned)((batch + kSeqs - 1) / kSeqs)),
                               dim3(swa::kPrefixThreads), 0, s, (const int32_t *)tokens, draft,
                               accepted, batch, q_len);
        if (e != cudaSuccess) return swa::api_cuda_fail(e, "accepted prefix kernel launch");
    }
    return swa::api_ok();
}
