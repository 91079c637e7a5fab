// Launches of the CUDA-core kernel, for the translation unit of each variant
// (SK: the first positions stay visible as sinks).
#pragma once

#include "swa_host.h"
#include "swa_simt.cuh"
#include "swa_tc_host.h"

namespace swa {
namespace {

template <int D, int RPW, int NRG, bool AP, bool SK>
cudaError_t launch_simt_ap(const AttnParams &P, cudaStream_t stream) {
    using C = SimtCfg<D, RPW, NRG>;
    auto kern = swa_simt_kernel<D, RPW, NRG, AP, SK>;
    static std::atomic<bool> attr_done[kMaxDevices];
    cudaError_t e = raise_smem_limit(kern, C::SMEM_BYTES, attr_done);
    if (e != cudaSuccess) return e;
    dim3 grid(P.splits, P.Hkv * P.row_tiles, P.B);
    return launch_kernel(kern, grid, dim3(kSimtThreads), C::SMEM_BYTES, stream, P);
}

// The plain kernel, or (fused append) its variant.
template <int D, int RPW, int NRG, bool SK>
cudaError_t launch_simt(const AttnParams &P, cudaStream_t stream) {
    return P.k_new != nullptr ? launch_simt_ap<D, RPW, NRG, true, SK>(P, stream)
                              : launch_simt_ap<D, RPW, NRG, false, SK>(P, stream);
}

template <int D, bool SK>
cudaError_t launch_simt_d(const AttnParams &P, int rpw, int nrg, cudaStream_t s) {
    if (rpw == 4) return launch_simt<D, 4, 1, SK>(P, s);
    if (nrg == 1) return launch_simt<D, 8, 1, SK>(P, s);
    if (nrg == 2) return launch_simt<D, 8, 2, SK>(P, s);
    return launch_simt<D, 8, 4, SK>(P, s);
}

// `rpw` rows per warp and `nrg` row groups, as the plan lays the rows out.
template <bool SK>
cudaError_t launch_simt_kernel(const AttnParams &P, int D, int rpw, int nrg, cudaStream_t s) {
    return D == 64    ? launch_simt_d<64, SK>(P, rpw, nrg, s)
           : D == 128 ? launch_simt_d<128, SK>(P, rpw, nrg, s)
                      : launch_simt_d<256, SK>(P, rpw, nrg, s);
}

}  // namespace
}  // namespace swa
