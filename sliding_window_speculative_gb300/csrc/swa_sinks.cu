// The attention kernels' sink variants: the first positions of a sequence stay
// visible behind the window (swa_sink_verify_attn).
#include <cuda_runtime.h>

#include "swa_simt_launch.cuh"
#include "swa_tc_launch.cuh"

cudaError_t swa::tc_launch_sinks(const TcLaunch &L, const TcMaps &maps, cudaStream_t stream) {
    return launch_kernels<true>(L, maps, stream);
}

cudaError_t swa::simt_launch_sinks(const AttnParams &P, int D, int rpw, int nrg,
                                   cudaStream_t stream) {
    return launch_simt_kernel<true>(P, D, rpw, nrg, stream);
}
