// Host side of the attention over the 8-bit cache on the fp8 tensor cores:
// tensor maps and the persistent launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>

#include "swa_host.h"
#include "swa_q8_host.h"
#include "swa_q8_tc.cuh"
#include "swa_tc_host.h"

namespace swa {
namespace {

template <int HD, int N>
cudaError_t launch(const Q8TcParams &A, const TcMaps &maps, int grid, cudaStream_t stream) {
    constexpr int D = HD < 128 ? 128 : HD;
    constexpr int NT = D == 256 ? 5 : 10;  // ring slots within 227 KB of shared memory
    using C = Q8Cfg<D, N, NT>;
    auto kern = swa_q8_tc_kernel<HD, N, NT>;
    static std::atomic<bool> attr_done[kMaxDevices];
    const cudaError_t e = raise_smem_limit(kern, C::SMEM_BYTES, attr_done);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(grid), dim3(kQ8TcThreads), C::SMEM_BYTES, stream, A, maps);
}

template <int D>
cudaError_t launch_n(const Q8TcParams &A, const TcMaps &maps, int n, int grid, cudaStream_t s) {
    switch (n) {
        case 16: return launch<D, 16>(A, maps, grid, s);
        case 32: return launch<D, 32>(A, maps, grid, s);
        default: return cudaErrorInvalidConfiguration;
    }
}

}  // namespace

cudaError_t q8_tc_launch(const Q8TcLaunch &L, cudaStream_t stream, char *err, size_t errlen) {
    const auto encode = tc_encode();
    if (encode == nullptr) {
        snprintf(err, errlen, "cuTensorMapEncodeTiled is not available from the driver");
        return cudaErrorNotSupported;
    }
    const int D = L.head_dim;
    // the cache as rows of D bytes: maps as for the bf16 cache, with 128-byte
    // slabs of 128 elements; of rows of 64 the box's other half is past the end, which
    // fills it with zeros
    TcMaps maps{};
    const cuuint64_t rows = (cuuint64_t)L.cache_rows;
    const cuuint32_t slabs = D == 256 ? 2 : 1;
    for (int kv = 0; kv < 2; ++kv) {
        CUtensorMap *m4 = kv ? maps.v_atoms : maps.k_atoms;
        for (int bi = 0; bi < 5; ++bi) {
            const bool atom = bi == 4;
            const cuuint32_t boxes = atom ? 1u : (16u >> bi);
            cuuint64_t dims[4] = {(cuuint64_t)(D < 128 ? D : 128), rows, slabs, 16};
            cuuint64_t strides[3] = {(cuuint64_t)D, 128, (cuuint64_t)D * 8};
            cuuint32_t box[4] = {128, 8, slabs, boxes};
            cuuint32_t es[4] = {1, 1, 1, 1};
            const CUresult r =
                encode(atom ? (kv ? &maps.v_atom : &maps.k_atom) : &m4[bi],
                       CU_TENSOR_MAP_DATA_TYPE_UINT8, atom ? 3 : 4,
                       const_cast<void *>(kv ? L.v : L.k), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            if (r != CUDA_SUCCESS) {
                snprintf(err, errlen, "cuTensorMapEncodeTiled(8-bit %s cache, %u-atom box) failed: %d",
                         kv ? "V" : "K", (unsigned)boxes, (int)r);
                return cudaErrorInvalidValue;
            }
        }
    }
    const Q8TcParams A{L.T, L.k_exp, L.v_exp};
    return D == 256   ? launch_n<256>(A, maps, L.n, L.grid, stream)
           : D == 128 ? launch_n<128>(A, maps, L.n, L.grid, stream)
                      : launch_n<64>(A, maps, L.n, L.grid, stream);
}

}  // namespace swa
