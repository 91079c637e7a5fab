// Host side of the tensor-core path: per-configuration constants, TMA tensor
// maps for the cache and the queries, and the persistent launch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <mutex>

#include "swa_pair.cuh"
#include "swa_rows.cuh"
#include "swa_tc.cuh"
#include "swa_tc_host.h"
#include "swa_tc_launch.cuh"

namespace swa {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool load_encode() {
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// CTA-pair kernel: clusters of two CTAs, as many pairs as the plan's grid
// holds and the device runs at once (queried once per device).
template <int D>
cudaError_t launch_pairs(const TcLaunch &L, const TcMaps &maps, const PairMaps &pm,
                         cudaStream_t stream) {
    using C = PairCfg<D, kPairSlots>;
    auto kern = swa_pair_kernel<D, kPairSlots>;
    static std::atomic<bool> attr_done[64];
    static std::atomic<int> max_pairs[64];
    cudaError_t e = raise_smem_limit(kern, C::SMEM_BYTES, attr_done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int fit = dev >= 0 && dev < 64 ? max_pairs[dev].load(std::memory_order_acquire) : 0;
    if (fit == 0) {
        cfg.gridDim = dim3((unsigned)L.grid);
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (fit < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 64) max_pairs[dev].store(fit, std::memory_order_release);
    }
    const int pairs = L.grid / 2 < fit ? L.grid / 2 : fit;
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    if (launch_fault_due()) return cudaErrorLaunchOutOfResources;
    return cudaLaunchKernelEx(&cfg, kern, L.T, maps, pm);
}

template <int D, int N>
void conf_info(TcConfInfo *c) {
    using C = typename Conf<D, N>::C;
    c->nslot = Conf<D, N>::NT;
    c->smem_bytes = C::SMEM_BYTES;
    c->tmem_cols = C::TMEM_COLS;
    c->ctas_per_sm = 1;  // persistent: one CTA per SM
}

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 tc_encode() { return load_encode() ? g_encode : nullptr; }

bool tc_conf(int D, int N, TcConfInfo *c) {
    if (D == 256) {
        switch (N) {
            case 16: conf_info<256, 16>(c); return true;
            case 32: conf_info<256, 32>(c); return true;
            case 64: conf_info<256, 64>(c); return true;
        }
    } else if (D == 128) {
        switch (N) {
            case 16: conf_info<128, 16>(c); return true;
            case 32: conf_info<128, 32>(c); return true;
            case 64: conf_info<128, 64>(c); return true;
        }
    }
    return false;
}

cudaError_t tc_launch(const TcLaunch &L, cudaStream_t stream, char *err, size_t errlen) {
    if (!load_encode()) {
        snprintf(err, errlen, "cuTensorMapEncodeTiled is not available from the driver");
        return cudaErrorNotSupported;
    }
    const AttnParams &P = L.T.a;
    const int D = L.D;
    // K and V cache viewed as rows of D bf16 (B * Hkv * L rows, or every
    // page's rows of a paged cache).  4D maps
    // (x = 64 dims, y = row, z = 64-dim slab, w = 8-row atom; strides D*2,
    // 128 and 8*D*2 bytes) with boxes of 16, 8, 4 and 2 atoms, and a 3D
    // one-atom map (x, y, z) whose rows are bounds-checked one by one.
    // Both land as [atom][slab][8 rows][128 bytes], 128-byte swizzled.
    TcMaps maps{};
    const cuuint64_t rows = (cuuint64_t)L.cache_rows;
    const cuuint32_t slabs = (cuuint32_t)(D / 64);
    for (int kv = 0; kv < 2; ++kv) {
        const void *base = kv ? L.v : L.k;
        CUtensorMap *m4 = kv ? maps.v_atoms : maps.k_atoms;
        for (int bi = 0; bi < 5; ++bi) {
            const bool atom = bi == 4;
            const cuuint32_t A = atom ? 1u : (16u >> bi);
            cuuint64_t dims[4] = {64, rows, slabs, 16};
            cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 2 * 8};
            cuuint32_t box[4] = {64, 8, slabs, A};
            cuuint32_t es[4] = {1, 1, 1, 1};
            CUresult r = g_encode(atom ? (kv ? &maps.v_atom : &maps.k_atom) : &m4[bi],
                                  CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, atom ? 3 : 4,
                                  const_cast<void *>(base), dims, strides, box, es,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            if (r != CUDA_SUCCESS) {
                snprintf(err, errlen, "cuTensorMapEncodeTiled(%s cache, %u-atom box) failed: %d",
                         kv ? "V" : "K", (unsigned)A, (int)r);
                return cudaErrorInvalidValue;
            }
        }
    }
    {
        cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)P.Hq, (cuuint64_t)P.B * P.q_len};
        cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)P.Hq * D * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)P.G, (cuuint32_t)L.T.q_rows_per_tile};
        cuuint32_t es[3] = {1, 1, 1};
        CUresult r = g_encode(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                              const_cast<void *>(L.q), dims, strides, box, es,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) {
            snprintf(err, errlen, "cuTensorMapEncodeTiled(q) failed: %d", (int)r);
            return cudaErrorInvalidValue;
        }
    }
    if (P.k_new != nullptr) {
        for (int kv = 0; kv < 2; ++kv) {
            cuuint64_t dims[5] = {64, (cuuint64_t)P.q_len, slabs, (cuuint64_t)P.Hkv,
                                  (cuuint64_t)P.B};
            cuuint64_t strides[4] = {(cuuint64_t)P.Hkv * D * 2, 128, (cuuint64_t)D * 2,
                                     (cuuint64_t)P.q_len * P.Hkv * D * 2};
            cuuint32_t box[5] = {64, 8, slabs, 1, 1};
            cuuint32_t es[5] = {1, 1, 1, 1, 1};
            CUresult r = g_encode(kv ? &maps.vn_atom : &maps.kn_atom,
                                  CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                                  const_cast<__nv_bfloat16 *>(kv ? P.v_new : P.k_new), dims,
                                  strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            if (r != CUDA_SUCCESS) {
                snprintf(err, errlen, "cuTensorMapEncodeTiled(%s new rows) failed: %d",
                         kv ? "V" : "K", (int)r);
                return cudaErrorInvalidValue;
            }
        }
    }
    if (L.pairs) {
        // V as D / 2 head dims per CTA: boxes of half the slabs, otherwise as
        // the full maps above
        if (D != 256 || L.grid < 2) return cudaErrorInvalidConfiguration;
        PairMaps pm{};
        for (int bi = 0; bi < 5; ++bi) {
            const bool atom = bi == 4;
            const cuuint32_t A = atom ? 1u : (16u >> bi);
            cuuint64_t dims[4] = {64, rows, slabs, 16};
            cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 2 * 8};
            cuuint32_t box[4] = {64, 8, slabs / 2, A};
            cuuint32_t es[4] = {1, 1, 1, 1};
            CUresult r = g_encode(atom ? &pm.vh_atom : &pm.vh_atoms[bi],
                                  CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, atom ? 3 : 4,
                                  const_cast<void *>(L.v), dims, strides, box, es,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            if (r != CUDA_SUCCESS) {
                snprintf(err, errlen, "cuTensorMapEncodeTiled(V cache halves, %u-atom box) failed: %d",
                         (unsigned)A, (int)r);
                return cudaErrorInvalidValue;
            }
        }
        if (P.G <= 32 && 32 % P.G == 0) {
            cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)P.Hq, (cuuint64_t)P.B * P.q_len};
            cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)P.Hq * D * 2};
            cuuint32_t box[3] = {32, (cuuint32_t)P.G, (cuuint32_t)(32 / P.G)};
            cuuint32_t es[3] = {1, 1, 1};
            CUresult r = g_encode(&pm.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, P.out, dims, strides,
                                  box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            if (r != CUDA_SUCCESS) {
                snprintf(err, errlen, "cuTensorMapEncodeTiled(out) failed: %d", (int)r);
                return cudaErrorInvalidValue;
            }
            pm.out_ok = 1;
        }
        return launch_pairs<256>(L, maps, pm, stream);
    }
    return P.sinks > 0 ? tc_launch_sinks(L, maps, stream) : launch_kernels<false>(L, maps, stream);
}

}  // namespace swa
