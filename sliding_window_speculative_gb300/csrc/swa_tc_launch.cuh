// Per-configuration constants and launches of the key-major and rows-major
// tensor-core kernels, for the translation unit of each variant (SK: the first
// positions stay visible as sinks).
#pragma once

#include "swa_rows.cuh"
#include "swa_tc.cuh"
#include "swa_tc_host.h"

namespace swa {
namespace {

// Per (head_dim, padded rows): ring slots of one 128-key tile and Q / P
// buffer counts, sized to one CTA per SM (at most 227 KB of shared memory).
template <int D, int N>
struct Conf {
    // A ring of three K-or-V tiles lets V(t+1) load while V(t) waits for its
    // PV; at head_dim 256 (64 KB tiles) that leaves room for one Q and one P
    // buffer beside it (two at 16 rows).  O^T (2N columns per head-dim half)
    // is double-buffered unless TMEM runs out (head_dim 256, 64 rows).
    static constexpr int NT = D == 256 ? (N <= 32 ? 3 : 2) : 5;
    static constexpr int QB = (D == 256 && N >= 32) ? 1 : (D == 128 && N == 64) ? 1 : 2;
    static constexpr int PB = (D == 256 && N >= 32) ? 1 : (N == 64) ? 1 : 2;
    static constexpr int OB = (D == 256 && N == 64) ? 1 : 2;
    using C = TcCfg<D, N, NT, QB, PB, OB>;
};

template <int D, int N, bool AP, bool SK>
cudaError_t launch_ap(const TcLaunch &L, const TcMaps &maps, cudaStream_t stream) {
    using Cf = Conf<D, N>;
    using C = typename Cf::C;
    auto kern = swa_tc_kernel<D, N, Cf::NT, Cf::QB, Cf::PB, Cf::OB, AP, SK>;
    static std::atomic<bool> attr_done[64];
    cudaError_t e = raise_smem_limit(kern, C::SMEM_BYTES, attr_done);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(L.grid), dim3(AP ? kTcThreads + 32 : kTcThreads),
                         C::SMEM_BYTES, stream, L.T, maps);
}

// The plain kernel, or (fused append) its variant with the append warp.
template <int D, int N, bool SK>
cudaError_t launch(const TcLaunch &L, const TcMaps &maps, cudaStream_t stream) {
    return L.T.a.k_new != nullptr ? launch_ap<D, N, true, SK>(L, maps, stream)
                                  : launch_ap<D, N, false, SK>(L, maps, stream);
}

// Rows-major kernel: per (head_dim, Q rows) the ring tiles and Q buffers
// that fit one CTA per SM.
template <int D, int QR>
struct RowsConf {
    static constexpr int NT = D == 256 ? (QR == 32 ? 3 : 2) : (QR == 128 ? 5 : 6);
    static constexpr int QB = D == 256 ? (QR == 64 ? 2 : 1) : (QR == 32 ? 2 : 1);
    using C = RowsCfg<D, QR, NT, QB>;
};

template <int D, int QR, bool AP, bool SK>
cudaError_t launch_rows_ap(const TcLaunch &L, const TcMaps &maps, cudaStream_t stream) {
    using Cf = RowsConf<D, QR>;
    using C = typename Cf::C;
    auto kern = swa_rows_kernel<D, QR, Cf::NT, Cf::QB, AP, SK>;
    static std::atomic<bool> attr_done[64];
    cudaError_t e = raise_smem_limit(kern, C::SMEM_BYTES, attr_done);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(L.grid), dim3(AP ? kRowsThreads + 32 : kRowsThreads),
                         C::SMEM_BYTES, stream, L.T, maps);
}

template <int D, int QR, bool SK>
cudaError_t launch_rows(const TcLaunch &L, const TcMaps &maps, cudaStream_t stream) {
    return L.T.a.k_new != nullptr ? launch_rows_ap<D, QR, true, SK>(L, maps, stream)
                                  : launch_rows_ap<D, QR, false, SK>(L, maps, stream);
}

template <int D, bool SK>
cudaError_t launch_rows_d(const TcLaunch &L, const TcMaps &maps, cudaStream_t s) {
    switch (L.N) {
        case 32: return launch_rows<D, 32, SK>(L, maps, s);
        case 64: return launch_rows<D, 64, SK>(L, maps, s);
        case 128: return launch_rows<D, 128, SK>(L, maps, s);
        default: return cudaErrorInvalidConfiguration;
    }
}

template <int D, bool SK>
cudaError_t launch_d(const TcLaunch &L, const TcMaps &maps, cudaStream_t s) {
    switch (L.N) {
        case 16: return launch<D, 16, SK>(L, maps, s);
        case 32: return launch<D, 32, SK>(L, maps, s);
        case 64: return launch<D, 64, SK>(L, maps, s);
        default: return cudaErrorInvalidConfiguration;
    }
}

template <bool SK>
cudaError_t launch_kernels(const TcLaunch &L, const TcMaps &maps, cudaStream_t s) {
    if (L.rows_major)
        return L.D == 256 ? launch_rows_d<256, SK>(L, maps, s) : launch_rows_d<128, SK>(L, maps, s);
    return L.D == 256 ? launch_d<256, SK>(L, maps, s) : launch_d<128, SK>(L, maps, s);
}

}  // namespace
}  // namespace swa
