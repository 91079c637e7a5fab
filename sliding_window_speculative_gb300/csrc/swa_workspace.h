// Device memory of one purpose on one device that grows with the calls using
// it: the attention's split partials, the greedy acceptance's scratch.  Plain
// host code on the CUDA runtime's C interface (tests run it against a counting
// stand-in).
//
// A buffer that a captured call was given has to outlive the graph, which may
// be replayed at any time, so it is kept when a larger call outgrows it.  Any
// other outgrown buffer is freed before the larger one is allocated: cudaFree
// waits for the calls that use it, and a call finds as much room as if it
// were the first.  So what is held is the current buffer and those that
// captures have seen, each over a quarter larger than the one before where
// memory allows.
#pragma once

#include <cuda_runtime_api.h>

#include <cstddef>
#include <new>

namespace swa {

struct Workspace {
    struct Kept {
        void *ptr;
        Kept *next;
    };
    void *ptr = nullptr;
    size_t bytes = 0;
    bool owned = false;     // allocated here (else the caller's, or none)
    bool captured = false;  // a captured call was given it
    Kept *kept = nullptr;   // outgrown, but captured
};

// Whether `stream` is capturing.  Without an answer (the legacy stream while
// another stream captures) it counts as capturing: the buffer is kept.
inline bool stream_capturing(cudaStream_t stream) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) {
        (void)cudaGetLastError();
        return true;
    }
    return cap != cudaStreamCaptureStatusNone;
}

// Frees what was allocated here, outgrown buffers too; the first error.
inline cudaError_t workspace_free(Workspace &w) {
    cudaError_t first = cudaSuccess;
    while (w.kept != nullptr) {
        Workspace::Kept *k = w.kept;
        w.kept = k->next;
        const cudaError_t e = cudaFree(k->ptr);
        if (first == cudaSuccess) first = e;
        delete k;
    }
    if (w.owned && w.ptr != nullptr) {
        const cudaError_t e = cudaFree(w.ptr);
        if (first == cudaSuccess) first = e;
        w.ptr = nullptr;
        w.bytes = 0;
        w.owned = w.captured = false;
    }
    return first;
}

// A buffer of at least `need` bytes (more than it has), outside stream capture
// and not the caller's: a quarter more than needed, or exactly that where the
// quarter does not fit.  On an error a captured buffer, or one that could not be
// freed (another stream captures), stays the current one.
inline cudaError_t workspace_grow(Workspace &w, size_t need) {
    Workspace::Kept *node = nullptr;
    if (w.ptr != nullptr && w.captured) {
        node = new (std::nothrow) Workspace::Kept{w.ptr, w.kept};
        if (node == nullptr) return cudaErrorMemoryAllocation;
    } else if (w.ptr != nullptr) {
        const cudaError_t e = cudaFree(w.ptr);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        w.ptr = nullptr;
        w.bytes = 0;
        w.owned = false;
    }
    size_t bytes = need + need / 4;
    void *ptr = nullptr;
    cudaError_t e = cudaMalloc(&ptr, bytes);
    if (e == cudaErrorMemoryAllocation) {
        (void)cudaGetLastError();
        bytes = need;
        e = cudaMalloc(&ptr, bytes);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        delete node;
        return e;
    }
    if (node != nullptr) w.kept = node;
    w.ptr = ptr;
    w.bytes = bytes;
    w.owned = true;
    w.captured = false;
    return cudaSuccess;
}

}  // namespace swa
