"""The library-owned workspace without a GPU: its growth (csrc/swa_workspace.h)
compiled against a stand-in for the CUDA runtime that counts what is held and
refuses what does not fit."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <map>
#include "swa_workspace.h"

static size_t room, held, frees;
static std::map<void *, size_t> live;
static bool capturing, unanswered, unfreeable;
static size_t next_ptr = 4096;

extern "C" {
cudaError_t cudaMalloc(void **p, size_t n) {
    if (held + n > room) return cudaErrorMemoryAllocation;
    *p = (void *)next_ptr;
    next_ptr += (n + 4095) / 4096 * 4096;
    live[*p] = n;
    held += n;
    return cudaSuccess;
}
cudaError_t cudaFree(void *p) {
    if (unfreeable) return cudaErrorStreamCaptureUnsupported;
    if (live.find(p) == live.end()) return cudaErrorInvalidValue;
    held -= live[p];
    live.erase(p);
    ++frees;
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, enum cudaStreamCaptureStatus *s) {
    if (unanswered) return cudaErrorStreamCaptureImplicit;
    *s = capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
}

#define CHECK(x) if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
    using swa::Workspace;
    {   // eager calls that grow hold one buffer, and find the room of the old one
        Workspace w;
        room = 1250;
        CHECK(swa::workspace_grow(w, 400) == cudaSuccess && w.bytes == 500 && held == 500);
        CHECK(swa::workspace_grow(w, 1000) == cudaSuccess && w.bytes == 1250 && held == 1250);
        CHECK(frees == 1 && live.size() == 1 && live.count(w.ptr) == 1);
        CHECK(swa::workspace_free(w) == cudaSuccess && held == 0 && w.ptr == nullptr);
    }
    {   // exactly what is needed where a quarter more does not fit
        Workspace w;
        room = 1100;
        CHECK(swa::workspace_grow(w, 600) == cudaSuccess && w.bytes == 750);
        CHECK(swa::workspace_grow(w, 1000) == cudaSuccess && w.bytes == 1000 && held == 1000);
        // and an error without anything held where that does not fit either
        CHECK(swa::workspace_grow(w, 1200) == cudaErrorMemoryAllocation);
        CHECK(held == 0 && w.ptr == nullptr && w.bytes == 0 && !w.owned);
        CHECK(swa::workspace_grow(w, 100) == cudaSuccess && w.bytes == 125);
        CHECK(swa::workspace_free(w) == cudaSuccess && held == 0);
    }
    {   // a captured call's buffer stays, whatever the growth does
        Workspace w;
        room = 2000;
        CHECK(swa::workspace_grow(w, 400) == cudaSuccess);
        void *graph = w.ptr;
        w.captured = true;
        CHECK(swa::workspace_grow(w, 3000) == cudaErrorMemoryAllocation);
        CHECK(w.ptr == graph && w.bytes == 500 && w.captured && held == 500);
        CHECK(swa::workspace_grow(w, 1000) == cudaSuccess && w.bytes == 1250);
        CHECK(live.count(graph) == 1 && held == 1750 && !w.captured);
        // the one after it was not captured: it goes
        void *eager = w.ptr;
        CHECK(swa::workspace_grow(w, 1400) == cudaSuccess && w.bytes == 1400);
        CHECK(live.count(graph) == 1 && live.count(eager) == 0 && held == 1900);
        CHECK(swa::workspace_free(w) == cudaSuccess && held == 0 && w.kept == nullptr);
    }
    {   // a buffer that cannot be freed now stays in use
        Workspace w;
        room = 2000;
        CHECK(swa::workspace_grow(w, 400) == cudaSuccess);
        void *before = w.ptr;
        unfreeable = true;
        CHECK(swa::workspace_grow(w, 800) == cudaErrorStreamCaptureUnsupported);
        unfreeable = false;
        CHECK(w.ptr == before && w.bytes == 500 && w.owned && held == 500);
        CHECK(swa::workspace_grow(w, 800) == cudaSuccess && held == 1000);
        CHECK(swa::workspace_free(w) == cudaSuccess && held == 0);
    }
    {   // any number of captured buffers
        Workspace w;
        room = (size_t)1 << 60;
        for (int i = 0; i < 1000; ++i) {
            CHECK(swa::workspace_grow(w, w.bytes + 1) == cudaSuccess || w.bytes > room / 8);
            w.captured = true;
            if (w.bytes > room / 16) break;
        }
        CHECK(live.size() > 100);
        CHECK(swa::workspace_free(w) == cudaSuccess && held == 0);
    }
    CHECK(!swa::stream_capturing(nullptr));
    capturing = true;
    CHECK(swa::stream_capturing(nullptr));
    capturing = false;
    unanswered = true;
    CHECK(swa::stream_capturing(nullptr));
    puts("ok");
    return 0;
}
"""


def test_growth_against_a_counting_runtime(tmp_path):
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("no CUDA headers")
    src, exe = tmp_path / "workspace.cpp", tmp_path / "workspace"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-I", cuda, "-I",
                        os.path.join(ROOT, "sliding_window_speculative_gb300", "csrc"), str(src),
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
