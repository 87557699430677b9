// launch.cuh — host helpers that the memory-bound operators (norm.cu, embedding.cu)
// share: argument checks, launches, status.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "zb_internal.h"

namespace {

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// Launches a kernel that waits for the one before it in the stream by itself
// (grid_dependency_wait before its first access to global memory), so that its blocks
// may be set up while that one's last blocks run (unless ZB_GEMM_PDL=0 says no).
template <typename K, typename... Args>
cudaError_t launch_after(K kern, long long blocks, int threads, size_t smem, void* stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = zb::dependent_launches();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

zb_status launched(const char* who, cudaError_t e) {
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string(who) + " launch: " + cudaGetErrorString(e));
    zb::clear_error();
    return ZB_OK;
}

zb_status done() {
    zb::clear_error();
    return ZB_OK;
}

}  // namespace
