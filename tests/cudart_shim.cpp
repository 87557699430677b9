// A stand-in for some calls of the CUDA runtime, preloaded into a child process of
// the tests.  Every launch is written to the file SHIM_LOG: blocks, threads, cluster,
// programmatic launch allowed or not, and SHIM_BYTES bytes of argument SHIM_ARG.
//   SHIM_FAKE=1      nothing reaches a device: launches succeed at once (152 SMs)
//   SHIM_CLUSTERS=n  no cluster of more than n blocks can be resident
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <dlfcn.h>

#include <cstdio>
#include <cstdlib>

namespace {
int number(const char* name, int otherwise) {
    const char* v = std::getenv(name);
    return v ? std::atoi(v) : otherwise;
}
bool fake() { return number("SHIM_FAKE", 0) != 0; }
template <typename F>
F real(F, const char* name) {
    void* lib = dlopen("libcudart.so.13", RTLD_LAZY | RTLD_NOLOAD);
    return reinterpret_cast<F>(lib ? dlsym(lib, name) : nullptr);
}
int cluster_of(const cudaLaunchConfig_t* c) {
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return static_cast<int>(c->attrs[i].val.clusterDim.x);
    return 1;
}
CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
unsigned char word[256];
}  // namespace

#define REAL(name) real(&name, #name)

extern "C" cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
    if (const char* path = std::getenv("SHIM_LOG")) {
        int programmatic = 0;
        for (unsigned i = 0; i < c->numAttrs; ++i)
            if (c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization)
                programmatic = c->attrs[i].val.programmaticStreamSerializationAllowed;
        if (FILE* out = std::fopen(path, "a")) {
            std::fprintf(out, "%u %u %d %d ", c->gridDim.x, c->blockDim.x, cluster_of(c), programmatic);
            const int bytes = number("SHIM_BYTES", 0);
            for (int i = 0; i < bytes; ++i)
                std::fprintf(out, "%02x", static_cast<const unsigned char*>(args[number("SHIM_ARG", 0)])[i]);
            std::fprintf(out, "\n");
            std::fclose(out);
        }
    }
    return fake() ? cudaSuccess : REAL(cudaLaunchKernelExC)(c, f, args);
}

extern "C" cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
    const int size = cluster_of(c);
    *n = 0;
    if (size > number("SHIM_CLUSTERS", 16)) return cudaSuccess;
    if (!fake()) return REAL(cudaOccupancyMaxActiveClusters)(n, f, c);
    *n = 152 / size;
    return cudaSuccess;
}

extern "C" cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
    return fake() ? cudaSuccess : REAL(cudaFuncSetAttribute)(f, a, v);
}

extern "C" cudaError_t cudaGetLastError() { return fake() ? cudaSuccess : REAL(cudaGetLastError)(); }

extern "C" cudaError_t cudaGetDevice(int* dev) {
    if (!fake()) return REAL(cudaGetDevice)(dev);
    *dev = 0;
    return cudaSuccess;
}

extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int dev) {
    if (!fake()) return REAL(cudaDeviceGetAttribute)(v, a, dev);
    *v = 152;
    return cudaSuccess;
}

extern "C" cudaError_t cudaGetSymbolAddress(void** p, const void* symbol) {
    if (!fake()) return REAL(cudaGetSymbolAddress)(p, symbol);
    *p = word;
    return cudaSuccess;
}

extern "C" cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** p, unsigned int version,
                                                        unsigned long long flags, cudaDriverEntryPointQueryResult* q) {
    if (!fake()) return REAL(cudaGetDriverEntryPointByVersion)(name, p, version, flags, q);
    *p = reinterpret_cast<void*>(&fake_encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
