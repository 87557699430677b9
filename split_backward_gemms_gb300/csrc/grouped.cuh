// grouped.cuh — what the products grouped by expert share (grouped.cu, fp8.cu):
// offsets in shared memory, the walk over ragged tiles, tensor maps of stacked
// matrices and launch configurations.
#pragma once

#include <algorithm>
#include <atomic>
#include <string>

#include "gemm_core.cuh"

namespace {

constexpr int MAX_EXPERTS = 256;

// A role's walk over the tiles of a product grouped by expert: expert e has nt
// tiles of `tr` rows (the last one fewer) x tiles_f of columns.  EVEN: its rows
// are spread over the tiles (in steps of 32); else every tile but the last has
// TILE_T.
template <int TILE_T, bool EVEN>
struct Walk {
    const int* off;
    int experts, tiles_f;
    int e, first, nt, tr;
    __device__ Walk(const int* off_, int experts_, int tiles_f_)
        : off(off_), experts(experts_), tiles_f(tiles_f_), e(-1), first(0), nt(0), tr(0) {}
    // Moves to tile t (ascending calls); false past the last one.
    __device__ __forceinline__ bool to(int t, int& row0, int& nrows, int& fb) {
        while (t >= first + nt * tiles_f) {
            first += nt * tiles_f;
            if (++e >= experts) return false;
            const int n = off[e + 1] - off[e];
            nt = (n + TILE_T - 1) / TILE_T;
            tr = !EVEN ? TILE_T : nt ? ((n + nt - 1) / nt + 31) / 32 * 32 : 0;
        }
        int tb;
        tile_coords(t - first, nt, tiles_f, 16, tb, fb);
        row0 = off[e] + tb * tr;
        nrows = min(tr, off[e + 1] - row0);
        return true;
    }
};

// off[0..experts] in shared memory from the caller's offsets, made legal:
// inside [0, rows] and ascending (a running maximum, 32 at a time).
__device__ __forceinline__ void load_offsets(int* off, const int* offsets, int experts, int rows) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int carry = 0;
        for (int i0 = 0; i0 <= experts; i0 += 32) {
            const int i = i0 + lane;
            int v = max(carry, i <= experts ? min(max(offsets[i], 0), rows) : 0);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v = max(v, u);
            }
            if (i <= experts) off[i] = v;
            carry = __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- host side
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// 3-D map of a stack of `count` matrices [outer, inner], dense, of elements of
// `es` bytes; 128-byte swizzle.
bool make_map3(CUtensorMap* m, const void* base, CUtensorMapDataType type, uint64_t es, uint64_t inner,
               uint64_t outer, uint64_t count, uint32_t box_inner, uint32_t box_outer, std::string* why) {
    EncodeTiledFn fn = encode_fn(why);
    if (!fn) return false;
    cuuint64_t dims[3] = {inner, outer, count};
    cuuint64_t strides[2] = {inner * es, inner * outer * es};
    cuuint32_t box[3] = {box_inner, box_outer, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        if (why) *why = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string(static_cast<int>(r));
        return false;
    }
    return true;
}

// Shared-memory limit of a kernel, set once per device, and the CTAs of a
// full grid of its clusters.
template <typename K>
zb_status full_grid(K kern, std::atomic<int>* cache, size_t smem, int threads, int cg, int* ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return zb::fail(ZB_ERR_CUDA, "cudaGetDevice failed");
    if (!cache[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess)
            return zb::fail(ZB_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
        int n = sm_count();
        if (cg == 2) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(512);
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 2;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int clusters = 0;
            e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
            if (e != cudaSuccess || clusters <= 0)
                return zb::fail(ZB_ERR_UNSUPPORTED, std::string("no co-resident CTA pairs: ") + cudaGetErrorString(e));
            n = 2 * clusters;
        }
        if (n <= 0) return zb::fail(ZB_ERR_CUDA, "cannot query the SM count");
        cache[dev].store(n, std::memory_order_relaxed);
    }
    *ctas = cache[dev].load(std::memory_order_relaxed);
    return ZB_OK;
}

struct LaunchCfg {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    LaunchCfg(int grid, int threads, size_t smem, int cg, void* stream) {
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = static_cast<cudaStream_t>(stream);
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cg;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cg == 2 ? 2 : 1;
    }
};

}  // namespace
