// norm.cu — layer norm split like the block it stands before: F, the gradient
// of its input (B) and of its weights (the deferrable W).
//   mean = sum x / n, rstd = (sum (x - mean)^2 / n + eps)^-1/2, xh = (x - mean) rstd
//   F:  y = gamma xh + beta
//   B:  u = gamma dy;  dx = rstd (u - mean(u) - xh mean(u xh)) + dR
//   W:  dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "ptx.cuh"
#include "zb_internal.h"

namespace {

constexpr int MAX_WIDTH = 32768;

// 8 consecutive values.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A row belongs to G warps, a lane of which holds V vectors of 8 values (lane,
// lane + 32 G, ...).  A block has 8 warps, or 16 where G is 16.
template <int G>
struct Team {
    static constexpr int THREADS = G > 8 ? 32 * G : 256;
    static constexpr int ROWS = THREADS / (32 * G);
};

// Sums of a row's warps, the same in all of them: the warps' sums in order.
template <int G, int N>
__device__ __forceinline__ void team_sum(float (&x)[N], float (*part)[G][N], int team) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
    if (G == 1) return;
    const int w = (threadIdx.x >> 5) % G;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[team][w][i] = x[i];
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * G) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = part[team][0][i];
#pragma unroll
        for (int k = 1; k < G; ++k) x[i] += part[team][k][i];
    }
}

template <typename T, int V, int G>
__global__ void __launch_bounds__(Team<G>::THREADS)
    zb_layernorm_forward_kernel(const T* __restrict__ X, const __nv_bfloat16* __restrict__ gamma,
                                const __nv_bfloat16* __restrict__ beta, __nv_bfloat16* __restrict__ Y,
                                float* __restrict__ mean_out, float* __restrict__ rstd_out, long long rows, int width,
                                float eps) {
    __shared__ float part[2][Team<G>::ROWS][G][1];
    const int team = threadIdx.x / (32 * G), at = threadIdx.x % (32 * G);
    const long long row = static_cast<long long>(blockIdx.x) * Team<G>::ROWS + team;
    if (row >= rows) return;
    const T* x = X + row * width;
    const int nv = width / 8;
    float v[V][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * 32 * G;
        if (k < nv) {
            load8(x + 8 * k, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] += v[i][j];
    team_sum<G, 1>(sum, part[0], team);
    const float mean = sum[0] / static_cast<float>(width);
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (at + i * 32 * G < nv)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mean;
                sq[0] = fmaf(v[i][j], v[i][j], sq[0]);
            }
    team_sum<G, 1>(sq, part[1], team);
    const float rstd = 1.0f / sqrtf(sq[0] / static_cast<float>(width) + eps);
    if (at == 0 && mean_out) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * 32 * G;
        if (k >= nv) break;
        float g[8], b[8] = {};
        load8(gamma + 8 * k, g);
        if (beta) load8(beta + 8 * k, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, g[j], b[j]);
        store8(Y + row * width + 8 * k, v[i]);
    }
}

template <typename T, int V, int G>
__global__ void __launch_bounds__(Team<G>::THREADS)
    zb_layernorm_backward_input_kernel(const __nv_bfloat16* __restrict__ dY, const T* __restrict__ X,
                                       const __nv_bfloat16* __restrict__ gamma, const float* __restrict__ mean_in,
                                       const float* __restrict__ rstd_in, const T* dR, T* dX,
                                       __nv_bfloat16* __restrict__ dX16, long long rows, int width) {
    __shared__ float part[Team<G>::ROWS][G][2];
    const int team = threadIdx.x / (32 * G), at = threadIdx.x % (32 * G);
    const long long row = static_cast<long long>(blockIdx.x) * Team<G>::ROWS + team;
    if (row >= rows) return;
    const int nv = width / 8;
    const float mean = mean_in[row], rstd = rstd_in[row];
    float xh[V][8], u[V][8];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * 32 * G;
        if (k < nv) {
            load8(X + row * width + 8 * k, xh[i]);
            load8(dY + row * width + 8 * k, u[i]);
            float g[8];
            load8(gamma + 8 * k, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] = (xh[i][j] - mean) * rstd;
                u[i][j] *= g[j];
                sum[0] += u[i][j];
                sum[1] = fmaf(u[i][j], xh[i][j], sum[1]);
            }
        }
    }
    team_sum<G, 2>(sum, part, team);
    const float mu = sum[0] / static_cast<float>(width), along = sum[1] / static_cast<float>(width);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * 32 * G;
        if (k >= nv) break;
        float r[8] = {};
        if (dR) load8(dR + row * width + 8 * k, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = fmaf(rstd, u[i][j] - mu - xh[i][j] * along, r[j]);
        store8(dX + row * width + 8 * k, r);
        if (dX16) store8(dX16 + row * width + 8 * k, r);
    }
}

// W: a cluster of 8 blocks takes 64 columns (a 128-byte line of a row in bf16),
// each block an eighth of the rows, 32 of them at a time (8 lanes a row); the
// blocks' sums meet in the first one's, in order.
constexpr int W_SPLIT = 8;
constexpr int W_COLS = 64;
constexpr int W_THREADS = 256;

template <typename T>
__global__ void __cluster_dims__(W_SPLIT, 1, 1) __launch_bounds__(W_THREADS)
    zb_layernorm_backward_weight_kernel(const __nv_bfloat16* __restrict__ dY, const T* __restrict__ X,
                                        const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                                        float* __restrict__ dgamma, float* __restrict__ dbeta, long long rows,
                                        int width, int accumulate) {
    __shared__ float part[W_THREADS / 32][2][W_COLS];
    __shared__ float block_sum[2][W_COLS];
    const uint32_t rank = zbp::cluster_ctarank();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c0 = (blockIdx.x / W_SPLIT) * W_COLS, col = c0 + (lane & 7) * 8;
    const long long lo = rows * rank / W_SPLIT, hi = rows * (rank + 1) / W_SPLIT;
    float dg[8] = {}, db[8] = {};
    if (col < width) {
#pragma unroll 4
        for (long long r = lo + (threadIdx.x >> 3); r < hi; r += W_THREADS / 8) {
            float x[8], dy[8];
            load8(X + r * width + col, x);
            load8(dY + r * width + col, dy);
            const float mean = mean_in[r], rstd = rstd_in[r];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dg[j] = fmaf(dy[j], (x[j] - mean) * rstd, dg[j]);
                db[j] += dy[j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        dg[j] += __shfl_xor_sync(0xffffffffu, dg[j], 8);
        db[j] += __shfl_xor_sync(0xffffffffu, db[j], 8);
        dg[j] += __shfl_xor_sync(0xffffffffu, dg[j], 16);
        db[j] += __shfl_xor_sync(0xffffffffu, db[j], 16);
        if (lane < 8) {
            part[w][0][lane * 8 + j] = dg[j];
            part[w][1][lane * 8 + j] = db[j];
        }
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < 2 * W_COLS) {
        float s = part[0][t / W_COLS][t % W_COLS];
#pragma unroll
        for (int k = 1; k < W_THREADS / 32; ++k) s += part[k][t / W_COLS][t % W_COLS];
        block_sum[t / W_COLS][t % W_COLS] = s;
    }
    zbp::cluster_sync();
    if (rank == 0 && t < 2 * W_COLS) {
        const int c = c0 + t % W_COLS;
        float* out = t < W_COLS ? dgamma : dbeta;
        if (c < width && out) {
            const uint32_t here = zbp::smem_u32(&block_sum[t / W_COLS][t % W_COLS]);
            float s = 0.0f;
#pragma unroll
            for (int b = 0; b < W_SPLIT; ++b) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(zbp::mapa_shared(here, b)) : "memory");
                s += v;
            }
            out[c] = accumulate ? out[c] + s : s;
        }
    }
    zbp::cluster_sync();  // no block leaves while the first may still read it
}

// ---------------------------------------------------------------- host side
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

zb_status check_norm(const char* who, const zb_layernorm* n) {
    const std::string w = who;
    if (!n) return zb::fail(ZB_ERR_INVALID_ARG, w + ": descriptor is NULL");
    if (n->rows < 0 || n->rows > (1LL << 30)) return zb::fail(ZB_ERR_SHAPE, w + ": rows must be in [0, 2^30]");
    if (n->width < 1 || n->width > MAX_WIDTH) return zb::fail(ZB_ERR_SHAPE, w + ": width must be in [1, 32768]");
    if (n->width % 8) return zb::fail(ZB_ERR_ALIGN, w + ": width must be a multiple of 8");
    if (n->dtype != ZB_DT_BF16 && n->dtype != ZB_DT_F32) return zb::fail(ZB_ERR_DTYPE, w + ": unknown dtype");
    if (!(n->eps > 0.0f) || std::isinf(n->eps)) return zb::fail(ZB_ERR_INVALID_ARG, w + ": eps must be positive");
    return ZB_OK;
}

zb_status launched(const char* who) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string(who) + " launch: " + cudaGetErrorString(e));
    zb::clear_error();
    return ZB_OK;
}

zb_status done() {
    zb::clear_error();
    return ZB_OK;
}

// Calls f(V, G) with the vectors a lane and the warps a row of `width` values.
template <typename F>
void by_width(int64_t width, F&& f) {
    const int nv = static_cast<int>(width / 8);
    using std::integral_constant;
#define ZB_CASE(v, g) f(integral_constant<int, v>(), integral_constant<int, g>())
    if (nv <= 32) ZB_CASE(1, 1);
    else if (nv <= 64) ZB_CASE(2, 1);
    else if (nv <= 128) ZB_CASE(4, 1);
    else if (nv <= 256) ZB_CASE(4, 2);
    else if (nv <= 512) ZB_CASE(4, 4);
    else if (nv <= 1024) ZB_CASE(4, 8);
    else if (nv <= 2048) ZB_CASE(4, 16);
    else ZB_CASE(8, 16);
#undef ZB_CASE
}

unsigned blocks_of(int64_t rows, int per) { return static_cast<unsigned>((rows + per - 1) / per); }

}  // namespace

extern "C" zb_status zb_layernorm_forward(const zb_layernorm* n, const void* X, const void* gamma, const void* beta,
                                          void* Y, float* mean, float* rstd, void* stream) {
    zb_status s = check_norm("zb_layernorm_forward", n);
    if (s != ZB_OK) return s;
    if (n->rows == 0) return done();
    if (!X || !gamma || !Y || !mean != !rstd)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_layernorm_forward: required pointer is NULL");
    if (off16(X) || off16(gamma) || off16(beta) || off16(Y) || off4(mean) || off4(rstd))
        return zb::fail(ZB_ERR_ALIGN, "zb_layernorm_forward: pointers must be 16-byte aligned (mean, rstd: 4)");
    auto go = [&](auto zero) {
        using T = decltype(zero);
        by_width(n->width, [&](auto v, auto g) {
            constexpr int V = v(), G = g();
            zb_layernorm_forward_kernel<T, V, G>
                <<<blocks_of(n->rows, Team<G>::ROWS), Team<G>::THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
                    static_cast<const T*>(X), static_cast<const __nv_bfloat16*>(gamma),
                    static_cast<const __nv_bfloat16*>(beta), static_cast<__nv_bfloat16*>(Y), mean, rstd, n->rows,
                    static_cast<int>(n->width), n->eps);
        });
    };
    if (n->dtype == ZB_DT_BF16)
        go(__nv_bfloat16());
    else
        go(float());
    return launched("zb_layernorm_forward");
}

extern "C" zb_status zb_layernorm_backward_input(const zb_layernorm* n, const void* dY, const void* X,
                                                 const void* gamma, const float* mean, const float* rstd,
                                                 const void* dR, void* dX, void* dX16, void* stream) {
    zb_status s = check_norm("zb_layernorm_backward_input", n);
    if (s != ZB_OK) return s;
    if (n->rows == 0) return done();
    if (!dY || !X || !gamma || !mean || !rstd || !dX)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_layernorm_backward_input: required pointer is NULL");
    if (off16(dY) || off16(X) || off16(gamma) || off4(mean) || off4(rstd) || off16(dR) || off16(dX) || off16(dX16))
        return zb::fail(ZB_ERR_ALIGN, "zb_layernorm_backward_input: pointers must be 16-byte aligned (mean, rstd: 4)");
    auto go = [&](auto zero) {
        using T = decltype(zero);
        by_width(n->width, [&](auto v, auto g) {
            constexpr int V = v(), G = g();
            zb_layernorm_backward_input_kernel<T, V, G>
                <<<blocks_of(n->rows, Team<G>::ROWS), Team<G>::THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
                    static_cast<const __nv_bfloat16*>(dY), static_cast<const T*>(X),
                    static_cast<const __nv_bfloat16*>(gamma), mean, rstd, static_cast<const T*>(dR),
                    static_cast<T*>(dX), static_cast<__nv_bfloat16*>(dX16), n->rows, static_cast<int>(n->width));
        });
    };
    if (n->dtype == ZB_DT_BF16)
        go(__nv_bfloat16());
    else
        go(float());
    return launched("zb_layernorm_backward_input");
}

extern "C" zb_status zb_layernorm_backward_weight(const zb_layernorm* n, const void* dY, const void* X,
                                                  const float* mean, const float* rstd, float* dgamma, float* dbeta,
                                                  int accumulate, void* stream) {
    zb_status s = check_norm("zb_layernorm_backward_weight", n);
    if (s != ZB_OK) return s;
    if (!dgamma || (n->rows > 0 && (!dY || !X || !mean || !rstd)))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_layernorm_backward_weight: required pointer is NULL");
    if (off16(dY) || off16(X) || off4(mean) || off4(rstd) || off4(dgamma) || off4(dbeta))
        return zb::fail(ZB_ERR_ALIGN,
                        "zb_layernorm_backward_weight: dY and X must be 16-byte aligned (fp32 vectors: 4)");
    const unsigned blocks = blocks_of(n->width, W_COLS) * W_SPLIT;
    auto go = [&](auto zero) {
        using T = decltype(zero);
        zb_layernorm_backward_weight_kernel<T><<<blocks, W_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
            static_cast<const __nv_bfloat16*>(dY), static_cast<const T*>(X), mean, rstd, dgamma, dbeta, n->rows,
            static_cast<int>(n->width), accumulate != 0);
    };
    if (n->dtype == ZB_DT_BF16)
        go(__nv_bfloat16());
    else
        go(float());
    return launched("zb_layernorm_backward_weight");
}
