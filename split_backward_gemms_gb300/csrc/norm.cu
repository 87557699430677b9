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

#include "launch.cuh"
#include "ptx.cuh"

namespace {

constexpr int MAX_WIDTH = 32768;

// 8 consecutive values as they lie in memory, so that what a lane has in flight or
// keeps for later takes few registers.
template <typename T>
struct Raw8 {
    static constexpr int WORDS = static_cast<int>(sizeof(T)) * 2;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = q.x;
            w[4 * i + 1] = q.y;
            w[4 * i + 2] = q.z;
            w[4 * i + 3] = q.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float operator[](int j) const {
        if (WORDS == 8) return __uint_as_float(w[WORDS == 8 ? j : 0]);
        return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
};
using Raw16 = Raw8<__nv_bfloat16>;

// Two fp32 values in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pk2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void up2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
template <typename R>
__device__ __forceinline__ f32x2 pair(const R& v, int j) {
    return pk2(v[2 * j], v[2 * j + 1]);
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

// F: x in registers, two sums over the row (the mean, then the squares around it),
// one read and one write; HBM bounds it.  8192 x 4096: 26 us in bf16 (5.2 TB/s), 32 in
// fp32 (6.3).  Half the vectors a lane and twice the warps a row: 28 and 35; gamma and
// beta asked for with x: no faster; a persistent grid with the next row asked for ahead
// (spills): 40 and 57; the warps' sums joined in one meeting: 27 and 33.
template <typename T, int V, int G>
__global__ void __launch_bounds__(Team<G>::THREADS)
    zb_layernorm_forward_kernel(const T* __restrict__ X, const __nv_bfloat16* __restrict__ gamma,
                                const __nv_bfloat16* __restrict__ beta, __nv_bfloat16* __restrict__ Y,
                                float* __restrict__ mean_out, float* __restrict__ rstd_out, long long rows, int width,
                                float eps) {
    __shared__ float part[2][Team<G>::ROWS][G][1];
    const int team = threadIdx.x / (32 * G), at = threadIdx.x % (32 * G);
    const long long row = static_cast<long long>(blockIdx.x) * Team<G>::ROWS + team;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    if (row >= rows) return;
    const int nv = width / 8;
    Raw8<T> x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * 32 * G;
        x[i].zero();
        if (k < nv) x[i].load(X + row * width + 8 * k);
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] += x[i][j];
    team_sum<G, 1>(sum, part[0], team);
    const float mean = sum[0] / static_cast<float>(width);
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (at + i * 32 * G < nv)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = x[i][j] - mean;
                sq[0] = fmaf(d, d, sq[0]);
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
        Raw16 g, b;
        g.load(gamma + 8 * k);
        b.zero();
        if (beta) b.load(beta + 8 * k);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fmaf((x[i][j] - mean) * rstd, g[j], b[j]);
        store8(Y + row * width + 8 * k, y);
    }
}

// B.  Everything a lane reads is asked for before the first sum, gamma and the
// residual's gradient too, so that a row waits for memory once.  HBM bounds it: 8192 x
// 4096 42 us in bf16 (6.4 TB/s), 77 in fp32 with the bf16 copy (6.9); with the values
// kept as fp32 and dR asked for after the sums 82 and 105.
template <typename T, int V, int G>
__global__ void __launch_bounds__(Team<G>::THREADS)
    zb_layernorm_backward_input_kernel(const __nv_bfloat16* __restrict__ dY, const T* __restrict__ X,
                                       const __nv_bfloat16* __restrict__ gamma, const float* __restrict__ mean_in,
                                       const float* __restrict__ rstd_in, const T* dR, T* dX,
                                       __nv_bfloat16* __restrict__ dX16, long long rows, int width) {
    __shared__ float part[Team<G>::ROWS][G][2];
    const int team = threadIdx.x / (32 * G), at = threadIdx.x % (32 * G);
    const long long row = static_cast<long long>(blockIdx.x) * Team<G>::ROWS + team;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    if (row >= rows) return;
    const int nv = width / 8;
    Raw8<T> x[V], r[V];
    Raw16 dy[V], g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * 32 * G;
        r[i].zero();
        if (k < nv) {
            x[i].load(X + row * width + 8 * k);
            dy[i].load(dY + row * width + 8 * k);
            if (dR) r[i].load(dR + row * width + 8 * k);
            g[i].load(gamma + 8 * k);
        }
    }
    const float mean = mean_in[row], rstd = rstd_in[row];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (at + i * 32 * G < nv)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = dy[i][j] * g[i][j];
                sum[0] += u;
                sum[1] = fmaf(u, (x[i][j] - mean) * rstd, sum[1]);
            }
    team_sum<G, 2>(sum, part, team);
    const float mu = sum[0] / static_cast<float>(width), along = sum[1] / static_cast<float>(width);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * 32 * G;
        if (k >= nv) break;
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            d[j] = fmaf(rstd, dy[i][j] * g[i][j] - mu - (x[i][j] - mean) * rstd * along, r[i][j]);
        store8(dX + row * width + 8 * k, d);
        if (dX16) store8(dX16 + row * width + 8 * k, d);
    }
}

// W: a cluster of 8 blocks takes `vecs` (a power of two) vectors of 8 columns, its
// blocks in turn as many rows at a time as they have threads for.  The rows go from
// the last to the first: where W follows B, the last ones are still in L2 (8191 x
// 2048 bf16 after B: B and W 37.0 us from the first row on, 36.3 from the last).
// Lanes of a warp that hold the same columns meet by shuffles, warps in shared
// memory, and blocks in each other's: block r adds the eighth part r of the columns.
// All sums in a fixed order.  8192 x 4096: 28 us in bf16 (4.8 TB/s), 35 in fp32 (5.8);
// some 4 us are the clusters' start and exchange.  256 threads a block 29, 16 clusters
// of 512 threads 44, more rows in flight a thread and so one block an SM 39 (bf16).
constexpr int W_SPLIT = 8;
constexpr int W_THREADS = 512;
constexpr int W_WARPS = W_THREADS / 32;
constexpr int W_COLS = 1024;  // of a cluster, at most

template <typename T>
__global__ void __cluster_dims__(W_SPLIT, 1, 1) __launch_bounds__(W_THREADS)
    zb_layernorm_backward_weight_kernel(const __nv_bfloat16* __restrict__ dY, const T* __restrict__ X,
                                        const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                                        float* __restrict__ dgamma, float* __restrict__ dbeta, long long rows,
                                        int width, int vecs, int accumulate) {
    __shared__ float part[W_WARPS][2][256];  // a warp's columns: 8 for each of its first min(32, vecs) lanes
    __shared__ float block_sum[2][W_COLS];
    const uint32_t rank = zbp::cluster_ctarank();
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int c0 = (blockIdx.x / W_SPLIT) * vecs * 8, col = c0 + (t & (vecs - 1)) * 8;
    const int slots = W_THREADS / vecs;  // rows of a block at a time
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    f32x2 dg2[4] = {0, 0, 0, 0}, db2[4] = {0, 0, 0, 0};
    if (col < width) {
#pragma unroll 4
        for (long long r = rows - 1 - (static_cast<long long>(rank) * slots + t / vecs); r >= 0; r -= W_SPLIT * slots) {
            Raw8<T> x;
            Raw16 dy;
            x.load(X + r * width + col);
            dy.load(dY + r * width + col);
            const float mean = mean_in[r], rstd = rstd_in[r];
            const f32x2 minus = pk2(-mean, -mean), scale = pk2(rstd, rstd);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x2 d = pair(dy, j);
                dg2[j] = fma2(d, mul2(add2(pair(x, j), minus), scale), dg2[j]);
                db2[j] = add2(db2[j], d);
            }
        }
    }
    float dg[8], db[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        up2(dg2[j], dg[2 * j], dg[2 * j + 1]);
        up2(db2[j], db[2 * j], db[2 * j + 1]);
    }
    for (int o = vecs; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dg[j] += __shfl_xor_sync(0xffffffffu, dg[j], o);
            db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
        }
    if (lane < vecs) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            part[w][0][lane * 8 + j] = dg[j];
            part[w][1][lane * 8 + j] = db[j];
        }
    }
    __syncthreads();
    // warps w, w + groups, ... hold the same columns
    const int groups = vecs > 32 ? vecs / 32 : 1, cols = vecs * 8;
    for (int i = t; i < 2 * cols; i += W_THREADS) {
        const int kind = i / cols, c = i - kind * cols;
        float s = 0.0f;
        for (int k = c / 256; k < W_WARPS; k += groups) s += part[k][kind][c % 256];
        block_sum[kind][c] = s;
    }
    zbp::cluster_sync();
    for (int i = static_cast<int>(rank) * cols / 4 + t; i < static_cast<int>(rank + 1) * cols / 4; i += W_THREADS) {
        const int kind = i / cols, c = i - kind * cols;
        float* out = kind ? dbeta : dgamma;
        if (c0 + c >= width || !out) continue;
        const uint32_t here = zbp::smem_u32(&block_sum[kind][c]);
        float s = 0.0f;
#pragma unroll
        for (int b = 0; b < W_SPLIT; ++b) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(zbp::mapa_shared(here, b)) : "memory");
            s += v;
        }
        out[c0 + c] = accumulate ? out[c0 + c] + s : s;
    }
    zbp::cluster_sync();  // no block leaves while another may still read its sums
}

// ---------------------------------------------------------------- host side
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

// Calls f(V, G) with the vectors a lane and the warps a row of `width` values.
template <typename F>
void forward_by_width(int64_t width, F&& f) {
    const int nv = static_cast<int>(width / 8);
    using std::integral_constant;
#define ZB_CASE(v, g) f(integral_constant<int, v>(), integral_constant<int, g>())
    if (nv <= 32) ZB_CASE(1, 1);
    else if (nv <= 64) ZB_CASE(2, 1);
    else if (nv <= 128) ZB_CASE(4, 1);
    else if (nv <= 192) ZB_CASE(3, 2);
    else if (nv <= 256) ZB_CASE(4, 2);
    else if (nv <= 384) ZB_CASE(3, 4);
    else if (nv <= 512) ZB_CASE(4, 4);
    else if (nv <= 768) ZB_CASE(3, 8);
    else if (nv <= 1024) ZB_CASE(4, 8);
    else if (nv <= 1536) ZB_CASE(3, 16);
    else if (nv <= 2048) ZB_CASE(4, 16);
    else ZB_CASE(8, 16);
}

template <typename F>
void backward_by_width(int64_t width, F&& f) {
    const int nv = static_cast<int>(width / 8);
    using std::integral_constant;
    if (nv <= 32) ZB_CASE(1, 1);
    else if (nv <= 64) ZB_CASE(2, 1);
    else if (nv <= 96) ZB_CASE(3, 1);
    else if (nv <= 128) ZB_CASE(2, 2);
    else if (nv <= 192) ZB_CASE(3, 2);
    else if (nv <= 256) ZB_CASE(2, 4);
    else if (nv <= 384) ZB_CASE(3, 4);
    else if (nv <= 512) ZB_CASE(2, 8);
    else if (nv <= 768) ZB_CASE(3, 8);
    else if (nv <= 1024) ZB_CASE(2, 16);
    else if (nv <= 1536) ZB_CASE(3, 16);
    else if (nv <= 2048) ZB_CASE(4, 16);
    else ZB_CASE(8, 16);
#undef ZB_CASE
}

// Vectors of 8 columns a cluster of W takes: the fewest, at least 4 (64 bytes a
// row), that leave no more than 32 clusters, which are resident at once.
int w_vecs(int64_t width) {
    int v = 4;
    while (width / 8 > 32LL * v) v *= 2;
    return v;
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
    cudaError_t err = cudaSuccess;
    auto go = [&](auto zero) {
        using T = decltype(zero);
        forward_by_width(n->width, [&](auto v, auto g) {
            constexpr int V = v(), G = g();
            err = launch_after(
                zb_layernorm_forward_kernel<T, V, G>, blocks_of(n->rows, Team<G>::ROWS), Team<G>::THREADS, 0, stream,
                    static_cast<const T*>(X), static_cast<const __nv_bfloat16*>(gamma),
                    static_cast<const __nv_bfloat16*>(beta), static_cast<__nv_bfloat16*>(Y), mean, rstd, n->rows,
                    static_cast<int>(n->width), n->eps);
        });
    };
    if (n->dtype == ZB_DT_BF16)
        go(__nv_bfloat16());
    else
        go(float());
    return launched("zb_layernorm_forward", err);
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
    cudaError_t err = cudaSuccess;
    auto go = [&](auto zero) {
        using T = decltype(zero);
        backward_by_width(n->width, [&](auto v, auto g) {
            constexpr int V = v(), G = g();
            err = launch_after(
                zb_layernorm_backward_input_kernel<T, V, G>, blocks_of(n->rows, Team<G>::ROWS), Team<G>::THREADS, 0,
                stream, static_cast<const __nv_bfloat16*>(dY), static_cast<const T*>(X),
                    static_cast<const __nv_bfloat16*>(gamma), mean, rstd, static_cast<const T*>(dR),
                    static_cast<T*>(dX), static_cast<__nv_bfloat16*>(dX16), n->rows, static_cast<int>(n->width));
        });
    };
    if (n->dtype == ZB_DT_BF16)
        go(__nv_bfloat16());
    else
        go(float());
    return launched("zb_layernorm_backward_input", err);
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
    const int vecs = w_vecs(n->width);
    const unsigned blocks = blocks_of(n->width, vecs * 8) * W_SPLIT;
    cudaError_t err = cudaSuccess;
    auto go = [&](auto zero) {
        using T = decltype(zero);
        err = launch_after(
            zb_layernorm_backward_weight_kernel<T>, blocks, W_THREADS, 0, stream, static_cast<const __nv_bfloat16*>(dY), static_cast<const T*>(X), mean, rstd, dgamma, dbeta, n->rows,
            static_cast<int>(n->width), vecs, accumulate != 0);
    };
    if (n->dtype == ZB_DT_BF16)
        go(__nv_bfloat16());
    else
        go(float());
    return launched("zb_layernorm_backward_weight", err);
}
