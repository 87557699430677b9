// fp8.cu — products in 8-bit floating point (e4m3) with an fp32 scale for each
// block of 128, dense or grouped by expert, and the quantisers that make their
// operands.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <string>

#include "gemm_core.cuh"

namespace {

constexpr int MAX_EXPERTS = 256;
constexpr int BLK = 128;

// The least power of two s with amax / s <= 448 = 1.75 * 2^8, at least 2^-126;
// 1 for amax = 0 and NaN for amax = inf or NaN.  With amax = m 2^x, 1 <= m < 2,
// s = 2^(x - 8) when m <= 1.75, else 2^(x - 7).  inv = 1 / s, exact.
__device__ __forceinline__ void block_scale(float amax, float& s, float& inv) {
    const uint32_t u = __float_as_uint(amax);
    if (u == 0u) {
        s = inv = 1.0f;
        return;
    }
    if (u >= 0x7f800000u) {
        s = inv = __uint_as_float(0x7fc00000u);
        return;
    }
    int x = static_cast<int>(u >> 23) - 8 + ((u & 0x007fffffu) > 0x00600000u ? 1 : 0);
    x = max(x, 1);  // biased exponent of s
    s = __uint_as_float(static_cast<uint32_t>(x) << 23);
    inv = __uint_as_float(static_cast<uint32_t>(254 - x) << 23);
}

// |x| as an integer: larger |x|, larger value; NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(__nv_bfloat16 x) { return (__bfloat16_as_ushort(x) & 0x7fffu) << 16; }

__device__ __forceinline__ uint8_t to_e4m3(float x) {
    return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float from_e4m3(uint8_t q) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
}

// One warp per 1 x 128 block.
__global__ void __launch_bounds__(256)
    zb_fp8_quantize_rows_kernel(const __nv_bfloat16* X, uint8_t* Q, float* S, long long rows, int cols, int blocks) {
    const long long item = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
    if (item >= rows * blocks) return;
    const int lane = threadIdx.x % 32;
    const long long r = item / blocks;
    const int b = static_cast<int>(item - r * blocks);
    uint32_t top = 0;
    for (int c = b * BLK + lane; c < min((b + 1) * BLK, cols); c += 32) top = max(top, magnitude(X[r * cols + c]));
    float s, inv;
    block_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, top)), s, inv);
    for (int c = b * BLK + lane; c < min((b + 1) * BLK, cols); c += 32)
        Q[r * cols + c] = to_e4m3(__bfloat162float(X[r * cols + c]) * inv);
    if (lane == 0) S[r * blocks + b] = s;
}

// One block of threads per 128 x 128 block.
__global__ void __launch_bounds__(256)
    zb_fp8_quantize_weight_kernel(const __nv_bfloat16* W, uint8_t* Q, float* S, uint8_t* QT, float* ST, int rows,
                                  int cols) {
    __shared__ uint32_t top;
    const int rb = blockIdx.y, cb = blockIdx.x;
    const int e = blockIdx.z;
    const long long base = static_cast<long long>(e) * rows * cols;
    const int r1 = min(rows, (rb + 1) * BLK), c1 = min(cols, (cb + 1) * BLK);
    if (threadIdx.x == 0) top = 0;
    __syncthreads();
    uint32_t m = 0;
    for (int r = rb * BLK + threadIdx.x / 128; r < r1; r += 2) {
        const int c = cb * BLK + threadIdx.x % 128;
        if (c < c1) m = max(m, magnitude(W[base + static_cast<long long>(r) * cols + c]));
    }
    atomicMax(&top, m);
    __syncthreads();
    float s, inv;
    block_scale(__uint_as_float(top), s, inv);
    for (int r = rb * BLK + threadIdx.x / 128; r < r1; r += 2) {
        const int c = cb * BLK + threadIdx.x % 128;
        if (c >= c1) continue;
        const uint8_t q = to_e4m3(__bfloat162float(W[base + static_cast<long long>(r) * cols + c]) * inv);
        if (Q) Q[base + static_cast<long long>(r) * cols + c] = q;
        if (QT) QT[base + static_cast<long long>(c) * rows + r] = q;
    }
    if (threadIdx.x == 0) {
        const int RB = gridDim.y, CB = gridDim.x;
        if (Q) S[(static_cast<long long>(e) * RB + rb) * CB + cb] = s;
        if (QT) ST[(static_cast<long long>(e) * CB + cb) * RB + rb] = s;
    }
}

struct MatmulArgs {
    const uint8_t *A, *B;
    const float *sa, *sb;
    const __nv_bfloat16 *bias, *aux;
    __nv_bfloat16 *out0, *out1;
    const int* offsets;
    int rows, N, K, epi, act;
};

__global__ void __launch_bounds__(256) zb_fp8_simple_kernel(const MatmulArgs a) {
    constexpr int TM = 64, TN = 64, TK = 16;
    __shared__ float As[TK][TM + 4], Bs[TK][TN + 4];
    const int e = blockIdx.y;
    int lo = 0, hi = a.rows;
    if (a.offsets) {
        lo = min(max(a.offsets[e], 0), a.rows);
        hi = max(min(a.offsets[e + 1], a.rows), lo);
    }
    const int KB = (a.K + BLK - 1) / BLK, NB = (a.N + BLK - 1) / BLK;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int n0 = blockIdx.x * TN;
    const uint8_t* B = a.B + static_cast<long long>(e) * a.N * a.K;
    const float* sb = a.sb + static_cast<long long>(e) * NB * KB;
    for (int m0 = lo + blockIdx.z * TM; m0 < hi; m0 += gridDim.z * TM) {
        float acc[4][4] = {}, part[4][4] = {};
        for (int k0 = 0; k0 < a.K; k0 += TK) {
            for (int i = tid; i < TK * TM; i += 256) {
                const int k = k0 + i % TK, m = m0 + i / TK, n = n0 + i / TK;
                As[i % TK][i / TK] = m < hi && k < a.K ? from_e4m3(a.A[static_cast<long long>(m) * a.K + k]) : 0.0f;
                Bs[i % TK][i / TK] = n < a.N && k < a.K ? from_e4m3(B[static_cast<long long>(n) * a.K + k]) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < TK; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], part[i][j]);
            __syncthreads();
            if ((k0 + TK) % BLK == 0 || k0 + TK >= a.K) {
                const int kb = k0 / BLK;
                for (int i = 0; i < 4; ++i) {
                    const int m = m0 + ty * 4 + i;
                    const float s = m < hi ? a.sa[static_cast<long long>(m) * KB + kb] : 0.0f;
                    for (int j = 0; j < 4; ++j) {
                        const int n = n0 + tx * 4 + j;
                        if (n < a.N) acc[i][j] = fmaf(s * sb[static_cast<long long>(n / BLK) * KB + kb], part[i][j], acc[i][j]);
                        part[i][j] = 0.0f;
                    }
                }
            }
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (m >= hi || n >= a.N) continue;
                const long long at = static_cast<long long>(m) * a.N + n;
                float x = acc[i][j];
                const bool tanh_form = a.act == ZB_ACT_GELU_TANH;
                if (a.bias) x += __bfloat162float(a.bias[static_cast<long long>(e) * a.N + n]);
                if (a.epi == ZB_FP8_GELU_GRAD) {
                    const float h = __bfloat162float(a.aux[at]);
                    x *= tanh_form ? gelu_grad_t<true>(h) : gelu_grad_t<false>(h);
                }
                a.out0[at] = __float2bfloat16_rn(x);
                if (a.epi == ZB_FP8_GELU) a.out1[at] = __float2bfloat16_rn(tanh_form ? gelu_t<true>(x) : gelu_t<false>(x));
            }
    }
}

// ---------------------------------------------------------------- host side
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

zb_status launched(const char* who) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string(who) + " launch: " + cudaGetErrorString(e));
    zb::clear_error();
    return ZB_OK;
}

}  // namespace

extern "C" zb_status zb_fp8_quantize_rows(int64_t rows, int64_t cols, const void* X, void* Q, float* S, void* stream) {
    if (rows < 0 || rows > (1LL << 30) || cols < 1 || cols > (1LL << 20))
        return zb::fail(ZB_ERR_SHAPE, "zb_fp8_quantize_rows: rows must be in [0, 2^30], cols in [1, 2^20]");
    if (cols % 16) return zb::fail(ZB_ERR_ALIGN, "zb_fp8_quantize_rows: cols must be a multiple of 16");
    if (rows == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    if (!X || !Q || !S) return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_quantize_rows: required pointer is NULL");
    if (off16(X) || off16(Q) || off4(S))
        return zb::fail(ZB_ERR_ALIGN, "zb_fp8_quantize_rows: pointers must be 16-byte aligned (S: 4)");
    const int blocks = static_cast<int>((cols + BLK - 1) / BLK);
    const long long grid = (rows * blocks + 7) / 8;
    if (grid > 0x7fffffffLL) return zb::fail(ZB_ERR_SHAPE, "zb_fp8_quantize_rows: too many elements");
    zb_fp8_quantize_rows_kernel<<<static_cast<unsigned>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const __nv_bfloat16*>(X), static_cast<uint8_t*>(Q), S, rows, static_cast<int>(cols), blocks);
    return launched("zb_fp8_quantize_rows");
}

extern "C" zb_status zb_fp8_quantize_weight(int32_t experts, int64_t rows, int64_t cols, const void* W, void* Q,
                                            float* S, void* QT, float* ST, void* stream) {
    if (experts < 1 || experts > MAX_EXPERTS || rows < 1 || cols < 1 || rows > (1LL << 20) || cols > (1LL << 20))
        return zb::fail(ZB_ERR_SHAPE, "zb_fp8_quantize_weight: experts must be in [1, 256], rows and cols in [1, 2^20]");
    if (rows % 16 || cols % 16)
        return zb::fail(ZB_ERR_ALIGN, "zb_fp8_quantize_weight: rows and cols must be multiples of 16");
    if (!W || (!Q && !QT) || !Q != !S || !QT != !ST)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_quantize_weight: W and a pair (Q, S) or (QT, ST) are required");
    if (off16(W) || off16(Q) || off16(QT) || off4(S) || off4(ST))
        return zb::fail(ZB_ERR_ALIGN, "zb_fp8_quantize_weight: pointers must be 16-byte aligned (S, ST: 4)");
    const dim3 grid(static_cast<unsigned>((cols + BLK - 1) / BLK), static_cast<unsigned>((rows + BLK - 1) / BLK),
                    static_cast<unsigned>(experts));
    zb_fp8_quantize_weight_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const __nv_bfloat16*>(W), static_cast<uint8_t*>(Q), S, static_cast<uint8_t*>(QT), ST,
        static_cast<int>(rows), static_cast<int>(cols));
    return launched("zb_fp8_quantize_weight");
}

extern "C" zb_status zb_fp8_matmul(const zb_fp8_gemm* g, const int32_t* offsets, const void* Xq, const float* xs,
                                   const void* Wq, const float* ws, const void* bias, const void* H, void* out0,
                                   void* out1, void* stream) {
    if (!g) return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: descriptor is NULL");
    if (g->reserved) return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: reserved must be 0");
    if (g->epilogue < ZB_FP8_STORE || g->epilogue > ZB_FP8_GELU_GRAD)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: unknown epilogue");
    if (g->epilogue != ZB_FP8_STORE && g->act != ZB_ACT_GELU_ERF && g->act != ZB_ACT_GELU_TANH)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: a GeLU epilogue needs a GeLU activation");
    if (g->experts < 1 || g->experts > MAX_EXPERTS || g->M < 0 || g->M > (1LL << 30) || g->N < 1 || g->K < 1 ||
        g->N > (1LL << 20) || g->K > (1LL << 20))
        return zb::fail(ZB_ERR_SHAPE, "zb_fp8_matmul: experts in [1, 256], M in [0, 2^30], N and K in [1, 2^20]");
    if (g->K % 16 || g->N % 8) return zb::fail(ZB_ERR_ALIGN, "zb_fp8_matmul: K must be a multiple of 16, N of 8");
    if (g->M == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    if (!Xq || !xs || !Wq || !ws || !out0 || (!offsets && g->experts != 1) || (g->epilogue == ZB_FP8_GELU && !out1) ||
        (g->epilogue == ZB_FP8_GELU_GRAD && !H))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: required pointer is NULL");
    if (bias && g->epilogue == ZB_FP8_GELU_GRAD)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: the GeLU' epilogue takes no bias");
    if (off16(offsets) || off16(Xq) || off4(xs) || off16(Wq) || off4(ws) || off16(bias) || off16(H) || off16(out0) ||
        off16(out1))
        return zb::fail(ZB_ERR_ALIGN, "zb_fp8_matmul: pointers must be 16-byte aligned (scales: 4)");
    MatmulArgs a;
    a.A = static_cast<const uint8_t*>(Xq);
    a.B = static_cast<const uint8_t*>(Wq);
    a.sa = xs;
    a.sb = ws;
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.aux = static_cast<const __nv_bfloat16*>(H);
    a.out0 = static_cast<__nv_bfloat16*>(out0);
    a.out1 = static_cast<__nv_bfloat16*>(out1);
    a.offsets = offsets;
    a.rows = static_cast<int>(g->M);
    a.N = static_cast<int>(g->N);
    a.K = static_cast<int>(g->K);
    a.epi = g->epilogue;
    a.act = g->act;
    const dim3 grid(static_cast<unsigned>((g->N + 63) / 64), static_cast<unsigned>(g->experts), 8);
    zb_fp8_simple_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched("zb_fp8_matmul");
}
