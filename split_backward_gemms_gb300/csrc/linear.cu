// linear.cu — a linear map with its epilogue: D = X W (or X W^T) with bias,
// GeLU or GeLU', and a residual.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <string>

#include "gemm_core.cuh"

namespace {

struct LinearArgs {
    const __nv_bfloat16 *X, *W, *bias, *H;
    const void* R;
    void *out0, *out1;
    long long ldx, ldr, ldh, ldo, sk, sn;  // sk, sn: strides of W along K and N
    int M, N, K, epilogue, tanh_form, f32;
};

// 64 x 64 outputs a block, 16 along K at a time, 4 x 4 a thread.
__global__ void __launch_bounds__(256) zb_linear_simple_kernel(const LinearArgs a) {
    __shared__ float xs[16][65], ws[16][65];
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i / 16, k = i % 16;
            xs[k][r] = m0 + r < a.M && k0 + k < a.K ? __bfloat162float(a.X[(m0 + r) * a.ldx + k0 + k]) : 0.0f;
            ws[k][r] = n0 + r < a.N && k0 + k < a.K ? __bfloat162float(a.W[(k0 + k) * a.sk + (n0 + r) * a.sn]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long r = m0 + ty * 4 + i;
            const int n = n0 + tx * 4 + j;
            if (r >= a.M || n >= a.N) continue;
            float d = acc[i][j] + (a.bias ? __bfloat162float(a.bias[n]) : 0.0f);
            void* out = a.out0;
            if (a.epilogue == ZB_LINEAR_GELU) {
                if (a.out0) static_cast<__nv_bfloat16*>(a.out0)[r * a.ldo + n] = __float2bfloat16(d);
                d = a.tanh_form ? gelu_t<true>(d) : gelu_t<false>(d);
                out = a.out1;
            } else if (a.epilogue == ZB_LINEAR_GELU_GRAD) {
                const float h = __bfloat162float(a.H[r * a.ldh + n]);
                d *= a.tanh_form ? gelu_grad_t<true>(h) : gelu_grad_t<false>(h);
            }
            if (a.f32) {
                if (a.R) d += static_cast<const float*>(a.R)[r * a.ldr + n];
                static_cast<float*>(out)[r * a.ldo + n] = d;
            } else {
                if (a.R) d += __bfloat162float(static_cast<const __nv_bfloat16*>(a.R)[r * a.ldr + n]);
                static_cast<__nv_bfloat16*>(out)[r * a.ldo + n] = __float2bfloat16(d);
            }
        }
}

bool mis16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// A row stride given as 0 is the row's width; false if it is not legal.
bool stride(int64_t* ld, int64_t width) {
    if (*ld == 0) *ld = width;
    return *ld >= width && *ld <= (1LL << 30);
}

}  // namespace

extern "C" zb_status zb_linear_product(const zb_linear* g, const void* X, const void* W, const void* bias,
                                       const void* R, const void* H, void* out0, void* out1, void* stream) {
    if (!g) return zb::fail(ZB_ERR_INVALID_ARG, "zb_linear_product: descriptor is NULL");
    constexpr int64_t most = 1LL << 30;
    if (g->M < 0 || g->M > most || g->N < 1 || g->N > most || g->K < 1 || g->K > most)
        return zb::fail(ZB_ERR_SHAPE, "zb_linear_product: M must be in [0, 2^30], N and K in [1, 2^30]");
    if (g->N % 8 || g->K % 8) return zb::fail(ZB_ERR_ALIGN, "zb_linear_product: N and K must be multiples of 8");
    if ((g->transposed & ~1) || g->epilogue < ZB_LINEAR_STORE || g->epilogue > ZB_LINEAR_GELU_GRAD)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_linear_product: unknown transposed or epilogue");
    if (g->epilogue != ZB_LINEAR_STORE && g->act != ZB_ACT_GELU_ERF && g->act != ZB_ACT_GELU_TANH)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_linear_product: the GeLU epilogues need a GeLU activation");
    if (g->dtype != ZB_DT_BF16 && (g->dtype != ZB_DT_F32 || g->epilogue != ZB_LINEAR_STORE))
        return zb::fail(ZB_ERR_DTYPE, "zb_linear_product: dtype must be bf16, or fp32 with ZB_LINEAR_STORE");
    int64_t ldx = g->ldx, ldw = g->ldw, ldr = g->ldr, ldh = g->ldh, ldo = g->ldo;
    if (!stride(&ldx, g->K) || !stride(&ldw, g->transposed ? g->K : g->N) || !stride(&ldr, g->N) ||
        !stride(&ldh, g->N) || !stride(&ldo, g->N))
        return zb::fail(ZB_ERR_SHAPE, "zb_linear_product: a row stride is shorter than its row or above 2^30");
    if (ldx % 8 || ldw % 8 || ldr % 8 || ldh % 8 || ldo % 8)
        return zb::fail(ZB_ERR_ALIGN, "zb_linear_product: row strides must be multiples of 8");
    const bool grad = g->epilogue == ZB_LINEAR_GELU_GRAD, gelu = g->epilogue == ZB_LINEAR_GELU;
    if (grad && bias) return zb::fail(ZB_ERR_INVALID_ARG, "zb_linear_product: ZB_LINEAR_GELU_GRAD takes no bias");
    if (g->M == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    if (!X || !W || (grad && !H) || !(gelu ? out1 : out0))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_linear_product: required pointer is NULL");
    if (mis16(X) || mis16(W) || mis16(bias) || mis16(R) || mis16(H) || mis16(out0) || mis16(out1))
        return zb::fail(ZB_ERR_ALIGN, "zb_linear_product: pointers must be 16-byte aligned");
    LinearArgs a;
    a.X = static_cast<const __nv_bfloat16*>(X);
    a.W = static_cast<const __nv_bfloat16*>(W);
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.H = static_cast<const __nv_bfloat16*>(H);
    a.R = R;
    a.out0 = out0;
    a.out1 = out1;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldo = ldo;
    a.sk = g->transposed ? 1 : ldw;
    a.sn = g->transposed ? ldw : 1;
    a.M = static_cast<int>(g->M);
    a.N = static_cast<int>(g->N);
    a.K = static_cast<int>(g->K);
    a.epilogue = g->epilogue;
    a.tanh_form = g->act == ZB_ACT_GELU_TANH;
    a.f32 = g->dtype == ZB_DT_F32;
    const int64_t by = (g->M + 63) / 64;
    if (by > 65535) return zb::fail(ZB_ERR_SHAPE, "zb_linear_product: M too large");
    zb_linear_simple_kernel<<<dim3(static_cast<unsigned>((g->N + 63) / 64), static_cast<unsigned>(by)), 256, 0,
                              static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return zb::fail(ZB_ERR_CUDA, std::string("zb_linear_product launch: ") + cudaGetErrorString(e));
    zb::clear_error();
    return ZB_OK;
}
