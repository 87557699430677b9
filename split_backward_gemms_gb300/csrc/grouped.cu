// grouped.cu — matrix products grouped by expert with ragged rows: F, B and W
// of a mixture-of-experts stage's blocks.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <string>

#include "gemm_core.cuh"

namespace {

constexpr int MAX_EXPERTS = 256;
constexpr int TM = 64, TN = 64, TK = 16;

// Rows [lo, hi) of expert e, kept inside [0, rows] whatever the offsets say.
__device__ __forceinline__ void expert_rows(const int* offsets, int e, int rows, int& lo, int& hi) {
    lo = min(max(offsets[e], 0), rows);
    hi = max(min(offsets[e + 1], rows), lo);
}

struct SimpleArgs {
    const __nv_bfloat16* A;   // [rows, K]
    const __nv_bfloat16* W;   // element (k, n) of expert e at e * K * N + k * sk + n * sn
    long long sk, sn;
    const __nv_bfloat16* bias;  // [E, N]
    const __nv_bfloat16* aux;   // [rows, N]
    __nv_bfloat16 *out0, *out1;
    const int* offsets;
    int rows, N, K, epi, act;
};

__device__ __forceinline__ float gelu_of(float x, int act) {
    return act == ZB_ACT_GELU_TANH ? gelu_t<true>(x) : gelu_t<false>(x);
}
__device__ __forceinline__ float gelu_grad_of(float x, int act) {
    return act == ZB_ACT_GELU_TANH ? gelu_grad_t<true>(x) : gelu_grad_t<false>(x);
}

__global__ void __launch_bounds__(256) zb_moe_rows_simple_kernel(const SimpleArgs a) {
    __shared__ float As[TK][TM + 4], Bs[TK][TN + 4];
    int lo, hi;
    expert_rows(a.offsets, blockIdx.y, a.rows, lo, hi);
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int n0 = blockIdx.x * TN;
    const __nv_bfloat16* W = a.W + static_cast<long long>(blockIdx.y) * a.K * a.N;
    for (int m0 = lo + blockIdx.z * TM; m0 < hi; m0 += gridDim.z * TM) {
        float acc[4][4] = {};
        for (int k0 = 0; k0 < a.K; k0 += TK) {
            for (int i = tid; i < TK * TM; i += 256) {
                const int m = m0 + i / TK, k = k0 + i % TK;
                As[i % TK][i / TK] = m < hi && k < a.K ? __bfloat162float(a.A[static_cast<long long>(m) * a.K + k]) : 0.0f;
                const int n = n0 + i % TN, kb = k0 + i / TN;
                Bs[i / TN][i % TN] = n < a.N && kb < a.K ? __bfloat162float(W[kb * a.sk + n * a.sn]) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < TK; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], acc[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (m >= hi || n >= a.N) continue;
                const long long at = static_cast<long long>(m) * a.N + n;
                float x = acc[i][j];
                if (a.bias) x += __bfloat162float(a.bias[static_cast<long long>(blockIdx.y) * a.N + n]);
                if (a.epi == zb::EPI_GELU_BWD) x *= gelu_grad_of(__bfloat162float(a.aux[at]), a.act);
                a.out0[at] = __float2bfloat16_rn(x);
                if (a.epi == zb::EPI_GELU_DUAL) a.out1[at] = __float2bfloat16_rn(gelu_of(x, a.act));
            }
    }
}

// dW[e][m][n] (+)= sum over the rows r of e of A[r][m] B[r][n]
__global__ void __launch_bounds__(256)
    zb_moe_wgrad_simple_kernel(const __nv_bfloat16* A, const __nv_bfloat16* B, float* dW, const int* offsets, int rows,
                               int M, int N, int accumulate) {
    __shared__ float As[TK][TM], Bs[TK][TN];
    int lo, hi;
    expert_rows(offsets, blockIdx.z, rows, lo, hi);
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TN;
    float acc[4][4] = {};
    for (int r0 = lo; r0 < hi; r0 += TK) {
        for (int i = tid; i < TK * TM; i += 256) {
            const int r = r0 + i / TM, m = m0 + i % TM, n = n0 + i % TN;
            As[i / TM][i % TM] = r < hi && m < M ? __bfloat162float(A[static_cast<long long>(r) * M + m]) : 0.0f;
            Bs[i / TN][i % TN] = r < hi && n < N ? __bfloat162float(B[static_cast<long long>(r) * N + n]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < TK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= M || n >= N) continue;
            float* d = dW + (static_cast<long long>(blockIdx.z) * M + m) * N + n;
            *d = accumulate ? *d + acc[i][j] : acc[i][j];
        }
}

// db[e][n] (+)= sum over the rows of e of X[r][n]: a block takes 64 columns of
// one expert; 4 row groups in ascending rows, then added in group order.
__global__ void __launch_bounds__(256)
    zb_moe_colsum_kernel(const __nv_bfloat16* X, float* db, const int* offsets, int rows, int N, int accumulate) {
    __shared__ float part[4][64];
    int lo, hi;
    expert_rows(offsets, blockIdx.y, rows, lo, hi);
    const int c = threadIdx.x % 64, g = threadIdx.x / 64, n = blockIdx.x * 64 + c;
    float s = 0.0f;
    if (n < N)
#pragma unroll 8
        for (int r = lo + g; r < hi; r += 4) s += __bfloat162float(X[static_cast<long long>(r) * N + n]);
    part[g][c] = s;
    __syncthreads();
    if (g == 0 && n < N) {
        s = ((part[0][c] + part[1][c]) + part[2][c]) + part[3][c];
        float* d = db + static_cast<long long>(blockIdx.y) * N + n;
        *d = accumulate ? *d + s : s;
    }
}

// ---------------------------------------------------------------- host side
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

zb_status check_moe(const zb_moe* m) {
    if (!m) return zb::fail(ZB_ERR_INVALID_ARG, "moe is NULL");
    if (m->flags) return zb::fail(ZB_ERR_INVALID_ARG, "moe.flags must be 0");
    if (m->act < ZB_ACT_NONE || m->act > ZB_ACT_GELU_TANH) return zb::fail(ZB_ERR_INVALID_ARG, "unknown activation");
    if (m->has_bias != 0 && m->has_bias != 1) return zb::fail(ZB_ERR_INVALID_ARG, "has_bias must be 0 or 1");
    if (m->experts < 1 || m->experts > MAX_EXPERTS) return zb::fail(ZB_ERR_SHAPE, "experts must be in [1, 256]");
    if (m->rows < 0 || m->rows > (1LL << 30)) return zb::fail(ZB_ERR_SHAPE, "rows must be in [0, 2^30]");
    if (m->h < 1 || m->f < 1 || m->h > (1LL << 20) || m->f > (1LL << 20))
        return zb::fail(ZB_ERR_SHAPE, "h and f must be in [1, 2^20]");
    if (m->h % 8 || m->f % 8) return zb::fail(ZB_ERR_ALIGN, "h and f must be multiples of 8");
    return ZB_OK;
}

zb_status launched(const char* who) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string(who) + " launch: " + cudaGetErrorString(e));
    return ZB_OK;
}

zb_status rows_product(const zb_moe& m, const int32_t* offsets, const void* A, const void* W, bool transposed,
                       int64_t N, int64_t K, const void* bias, const void* aux, int epi, void* out0, void* out1,
                       void* stream) {
    SimpleArgs a;
    a.A = static_cast<const __nv_bfloat16*>(A);
    a.W = static_cast<const __nv_bfloat16*>(W);
    a.sk = transposed ? 1 : N;
    a.sn = transposed ? K : 1;
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.aux = static_cast<const __nv_bfloat16*>(aux);
    a.out0 = static_cast<__nv_bfloat16*>(out0);
    a.out1 = static_cast<__nv_bfloat16*>(out1);
    a.offsets = offsets;
    a.rows = static_cast<int>(m.rows);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.epi = epi;
    a.act = m.act;
    const dim3 grid(static_cast<unsigned>((N + TN - 1) / TN), m.experts, 8);
    zb_moe_rows_simple_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched("grouped product");
}

}  // namespace

extern "C" zb_status zb_moe_forward(const zb_moe* m, const int32_t* offsets, const void* X, const void* W1,
                                    const void* W2, const void* b1, const void* b2, void* H_save, void* A_save,
                                    void* Y, void* stream) {
    zb_status s = check_moe(m);
    if (s != ZB_OK) return s;
    if (m->rows == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    const bool mlp = m->act != ZB_ACT_NONE;
    if (!offsets || !X || !W1 || !Y || (mlp && (!W2 || !H_save || !A_save)))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_forward: required pointer is NULL");
    if (m->has_bias && (!b1 || (mlp && !b2))) return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_forward: bias pointer is NULL");
    if (off16(offsets) || off16(X) || off16(W1) || off16(W2) || off16(b1) || off16(b2) || off16(H_save) ||
        off16(A_save) || off16(Y))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_forward: pointers must be 16-byte aligned");
    const void* bias1 = m->has_bias ? b1 : nullptr;
    if (!mlp) {
        s = rows_product(*m, offsets, X, W1, false, m->f, m->h, bias1, nullptr, zb::EPI_STORE_BF16, Y, nullptr, stream);
    } else {
        s = rows_product(*m, offsets, X, W1, false, m->f, m->h, bias1, nullptr, zb::EPI_GELU_DUAL, H_save, A_save, stream);
        if (s == ZB_OK)
            s = rows_product(*m, offsets, A_save, W2, false, m->h, m->f, m->has_bias ? b2 : nullptr, nullptr,
                             zb::EPI_STORE_BF16, Y, nullptr, stream);
    }
    if (s == ZB_OK) zb::clear_error();
    return s;
}

extern "C" zb_status zb_moe_backward_input(const zb_moe* m, const int32_t* offsets, const void* dY, const void* W1,
                                           const void* W2, const void* H_save, void* dH_out, void* dX, void* stream) {
    zb_status s = check_moe(m);
    if (s != ZB_OK) return s;
    if (m->rows == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    const bool mlp = m->act != ZB_ACT_NONE;
    if (!offsets || !dY || !W1 || !dX || (mlp && (!W2 || !H_save || !dH_out)))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_backward_input: required pointer is NULL");
    if (off16(offsets) || off16(dY) || off16(W1) || off16(W2) || off16(H_save) || off16(dH_out) || off16(dX))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_backward_input: pointers must be 16-byte aligned");
    if (!mlp) {
        s = rows_product(*m, offsets, dY, W1, true, m->h, m->f, nullptr, nullptr, zb::EPI_STORE_BF16, dX, nullptr, stream);
    } else {
        s = rows_product(*m, offsets, dY, W2, true, m->f, m->h, nullptr, H_save, zb::EPI_GELU_BWD, dH_out, nullptr, stream);
        if (s == ZB_OK)
            s = rows_product(*m, offsets, dH_out, W1, true, m->h, m->f, nullptr, nullptr, zb::EPI_STORE_BF16, dX,
                             nullptr, stream);
    }
    if (s == ZB_OK) zb::clear_error();
    return s;
}

extern "C" size_t zb_moe_workspace_bytes(const zb_moe* m) {
    if (check_moe(m) != ZB_OK) return 0;
    return static_cast<size_t>(m->experts) * 4 * 128;
}

extern "C" zb_status zb_moe_backward_weight(const zb_moe* m, const int32_t* offsets, const void* X, const void* A_save,
                                            const void* dH, const void* dY, float* dW1, float* dW2, float* db1,
                                            float* db2, int accumulate, void* workspace, size_t ws_bytes,
                                            void* stream) {
    zb_status s = check_moe(m);
    if (s != ZB_OK) return s;
    const bool mlp = m->act != ZB_ACT_NONE;
    if (!offsets || !dW1 || (mlp && !dW2) || (m->rows > 0 && (!X || !dY || (mlp && (!A_save || !dH)))))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_backward_weight: required pointer is NULL");
    if (m->has_bias && (!db1 || (mlp && !db2)))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_backward_weight: bias-gradient pointer is NULL");
    if (off16(offsets) || off16(X) || off16(A_save) || off16(dH) || off16(dY) || off16(dW1) || off16(dW2) ||
        off16(db1) || off16(db2))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_backward_weight: pointers must be 16-byte aligned");
    if (!workspace || ws_bytes < zb_moe_workspace_bytes(m))
        return zb::fail(ZB_ERR_WORKSPACE, "zb_moe_backward_weight: workspace missing or too small: need " +
                                              std::to_string(zb_moe_workspace_bytes(m)) + " bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_backward_weight: workspace must be 256-byte aligned");
    const int rows = static_cast<int>(m->rows), h = static_cast<int>(m->h), f = static_cast<int>(m->f);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto product = [&](const void* A, const void* B, float* dW, int M, int N) {
        const dim3 grid((N + TN - 1) / TN, (M + TM - 1) / TM, m->experts);
        zb_moe_wgrad_simple_kernel<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(A),
                                                         static_cast<const __nv_bfloat16*>(B), dW, offsets, rows, M, N,
                                                         accumulate ? 1 : 0);
        return launched("grouped weight gradient");
    };
    auto colsum = [&](const void* A, float* db, int N) {
        zb_moe_colsum_kernel<<<dim3((N + 63) / 64, m->experts), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(A), db,
                                                                              offsets, rows, N, accumulate ? 1 : 0);
        return launched("grouped column sums");
    };
    if (mlp) s = product(A_save, dY, dW2, f, h);
    if (s == ZB_OK) s = product(X, mlp ? dH : dY, dW1, h, f);
    if (s == ZB_OK && m->has_bias) s = colsum(mlp ? dH : dY, db1, f);
    if (s == ZB_OK && m->has_bias && mlp) s = colsum(dY, db2, h);
    if (s == ZB_OK) zb::clear_error();
    return s;
}
