// moe_route.cu — the router of a mixture-of-experts stage and what carries
// tokens to their rows and back: top-k gates, the order of rows by expert,
// dispatch, combine, and their gradients.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "ptx.cuh"
#include "zb_internal.h"

namespace {

constexpr int MAX_EXPERTS = 256;
constexpr int MAX_TOPK = 32;
constexpr unsigned FULL = 0xffffffffu;

// ---------------------------------------------------------------- top k
// Order-preserving key of a logit: larger logit, larger key.  0: no such
// expert (or already chosen); 1: -inf, never chosen; 2: NaN, chosen last.
// -0 and +0 are one value, so that their tie goes to the lower index.
__device__ __forceinline__ uint32_t key_of(float z) {
    if (z != z) return 2u;
    if (z == -INFINITY) return 1u;
    const uint32_t u = __float_as_uint(z + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return key == 2u ? __uint_as_float(0x7fc00000u)
                     : __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

template <typename T>
__device__ __forceinline__ float ld_logit(const T* p);
template <>
__device__ __forceinline__ float ld_logit<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float ld_logit<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

struct RouteArgs {
    const void* logits;
    long long tokens;
    int experts, topk, renorm, per_block;  // per_block: tokens of one block
    float* gates;
    int* expert;
    int* offsets;
    int* row_of;
    int* token_of;
    int* hist;  // [blocks, experts]
};

// A token's logits, element v * 32 + lane in z[v].
template <int VPL, typename T>
__device__ __forceinline__ void load_row(const RouteArgs& a, long long t, int lane, float (&z)[VPL]) {
    const T* p = static_cast<const T*>(a.logits) + t * a.experts;
#pragma unroll
    for (int v = 0; v < VPL; ++v) z[v] = v * 32 + lane < a.experts ? ld_logit<T>(p + v * 32 + lane) : -INFINITY;
}

// One warp chooses for one token.  A lane first sorts its elements by
// descending key (adjacent exchanges of strictly larger keys, so equal ones
// stay in the order of their indices).  Each of the k rounds then takes the
// largest first key (a warp maximum) and among its holders the lowest index (a
// warp minimum), and that lane drops its first element; lane j keeps choice j.
// Softmax statistics and gates are fp32.  The work is instructions, not bytes:
// about 490 a warp and token with 128 experts and k = 8, against 0.5 KB read, and
// choosing for 16384 such tokens takes 12 us where reading them takes 1.6.
template <int VPL>
__device__ __forceinline__ void choose(const RouteArgs& a, long long t, int lane, const float (&z)[VPL], int* cnt) {
    uint32_t key[VPL], at[VPL];
    bool nan = false;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        key[v] = v * 32 + lane < a.experts ? key_of(z[v]) : 0u;
        at[v] = v;
        nan |= key[v] == 2u;
    }
    nan = __any_sync(FULL, nan);
#pragma unroll
    for (int n = VPL - 1; n > 0; --n)
#pragma unroll
        for (int v = 0; v < n; ++v) {
            const bool swap = key[v + 1] > key[v];
            const uint32_t k = key[v], i = at[v];
            key[v] = swap ? key[v + 1] : k;
            at[v] = swap ? at[v + 1] : i;
            key[v + 1] = swap ? k : key[v + 1];
            at[v + 1] = swap ? i : at[v + 1];
        }
    uint32_t order = 0;  // four bits an element, the first lowest
#pragma unroll
    for (int v = 0; v < VPL; ++v) order |= at[v] << (4 * v);
    int mine = -1;
    uint32_t won = 0u;
    for (int j = 0; j < a.topk; ++j) {
        const uint32_t m = __reduce_max_sync(FULL, key[0]);
        if (m < 2u) break;
        const int i = static_cast<int>((order & 15u) * 32u) + lane;
        const int e = __reduce_min_sync(FULL, key[0] == m ? i : 0x7fffffff);
        if (i == e) {
#pragma unroll
            for (int v = 0; v < VPL; ++v) key[v] = v + 1 < VPL ? key[v + 1] : 0u;
            order >>= 4;
        }
        if (lane == j) {
            mine = e;
            won = m;
        }
    }
    const float val = logit_of(won), top = __shfl_sync(FULL, val, 0);
    const float w = mine >= 0 ? expf(val - top) : 0.0f;
    float total = w;
    if (!a.renorm) {
        total = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) total += v * 32 + lane < a.experts ? expf(z[v] - top) : 0.0f;
    }
    total = warp_sum(total);
    if (lane < a.topk) {
        a.gates[t * a.topk + lane] = mine < 0 ? 0.0f : nan ? __uint_as_float(0x7fc00000u) : w / total;
        a.expert[t * a.topk + lane] = mine;
        if (mine >= 0) atomicAdd(&cnt[mine], 1);  // integer sums: no order
    }
}

// Every warp's tokens of [t0, t1); the next token's logits are on their way
// while one is worked on.
template <int VPL, typename T>
__device__ __forceinline__ void choose_all(const RouteArgs& a, long long t0, long long t1, int* cnt) {
    const int lane = threadIdx.x & 31, step = blockDim.x / 32;
    long long t = t0 + (threadIdx.x >> 5);
    float z[VPL], zn[VPL];
    if (t < t1) load_row<VPL, T>(a, t, lane, z);
    for (; t < t1; t += step) {
        if (t + step < t1) load_row<VPL, T>(a, t + step, lane, zn);
        choose<VPL>(a, t, lane, z, cnt);
#pragma unroll
        for (int v = 0; v < VPL; ++v) z[v] = zn[v];
    }
}

// Exclusive prefix of n[0..255] (one warp; n holds the prefixes after).
// Returns the total.
__device__ __forceinline__ int scan_experts(int* n, int lane) {
    int v[MAX_EXPERTS / 32], sum = 0;
#pragma unroll
    for (int i = 0; i < MAX_EXPERTS / 32; ++i) {
        v[i] = n[lane * (MAX_EXPERTS / 32) + i];
        sum += v[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += u;
    }
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < MAX_EXPERTS / 32; ++i) {
        n[lane * (MAX_EXPERTS / 32) + i] = run;
        run += v[i];
    }
    return __shfl_sync(FULL, incl, 31);
}

constexpr int ROUTE_THREADS = 1024;
constexpr int SUB = 128;  // tokens whose ranks are counted at once

// Rows of the tokens [t0, t1): base[e] is the first free row of expert e.  A
// token chooses an expert at most once, so a choice's rank among 128 tokens is
// the number of lower bits of its expert's 128-bit mask: no order of atomics
// can change it.
// Choices of 128 tokens that a thread has, at most (the small kernel's smaller
// blocks have no more than one a thread).
constexpr int PER_THREAD = SUB * MAX_TOPK / ROUTE_THREADS;

// The thread's choices among the tokens [s, min(s + SUB, t1)).
__device__ __forceinline__ int load_choices(const RouteArgs& a, long long s, long long t1, int (&e)[PER_THREAD]) {
    const int n = static_cast<int>(min(t1 - s, static_cast<long long>(SUB))) * a.topk;
#pragma unroll
    for (int u = 0; u < PER_THREAD; ++u) {
        const int i = threadIdx.x + u * blockDim.x;
        e[u] = i < n ? a.expert[s * a.topk + i] : -1;
    }
    return n;
}

// e: load_choices() of the first SUB tokens.
__device__ __forceinline__ void place(const RouteArgs& a, long long t0, long long t1, int (&e)[PER_THREAD], int* base,
                                      unsigned (*mask)[SUB / 32]) {
    const int tid = threadIdx.x;
    for (long long s = t0; s < t1; s += SUB) {
        if (s > t0) load_choices(a, s, t1, e);
        const int n = static_cast<int>(min(t1 - s, static_cast<long long>(SUB))) * a.topk;
        for (int i = tid; i < MAX_EXPERTS * (SUB / 32); i += blockDim.x) (&mask[0][0])[i] = 0u;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < PER_THREAD; ++u) {
            const int tl = (tid + u * static_cast<int>(blockDim.x)) / a.topk;
            if (e[u] >= 0) atomicOr(&mask[e[u]][tl >> 5], 1u << (tl & 31));
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < PER_THREAD; ++u) {
            const int i = tid + u * static_cast<int>(blockDim.x);
            if (i >= n) break;
            const int tl = i / a.topk;
            int row = -1;
            if (e[u] >= 0) {
                row = base[e[u]];
#pragma unroll
                for (int w = 0; w < SUB / 32; ++w) {
                    const unsigned m = mask[e[u]][w];
                    const int lo = tl - w * 32;  // tokens below this one in word w
                    row += __popc(lo >= 32 ? m : lo > 0 ? m & ((1u << lo) - 1u) : 0u);
                }
                a.token_of[row] = static_cast<int>(s + tl);
            }
            a.row_of[s * a.topk + i] = row;
        }
        __syncthreads();
        if (tid < MAX_EXPERTS) {
            int c = 0;
#pragma unroll
            for (int w = 0; w < SUB / 32; ++w) c += __popc(mask[tid][w]);
            base[tid] += c;
        }
        __syncthreads();
    }
}

// Kernel 1 of 2: choices and gates, and this block's count of each expert.
template <int VPL, typename T>
__global__ void __launch_bounds__(ROUTE_THREADS) zb_moe_choose_kernel(const RouteArgs a) {
    __shared__ int cnt[MAX_EXPERTS];
    const int tid = threadIdx.x;
    if (tid < MAX_EXPERTS) cnt[tid] = 0;
    zbp::allow_dependent_launch();
    __syncthreads();
    const long long t0 = static_cast<long long>(blockIdx.x) * a.per_block;
    const long long t1 = min(t0 + a.per_block, a.tokens);
    choose_all<VPL, T>(a, t0, t1, cnt);
    __syncthreads();
    if (tid < a.experts) a.hist[static_cast<long long>(blockIdx.x) * a.experts + tid] = cnt[tid];
}

// Kernel 2 of 2: every block sums the counts of all blocks (at most one per SM,
// so this is a few KB from L2 and cheaper than a third kernel), which gives the
// experts' offsets and the first row of each expert in this block.  Both kernels:
// 16.4 us for 16384 tokens, 128 experts, k = 8.
__global__ void __launch_bounds__(ROUTE_THREADS) zb_moe_place_kernel(const RouteArgs a) {
    __shared__ int base[MAX_EXPERTS], before[MAX_EXPERTS];
    __shared__ unsigned mask[MAX_EXPERTS][SUB / 32];
    __shared__ int total;
    const int tid = threadIdx.x;
    if (tid < MAX_EXPERTS) base[tid] = before[tid] = 0;
    __syncthreads();
    zbp::grid_dependency_wait();
    const long long t0 = static_cast<long long>(blockIdx.x) * a.per_block;
    const long long t1 = min(t0 + a.per_block, a.tokens);
    int mine[PER_THREAD];
    load_choices(a, t0, t1, mine);
    const int blocks = gridDim.x;
    // as many threads an expert as fit, each with every such-th block
    const int lg = 32 - __clz(a.experts - 1 | 1);  // 2^lg >= experts
    const int e = tid & ((1 << lg) - 1), step = ROUTE_THREADS >> lg;
    if (e < a.experts) {
        int all = 0, lower = 0;
#pragma unroll 8
        for (int b = tid >> lg; b < blocks; b += step) {
            const int c = a.hist[b * a.experts + e];
            all += c;
            lower += b < static_cast<int>(blockIdx.x) ? c : 0;
        }
        atomicAdd(&base[e], all);
        atomicAdd(&before[e], lower);
    }
    __syncthreads();
    if (tid < 32) {
        const int sum = scan_experts(base, tid);
        if (tid == 0) total = sum;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (tid < a.experts) a.offsets[tid] = base[tid];
        if (tid == 0) a.offsets[a.experts] = total;
    }
    const long long rows = a.tokens * a.topk;
    for (long long p = total + static_cast<long long>(blockIdx.x) * ROUTE_THREADS + tid; p < rows;
         p += static_cast<long long>(blocks) * ROUTE_THREADS)
        a.token_of[p] = -1;
    __syncthreads();
    if (tid < MAX_EXPERTS) base[tid] += before[tid];
    __syncthreads();
    place(a, t0, t1, mine, base, mask);
}

// Few tokens: one block does all of it in one launch, whose latency is what
// it costs (16 tokens, 64 experts, k = 6: 3.1 us, 5.7 with the call).
template <int VPL, typename T>
__global__ void __launch_bounds__(ROUTE_THREADS) zb_moe_route_small_kernel(const RouteArgs a) {
    __shared__ int base[MAX_EXPERTS];
    __shared__ unsigned mask[MAX_EXPERTS][SUB / 32];
    __shared__ int total;
    const int tid = threadIdx.x;
    if (tid < MAX_EXPERTS) base[tid] = 0;
    __syncthreads();
    choose_all<VPL, T>(a, 0, a.tokens, base);
    __syncthreads();  // also: the block's expert[] is visible to all of it
    int e[PER_THREAD];
    load_choices(a, 0, a.tokens, e);
    if (tid < 32) {
        const int sum = scan_experts(base, tid);
        if (tid == 0) total = sum;
    }
    __syncthreads();
    if (tid < a.experts) a.offsets[tid] = base[tid];
    if (tid == 0) a.offsets[a.experts] = total;
    for (long long p = total + tid; p < a.tokens * a.topk; p += blockDim.x) a.token_of[p] = -1;
    place(a, 0, a.tokens, e, base, mask);
}

// ---------------------------------------------------------------- gradient
__device__ __forceinline__ void st_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// One warp per token; lane j holds choice j, lane i mod 32 holds dz_i.  8191
// tokens of 60 bf16 logits, k = 4: 4.9 us, of which about 3 are any launch's.
template <int VPL, typename T>
__global__ void __launch_bounds__(256)
    zb_moe_route_backward_kernel(const T* __restrict__ logits, const int* __restrict__ expert,
                                 const float* __restrict__ gates, const float* __restrict__ dgates,
                                 T* __restrict__ dlogits, long long tokens, int experts, int topk, int renorm) {
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= tokens) return;
    int e = -1;
    float g = 0.0f, dg = 0.0f;
    if (lane < topk) {
        e = expert[t * topk + lane];
        if (e >= 0) {
            g = gates[t * topk + lane];
            dg = dgates[t * topk + lane];
        }
    }
    const float inner = warp_sum(e >= 0 ? g * dg : 0.0f);
    const float mine = renorm ? g * (dg - inner) : g * dg;
    float dz[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) dz[v] = 0.0f;
    if (!renorm) {
        float z[VPL], top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int i = v * 32 + lane;
            z[v] = i < experts ? ld_logit<T>(logits + t * experts + i) : -INFINITY;
            top = fmaxf(top, z[v]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
        unsigned live = 0u;  // a bit an element: not -inf
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            live |= (z[v] != -INFINITY ? 1u : 0u) << v;
            z[v] = expf(z[v] - top);
            total += z[v];
        }
        total = warp_sum(total);
        // Logits of -inf get zeros whatever total and inner are: a NaN or an
        // infinity times the weight of 0 would be NaN.
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const float d = -(z[v] / total) * inner;
            dz[v] = (live >> v) & 1u ? d : 0.0f;
        }
    }
    for (int j = 0; j < topk; ++j) {
        const int ej = __shfl_sync(FULL, e, j);
        const float d = __shfl_sync(FULL, mine, j);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (v * 32 + lane == ej) dz[v] += d;
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        if (v * 32 + lane < experts) st_logit(dlogits + t * experts + v * 32 + lane, dz[v]);
}

// ---------------------------------------------------------------- rows
__device__ __forceinline__ float2 bf2(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void fma8(float (&acc)[8], float g, const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf2(w[i]);
        acc[2 * i] = fmaf(g, f.x, acc[2 * i]);
        acc[2 * i + 1] = fmaf(g, f.y, acc[2 * i + 1]);
    }
}

// HBM-bound.  One warp copies up to 1024 columns of one token: 4 x 16 bytes a
// lane in flight, read once and stored to each of the token's rows.  8192 tokens
// of 4096 to 2 rows each: 33.3 us, 6.0 TB/s.
constexpr int COPY_U = 4;
__global__ void __launch_bounds__(256)
    zb_moe_dispatch_kernel(const uint4* __restrict__ X, const int* __restrict__ row_of, uint4* __restrict__ Xp,
                           long long tokens, int topk, int w8, int segs) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (item >= tokens * segs) return;
    const long long t = item / segs;
    const int c0 = static_cast<int>(item - t * segs) * 32 * COPY_U + lane;
    const long long rows = tokens * topk;
    const int mine = lane < topk ? row_of[t * topk + lane] : -1;
    uint4 v[COPY_U];
#pragma unroll
    for (int u = 0; u < COPY_U; ++u)
        if (c0 + u * 32 < w8) v[u] = __ldg(X + t * w8 + c0 + u * 32);
    for (int j = 0; j < topk; ++j) {
        const long long r = __shfl_sync(FULL, mine, j);
        if (r < 0 || r >= rows) continue;
#pragma unroll
        for (int u = 0; u < COPY_U; ++u)
            if (c0 + u * 32 < w8) Xp[r * w8 + c0 + u * 32] = v[u];
    }
}

// HBM-bound: a token's rows are read once and summed in fp32 in the order of its
// choices.  One warp takes up to 512 columns of a token, 2 x 16 bytes of each of 4
// rows in flight a lane (one, or all 8 rows at once, were no faster).  4099
// tokens, 8 rows of 2048 each: 29.2 us, 5.2 TB/s.
constexpr int SUM_U = 2;
__global__ void __launch_bounds__(256)
    zb_moe_combine_kernel(const uint4* __restrict__ Yp, const int* __restrict__ row_of,
                          const float* __restrict__ gates, uint4* __restrict__ Y, long long tokens, int topk,
                          int w8, int segs) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (item >= tokens * segs) return;
    const long long t = item / segs;
    const int c0 = static_cast<int>(item - t * segs) * 32 * SUM_U + lane;
    const long long rows = tokens * topk;
    int mine = -1;
    float gate = 1.0f;
    if (lane < topk) {
        mine = row_of[t * topk + lane];
        if (gates) gate = gates[t * topk + lane];
    }
    float acc[SUM_U][8];
#pragma unroll
    for (int u = 0; u < SUM_U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u][i] = 0.0f;
#pragma unroll 4
    for (int j = 0; j < topk; ++j) {
        const long long r = __shfl_sync(FULL, mine, j);
        const float g = __shfl_sync(FULL, gate, j);
        if (r < 0 || r >= rows) continue;
#pragma unroll
        for (int u = 0; u < SUM_U; ++u)
            if (c0 + u * 32 < w8) fma8(acc[u], g, __ldg(Yp + r * w8 + c0 + u * 32));
    }
#pragma unroll
    for (int u = 0; u < SUM_U; ++u)
        if (c0 + u * 32 < w8)
            Y[t * w8 + c0 + u * 32] = make_uint4(pack2(acc[u][0], acc[u][1]), pack2(acc[u][2], acc[u][3]),
                                                 pack2(acc[u][4], acc[u][5]), pack2(acc[u][6], acc[u][7]));
}

// dYp[row_j] = g_j dY, dg_j = <dY, Yp[row_j]>, both from one pass: HBM-bound (8192
// tokens, 2 rows of 4096 each: 54.2 us, 6.2 TB/s).  WPT warps share a token; each
// choice's dot product is summed over a lane's columns, the lanes (a fixed tree)
// and the warps in order.  dY is read again for each choice, from L1 or L2.
template <int WPT>
__global__ void __launch_bounds__(256)
    zb_moe_combine_backward_kernel(const uint4* __restrict__ dY, const uint4* __restrict__ Yp,
                                   const int* __restrict__ row_of, const float* __restrict__ gates,
                                   uint4* __restrict__ dYp, float* __restrict__ dgates, long long tokens, int topk,
                                   int w8) {
    __shared__ float part[8][MAX_TOPK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t = static_cast<long long>(blockIdx.x) * (8 / WPT) + warp / WPT;
    const long long rows = tokens * topk;
    if (t < tokens) {
        int mine = -1;
        float gate = 0.0f;
        if (lane < topk) {
            mine = row_of[t * topk + lane];
            gate = gates[t * topk + lane];
        }
        for (int j = 0; j < topk; ++j) {
            const long long r = __shfl_sync(FULL, mine, j);
            const float g = __shfl_sync(FULL, gate, j);
            float dot = 0.0f;
            if (r >= 0 && r < rows) {
#pragma unroll 2
                for (int c = (warp % WPT) * 32 + lane; c < w8; c += WPT * 32) {
                    const uint4 d = __ldg(dY + t * w8 + c);
                    const uint4 y = __ldg(Yp + r * w8 + c);
                    const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, yw[4] = {y.x, y.y, y.z, y.w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = bf2(dw[i]), b = bf2(yw[i]);
                        dot = fmaf(a.x, b.x, dot);
                        dot = fmaf(a.y, b.y, dot);
                        o[i] = pack2(g * a.x, g * a.y);
                    }
                    dYp[r * w8 + c] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            dot = warp_sum(dot);
            if (lane == 0) part[warp][j] = dot;
        }
    }
    __syncthreads();
    if (t < tokens && warp % WPT == 0 && lane < topk) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WPT; ++w) s += part[warp + w][lane];
        dgates[t * topk + lane] = s;
    }
}

// ---------------------------------------------------------------- host side
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

zb_status check_router(const zb_router* r) {
    if (!r) return zb::fail(ZB_ERR_INVALID_ARG, "router is NULL");
    if (r->experts < 1 || r->experts > MAX_EXPERTS) return zb::fail(ZB_ERR_SHAPE, "experts must be in [1, 256]");
    if (r->topk < 1 || r->topk > MAX_TOPK || r->topk > r->experts)
        return zb::fail(ZB_ERR_SHAPE, "topk must be in [1, min(experts, 32)]");
    if (r->tokens < 0 || r->tokens > (1LL << 30) / r->topk)
        return zb::fail(ZB_ERR_SHAPE, "tokens * topk must be in [0, 2^30]");
    if (r->dtype != ZB_DT_F32 && r->dtype != ZB_DT_BF16) return zb::fail(ZB_ERR_DTYPE, "unknown dtype of the logits");
    if (r->renorm != 0 && r->renorm != 1) return zb::fail(ZB_ERR_INVALID_ARG, "renorm must be 0 or 1");
    return ZB_OK;
}

zb_status check_rows(const char* who, int64_t tokens, int32_t topk, int64_t width) {
    if (topk < 1 || topk > MAX_TOPK) return zb::fail(ZB_ERR_SHAPE, std::string(who) + ": topk must be in [1, 32]");
    if (tokens < 0 || tokens > (1LL << 30) / topk)
        return zb::fail(ZB_ERR_SHAPE, std::string(who) + ": tokens * topk must be in [0, 2^30]");
    if (width < 1 || width > (1LL << 24)) return zb::fail(ZB_ERR_SHAPE, std::string(who) + ": width must be in [1, 2^24]");
    if (width % 8) return zb::fail(ZB_ERR_ALIGN, std::string(who) + ": width must be a multiple of 8");
    return ZB_OK;
}

zb_status launched(const char* who) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string(who) + " launch: " + cudaGetErrorString(e));
    zb::clear_error();
    return ZB_OK;
}

constexpr int ROUTE_BLOCKS = 152;     // one block an SM
// Tokens that one block takes alone, a warp each.  64 experts, k = 6, on the device
// alone: 32 tokens 4.1 us against 5.2 in two kernels, 64 tokens 5.7 against 5.2,
// 128 tokens 9.0 against 5.3.
constexpr int ROUTE_SMALL = 32;

int tokens_per_block(long long tokens) {
    const long long n = (tokens + ROUTE_BLOCKS - 1) / ROUTE_BLOCKS;
    return static_cast<int>(n < 32 ? 32 : n);
}

template <int VPL, typename T>
zb_status route(const RouteArgs& a, cudaStream_t st) {
    if (a.tokens <= ROUTE_SMALL) {
        // a warp a token, no more warps than needed: their barriers cost time
        const unsigned threads = a.tokens <= 8 ? 256u : a.tokens <= 16 ? 512u : ROUTE_THREADS;
        zb_moe_route_small_kernel<VPL, T><<<1, threads, 0, st>>>(a);
        return launched("zb_moe_route");
    }
    const unsigned blocks = static_cast<unsigned>((a.tokens + a.per_block - 1) / a.per_block);
    zb_moe_choose_kernel<VPL, T><<<blocks, ROUTE_THREADS, 0, st>>>(a);
    zb_status s = launched("zb_moe_route");
    if (s != ZB_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(ROUTE_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = zb::dependent_launches();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, zb_moe_place_kernel, a);
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string("zb_moe_route launch: ") + cudaGetErrorString(e));
    return launched("zb_moe_route");
}

template <typename T>
zb_status route_by_width(const RouteArgs& a, cudaStream_t st) {
    if (a.experts <= 32) return route<1, T>(a, st);
    if (a.experts <= 64) return route<2, T>(a, st);
    if (a.experts <= 128) return route<4, T>(a, st);
    return route<8, T>(a, st);
}

template <int VPL, typename T>
void route_backward(const zb_router& r, const void* logits, const int32_t* expert, const float* gates,
                    const float* dgates, void* dlogits, cudaStream_t st) {
    zb_moe_route_backward_kernel<VPL, T><<<static_cast<unsigned>((r.tokens + 7) / 8), 256, 0, st>>>(
        static_cast<const T*>(logits), expert, gates, dgates, static_cast<T*>(dlogits), r.tokens, r.experts, r.topk,
        r.renorm);
}

template <typename T>
void route_backward_by_width(const zb_router& r, const void* logits, const int32_t* expert, const float* gates,
                             const float* dgates, void* dlogits, cudaStream_t st) {
    if (r.experts <= 32) route_backward<1, T>(r, logits, expert, gates, dgates, dlogits, st);
    else if (r.experts <= 64) route_backward<2, T>(r, logits, expert, gates, dgates, dlogits, st);
    else if (r.experts <= 128) route_backward<4, T>(r, logits, expert, gates, dgates, dlogits, st);
    else route_backward<8, T>(r, logits, expert, gates, dgates, dlogits, st);
}

}  // namespace

extern "C" size_t zb_moe_route_workspace_bytes(const zb_router* r) {
    if (check_router(r) != ZB_OK) return 0;
    return (static_cast<size_t>(ROUTE_BLOCKS) * r->experts * sizeof(int) + 15) & ~static_cast<size_t>(15);
}

extern "C" zb_status zb_moe_route(const zb_router* r, const void* logits, float* gates, int32_t* expert,
                                  int32_t* offsets, int32_t* row_of, int32_t* token_of, void* workspace,
                                  size_t ws_bytes, void* stream) {
    zb_status s = check_router(r);
    if (s != ZB_OK) return s;
    if (!offsets || (r->tokens > 0 && (!logits || !gates || !expert || !row_of || !token_of)))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_route: required pointer is NULL");
    if (off16(logits) || off16(gates) || off16(expert) || off16(offsets) || off16(row_of) || off16(token_of) ||
        off16(workspace))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_route: pointers must be 16-byte aligned");
    if (!workspace || ws_bytes < zb_moe_route_workspace_bytes(r))
        return zb::fail(ZB_ERR_WORKSPACE, "zb_moe_route: workspace missing or too small: need " +
                                              std::to_string(zb_moe_route_workspace_bytes(r)) + " bytes");
    RouteArgs a;
    a.logits = logits;
    a.tokens = r->tokens;
    a.experts = r->experts;
    a.topk = r->topk;
    a.renorm = r->renorm;
    a.per_block = tokens_per_block(r->tokens);
    a.gates = gates;
    a.expert = expert;
    a.offsets = offsets;
    a.row_of = row_of;
    a.token_of = token_of;
    a.hist = static_cast<int*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return r->dtype == ZB_DT_BF16 ? route_by_width<__nv_bfloat16>(a, st) : route_by_width<float>(a, st);
}

extern "C" zb_status zb_moe_route_backward(const zb_router* r, const void* logits, const int32_t* expert,
                                           const float* gates, const float* dgates, void* dlogits, void* stream) {
    zb_status s = check_router(r);
    if (s != ZB_OK) return s;
    if (r->tokens == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    if (!expert || !gates || !dgates || !dlogits || (!r->renorm && !logits))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_route_backward: required pointer is NULL");
    if (off16(logits) || off16(expert) || off16(gates) || off16(dgates) || off16(dlogits))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_route_backward: pointers must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (r->dtype == ZB_DT_BF16)
        route_backward_by_width<__nv_bfloat16>(*r, logits, expert, gates, dgates, dlogits, st);
    else
        route_backward_by_width<float>(*r, logits, expert, gates, dgates, dlogits, st);
    return launched("zb_moe_route_backward");
}

extern "C" zb_status zb_moe_dispatch(int64_t tokens, int32_t topk, int64_t width, const void* X,
                                     const int32_t* row_of, void* Xp, void* stream) {
    zb_status s = check_rows("zb_moe_dispatch", tokens, topk, width);
    if (s != ZB_OK) return s;
    if (tokens == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    if (!X || !row_of || !Xp) return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_dispatch: required pointer is NULL");
    if (off16(X) || off4(row_of) || off16(Xp))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_dispatch: pointers must be 16-byte aligned (row_of: 4)");
    const int w8 = static_cast<int>(width / 8);
    const int segs = (w8 + 32 * COPY_U - 1) / (32 * COPY_U);
    const long long blocks = (tokens * segs + 7) / 8;
    if (blocks > 0x7fffffffLL) return zb::fail(ZB_ERR_SHAPE, "zb_moe_dispatch: too many elements");
    zb_moe_dispatch_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(X), row_of, static_cast<uint4*>(Xp), tokens, topk, w8, segs);
    return launched("zb_moe_dispatch");
}

extern "C" zb_status zb_moe_combine(int64_t tokens, int32_t topk, int64_t width, const void* Yp,
                                    const int32_t* row_of, const float* gates, void* Y, void* stream) {
    zb_status s = check_rows("zb_moe_combine", tokens, topk, width);
    if (s != ZB_OK) return s;
    if (tokens == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    if (!Yp || !row_of || !Y) return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_combine: required pointer is NULL");
    if (off16(Yp) || off4(row_of) || off4(gates) || off16(Y))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_combine: pointers must be 16-byte aligned (row_of, gates: 4)");
    const int w8 = static_cast<int>(width / 8);
    const int segs = (w8 + 32 * SUM_U - 1) / (32 * SUM_U);
    const long long blocks = (tokens * segs + 7) / 8;
    if (blocks > 0x7fffffffLL) return zb::fail(ZB_ERR_SHAPE, "zb_moe_combine: too many elements");
    zb_moe_combine_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(Yp), row_of, gates, static_cast<uint4*>(Y), tokens, topk, w8, segs);
    return launched("zb_moe_combine");
}

extern "C" zb_status zb_moe_combine_backward(int64_t tokens, int32_t topk, int64_t width, const void* dY,
                                             const void* Yp, const int32_t* row_of, const float* gates, void* dYp,
                                             float* dgates, void* stream) {
    zb_status s = check_rows("zb_moe_combine_backward", tokens, topk, width);
    if (s != ZB_OK) return s;
    if (tokens == 0) {
        zb::clear_error();
        return ZB_OK;
    }
    if (!dY || !Yp || !row_of || !gates || !dYp || !dgates)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_moe_combine_backward: required pointer is NULL");
    if (off16(dY) || off16(Yp) || off4(row_of) || off4(gates) || off16(dYp) || off4(dgates))
        return zb::fail(ZB_ERR_ALIGN,
                        "zb_moe_combine_backward: pointers must be 16-byte aligned (row_of, gates, dgates: 4)");
    const int w8 = static_cast<int>(width / 8);
    // A warp a token leaves wide tokens' reads one after the other (8192 tokens, 2
    // rows of 4096: 71 us, with 8 warps 55); more warps than a row has pieces for
    // are idle (16384 tokens, 4 rows of 512: 61 us with 8 warps, 33 with one).
    const int wpt = w8 <= 64 ? 1 : w8 <= 128 ? 2 : w8 <= 256 ? 4 : 8;
    const long long blocks = (tokens * wpt + 7) / 8;
    if (blocks > 0x7fffffffLL) return zb::fail(ZB_ERR_SHAPE, "zb_moe_combine_backward: too many tokens");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto kern) {
        kern<<<static_cast<unsigned>(blocks), 256, 0, st>>>(static_cast<const uint4*>(dY), static_cast<const uint4*>(Yp),
                                                            row_of, gates, static_cast<uint4*>(dYp), dgates, tokens,
                                                            topk, w8);
    };
    if (wpt == 1) go(zb_moe_combine_backward_kernel<1>);
    else if (wpt == 2) go(zb_moe_combine_backward_kernel<2>);
    else if (wpt == 4) go(zb_moe_combine_backward_kernel<4>);
    else go(zb_moe_combine_backward_kernel<8>);
    return launched("zb_moe_combine_backward");
}
