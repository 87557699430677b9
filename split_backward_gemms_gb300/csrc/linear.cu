// linear.cu — a linear map with its epilogue: D = X W (or X W^T) with bias,
// GeLU or GeLU', and a residual (zb_linear_product).
//
// Two kernels (use_rows says which):
//   zb_linear_tiles_kernel  persistent CTA pairs over tiles of 256 rows;
//   zb_linear_rows_kernel   one tile of 32, 64 or 128 rows x 128 columns a
//                           cluster, whose CTAs split K, for few rows or few tiles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <string>

#include "grouped.cuh"

namespace {

enum Form { STORE = 0, GELU = 1, GRAD = 2, STORE32 = 3 };

struct LinearArgs {
    const __nv_bfloat16 *bias, *H;
    const void* R;
    void *out0, *out1;  // out1: GELU's output
    long long ldr, ldh, ldo;
    int M, N, K;
    int save, tanh_form;
    int hint_a, hint_b, hint_out;  // L2 priorities of the copies (choose_l2_hints)
    int hint_once;                 // of H's and the residual's, which are read once
    int tile_n;                    // tiles kernel: columns of a tile, a multiple of 32
    int tiles_n, split;            // rows kernel: column tiles, CTAs along K
    int stages;                    // rows kernel: of the ring
    unsigned int* err;
};

// GeLU and GeLU' of pairs, with few instructions: at K = 1024 a tile's epilogue
// takes longer than its MMAs.  With a = |x| and q = Phi(-a) = e t (a1 + t (a2 +
// ...)) / 2, e = exp(-a^2 / 2), t = 1 / (1 + p a / sqrt 2) (Abramowitz & Stegun
// 7.1.26, as in gemm_core.cuh):
//   GeLU(x)  = max(x, 0) - a q
//   GeLU'(x) = 1/2 + sign(x) (1/2 - g),  g = q - a phi(a)
// The .ftz forms of ex2 and rcp are single instructions (the others also scale
// subnormal numbers, which neither e's place in these sums nor a denominator of at
// least 1 needs): 4096 x 4096, K 1024 with GeLU' and
// residual executes 16.5 million warp instructions with the forms of gemm_core.cuh,
// 10.7 million with these (45.6 and 41.5 us).
__device__ __forceinline__ float ex2_ftz(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_ftz(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pk2(v, v); }

// a, e and 2 q / e of the pair (x0, x1).
__device__ __forceinline__ void tail_pair(float x0, float x1, f32x2& A, f32x2& E, f32x2& Q) {
    using C = AS71_26;
    // e is 0 from 14 on; a finite a keeps an infinity out of its neighbour's t and of a e
    const float a0 = fminf(fabsf(x0), 32.0f), a1 = fminf(fabsf(x1), 32.0f);
    A = pk2(a0, a1);
    const f32x2 X = pk2(x0, x1);
    float v0, v1;
    up2(mul2(mul2(X, X), both(-0.7213475204444817f)), v0, v1);  // exp(v) = 2^(v / ln 2)
    E = pk2(ex2_ftz(v0), ex2_ftz(v1));
    constexpr float pz = C::p * 0.7071067811865476f;
    up2(fma2(A, both(pz), both(1.0f)), v0, v1);
    // one reciprocal for both: 1 / v0 = v1 / (v0 v1)
    const f32x2 T = mul2(both(rcp_ftz(v0 * v1)), pk2(v1, v0));
    f32x2 P = fma2(T, both(C::a5), both(C::a4));
    P = fma2(T, P, both(C::a3));
    P = fma2(T, P, both(C::a2));
    P = fma2(T, P, both(C::a1));
    Q = mul2(T, P);
}

// The tanh form, with its limits at the infinities (there the formula is 0 times an
// infinity; a NaN stays one).
__device__ __forceinline__ float gelu_tanh(float x) { return x < -32.0f ? 0.0f : gelu_t<true>(x); }
__device__ __forceinline__ float gelu_tanh_grad(float x) {
    return fabsf(x) > 32.0f ? (x > 0.0f ? 1.0f : 0.0f) : gelu_grad_t<true>(x);
}

// GeLU of N values in place (an even number of them), in fp32.
template <bool TANH, int N>
__device__ __forceinline__ void gelu_values(float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        if (TANH) {
            x[i] = gelu_tanh(x[i]);
            x[i + 1] = gelu_tanh(x[i + 1]);
        } else {
            f32x2 A, E, Q;
            tail_pair(x[i], x[i + 1], A, E, Q);
            const f32x2 relu = pk2(fmaxf(x[i], 0.0f), fmaxf(x[i + 1], 0.0f));
            up2(fma2(mul2(A, E), mul2(Q, both(-0.5f)), relu), x[i], x[i + 1]);
        }
    }
}

// x *= GeLU'(h) for N values (h: pairs of bf16).
template <bool TANH, int N>
__device__ __forceinline__ void gelu_grad_values(float (&x)[N], const uint32_t (&h)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float h0 = __uint_as_float(h[i / 2] << 16), h1 = __uint_as_float(h[i / 2] & 0xffff0000u);
        if (TANH) {
            x[i] *= gelu_tanh_grad(h0);
            x[i + 1] *= gelu_tanh_grad(h1);
        } else {
            f32x2 A, E, Q;
            tail_pair(h0, h1, A, E, Q);
            // 1/2 - g = 1/2 - e (Q / 2 - a / sqrt(2 pi))
            const f32x2 U = fma2(Q, both(-0.5f), mul2(A, both(0.3989422804014327f)));
            float g0, g1;
            up2(fma2(E, U, both(0.5f)), g0, g1);
            const f32x2 G = add2(pk2(copysignf(g0, h0), copysignf(g1, h1)), both(0.5f));
            up2(mul2(pk2(x[i], x[i + 1]), G), x[i], x[i + 1]);
        }
    }
}

// x += r for 8 values of bf16.
__device__ __forceinline__ void add_bf16(float* x, const float4& r) {
    const uint32_t w[4] = {__float_as_uint(r.x), __float_as_uint(r.y), __float_as_uint(r.z), __float_as_uint(r.w)};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        up2(add2(pk2(x[2 * j], x[2 * j + 1]), pk2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u))),
            x[2 * j], x[2 * j + 1]);
}

// ---------------------------------------------------------------- large problems
// The roles of the dense kernel (gemm_tc.cu) on CTA pairs: warp 0 copies, warp
// 1 of the even CTA issues MMAs of 256 rows x up to 256 columns into one of two
// accumulators, warps 2-9 drain (a TMEM lane is a row; a warp has 32 rows and half
// of the columns, in chunks of 32).  H and the residual come by TMA, the residual
// into the staging box that the chunk's results then leave from: a thread adds its
// row's values and writes the sums back to where they lay.  So their bytes cost no
// registers and no waiting loads, and an output that is the residual itself needs
// no care (each of its elements is read and written by one warp, in this order).
// The boxes are a ring over the chunks of all of a CTA's tiles, asked for again as
// soon as the stores have read them.
//
// 5 stages and 4 boxes a warp or 4 and 6, us of 4096 x 4096 (8192 x 4096) with
// residual: GeLU' K 64 31.9, 30.0; K 1024 38.8, 42.4; K 4096 (180, 189).  16
// epilogue warps with 2 boxes each: 33.2, 39.0 (179); fp32 K 1024 43.1 for 40.9.  H
// and R asked for in L2 a tile ahead: no faster at K 64, 41.3 for 39.5 at K 1024.
// With K 4096 the store without residual runs at 1.81-1.97 PF/s, with it at 1.67-1.74;
// at K 1024 the epilogue's bytes take as long as the MMAs.
//
// fp32 outputs (STORE32): the tensor core cuts off low bits as it adds, so the
// accumulators take SEG blocks of K each and the epilogue adds them in registers,
// rounding to nearest, as the experts' W does (grouped.cu has both sides' errors).
template <int FORM>
struct TileCfg {
    static constexpr bool F32 = FORM == STORE32;
    static constexpr int COLS = F32 ? 16 : 32;  // of a box: 32 rows of 64 bytes
    // F32's 128 sums a thread need the registers that warps 0-3 (2 and 3 idle) give up
    static constexpr int THREADS = F32 ? 384 : NUM_THREADS;
    static constexpr int FIRST = F32 ? 4 : 2;  // first epilogue warp
};
// (fp32 kernels are compiled to 168 registers a thread, what 384 threads leave)
constexpr int REGS_LOW = 56, REGS_HIGH = 224;
static_assert(128 * REGS_LOW + 256 * REGS_HIGH <= 384 * 168, "register split");
constexpr int SEG = 8;            // fp32 outputs: blocks of 64 along K an accumulator takes
constexpr int TILE_STAGES = 5;    // of the ring: 16 KiB of X, up to 16 of W
constexpr int TILE_WARPS = 8;     // of the epilogue
constexpr int WARP_COLS = 128;    // columns of a warp, at most
constexpr uint32_t TILE_BOXES = 4;  // staging boxes a warp
constexpr uint32_t T_BOX = 32 * 64;
constexpr uint32_t T_STAGE = Cfg<2>::STAGE_BYTES;

struct TileCtl {
    uint64_t full[TILE_STAGES], empty[TILE_STAGES], tfull[2], tempty[2], drain;
    uint64_t rbar[TILE_WARPS][TILE_BOXES];  // a chunk's H and residual have landed
    uint32_t tmem_base;
    int abort_flag;
};
constexpr size_t TILE_SMEM = 1024 + TILE_STAGES * T_STAGE + TILE_WARPS * TILE_BOXES * T_BOX + sizeof(TileCtl);
static_assert(TILE_SMEM <= 232448, "shared memory");

template <int FORM, int W_MN>
__global__ void __launch_bounds__(TileCfg<FORM>::THREADS, 1)
    zb_linear_tiles_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                           const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmH,
                           const __grid_constant__ CUtensorMap tmR, const LinearArgs args) {
    using T = TileCfg<FORM>;
    constexpr int STAGES = TILE_STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + STAGES * T_STAGE;
    TileCtl* ctl = reinterpret_cast<TileCtl*>(staging + TILE_WARPS * TILE_BOXES * T_BOX);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = zbp::cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = blockIdx.x / 2, clusters = gridDim.x / 2;
    const int tile_n = args.tile_n;
    const int tiles_m = (args.M + 255) / 256, tiles_n = (args.N + tile_n - 1) / tile_n, num_tiles = tiles_m * tiles_n;
    const uint32_t w_bytes = static_cast<uint32_t>(tile_n / 2) * BK * 2u;  // of a stage in one CTA
    const int num_kb = (args.K + BK - 1) / BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            zbp::mbar_init(zbp::smem_u32(&ctl->full[s]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            zbp::mbar_init(zbp::smem_u32(&ctl->tfull[b]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->tempty[b]), 2 * TILE_WARPS);
        }
        zbp::mbar_init(zbp::smem_u32(&ctl->drain), 1);
        for (int w = 0; w < TILE_WARPS; ++w)
            for (int b = 0; b < static_cast<int>(TILE_BOXES); ++b) zbp::mbar_init(zbp::smem_u32(&ctl->rbar[w][b]), 1);
        ctl->abort_flag = 0;
        zbp::fence_mbar_init();
        zbp::tma_prefetch_desc(&tmX);
        zbp::tma_prefetch_desc(&tmW);
        zbp::tma_prefetch_desc(&tmO);
        if (args.R) zbp::tma_prefetch_desc(&tmR);
        if (FORM == GRAD || (FORM == GELU && args.save)) zbp::tma_prefetch_desc(&tmH);
    }
    if (warp == 1) {
        zbp::tmem_alloc_pair(zbp::smem_u32(&ctl->tmem_base), TMEM_COLS);
        zbp::tmem_relinquish_pair();
    }
    zbp::tc_fence_before();
    __syncthreads();
    zbp::cluster_sync();
    zbp::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();

    if (T::F32 && warp < T::FIRST) zbp::regs_dec<REGS_LOW>();
    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
        const uint32_t full0_lead = zbp::mapa_shared(full0, 0), sa0 = zbp::smem_u32(smem);
        const uint64_t pol_x = zbp::l2_policy(args.hint_a), pol_w = zbp::l2_policy(args.hint_b);
        uint32_t s = 0, sp = 1, it = 0;  // stage and the phase of its last release; stages filled
        bool ok = true;
        for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
            int mb, nb;
            tile_coords(tile, tiles_m, tiles_n, Cfg<2>::GROUP_M, mb, nb);
            const int m0 = mb * 256 + static_cast<int>(rank) * BM;
            const int n0 = nb * tile_n + static_cast<int>(rank) * (tile_n / 2);
            for (int kb = 0; kb < num_kb; ++kb, ++it) {
                if (!wait_bar<false>(empty0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_PRODUCER, WAIT_LIMIT_NS, true)) {
                    ok = false;
                    break;
                }
                if (zbp::elect_one()) {
                    const uint32_t full = full0_lead + s * 8u, sa = sa0 + s * T_STAGE, sb = sa + A_BYTES;
                    const int k0 = kb * BK;
                    if (leader) zbp::mbar_arrive_expect_tx(full0 + s * 8u, 2 * (A_BYTES + w_bytes));
                    zbp::tma_load_2d_pair_hint(sa, &tmX, full, k0, m0, pol_x);
                    if (W_MN) {
                        zbp::tma_load_2d_pair_hint(sb, &tmW, full, n0, k0, pol_w);
                        if (tile_n == BN) zbp::tma_load_2d_pair_hint(sb + MN_ATOM_BYTES, &tmW, full, n0 + 64, k0, pol_w);
                    } else {
                        zbp::tma_load_2d_pair_hint(sb, &tmW, full, k0, n0, pol_w);
                    }
                }
                __syncwarp();
                if (++s == STAGES) {
                    s = 0;
                    sp ^= 1u;
                }
            }
        }
        if (!ok && leader) {
            // wait for the copies that were issued but may not have landed
            const uint32_t first = it > STAGES ? it - STAGES : 0;
            for (uint32_t i = first; i < it; ++i)
                wait_bar<false>(full0 + (i % STAGES) * 8u, (i / STAGES) & 1u, abort_flag, args.err, ERR_WAIT_PRODUCER,
                                DRAIN_LIMIT_NS, false);
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------ MMA issuer
            const uint32_t idesc = zbp::idesc_bf16_f32(256, static_cast<uint32_t>(tile_n), 0, W_MN);
            constexpr uint32_t W_STEP = W_MN ? 2048 >> 4 : 32 >> 4, hi = zbp::desc_hi(1024);
            const uint32_t a0 = zbp::desc_lo(zbp::smem_u32(smem), 16);
            const uint32_t b0 = zbp::desc_lo(zbp::smem_u32(smem) + A_BYTES, W_MN ? MN_ATOM_BYTES : 16);
            const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
            uint32_t s = 0, sp = 0, local = 0;  // stage and its phase; accumulators filled
            bool ok = true;
            for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
                for (int kb0 = 0; kb0 < num_kb && ok; kb0 += T::F32 ? SEG : num_kb) {
                    const uint32_t buf = local & 1u, tr = local >> 1;
                    ++local;
                    if (!wait_bar<false>(zbp::smem_u32(&ctl->tempty[buf]), (tr & 1u) ^ 1u, abort_flag, args.err,
                                         ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        break;
                    }
                    zbp::tc_fence_after();
                    const uint32_t d_tmem = tmem_base + buf * ACC_COLS;
                    const int kb1 = T::F32 ? min(kb0 + SEG, num_kb) : num_kb;
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!wait_bar<false>(full0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                            ok = false;
                            break;
                        }
                        zbp::tc_fence_after();
                        if (zbp::elect_one()) {
                            const uint32_t off = s * (T_STAGE >> 4);
                            zbp::mma4_f16_pair<2, W_STEP>(d_tmem, a0 + off, hi, b0 + off, hi, idesc, kb != kb0);
                            zbp::tc_commit_pair_multicast(empty0 + s * 8u, 0x3);
                            if (kb + 1 == kb1) zbp::tc_commit_pair_multicast(zbp::smem_u32(&ctl->tfull[buf]), 0x3);
                        }
                        __syncwarp();
                        if (++s == STAGES) {
                            s = 0;
                            sp ^= 1u;
                        }
                    }
                }
            }
            // every MMA issued here completes before TMEM is released
            if (zbp::elect_one()) zbp::tc_commit_pair(zbp::smem_u32(&ctl->drain));
            __syncwarp();
            wait_bar<false>(zbp::smem_u32(&ctl->drain), 0, abort_flag, args.err, ERR_WAIT_MMA, DRAIN_LIMIT_NS, false);
        }
    } else if (warp >= T::FIRST) {
        // ---------------------------------------------------- epilogue
        if (T::F32) zbp::regs_inc<REGS_HIGH>();
        constexpr int CH = WARP_COLS / T::COLS;  // chunks of a warp's columns
        const int ew = warp - T::FIRST, q = warp & 3, half = (tile_n / 2 + 31) / 32 * 32, c_lo = (ew >> 2) * half;
        const uint32_t stg0 = zbp::smem_u32(staging) + static_cast<uint32_t>(ew) * TILE_BOXES * T_BOX;
        const uint32_t rbar0 = zbp::smem_u32(&ctl->rbar[ew][0]);
        const uint64_t pol_out = zbp::l2_policy(args.hint_out), pol_once = zbp::l2_policy(args.hint_once);
        const bool res = args.R != nullptr, save = FORM == GELU && args.save;
        // The boxes are a ring of chunks: one box a chunk, for the residual, which the
        // results leave from; or two where GELU keeps H, whose box comes first.  Without
        // a residual GRAD's results leave from H's box.  With one, H has the last box to
        // itself: it is free as soon as H is in registers, so one is enough, and three
        // are left to the residual, which hold it until the results are stored.
        const bool h_box = FORM == GRAD && res, inputs = !T::F32 && (res || FORM == GRAD);
        const uint32_t per = save ? 2 : 1, ring = save ? TILE_BOXES / 2 : h_box ? TILE_BOXES - 1 : TILE_BOXES;
        const uint32_t hat = stg0 + (TILE_BOXES - 1) * T_BOX, hbar = rbar0 + (TILE_BOXES - 1) * 8u;
        auto boxes_of = [&](uint32_t slot) { return stg0 + slot * per * T_BOX; };
        auto place = [&](int tile, int& row0, int& n0) {  // a tile's first row and column of this warp; its live chunks
            int mb, nb;
            tile_coords(tile, tiles_m, tiles_n, Cfg<2>::GROUP_M, mb, nb);
            row0 = mb * 256 + static_cast<int>(rank) * BM + q * 32;
            n0 = nb * tile_n + c_lo;
            const int cols = min(args.N - n0, min(half, tile_n - c_lo));
            return row0 < args.M ? min(CH, max(0, (cols + T::COLS - 1) / T::COLS)) : 0;
        };
        // a walk over the chunks of all tiles, ahead of the one that stores them
        struct Cursor {
            int tile, c, chunks, row0, n0;
        };
        auto next = [&](Cursor& a) {
            while (a.c >= a.chunks) {
                if (a.tile >= num_tiles) return false;
                a.tile += clusters;
                if (a.tile >= num_tiles) return false;
                a.c = 0;
                a.chunks = place(a.tile, a.row0, a.n0);
            }
            return true;
        };
        Cursor ahead = {cluster - clusters, 0, 0, 0, 0}, h_ahead = ahead;
        uint32_t asked = 0, used = 0, h_asked = 0;  // chunks asked for, chunks stored
        uint32_t a_slot = 0, slot = 0, turn = 0;     // their places in the ring; parity of the ring's turn
        auto ask = [&]() {
            if (!next(ahead)) return;
            if (lane == 0) {
                const uint32_t bar = rbar0 + a_slot * 8u, at = boxes_of(a_slot) + (per - 1) * T_BOX;
                zbp::mbar_arrive_expect_tx(bar, T_BOX);
                zbp::tma_load_2d_hint(at, res ? &tmR : &tmH, bar, ahead.n0 + ahead.c * T::COLS, ahead.row0, pol_once);
            }
            ++ahead.c;
            ++asked;
            a_slot = a_slot + 1 == ring ? 0 : a_slot + 1;
        };
        auto ask_h = [&]() {
            if (!next(h_ahead)) return;
            if (lane == 0) {
                zbp::mbar_arrive_expect_tx(hbar, T_BOX);
                zbp::tma_load_2d_hint(hat, &tmH, hbar, h_ahead.n0 + h_ahead.c * T::COLS, h_ahead.row0, pol_once);
            }
            ++h_ahead.c;
            ++h_asked;
        };
        bool owed = false;  // the last chunk's boxes have not been asked for again
        // once the stores so far have read their boxes
        auto ask_on = [&]() {
            if (lane == 0) zbp::bulk_wait_read<0>();
            __syncwarp();
            ask();
            owed = false;
        };
        if (h_box) ask_h();
        if (inputs)
            for (uint32_t k = 0; k < ring; ++k) ask();
        // this lane's 16-byte part k of its row in a box
        auto part = [&](uint32_t box, int k) { return box + static_cast<uint32_t>(lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)); };
        // fp32: the residual is added just before the tile's last accumulator, while whose
        // MMAs run; not after it, since the next tile's MMAs have but the other accumulator
        // until this one is read (4096 x 4096, K 1024 42.5 us for 38.8); nor first, which
        // would round every later sum at the residual's size (and saves 35.3 us for 36.4 at
        // K 512, nothing at K 1024).  Chunk c comes into box c mod 4.
        uint32_t on_way = 0, phases = 0;  // a bit a box: asked for and not read; phase of its barrier
        auto ask32 = [&](int c, int row0, int n0) {
            const uint32_t b = static_cast<uint32_t>(c) % TILE_BOXES;
            if (lane == 0) {
                zbp::mbar_arrive_expect_tx(rbar0 + b * 8u, T_BOX);
                zbp::tma_load_2d_hint(stg0 + b * T_BOX, &tmR, rbar0 + b * 8u, n0 + c * T::COLS, row0, pol_once);
            }
            on_way |= 1u << b;
        };
        auto ask32_tile = [&](int tile) {  // the first boxes of a tile
            int row0, n0;
            const int chunks = min(static_cast<int>(TILE_BOXES), tile < num_tiles ? place(tile, row0, n0) : 0);
            for (int c = 0; c < chunks; ++c) ask32(c, row0, n0);
        };
        if (T::F32 && res) ask32_tile(cluster);
        uint32_t local = 0;
        bool ok = true;
        for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
            int row0, n0;
            const int chunks = place(tile, row0, n0);
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c_lo);
            float acc[T::F32 ? CH : 1][16];
            uint32_t buf = 0;
            if constexpr (T::F32) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c][i] = 0.0f;
            }
            auto add_residual = [&]() {
                constexpr uint32_t B = TILE_BOXES;
#pragma unroll
                for (int c = 0; c < (T::F32 ? CH : 0); ++c) {
                    if (c >= chunks || !ok) continue;
                    const uint32_t b = static_cast<uint32_t>(c) % B, box = stg0 + b * T_BOX;
                    if (!wait_bar<false>(rbar0 + b * 8u, (phases >> b) & 1u, abort_flag, args.err, ERR_WAIT_EPI,
                                        WAIT_LIMIT_NS, true)) {
                        ok = false;
                        continue;
                    }
                    phases ^= 1u << b;
                    on_way &= ~(1u << b);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 r = zbp::ld_shared_v4(part(box, k));
                        acc[c][4 * k] += r.x;
                        acc[c][4 * k + 1] += r.y;
                        acc[c][4 * k + 2] += r.z;
                        acc[c][4 * k + 3] += r.w;
                    }
                    zbp::fence_proxy_async_smem();  // every lane has read the box
                    __syncwarp();
                    if (c + static_cast<int>(B) < chunks) ask32(c + static_cast<int>(B), row0, n0);
                }
            };
            // fp32 outputs add the accumulators' parts; the others have one, read piece by piece below
            for (int kb0 = 0; kb0 < num_kb; kb0 += T::F32 ? SEG : num_kb) {
                if (T::F32 && res && kb0 + SEG >= num_kb) {
                    add_residual();
                    if (!ok) break;
                }
                buf = local & 1u;
                const uint32_t tr = local >> 1;
                ++local;
                if (!wait_bar<false>(zbp::smem_u32(&ctl->tfull[buf]), tr & 1u, abort_flag, args.err, ERR_WAIT_EPI,
                                    WAIT_LIMIT_NS, true)) {
                    ok = false;
                    break;
                }
                zbp::tc_fence_after();
                if constexpr (T::F32) {
#pragma unroll
                    for (int c = 0; c < CH; c += 2) {
                        uint32_t v[32];
                        zbp::tmem_ld_32x32b_x32(taddr + buf * ACC_COLS + c * 16, v);
                        zbp::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            acc[c + i / 16][i % 16] += __uint_as_float(v[i]);
                        }
                    }
                    zbp::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) zbp::mbar_arrive_remote(zbp::mapa_shared(zbp::smem_u32(&ctl->tempty[buf]), 0));
                }
            }
            if (!ok) break;
            // 16 columns from col, the p-th of their boxes
            auto piece = [&](int p, int col, uint32_t box0, uint32_t box, const uint32_t (&w)[8], float (&x)[16]) {
                if (FORM == GRAD) {
                    if (args.tanh_form)
                        gelu_grad_values<true, 16>(x, w);
                    else
                        gelu_grad_values<false, 16>(x, w);
                } else if (args.bias) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (col + i * 8 < args.N)
                            add_bf16(x + i * 8, *reinterpret_cast<const float4*>(args.bias + col + i * 8));
                }
                auto put = [&](uint32_t to) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        zbp::st_shared_v4(part(to, 2 * p + k), pack_bf16x2(x[8 * k], x[8 * k + 1]),
                                          pack_bf16x2(x[8 * k + 2], x[8 * k + 3]), pack_bf16x2(x[8 * k + 4], x[8 * k + 5]),
                                          pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
                };
                if (FORM == GELU) {
                    if (save) put(box0);
                    if (args.tanh_form)
                        gelu_values<true, 16>(x);
                    else
                        gelu_values<false, 16>(x);
                }
                if constexpr (T::F32) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        zbp::st_shared_v4(part(box, k), __float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]),
                                          __float_as_uint(x[4 * k + 2]), __float_as_uint(x[4 * k + 3]));
                    }
                } else {
                    if (res)
#pragma unroll
                        for (int k = 0; k < 2; ++k) add_bf16(x + 8 * k, zbp::ld_shared_v4(part(box, 2 * p + k)));
                    put(box);
                }
            };
            auto chunk = [&](int c, float (&sums)[16]) {
                const int col0 = n0 + c * T::COLS;
                const uint32_t box0 = boxes_of(slot), box = box0 + (per - 1) * T_BOX;
                uint32_t v[T::F32 ? 1 : 32];  // bf16: the chunk's sums, on their way while the inputs are waited for
                if constexpr (!T::F32) zbp::tmem_ld_32x32b_x32(taddr + buf * ACC_COLS + c * 32, v);
                if (inputs) {
                    if (owed) ask_on();
                    if (!wait_bar<false>(rbar0 + slot * 8u, turn, abort_flag, args.err, ERR_WAIT_EPI, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        return;
                    }
                } else {
                    if (lane == 0) {
                        if (per == 2)
                            zbp::bulk_wait_read<TILE_BOXES / 2 - 1>();
                        else
                            zbp::bulk_wait_read<TILE_BOXES - 1>();
                    }
                    __syncwarp();
                }
                uint32_t w[2][8];  // H
                if (FORM == GRAD) {
                    if (h_box && !wait_bar<false>(hbar, used & 1u, abort_flag, args.err, ERR_WAIT_EPI, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        return;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 h = zbp::ld_shared_v4(part(h_box ? hat : box0, k));
                        w[k / 2][k % 2 * 4] = __float_as_uint(h.x);
                        w[k / 2][k % 2 * 4 + 1] = __float_as_uint(h.y);
                        w[k / 2][k % 2 * 4 + 2] = __float_as_uint(h.z);
                        w[k / 2][k % 2 * 4 + 3] = __float_as_uint(h.w);
                    }
                    if (h_box) {
                        zbp::fence_proxy_async_smem();  // every lane has read the box
                        __syncwarp();
                        ask_h();
                    }
                }
                if constexpr (T::F32) {
                    piece(0, col0, box0, box, w[0], sums);
                } else {
                    zbp::tmem_ld_wait();
                    float x[2][16];
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i / 16][i % 16] = __uint_as_float(v[i]);
                    piece(0, col0, box0, box, w[0], x[0]);
                    piece(1, col0 + 16, box0, box, w[1], x[1]);
                }
                zbp::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (save) zbp::tma_store_2d_hint(&tmH, box0, col0, row0, pol_out);
                    zbp::tma_store_2d_hint(&tmO, box, col0, row0, pol_out);
                    zbp::bulk_commit();
                }
                owed = inputs;
                ++used;
                if (++slot == ring) {
                    slot = 0;
                    turn ^= 1u;
                }
            };
            if constexpr (T::F32) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    if (c < chunks && ok) chunk(c, acc[c]);
            } else {
#pragma unroll 1
                for (int c = 0; c < chunks && ok; ++c) {
                    chunk(c, acc[0]);
                }
                zbp::tc_fence_before();
                __syncwarp();
                if (lane == 0) zbp::mbar_arrive_remote(zbp::mapa_shared(zbp::smem_u32(&ctl->tempty[buf]), 0));
            }
            if (owed) ask_on();
            if (T::F32 && res) {
                if (lane == 0) zbp::bulk_wait_read<0>();
                __syncwarp();
                ask32_tile(tile + clusters);
            }
        }
        zbp::tmem_ld_wait();  // (a chunk's sums may be on their way after an abort)
        // inputs asked for and not used (after an abort)
        for (uint32_t b = 0; T::F32 && b < TILE_BOXES; ++b)
            if ((on_way >> b) & 1u)
                wait_bar<false>(rbar0 + b * 8u, (phases >> b) & 1u, abort_flag, args.err, ERR_WAIT_EPI, DRAIN_LIMIT_NS, false);
        if (h_box && h_asked > used)
            wait_bar<false>(hbar, (h_asked - 1) & 1u, abort_flag, args.err, ERR_WAIT_EPI, DRAIN_LIMIT_NS, false);
        for (; inputs && used < asked; ++used) {
            wait_bar<false>(rbar0 + slot * 8u, turn, abort_flag, args.err, ERR_WAIT_EPI, DRAIN_LIMIT_NS, false);
            if (++slot == ring) {
                slot = 0;
                turn ^= 1u;
            }
        }
        // the staging boxes must not be released while a bulk store reads them
        if (lane == 0) zbp::bulk_wait<0>();
        __syncwarp();
    }

    __syncthreads();
    zbp::cluster_sync();  // no remote arrivals or copies remain
    if (warp == 1) {
        zbp::tc_fence_after();
        zbp::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------- few tiles
// One tile of ROWS rows x 128 columns a cluster of `split` CTAs, which share its K
// range.  The product is transposed (as in grouped.cu): the weight's columns are
// the MMA's M side, the rows its N side, so a few rows cost little more than
// streaming the weight, and the split lets as many SMs stream it as there are.
// Each CTA leaves its fp32 partial tile in its own shared memory (its ring, idle
// by then), [row][column]; after a cluster barrier CTA r adds the partials of the
// r-th part of the rows through distributed shared memory, in the order of the
// CTAs (so the same inputs give the same bits), applies the epilogue and stores.
//
// At least R_SMEM of shared memory are asked for whatever the ring needs, so that
// an SM holds one CTA: two CTAs of different clusters on an SM could each wait for
// the other's tensor memory while their own clusters wait for them.
//
// 16 x 1024, K 4096 takes 5.0 us in a graph of such calls, of which streaming the
// weight is 1.3: the rest is the chain of launch, first loads, MMAs, exchange.
//
// fp32 outputs: an accumulator takes at most SEG blocks of K, as above.  Tensor memory
// holds 512 columns / ROWS of them; when all are full, the epilogue adds them to its
// registers and they are filled again.
constexpr int R_THREADS = NUM_THREADS;
constexpr int R_EPI_WARPS = R_THREADS / 32 - 2;
constexpr int R_STAGES = 10;
constexpr int R_MIN_KB = 2;  // blocks of K a CTA, at least
constexpr uint32_t R_SMEM = 120 * 1024;
constexpr uint32_t R_W_BYTES = 128 * BK * 2;
constexpr uint32_t rows_stage(int rows) { return R_W_BYTES + static_cast<uint32_t>(rows) * BK * 2; }

struct RowsCtl {
    uint64_t full[R_STAGES], empty[R_STAGES], tfull, tempty, drain;
    uint32_t tmem_base;
    int abort_flag;
};

// The epilogue of 4 consecutive columns of a row (all inside the matrix).
template <int FORM>
__device__ __forceinline__ void finish4(const LinearArgs& a, long long row, int col, float (&x)[4]) {
    auto four = [](const __nv_bfloat16* p, float (&v)[4]) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const float2 lo = unpack_bf16x2(u.x), hi = unpack_bf16x2(u.y);
        v[0] = lo.x;
        v[1] = lo.y;
        v[2] = hi.x;
        v[3] = hi.y;
    };
    auto put = [](void* p, long long at, const float (&v)[4]) {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    };
    // the residual before anything is stored: an output may take its place
    float r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (FORM == STORE32) {
        if (a.R) {
            const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.R) + row * a.ldr + col);
            r[0] = f.x;
            r[1] = f.y;
            r[2] = f.z;
            r[3] = f.w;
        }
    } else if (a.R) {
        four(static_cast<const __nv_bfloat16*>(a.R) + row * a.ldr + col, r);
    }
    if (FORM != GRAD && a.bias) {
        float b[4];
        four(a.bias + col, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += b[i];
    }
    if (FORM == GELU) {
        if (a.save) put(a.out0, row * a.ldo + col, x);
        if (a.tanh_form)
            gelu_values<true, 4>(x);
        else
            gelu_values<false, 4>(x);
    }
    if (FORM == GRAD) {
        const uint2 u = *reinterpret_cast<const uint2*>(a.H + row * a.ldh + col);
        const uint32_t h[2] = {u.x, u.y};
        if (a.tanh_form)
            gelu_grad_values<true, 4>(x, h);
        else
            gelu_grad_values<false, 4>(x, h);
    }
    if (a.R)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += r[i];
    if (FORM == STORE32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out0) + row * a.ldo + col) = make_float4(x[0], x[1], x[2], x[3]);
    else
        put(FORM == GELU ? a.out1 : a.out0, row * a.ldo + col, x);
}

template <int FORM, int W_MN, int ROWS>
__global__ void __launch_bounds__(R_THREADS, 1)
    zb_linear_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                          const LinearArgs args) {
    constexpr uint32_t STAGE = rows_stage(ROWS);
    constexpr bool F32 = FORM == STORE32;
    constexpr int PARTS = F32 ? 512 / ROWS : 1;  // accumulators
    constexpr uint32_t TMEM = PARTS * ROWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ RowsCtl ctl_shared;
    RowsCtl* ctl = &ctl_shared;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int split = args.split, stages = args.stages;
    const int rank = split > 1 ? static_cast<int>(zbp::cluster_ctarank()) : 0;
    const int tile = blockIdx.x / split;
    const int mb = tile / args.tiles_n, n0 = (tile - mb * args.tiles_n) * 128;
    const int m0 = mb * ROWS, live = min(ROWS, args.M - m0);
    const int num_kb_all = (args.K + BK - 1) / BK;
    const int kb0 = static_cast<int>(static_cast<long long>(num_kb_all) * rank / split);
    const int num_kb = static_cast<int>(static_cast<long long>(num_kb_all) * (rank + 1) / split) - kb0;
    const int fills = F32 ? (num_kb + SEG - 1) / SEG : 1, seg = (num_kb + fills - 1) / fills;  // blocks of K a filling

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            zbp::mbar_init(zbp::smem_u32(&ctl->full[s]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->empty[s]), 1);
        }
        zbp::mbar_init(zbp::smem_u32(&ctl->tfull), 1);
        zbp::mbar_init(zbp::smem_u32(&ctl->tempty), R_EPI_WARPS);
        zbp::mbar_init(zbp::smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        zbp::fence_mbar_init();
        zbp::tma_prefetch_desc(&tmX);
        zbp::tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        zbp::tmem_alloc(zbp::smem_u32(&ctl->tmem_base), TMEM);
        zbp::tmem_relinquish();
    }
    zbp::tc_fence_before();
    __syncthreads();
    zbp::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();

    const uint32_t ring = zbp::smem_u32(smem);
    const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        int s = 0;
        uint32_t sp = 1, it = 0;
        bool ok = true;
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
            if (!wait_bar<false>(empty0 + static_cast<uint32_t>(s) * 8u, sp, abort_flag, args.err, ERR_WAIT_PRODUCER,
                                WAIT_LIMIT_NS, true)) {
                ok = false;
                break;
            }
            if (zbp::elect_one()) {
                const uint32_t full = full0 + static_cast<uint32_t>(s) * 8u;
                const uint32_t sa = ring + static_cast<uint32_t>(s) * STAGE, sb = sa + R_W_BYTES;
                const int k0 = (kb0 + kb) * BK;
                zbp::mbar_arrive_expect_tx(full, STAGE);
                if (W_MN) {
                    zbp::tma_load_2d(sa, &tmW, full, n0, k0);
                    zbp::tma_load_2d(sa + MN_ATOM_BYTES, &tmW, full, n0 + 64, k0);
                } else {
                    zbp::tma_load_2d(sa, &tmW, full, k0, n0);
                }
                zbp::tma_load_2d(sb, &tmX, full, k0, m0);
            }
            __syncwarp();
            if (++s == stages) {
                s = 0;
                sp ^= 1u;
            }
        }
        if (!ok) {
            // wait for the copies that were issued but may not have landed
            const uint32_t n = static_cast<uint32_t>(stages), first = it > n ? it - n : 0;
            for (uint32_t i = first; i < it; ++i)
                wait_bar<false>(full0 + (i % n) * 8u, (i / n) & 1u, abort_flag, args.err, ERR_WAIT_PRODUCER,
                                DRAIN_LIMIT_NS, false);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        constexpr uint32_t idesc = zbp::idesc_bf16_f32(128, ROWS, W_MN, 0);
        constexpr uint32_t W_STEP = W_MN ? 2048 >> 4 : 32 >> 4, hi = zbp::desc_hi(1024);
        const uint32_t a0 = zbp::desc_lo(ring, W_MN ? MN_ATOM_BYTES : 16), b0 = zbp::desc_lo(ring + R_W_BYTES, 16);
        int s = 0;
        uint32_t sp = 0, turn = 0;  // turn: phase of the accumulators' next release
        bool ok = true;
        for (int lo = 0; lo < num_kb && ok; lo += PARTS * seg) {
            if (F32 && lo) {
                if (!wait_bar<false>(zbp::smem_u32(&ctl->tempty), turn, abort_flag, args.err, ERR_WAIT_MMA, WAIT_LIMIT_NS,
                                    true))
                    break;
                zbp::tc_fence_after();
                turn ^= 1u;
            }
            const int given = min(num_kb, lo + PARTS * seg);  // the accumulators are then handed to the epilogue
            uint32_t d_tmem = tmem_base;
            int in_part = 0;
            for (int kb = lo; kb < given; ++kb) {
                if (!wait_bar<false>(full0 + static_cast<uint32_t>(s) * 8u, sp, abort_flag, args.err, ERR_WAIT_MMA,
                                    WAIT_LIMIT_NS, true)) {
                    ok = false;
                    break;
                }
                zbp::tc_fence_after();
                if (zbp::elect_one()) {
                    const uint32_t off = static_cast<uint32_t>(s) * (STAGE >> 4);
                    zbp::mma4_f16<W_STEP, 2>(d_tmem, a0 + off, hi, b0 + off, hi, idesc, in_part != 0);
                    zbp::tc_commit(empty0 + static_cast<uint32_t>(s) * 8u);
                    if (kb + 1 == given) zbp::tc_commit(zbp::smem_u32(&ctl->tfull));
                }
                __syncwarp();
                if (++in_part == seg) {
                    in_part = 0;
                    d_tmem += ROWS;
                }
                if (++s == stages) {
                    s = 0;
                    sp ^= 1u;
                }
            }
        }
        // every MMA issued here completes before TMEM is released
        if (zbp::elect_one()) zbp::tc_commit(zbp::smem_u32(&ctl->drain));
        __syncwarp();
        wait_bar<false>(zbp::smem_u32(&ctl->drain), 0, abort_flag, args.err, ERR_WAIT_MMA, DRAIN_LIMIT_NS, false);
    } else {
        // ---------------------------------------------------- partial tile to shared memory
        constexpr int CHUNKS = ROWS > 64 ? 2 : 1;  // of 32 rows a warp: hf and hf + 2
        const int q = warp & 3, hf = (warp - 2) >> 2;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        auto has = [&](int j) { return hf + 2 * j < ROWS / 32 && (hf + 2 * j) * 32 < live; };
        float x[CHUNKS][32];
        if constexpr (F32)
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
                for (int i = 0; i < 32; ++i) x[j][i] = 0.0f;
        uint32_t turn = 0;
        bool ok = true;
        for (int kb = 0; kb < num_kb; kb += PARTS * seg) {
            if (!wait_bar<false>(zbp::smem_u32(&ctl->tfull), turn, abort_flag, args.err, ERR_WAIT_EPI, WAIT_LIMIT_NS, true)) {
                ok = false;
                break;
            }
            turn ^= 1u;
            zbp::tc_fence_after();
            const int parts = F32 ? min(PARTS, (num_kb - kb + seg - 1) / seg) : 1;  // full ones
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j)
                if (has(j))
#pragma unroll 1
                    for (int p = 0; p < parts; ++p) {
                        uint32_t v[32];
                        zbp::tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(p * ROWS + (hf + 2 * j) * 32), v);
                        zbp::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[j][i] = F32 ? x[j][i] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
                    }
            zbp::tc_fence_before();
            __syncwarp();
            if (F32 && lane == 0) zbp::mbar_arrive(zbp::smem_u32(&ctl->tempty));
        }
        if (ok) {  // every MMA has read its stages, which the partial tile takes the place of
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j)
                if (has(j)) {
                    float* to = reinterpret_cast<float*>(smem) + (hf + 2 * j) * 32 * 128 + q * 32 + lane;
#pragma unroll
                    for (int i = 0; i < 32; ++i) to[i * 128] = x[j][i];
                }
        }
        __syncwarp();
    }

    __syncthreads();
    if (split > 1) zbp::cluster_sync();  // every partial is written
    if (!*abort_flag) {
        const int lo = live * rank / split, items = (live * (rank + 1) / split - lo) * 32;
        for (int i = threadIdx.x; i < items; i += R_THREADS) {
            const int r = lo + (i >> 5), c = (i & 31) * 4;
            if (n0 + c >= args.N) continue;
            const uint32_t at = ring + static_cast<uint32_t>(r * 512 + c * 4);
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (split == 1) {
                const float4 p = zbp::ld_shared_v4(at);
                x[0] = p.x;
                x[1] = p.y;
                x[2] = p.z;
                x[3] = p.w;
            } else {
                float4 p[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < split) p[k] = zbp::ld_shared_cluster_v4(zbp::mapa_shared(at, static_cast<uint32_t>(k)));
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < split) {
                        x[0] += p[k].x;
                        x[1] += p[k].y;
                        x[2] += p[k].z;
                        x[3] += p[k].w;
                    }
            }
            finish4<FORM>(args, m0 + r, n0 + c, x);
        }
    }
    __syncthreads();
    if (split > 1) zbp::cluster_sync();  // no CTA leaves while another may still read its partial
    if (warp == 1) {
        zbp::tc_fence_after();
        zbp::tmem_dealloc(tmem_base, TMEM);
    }
}

// ---------------------------------------------------------------- host side
template <int FORM, int W_MN>
zb_status launch_tiles(const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& o, const CUtensorMap& h,
                       const CUtensorMap& r, const LinearArgs& a, void* stream) {
    static std::atomic<int> cache[64];
    auto kern = zb_linear_tiles_kernel<FORM, W_MN>;
    int ctas = 0;
    const zb_status s = full_grid(kern, cache, TILE_SMEM, TileCfg<FORM>::THREADS, 2, &ctas);
    if (s != ZB_OK) return s;
    const long long tiles = (static_cast<long long>(a.M) + 255) / 256 * ((a.N + a.tile_n - 1) / a.tile_n);
    LaunchCfg cfg(static_cast<int>(std::min<long long>(2 * tiles, ctas)), TileCfg<FORM>::THREADS, TILE_SMEM, 2, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.cfg, kern, x, w, o, h, r, a);
    if (e != cudaSuccess)
        return zb::fail(ZB_ERR_CUDA, std::string("zb_linear_product launch: ") + cudaGetErrorString(e));
    return ZB_OK;
}

constexpr size_t rows_smem(int rows, int stages) {
    const size_t ring = static_cast<size_t>(stages) * rows_stage(rows), tile = static_cast<size_t>(rows) * 512;
    return std::max<size_t>(R_SMEM, 1024 + std::max(ring, tile));
}

template <int FORM, int W_MN, int ROWS>
zb_status launch_rows(const CUtensorMap& x, const CUtensorMap& w, LinearArgs a, void* stream) {
    auto kern = zb_linear_rows_kernel<FORM, W_MN, ROWS>;
    constexpr int MOST = std::min(R_STAGES, static_cast<int>((220 * 1024) / rows_stage(ROWS)));
    // co-resident clusters of 1, 2, 4 and 8 CTAs, per device
    static std::atomic<int> cache[64][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return zb::fail(ZB_ERR_CUDA, "zb_linear_product: cudaGetDevice failed");
    if (!cache[dev][0].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(rows_smem(ROWS, MOST)));
        if (e != cudaSuccess)
            return zb::fail(ZB_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
        for (int i = 3; i >= 0; --i) {
            int n = sm_count();
            if (i > 0) {
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(1024);
                cfg.blockDim = dim3(R_THREADS);
                cfg.dynamicSmemBytes = rows_smem(ROWS, MOST);
                cudaLaunchAttribute attr;
                attr.id = cudaLaunchAttributeClusterDimension;
                attr.val.clusterDim.x = 1u << i;
                attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
                cfg.attrs = &attr;
                cfg.numAttrs = 1;
                if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
                    cudaGetLastError();
                    n = 0;  // no clusters of this size
                }
            }
            if (i == 0 && n <= 0) return zb::fail(ZB_ERR_CUDA, "cannot query the SM count");
            cache[dev][i].store(n, std::memory_order_release);
        }
    }
    const long long tiles = (static_cast<long long>(a.M) + ROWS - 1) / ROWS * ((a.N + 127) / 128);
    const int num_kb = (a.K + BK - 1) / BK;
    // as many CTAs along K as are resident at once, with at least R_MIN_KB blocks each
    int split = 1;
    for (int i = 1; i <= 3; ++i)
        if (cache[dev][i].load(std::memory_order_relaxed) >= tiles && num_kb >= R_MIN_KB << i) split = 1 << i;
    a.tiles_n = (a.N + 127) / 128;
    a.split = split;
    a.stages = std::min(MOST, (num_kb + split - 1) / split);
    LaunchCfg cfg(static_cast<int>(tiles * split), R_THREADS, rows_smem(ROWS, a.stages), split, stream);
    cfg.cfg.numAttrs = split > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg.cfg, kern, x, w, a);
    if (e != cudaSuccess)
        return zb::fail(ZB_ERR_CUDA, std::string("zb_linear_product launch: ") + cudaGetErrorString(e));
    return ZB_OK;
}

bool mis16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// A row stride given as 0 is the row's width; false if it is not legal.
bool stride(int64_t* ld, int64_t width) {
    if (*ld == 0) *ld = width;
    return *ld >= width && *ld <= (1LL << 30);
}

// Columns of a tile: those for which the rounds of tiles that a CTA pair takes
// cost least; what a tile costs goes with the operands' bytes, 256 rows and its
// columns.  W's copies come in columns of 64 for each CTA of the pair unless it
// lies along K (transposed), so there the columns are 256 or 128.
// 256 and 224 columns, GeLU' with residual, K 1024 (and 1536): 4096 x 4096 39.0
// and 36.1 us, 2048 x 4096 23.5 and 22.0, 4096 x 6144 66.0 and 63.2.
int choose_tile_n(int64_t M, int64_t N, bool along_k) {
    const int64_t pairs = std::max(sm_count() / 2, 1), tm = (M + 255) / 256;
    int best = BN;
    int64_t least = INT64_MAX;
    for (int tn = BN; tn >= 128; tn -= along_k ? 32 : 128) {
        const int64_t cost = (tm * ((N + tn - 1) / tn) + pairs - 1) / pairs * (256 + tn);
        if (cost < least) {
            least = cost;
            best = tn;
        }
    }
    return best;
}

// The rows kernel's tile: as few rows as hold M, 128 at most.
int rows_of(int64_t M) { return M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// The rows kernel for up to 32 rows, for up to 64 unless its tiles outnumber the
// SMs, and for more where it can split K as often as pays.  us of the tiles and
// the rows kernel with residual:
//   16 x 1024    K 4096  20    5.3      16 x 16384   K 1024  12.7   8.2
//   64 x 4096    K 1024   6.5  5.6      64 x 32768   K 1024  17.6  25.1
//   256 x 1024   K 1024   6.6  5.9      512 x 1024   K  512   5.5   6.4
//   512 x 1024   K 1024   6.7  7.0      512 x 1024   K 4096  14.1   9.8
//   512 x 2048   K 1024   6.8  8.5      512 x 2048   K 4096  16.4  15.9
//   1024 x 2048  K 1024   7.6 10.1      1024 x 2048  K 4096  19.5  25.2
bool use_rows(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = (M + rows_of(M) - 1) / rows_of(M) * ((N + 127) / 128), sms = sm_count();
    if (M <= 32) return true;
    if (M <= 64) return tiles <= sms;
    return tiles <= sms / 8 || (tiles <= sms / 4 && K >= 2048) || (tiles <= sms / 2 && K >= 4096);
}

template <int FORM, int W_MN>
zb_status product(const zb_linear& g, int64_t ldx, int64_t ldw, const void* X, const void* W, LinearArgs a,
                  void* stream) {
    std::string why;
    CUtensorMap x, w, o, h, r;
    const bool rows = use_rows(g.M, g.N, g.K);
    a.tile_n = choose_tile_n(g.M, g.N, !W_MN);
    const uint32_t w_rows = rows ? 128 : static_cast<uint32_t>(a.tile_n / 2);
    const uint32_t x_rows = rows ? static_cast<uint32_t>(rows_of(g.M)) : 128;
    bool ok = make_map(&x, X, false, g.K, g.M, ldx, BK, x_rows, &why) &&
              (W_MN ? make_map(&w, W, false, g.N, g.K, ldw, 64, BK, &why)
                    : make_map(&w, W, false, g.K, g.N, ldw, BK, w_rows, &why));
    if (!ok) return zb::fail(ZB_ERR_CUDA, why);
    if (rows) {
        if (x_rows == 32) return launch_rows<FORM, W_MN, 32>(x, w, a, stream);
        if (x_rows == 64) return launch_rows<FORM, W_MN, 64>(x, w, a, stream);
        return launch_rows<FORM, W_MN, 128>(x, w, a, stream);
    }
    constexpr bool f32 = FORM == STORE32;
    constexpr CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_64B;
    constexpr uint32_t cols = TileCfg<FORM>::COLS;
    ok = make_map(&o, FORM == GELU ? a.out1 : a.out0, f32, g.N, g.M, a.ldo, cols, 32, &why, sw);
    h = r = o;
    if (ok && FORM == GELU && a.save) ok = make_map(&h, a.out0, false, g.N, g.M, a.ldo, cols, 32, &why, sw);
    if (ok && FORM == GRAD) ok = make_map(&h, a.H, false, g.N, g.M, a.ldh, cols, 32, &why, sw);
    if (ok && a.R) ok = make_map(&r, a.R, f32, g.N, g.M, a.ldr, cols, 32, &why, sw);
    if (!ok) return zb::fail(ZB_ERR_CUDA, why);
    zb::GemmBf16 gm;
    gm.Mg = g.M;
    gm.Ng = g.N;
    gm.Kg = g.K;
    gm.epi = f32 ? zb::EPI_F32 : zb::EPI_STORE_BF16;
    EpiArgs ea;
    choose_l2_hints(gm, 2, &ea);
    a.hint_a = ea.hint_a;
    a.hint_b = ea.hint_b;
    a.hint_out = ea.hint_out;
    a.hint_once = l2_hints() ? 1 : 0;
    return launch_tiles<FORM, W_MN>(x, w, o, h, r, a, stream);
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
    unsigned int* err = zb::device_error_word();
    if (!err) return ZB_ERR_CUDA;
    LinearArgs a = {};
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.H = static_cast<const __nv_bfloat16*>(H);
    a.R = R;
    a.out0 = out0;
    a.out1 = out1;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldo = ldo;
    a.M = static_cast<int>(g->M);
    a.N = static_cast<int>(g->N);
    a.K = static_cast<int>(g->K);
    a.save = gelu && out0 != nullptr;
    a.tanh_form = g->act == ZB_ACT_GELU_TANH;
    a.err = err;
    auto go = [&](auto form) {
        constexpr int F = form();
        return g->transposed ? product<F, 0>(*g, ldx, ldw, X, W, a, stream) : product<F, 1>(*g, ldx, ldw, X, W, a, stream);
    };
    zb_status s;
    if (g->dtype == ZB_DT_F32)
        s = go(std::integral_constant<int, STORE32>());
    else if (gelu)
        s = go(std::integral_constant<int, GELU>());
    else if (grad)
        s = go(std::integral_constant<int, GRAD>());
    else
        s = go(std::integral_constant<int, STORE>());
    if (s == ZB_OK) zb::clear_error();
    return s;
}
