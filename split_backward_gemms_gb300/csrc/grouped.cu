// grouped.cu — matrix products grouped by expert with ragged rows: F, B and W
// of a mixture-of-experts stage's blocks.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <string>

#include "grouped.cuh"

namespace {

constexpr int MAX_TOK = 32;  // tokens of one epilogue chunk

// Rows [lo, hi) of expert e, kept inside [0, rows] whatever the offsets say.
__device__ __forceinline__ void expert_rows(const int* offsets, int e, int rows, int& lo, int& hi) {
    lo = min(max(offsets[e], 0), rows);
    hi = max(min(offsets[e + 1], rows), lo);
}

// ---------------------------------------------------------------- F and B
// D[row, n] = sum_k A[row, k] W_e(k, n) for the rows of every expert e, as the
// transposed product D^T = W_e^T A^T: the weights' columns are the MMA's M side
// (128 for one CTA, 256 for a pair: always full but for the matrix edge) and
// an expert's rows its N side, whose extent is any multiple of 16 (32 for a
// pair) chosen per tile.  So a ragged expert costs its own rows rounded up to
// 16 or 32, not to 128 or 256, and one row (a decoding step) costs little more
// than streaming the weights.  The roles, the ring and the two accumulators
// are those of the dense kernel (gemm_tc.cu): warp 0 copies, warp 1 issues
// MMAs, warps 2-9 drain.  Tiles are walked in a fixed order; every role walks
// the experts' offsets (in shared memory) by itself.
//
// Epilogue: a TMEM lane is a column n of D and a TMEM column a row of D, so a
// chunk of 32 lanes x 32 columns is read as 8 x 8 fragments (16x256b loads),
// rounded to bf16 pairs of rows and transposed on its way to the staging box
// by stmatrix; H (for GeLU') comes the same way back, by TMA and ldmatrix.  A
// box of 32 rows leaves by a TMA store; the last, partial box of an expert by
// plain stores of its live rows, since the rows after it are another expert's.
//
// With a few rows an expert (SHAPE FEW) the weights are all that counts, and a
// CTA's rate is that of its MMA thread: a wait, four small MMAs and a commit take
// 370 cycles a K block, whatever the block's bytes, which the MMAs of larger
// tiles hide.  So a stage there has four K blocks (and 32 rows, not 128), one
// wait and one commit; and where tiles of 128 columns would leave half of the
// SMs idle, they have 64.  The MMA has 128 columns all the same: the upper 64 of
// a narrow tile are whatever lies behind its weights in the ring, and their
// products are not read back.  16 rows, 8 experts, K 4096, N 1024: 17.3 us with
// one block a stage, 13.8 with two, 12.1 with four (5.5 TB/s).
enum Shape { FEW = 0, ONE = 1, PAIRS = 2 };
template <int SHAPE>
struct RowsCfg {
    static constexpr int CG = SHAPE == PAIRS ? 2 : 1;
    static constexpr int TILE_T = SHAPE == FEW ? 32 : 128 * CG;  // rows of D per tile, at most
    static constexpr int N_STEP = 16 * CG;                       // granularity of the MMA's N
    static constexpr int KPS = SHAPE == FEW ? 4 : 1;             // K blocks of a stage
    static constexpr uint32_t STAGE = 32 * 1024;                 // 16 KiB of weights, 16 KiB of rows (not FEW)
    static constexpr uint32_t TMEM = 2 * TILE_T;
};
template <int EPI>
struct RowsEpi {
    static constexpr int STAGES = EPI == zb::EPI_GELU_BWD ? 5 : 6;
    static constexpr int BOXES = EPI == zb::EPI_GELU_BWD ? 4 : 2;  // staging boxes per warp
};
constexpr uint32_t ROW_BOX = 32 * 64;  // 32 rows x 32 columns of bf16
constexpr int EPI_WARPS = 8;
constexpr int MAX_STAGES = 16;

struct RowsCtl {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], drain;
    uint64_t hbar[EPI_WARPS][4];  // H boxes
    uint32_t tmem_base;
    int abort_flag;
    int off[MAX_EXPERTS + 1];  // legal, ascending
};

template <int EPI>
constexpr size_t rows_smem() {
    return 1024 + RowsEpi<EPI>::STAGES * RowsCfg<ONE>::STAGE + EPI_WARPS * RowsEpi<EPI>::BOXES * ROW_BOX + sizeof(RowsCtl);
}
static_assert(rows_smem<zb::EPI_GELU_BWD>() <= 232448 && rows_smem<zb::EPI_GELU_DUAL>() <= 232448, "shared memory");

struct RowsArgs {
    const int* offsets;
    const __nv_bfloat16* bias;  // [E, N] or nullptr
    __nv_bfloat16 *out0, *out1;
    int rows, experts, N, K, act;
    int tile_f;  // columns of D per tile: 128, 64 (FEW) or 256 (PAIRS)
    unsigned int* err;
};

template <int EPI, int A_MN, int SHAPE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    zb_moe_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA128,
                       const __grid_constant__ CUtensorMap tmA32, const __grid_constant__ CUtensorMap tmO0,
                       const __grid_constant__ CUtensorMap tmO1, const RowsArgs args) {
    using C = RowsCfg<SHAPE>;
    constexpr int CG = C::CG;
    constexpr bool PAIR = CG == 2;
    constexpr int BOXES = RowsEpi<EPI>::BOXES;
    constexpr uint32_t RING = RowsEpi<EPI>::STAGES * C::STAGE;
    const int tile_f = SHAPE == FEW ? args.tile_f : 128 * CG;
    const uint32_t w_bytes = static_cast<uint32_t>(tile_f / CG) * BK * 2u;  // of a stage in one CTA; the rows follow
    const uint32_t BLOCK = SHAPE == FEW ? w_bytes + 32u * BK * 2u : C::STAGE;  // a K block in the ring
    const uint32_t STAGE = C::KPS * BLOCK;
    const int STAGES = SHAPE == FEW ? min(MAX_STAGES, static_cast<int>(RING / STAGE)) : RowsEpi<EPI>::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + RING;
    RowsCtl* ctl = reinterpret_cast<RowsCtl*>(staging + EPI_WARPS * BOXES * ROW_BOX);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? zbp::cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
    const int tiles_f = (args.N + tile_f - 1) / tile_f;
    const int num_kb = (args.K + BK - 1) / BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            zbp::mbar_init(zbp::smem_u32(&ctl->full[s]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            zbp::mbar_init(zbp::smem_u32(&ctl->tfull[b]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->tempty[b]), EPI_WARPS * CG);
        }
        zbp::mbar_init(zbp::smem_u32(&ctl->drain), 1);
        if (EPI == zb::EPI_GELU_BWD)
            for (int w = 0; w < EPI_WARPS; ++w)
                for (int b = 0; b < 4; ++b) zbp::mbar_init(zbp::smem_u32(&ctl->hbar[w][b]), 1);
        ctl->abort_flag = 0;
        zbp::fence_mbar_init();
        zbp::tma_prefetch_desc(&tmW);
        zbp::tma_prefetch_desc(&tmA128);
        zbp::tma_prefetch_desc(&tmA32);
        zbp::tma_prefetch_desc(&tmO0);
        if (EPI != zb::EPI_STORE_BF16) zbp::tma_prefetch_desc(&tmO1);
    }
    if (warp == 1) {
        if (PAIR) {
            zbp::tmem_alloc_pair(zbp::smem_u32(&ctl->tmem_base), C::TMEM);
            zbp::tmem_relinquish_pair();
        } else {
            zbp::tmem_alloc(zbp::smem_u32(&ctl->tmem_base), C::TMEM);
            zbp::tmem_relinquish();
        }
    }
    zbp::tc_fence_before();
    __syncthreads();
    if (PAIR) zbp::cluster_sync();
    zbp::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    load_offsets(ctl->off, args.offsets, args.experts, args.rows);

    Walk<C::TILE_T, true> walk(ctl->off, args.experts, tiles_f);
    int row0 = 0, nrows = 0, fb = 0;
    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
        const uint32_t full0_lead = PAIR ? zbp::mapa_shared(full0, 0) : full0;
        const uint32_t sa0 = zbp::smem_u32(smem);
        uint32_t s = 0, sp = 1, it = 0;  // stage and the phase of its last release; stages filled
        bool ok = true;
        for (int tile = cluster; ok && walk.to(tile, row0, nrows, fb); tile += clusters) {
            const int f0 = fb * tile_f + static_cast<int>(rank) * 128;
            const int mma_n = (nrows + C::N_STEP - 1) / C::N_STEP * C::N_STEP;
            const int half = mma_n / CG;  // rows in this CTA
            const int r0 = row0 + static_cast<int>(rank) * half;
            const int boxes = (half + 31) / 32;
            const uint32_t bytes = CG * (w_bytes + static_cast<uint32_t>(boxes) * 32u * BK * 2u);
            for (int kb = 0; kb < num_kb; kb += C::KPS, ++it) {
                if (!wait_bar<false>(empty0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_PRODUCER, WAIT_LIMIT_NS, true)) {
                    ok = false;
                    break;
                }
                if (zbp::elect_one()) {
                    const uint32_t full = full0_lead + s * 8u;
                    const int blocks = min(C::KPS, num_kb - kb);
                    if (leader) zbp::mbar_arrive_expect_tx(full0 + s * 8u, bytes * static_cast<uint32_t>(blocks));
#pragma unroll
                    for (int j = 0; j < C::KPS; ++j) {
                        if (j >= blocks) break;
                        const uint32_t sa = sa0 + s * STAGE + static_cast<uint32_t>(j) * BLOCK, sb = sa + w_bytes;
                        const int k0 = (kb + j) * BK;
                        auto load_w = [&](uint32_t dst, int x, int y) {
                            if (PAIR)
                                zbp::tma_load_3d_pair(dst, &tmW, full, x, y, walk.e);
                            else
                                zbp::tma_load_3d(dst, &tmW, full, x, y, walk.e);
                        };
                        auto load_a = [&](uint32_t dst, const CUtensorMap* tm, int y) {
                            if (PAIR)
                                zbp::tma_load_2d_pair(dst, tm, full, k0, y);
                            else
                                zbp::tma_load_2d(dst, tm, full, k0, y);
                        };
                        if (A_MN) {
                            load_w(sa, f0, k0);
                            if (tile_f > 64) load_w(sa + MN_ATOM_BYTES, f0 + 64, k0);
                        } else {
                            load_w(sa, k0, f0);
                        }
                        if (boxes == 4) {
                            load_a(sb, &tmA128, r0);
                        } else {
#pragma unroll
                            for (int b = 0; b < 3; ++b)
                                if (b < boxes) load_a(sb + static_cast<uint32_t>(b) * 32u * BK * 2u, &tmA32, r0 + 32 * b);
                        }
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
                wait_bar<false>(zbp::smem_u32(&ctl->full[i % STAGES]), (i / STAGES) & 1u, abort_flag, args.err,
                                ERR_WAIT_PRODUCER, DRAIN_LIMIT_NS, false);
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t A_STEP = A_MN ? 2048 >> 4 : 32 >> 4, hi = zbp::desc_hi(1024);
            const uint32_t a0 = zbp::desc_lo(zbp::smem_u32(smem), A_MN ? MN_ATOM_BYTES : 16);
            const uint32_t b0 = zbp::desc_lo(zbp::smem_u32(smem) + w_bytes, 16);
            const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
            uint32_t s = 0, sp = 0, local = 0;  // stage and its phase; tile
            bool ok = true;
            for (int tile = cluster; ok && walk.to(tile, row0, nrows, fb); tile += clusters, ++local) {
                const uint32_t buf = local & 1u, tr = local >> 1;
                if (!wait_bar<false>(zbp::smem_u32(&ctl->tempty[buf]), (tr & 1u) ^ 1u, abort_flag, args.err,
                                     ERR_WAIT_MMA, WAIT_LIMIT_NS, true))
                    break;
                const uint32_t d_tmem = tmem_base + buf * C::TILE_T;
                const uint32_t mma_n = static_cast<uint32_t>((nrows + C::N_STEP - 1) / C::N_STEP * C::N_STEP);
                const uint32_t idesc = zbp::idesc_bf16_f32(128 * CG, mma_n, A_MN, 0);
                for (int kb = 0; kb < num_kb; kb += C::KPS) {
                    if (!wait_bar<false>(full0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        break;
                    }
                    zbp::tc_fence_after();
                    if (zbp::elect_one()) {
                        const uint32_t off = s * (STAGE >> 4);
                        if (PAIR) {
                            zbp::mma4_f16_pair<A_STEP, 2>(d_tmem, a0 + off, hi, b0 + off, hi, idesc, kb != 0);
                            zbp::tc_commit_pair_multicast(empty0 + s * 8u, 0x3);
                            if (kb + 1 == num_kb) zbp::tc_commit_pair_multicast(zbp::smem_u32(&ctl->tfull[buf]), 0x3);
                        } else {
                            zbp::mma4_f16<A_STEP, 2>(d_tmem, a0 + off, hi, b0 + off, hi, idesc, kb != 0);
#pragma unroll
                            for (int j = 1; j < C::KPS; ++j) {
                                const uint32_t o = off + static_cast<uint32_t>(j) * (BLOCK >> 4);
                                if (kb + j < num_kb) zbp::mma4_f16<A_STEP, 2>(d_tmem, a0 + o, hi, b0 + o, hi, idesc, 1);
                            }
                            zbp::tc_commit(empty0 + s * 8u);
                            if (kb + C::KPS >= num_kb) zbp::tc_commit(zbp::smem_u32(&ctl->tfull[buf]));
                        }
                    }
                    __syncwarp();
                    if (++s == STAGES) {
                        s = 0;
                        sp ^= 1u;
                    }
                }
            }
            // every MMA issued here completes before TMEM is released
            if (zbp::elect_one()) {
                if (PAIR)
                    zbp::tc_commit_pair(zbp::smem_u32(&ctl->drain));
                else
                    zbp::tc_commit(zbp::smem_u32(&ctl->drain));
            }
            __syncwarp();
            wait_bar<false>(zbp::smem_u32(&ctl->drain), 0, abort_flag, args.err, ERR_WAIT_MMA, DRAIN_LIMIT_NS, false);
        }
    } else {
        // ---------------------------------------------------- epilogue
        const int ew = warp - 2, q = warp & 3, hf = ew >> 2;
        const uint32_t stg0 = zbp::smem_u32(staging + ew * BOXES * ROW_BOX);
        // this lane's address in a box for the matrix moves: matrix lane/8 is
        // an 8-column block, memory row lane%8 a row of D (64-byte swizzle)
        const int mr = lane & 7, mb = lane >> 3;
        uint32_t local = 0;
        uint32_t g = 0;       // boxes filled so far (GeLU': chunks)
        uint32_t issued = 0;  // H boxes asked for
        bool ok = true;
        for (int tile = cluster; ok && walk.to(tile, row0, nrows, fb); tile += clusters, ++local) {
            const uint32_t buf = local & 1u, tr = local >> 1;
            const int n0 = fb * tile_f + static_cast<int>(rank) * 128 + q * 32;  // first column of D
            const int chunks = (nrows + MAX_TOK - 1) / MAX_TOK;
            const bool cols_live = n0 < args.N && (SHAPE != FEW || q * 32 < tile_f);
            const int mine = cols_live ? (chunks - hf + 1) / 2 : 0;  // chunks hf, hf + 2, ...
            auto ask_h = [&](int i) {  // chunk i of mine: H into box (g0 + i) % 4
                if (lane == 0) {
                    const uint32_t b = issued & 3u;
                    const uint32_t bar = zbp::smem_u32(&ctl->hbar[ew][b]);
                    zbp::mbar_arrive_expect_tx(bar, ROW_BOX);
                    zbp::tma_load_2d(stg0 + b * ROW_BOX, &tmO1, bar, n0, row0 + (hf + 2 * i) * MAX_TOK);
                }
                ++issued;
            };
            if (EPI == zb::EPI_GELU_BWD && mine > 0) {
                // at most the last two boxes' stores still read them
                if (lane == 0) zbp::bulk_wait_read<2>();
                ask_h(0);
                if (mine > 1) ask_h(1);
            }
            float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (EPI != zb::EPI_GELU_BWD && args.bias && cols_live) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = n0 + i * 8 + (lane >> 2);
                    if (n < args.N) bias[i] = __bfloat162float(args.bias[static_cast<long long>(walk.e) * args.N + n]);
                }
            }
            if (!wait_bar<false>(zbp::smem_u32(&ctl->tfull[buf]), tr & 1u, abort_flag, args.err, ERR_WAIT_EPI,
                                WAIT_LIMIT_NS, true))
                break;
            zbp::tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * C::TILE_T;
#pragma unroll 1
            for (int i = 0; i < mine; ++i) {
                const int c = hf + 2 * i;
                uint32_t v[2][16];
                zbp::tmem_ld_16x256b_x4(taddr + c * MAX_TOK, v[0]);
                zbp::tmem_ld_16x256b_x4(taddr + (16u << 16) + c * MAX_TOK, v[1]);
                const int row = row0 + c * MAX_TOK;
                const int live = nrows - c * MAX_TOK;  // rows of this chunk
                if (EPI == zb::EPI_GELU_BWD && i + 2 < mine) {
                    if (lane == 0) zbp::bulk_wait_read<1>();
                    ask_h(i + 2);
                }
                // one box of bf16 pairs: w[j][fb]: rows 8j + 2(t%4), +1 of column block fb
                auto store = [&](const CUtensorMap* tm, __nv_bfloat16* out, uint32_t stg, const uint32_t (&w)[4][4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int rr = 8 * j + mr;
                        zbp::stmatrix_x4_trans(stg + static_cast<uint32_t>(rr * 64 + ((mb ^ ((rr >> 1) & 3)) << 4)),
                                               w[j][0], w[j][1], w[j][2], w[j][3]);
                    }
                    if (live >= MAX_TOK) {
                        zbp::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            zbp::tma_store_2d(tm, stg, n0, row);
                            zbp::bulk_commit();
                        }
                    } else {
                        __syncwarp();
                        if (lane < live) {
                            __nv_bfloat16* o = out + static_cast<long long>(row + lane) * args.N + n0;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (n0 + 8 * k < args.N) {
                                    const float4 x = zbp::ld_shared_v4(
                                        stg + static_cast<uint32_t>(lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)));
                                    *reinterpret_cast<float4*>(o + 8 * k) = x;
                                }
                        }
                        zbp::fence_proxy_async_smem();  // the box may be a copy's target next
                        __syncwarp();
                        if (lane == 0) zbp::bulk_commit();  // an empty group: groups count boxes
                    }
                };
                uint32_t hw[4][4];
                uint32_t hstg = 0;
                if (EPI == zb::EPI_GELU_BWD) {
                    const uint32_t b = g & 3u;
                    if (!wait_bar<false>(zbp::smem_u32(&ctl->hbar[ew][b]), (g >> 2) & 1u, abort_flag, args.err,
                                         ERR_WAIT_EPI, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        break;
                    }
                    hstg = stg0 + b * ROW_BOX;
                    ++g;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int rr = 8 * j + mr;
                        zbp::ldmatrix_x4_trans(hstg + static_cast<uint32_t>(rr * 64 + ((mb ^ ((rr >> 1) & 3)) << 4)),
                                               hw[j][0], hw[j][1], hw[j][2], hw[j][3]);
                    }
                }
                zbp::tmem_ld_wait();
                // x[j * 8 + 2 fb + p]: row 8j + 2(t%4) + p, column block fb
                float x[32];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int f = 0; f < 4; ++f)
#pragma unroll
                        for (int p = 0; p < 2; ++p)
                            x[j * 8 + f * 2 + p] = __uint_as_float(v[f >> 1][4 * j + 2 * (f & 1) + p]) +
                                                   (EPI == zb::EPI_GELU_BWD ? 0.0f : bias[f]);
                if (EPI == zb::EPI_GELU_BWD) {
                    uint32_t hf32[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int f = 0; f < 4; ++f) hf32[j * 4 + f] = hw[j][f];
                    if (args.act == ZB_ACT_GELU_TANH)
                        gelu_grad_mul<true, 32>(x, hf32);
                    else
                        gelu_grad_mul<false, 32>(x, hf32);
                }
                uint32_t w[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int f = 0; f < 4; ++f) w[j][f] = pack_bf16x2(x[j * 8 + f * 2], x[j * 8 + f * 2 + 1]);
                if (EPI == zb::EPI_GELU_BWD) {
                    __syncwarp();  // every lane has read H from this box
                    store(&tmO0, args.out0, hstg, w);
                } else {
                    uint32_t stg = stg0 + (g & 1u) * ROW_BOX;
                    ++g;
                    staging_acquire(lane);
                    store(&tmO0, args.out0, stg, w);
                    if (EPI == zb::EPI_GELU_DUAL) {
                        uint32_t a[16];
                        if (args.act == ZB_ACT_GELU_TANH)
                            gelu_pack<true, 32>(x, a);
                        else
                            gelu_pack<false, 32>(x, a);
                        uint32_t w2[4][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int f = 0; f < 4; ++f) w2[j][f] = a[j * 4 + f];
                        stg = stg0 + (g & 1u) * ROW_BOX;
                        ++g;
                        staging_acquire(lane);
                        store(&tmO1, args.out1, stg, w2);
                    }
                }
            }
            if (!ok) break;
            zbp::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t te = zbp::smem_u32(&ctl->tempty[buf]);
                if (PAIR)
                    zbp::mbar_arrive_remote(zbp::mapa_shared(te, 0));
                else
                    zbp::mbar_arrive(te);
            }
        }
        if (EPI == zb::EPI_GELU_BWD)  // H boxes asked for and not used (after an abort)
            for (; g != issued; ++g)
                wait_bar<false>(zbp::smem_u32(&ctl->hbar[ew][g & 3u]), (g >> 2) & 1u, abort_flag, args.err, ERR_WAIT_EPI,
                                DRAIN_LIMIT_NS, false);
        // the staging boxes must not be released while a bulk store reads them
        if (lane == 0) zbp::bulk_wait<0>();
        __syncwarp();
    }

    __syncthreads();
    if (PAIR) zbp::cluster_sync();  // no remote arrivals or copies remain
    if (warp == 1) {
        zbp::tc_fence_after();
        if (PAIR)
            zbp::tmem_dealloc_pair(tmem_base, C::TMEM);
        else
            zbp::tmem_dealloc(tmem_base, C::TMEM);
    }
}

// ---------------------------------------------------------------- W
// dW[e][m][n] (+)= sum over the rows r of e of A[r][m] B[r][n], both of the
// pass's products in one launch.  The contraction runs over an expert's rows,
// so its last block of 64 must not see the next expert's: once a partial block
// has landed, warps 2 and 3 overwrite the rows past the expert's end with zeros
// in both operands (an infinity or NaN there would not vanish times zero).  Its
// copies complete on a barrier of their own CTA (part), and the two warps of
// each CTA arrive on the MMA's (edge).  Both operands are read as they lie
// (MN-major: a row of 64 values is a line of 128 bytes, whatever the swizzle).
//
// The tensor core cuts off low bits as it accumulates, so the error of one
// long accumulator grows with its length (1.0e-6 of the result after 1024 rows,
// 2.6e-6 after 2500, 1.9e-5 after 16384).  So an accumulator takes W_SEG
// blocks of rows only; the 8 epilogue warps (32 lanes x 128 columns each) add
// the partial sums in registers, rounding to nearest, while the MMAs of the
// next segment fill the other accumulator.  The fp32 tile goes out through 32 x
// 32 staging boxes, added in place by TMA reduce-adds when accumulating (one
// add per element: no order to vary).
//
// W_SEG trades error for time, since the epilogue reads an accumulator once a
// segment.  Error of experts of 512 to 16384 rows, and microseconds of W of 16384
// rows, 16 experts, h 1024, f 4096 (overwriting, accumulating) and of 8 experts, h
// 2048, f 8192 (the same):
//   W_SEG 4   2.3e-7 to 2.7e-7   255, 287   763, 791
//   W_SEG 6   3.1e-7 to 3.7e-7   230, 279   701, 756
//   W_SEG 8   4.6e-7 to 4.8e-7   226, 279   679, 753
// where a library product in fp32 is 1.6e-7 to 4.4e-7 off.  8 is the choice: an
// eleventh less time than 4 for twice its error, which is still a fifth of that of
// the dense block's W (2.4e-6).
//
// The stores share the copy unit with the next tile's loads and, issued at once,
// queue before them.  So a tile's four chunks a warp go out W_PACE cycles times
// its blocks of rows apart (at most W_PACE_MOST), which spreads them over about
// the time in which the MMAs fill the two accumulators anew.  W of 16384 rows,
// 16 experts, h 1024, f 4096: 249 us unpaced, 247 at 1000 cycles at most, 232 at
// 1500, 226 at 2200, 234 at 3500 (of 400 a block); of 24570 rows, 64 experts (6
// blocks each): 413, 406, 391, 386, 435.  Accumulating, the first is 308, 306, 296,
// 279 and 267: the reduce-adds take longer than stores and would bear a slower pace.
constexpr int W_SEG = 8;  // blocks of 64 rows
constexpr int W_PACE = 250, W_PACE_MOST = 2200;
// Warp 0 copies, warp 1 issues MMAs, warps 2 and 3 clear rows; warps 4-11 sum
// and store, with the registers that warps 0-3 give up (128 sums a thread).
constexpr int W_THREADS = 384;
constexpr int W_REGS_LOW = 40, W_REGS_HIGH = 232;
static_assert(128 * W_REGS_LOW + 256 * W_REGS_HIGH <= W_THREADS * 168, "register split");
constexpr uint32_t W_BOX = 32 * 128;  // 32 x 32 fp32
constexpr int W_BOXES = 2;            // staging boxes a warp
template <int CG>
struct WCfg {
    static constexpr int STAGES = CG == 1 ? 3 : 5;
};
struct WArgs {
    const int* offsets;
    int rows, experts, products;
    int M[2], N[2];
    int accumulate;
    unsigned int* err;
};
template <int CG>
struct WCtl {
    uint64_t full[6], empty[6], part[6], edge[6], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    int off[MAX_EXPERTS + 1];
};
template <int CG>
constexpr size_t w_smem() {
    return 1024 + WCfg<CG>::STAGES * Cfg<CG>::STAGE_BYTES + 8 * W_BOXES * W_BOX + sizeof(WCtl<CG>);
}
static_assert(w_smem<1>() <= 232448 && w_smem<2>() <= 232448, "shared memory");

template <int CG>
__global__ void __launch_bounds__(W_THREADS, 1)
    zb_moe_wgrad_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
                        const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB1,
                        const __grid_constant__ CUtensorMap tmO0, const __grid_constant__ CUtensorMap tmO1,
                        const WArgs args) {
    using C = Cfg<CG>;
    constexpr int STAGES = WCfg<CG>::STAGES;
    constexpr bool PAIR = CG == 2;
    constexpr int WARPS = 8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + STAGES * C::STAGE_BYTES;
    WCtl<CG>* ctl = reinterpret_cast<WCtl<CG>*>(staging + WARPS * W_BOXES * W_BOX);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? zbp::cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
    const int tm0 = (args.M[0] + C::TILE_M - 1) / C::TILE_M, tn0 = (args.N[0] + BN - 1) / BN;
    const int tm1 = args.products > 1 ? (args.M[1] + C::TILE_M - 1) / C::TILE_M : 0;
    const int tn1 = args.products > 1 ? (args.N[1] + BN - 1) / BN : 0;
    const int per = tm0 * tn0 + tm1 * tn1;  // tiles of one expert
    const int num_tiles = per * args.experts;
    // expert, product and block of a tile
    auto locate = [&](int tile, int& e, int& mb, int& nb) -> int {
        e = tile / per;
        int t = tile - e * per;
        if (t < tm0 * tn0) {
            tile_coords(t, tm0, tn0, C::GROUP_M, mb, nb);
            return 0;
        }
        tile_coords(t - tm0 * tn0, tm1, tn1, C::GROUP_M, mb, nb);
        return 1;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            zbp::mbar_init(zbp::smem_u32(&ctl->full[s]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->empty[s]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->part[s]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->edge[s]), 2 * CG);
        }
        for (int b = 0; b < 2; ++b) {
            zbp::mbar_init(zbp::smem_u32(&ctl->tfull[b]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->tempty[b]), WARPS * CG);
        }
        zbp::mbar_init(zbp::smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        zbp::fence_mbar_init();
        zbp::tma_prefetch_desc(&tmA0);
        zbp::tma_prefetch_desc(&tmB0);
        zbp::tma_prefetch_desc(&tmO0);
        if (args.products > 1) {
            zbp::tma_prefetch_desc(&tmA1);
            zbp::tma_prefetch_desc(&tmB1);
            zbp::tma_prefetch_desc(&tmO1);
        }
    }
    if (warp == 1) {
        if (PAIR) {
            zbp::tmem_alloc_pair(zbp::smem_u32(&ctl->tmem_base), TMEM_COLS);
            zbp::tmem_relinquish_pair();
        } else {
            zbp::tmem_alloc(zbp::smem_u32(&ctl->tmem_base), TMEM_COLS);
            zbp::tmem_relinquish();
        }
    }
    zbp::tc_fence_before();
    __syncthreads();
    if (PAIR) zbp::cluster_sync();
    zbp::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    load_offsets(ctl->off, args.offsets, args.experts, args.rows);
    auto blocks_of = [&](int e) { return (ctl->off[e + 1] - ctl->off[e] + BK - 1) / BK; };

    if (warp < 4) {
        zbp::regs_dec<W_REGS_LOW>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
            const uint32_t full0_lead = PAIR ? zbp::mapa_shared(full0, 0) : full0;
            const uint32_t sa0 = zbp::smem_u32(smem);
            const uint32_t part0 = zbp::smem_u32(&ctl->part[0]);
            uint32_t s = 0, sp = 1, it = 0;  // stage and the phase of its last release; stages filled
            uint32_t pending = 0, pp = 0;    // a bit a stage: last filled with a partial block; phase of part
            bool ok = true;
            for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
                int e, mb, nb;
                const int p = locate(tile, e, mb, nb);
                const int num_kb = blocks_of(e);
                if (num_kb == 0) continue;
                const int first = ctl->off[e], n = ctl->off[e + 1] - first;
                const int m0 = mb * C::TILE_M + static_cast<int>(rank) * BM;
                const int nb0 = nb * BN + static_cast<int>(rank) * C::B_ROWS;
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    if (!wait_bar<false>(empty0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_PRODUCER, WAIT_LIMIT_NS,
                                         true)) {
                        ok = false;
                        break;
                    }
                    const bool partial = kb * BK + BK > n;
                    // a stage is filled again after its partial block was used
                    if ((pending >> s) & 1u) pp ^= 1u << s;
                    pending = (pending & ~(1u << s)) | (partial ? 1u << s : 0u);
                    if (zbp::elect_one()) {
                        const uint32_t sa = sa0 + s * C::STAGE_BYTES, sb = sa + A_BYTES;
                        const uint32_t bar = partial ? part0 + s * 8u : full0_lead + s * 8u;
                        if (partial) {
                            zbp::mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
                            if (leader) zbp::mbar_arrive(full0 + s * 8u);
                        } else if (leader) {
                            zbp::mbar_arrive_expect_tx(full0 + s * 8u, C::STAGE_BYTES * CG);
                        }
                        const CUtensorMap* tma = p ? &tmA1 : &tmA0;
                        const CUtensorMap* tmb = p ? &tmB1 : &tmB0;
                        const int y = first + kb * BK;
                        auto load = [&](uint32_t dst, const CUtensorMap* tm, int x) {
                            if (PAIR && !partial)
                                zbp::tma_load_2d_pair(dst, tm, bar, x, y);
                            else
                                zbp::tma_load_2d(dst, tm, bar, x, y);
                        };
                        load(sa, tma, m0);
                        load(sa + MN_ATOM_BYTES, tma, m0 + 64);
#pragma unroll
                        for (int i = 0; i < C::B_ROWS / 64; ++i) load(sb + i * MN_ATOM_BYTES, tmb, nb0 + 64 * i);
                    }
                    __syncwarp();
                    if (++s == STAGES) {
                        s = 0;
                        sp ^= 1u;
                    }
                }
            }
            if (!ok) {
                // wait for the copies that were issued but may not have landed
                const uint32_t first = it > STAGES ? it - STAGES : 0;
                for (uint32_t i = first; i < it; ++i) {
                    const uint32_t st = i % STAGES;
                    if ((pending >> st) & 1u)
                        wait_bar<false>(part0 + st * 8u, (pp >> st) & 1u, abort_flag, args.err, ERR_WAIT_PRODUCER,
                                        DRAIN_LIMIT_NS, false);
                    else if (leader)
                        wait_bar<false>(full0 + st * 8u, (i / STAGES) & 1u, abort_flag, args.err, ERR_WAIT_PRODUCER,
                                        DRAIN_LIMIT_NS, false);
                }
            }
        } else if (warp >= 2) {
            // ------------------------------------------------ rows past an expert's end
            uint32_t it = 0, pp = 0;  // blocks so far; phase of each stage's part
            bool ok = true;
            for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
                const int e = tile / per, num_kb = blocks_of(e);
                it += static_cast<uint32_t>(num_kb);
                const int live = (ctl->off[e + 1] - ctl->off[e]) % BK;
                if (live == 0) continue;
                const uint32_t s = (it - 1) % STAGES;
                if (!wait_bar<false>(zbp::smem_u32(&ctl->part[s]), (pp >> s) & 1u, abort_flag, args.err,
                                     ERR_WAIT_PRODUCER, WAIT_LIMIT_NS, true)) {
                    ok = false;
                    break;
                }
                pp ^= 1u << s;
                uint8_t* at = smem + s * C::STAGE_BYTES + (lane & 7) * 16;
                for (int r = live + (warp - 2) * 4 + lane / 8; r < BK; r += 8)
#pragma unroll
                    for (int atom = 0; atom < static_cast<int>(C::STAGE_BYTES / MN_ATOM_BYTES); ++atom)
                        *reinterpret_cast<uint4*>(at + atom * MN_ATOM_BYTES + r * 128) = make_uint4(0, 0, 0, 0);
                zbp::fence_proxy_async_smem();  // the tensor core reads the zeros
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = zbp::smem_u32(&ctl->edge[s]);
                    if (PAIR)
                        zbp::mbar_arrive_cluster(zbp::mapa_shared(bar, 0));
                    else
                        zbp::mbar_arrive(bar);
                }
            }
        } else if (leader) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t idesc = zbp::idesc_bf16_f32(BM * CG, BN, 1, 1);
            constexpr uint32_t hi = zbp::desc_hi(1024);
            const uint32_t a0 = zbp::desc_lo(zbp::smem_u32(smem), MN_ATOM_BYTES);
            const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
            uint32_t s = 0, sp = 0, local = 0;  // stage and its phase; segment
            uint32_t ep = 0;                    // phase of each stage's edge
            bool ok = true;
            for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
                int e, mb, nb;
                locate(tile, e, mb, nb);
                const int num_kb = blocks_of(e), n = ctl->off[e + 1] - ctl->off[e];
                for (int kb0 = 0; kb0 < num_kb && ok; kb0 += W_SEG) {
                    const uint32_t buf = local & 1u, tr = local >> 1;
                    ++local;
                    if (!wait_bar<false>(zbp::smem_u32(&ctl->tempty[buf]), (tr & 1u) ^ 1u, abort_flag, args.err,
                                         ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        break;
                    }
                    const uint32_t d_tmem = tmem_base + buf * ACC_COLS;
                    const int kb1 = min(kb0 + W_SEG, num_kb);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!wait_bar<false>(full0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                            ok = false;
                            break;
                        }
                        if (kb * BK + BK > n) {
                            if (!wait_bar<true>(zbp::smem_u32(&ctl->edge[s]), (ep >> s) & 1u, abort_flag, args.err,
                                                ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                                ok = false;
                                break;
                            }
                            ep ^= 1u << s;
                        }
                        zbp::tc_fence_after();
                        if (zbp::elect_one()) {
                            const uint32_t a = a0 + s * (C::STAGE_BYTES >> 4), b = a + (A_BYTES >> 4);
                            if (PAIR) {
                                zbp::mma4_f16_pair<128, 128>(d_tmem, a, hi, b, hi, idesc, kb != kb0);
                                zbp::tc_commit_pair_multicast(empty0 + s * 8u, 0x3);
                                if (kb + 1 == kb1) zbp::tc_commit_pair_multicast(zbp::smem_u32(&ctl->tfull[buf]), 0x3);
                            } else {
                                zbp::mma4_f16<128, 128>(d_tmem, a, hi, b, hi, idesc, kb != kb0);
                                zbp::tc_commit(empty0 + s * 8u);
                                if (kb + 1 == kb1) zbp::tc_commit(zbp::smem_u32(&ctl->tfull[buf]));
                            }
                        }
                        __syncwarp();
                        if (++s == STAGES) {
                            s = 0;
                            sp ^= 1u;
                        }
                    }
                }
            }
            if (zbp::elect_one()) {
                if (PAIR)
                    zbp::tc_commit_pair(zbp::smem_u32(&ctl->drain));
                else
                    zbp::tc_commit(zbp::smem_u32(&ctl->drain));
            }
            __syncwarp();
            wait_bar<false>(zbp::smem_u32(&ctl->drain), 0, abort_flag, args.err, ERR_WAIT_MMA, DRAIN_LIMIT_NS, false);
        }
    } else {
        // ---------------------------------------------------- epilogue
        zbp::regs_inc<W_REGS_HIGH>();
        const int ew = warp - 4, q = warp & 3;
        const int c_lo = (ew >> 2) * (BN / 2);  // this warp's half of the tile's columns
        const uint32_t stg0 = zbp::smem_u32(staging + ew * W_BOXES * W_BOX);
        uint32_t local = 0, flip = 0;
        bool ok = true;
        for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
            int e, mb, nb;
            const int p = locate(tile, e, mb, nb);
            const int num_kb = blocks_of(e);
            if (num_kb == 0 && args.accumulate) continue;
            const int row0 = mb * C::TILE_M + static_cast<int>(rank) * BM + q * 32;
            const int n0 = nb * BN + c_lo;
            const int Mp = p ? args.M[1] : args.M[0], Np = p ? args.N[1] : args.N[0];
            const CUtensorMap* tmO = p ? &tmO1 : &tmO0;
            float sum[BN / 2];
#pragma unroll
            for (int i = 0; i < BN / 2; ++i) sum[i] = 0.0f;  // no rows: the gradient is zero
            for (int kb0 = 0; kb0 < num_kb; kb0 += W_SEG) {
                const uint32_t buf = local & 1u, tr = local >> 1;
                ++local;
                if (!wait_bar<false>(zbp::smem_u32(&ctl->tfull[buf]), tr & 1u, abort_flag, args.err, ERR_WAIT_EPI,
                                    WAIT_LIMIT_NS, true)) {
                    ok = false;
                    break;
                }
                zbp::tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * ACC_COLS + c_lo;
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t v[16];
                    zbp::tmem_ld_32x32b_x16(taddr + c * 16, v);
                    zbp::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[c * 16 + i] += __uint_as_float(v[i]);
                }
                zbp::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t te = zbp::smem_u32(&ctl->tempty[buf]);
                    if (PAIR)
                        zbp::mbar_arrive_remote(zbp::mapa_shared(te, 0));
                    else
                        zbp::mbar_arrive(te);
                }
            }
            if (!ok) break;
            const long long done = clock64();
            const int pace = tile + clusters < num_tiles ? min(W_PACE * num_kb, W_PACE_MOST) : 0;
#pragma unroll
            for (int c = 0; c < BN / 64; ++c) {
                const int col0 = n0 + c * 32;
                if (row0 >= Mp || col0 >= Np) continue;
                while (clock64() - done < c * pace) __nanosleep(64);
                uint32_t v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(sum[c * 32 + i]);
                const uint32_t stg = stg0 + flip * W_BOX;
                flip ^= 1u;
                staging_acquire(lane);
                stage_row(stg, lane, v);
                zbp::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (args.accumulate)
                        zbp::tma_reduce_add_3d(tmO, stg, col0, row0, e);
                    else
                        zbp::tma_store_3d(tmO, stg, col0, row0, e);
                    zbp::bulk_commit();
                }
            }
        }
        if (lane == 0) zbp::bulk_wait<0>();
        __syncwarp();
    }

    __syncthreads();
    if (PAIR) zbp::cluster_sync();
    if (warp == 1) {
        zbp::tc_fence_after();
        if (PAIR)
            zbp::tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else
            zbp::tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// db[e][n] (+)= sum over the rows of e of X[r][n].  HBM-bound: each value is read
// once, 16 bytes a load and 8 loads of a thread in flight.  A block takes 64
// columns of one expert and, where such blocks are few, one of up to 8 parts of
// its rows, the parts being a cluster whose first block adds the sums.  32 groups
// of 8 threads sum every 32nd row in ascending order; groups and parts are added
// in order, so the result does not vary.  The two sums of W (16384 rows, 16
// experts, h 1024, f 4096: 168 MB) take 44 us; one value a load in blocks of
// whole experts took 75.
__global__ void __launch_bounds__(256)
    zb_moe_colsum_kernel(const uint4* __restrict__ X, float* db, const int* offsets, int rows, int N, int accumulate) {
    __shared__ float part[32][65], sum[64];
    int lo, hi;
    expert_rows(offsets, blockIdx.y, rows, lo, hi);
    const int parts = gridDim.z, each = (hi - lo + parts - 1) / parts;
    lo = min(lo + static_cast<int>(blockIdx.z) * each, hi);
    hi = min(lo + each, hi);
    const int l = threadIdx.x & 7, g = threadIdx.x / 8, c0 = blockIdx.x * 64 + l * 8;
    float s[8] = {};
    auto add = [&](const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[2 * i] += __uint_as_float(w[i] << 16);
            s[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
        }
    };
    if (c0 < N) {
        const uint4* p = X + c0 / 8;
        const long long ld = N / 8;
        int r = lo + g;
        for (; r + 7 * 32 < hi; r += 8 * 32) {
            uint4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = __ldg(p + (r + u * 32) * ld);
#pragma unroll
            for (int u = 0; u < 8; ++u) add(v[u]);
        }
        for (; r < hi; r += 32) add(__ldg(p + r * ld));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[g][l * 8 + i] = s[i];
    __syncthreads();
    const int c = threadIdx.x, n = blockIdx.x * 64 + c;
    float t = 0.0f;
    if (c < 64) {
#pragma unroll
        for (int i = 0; i < 32; ++i) t += part[i][c];
        sum[c] = t;
    }
    if (parts > 1) zbp::cluster_sync();
    if (blockIdx.z == 0 && c < 64 && n < N) {
        for (int z = 1; z < parts; ++z) t += ld_shared_cluster_f32(zbp::mapa_shared(zbp::smem_u32(&sum[c]), z));
        float* d = db + static_cast<long long>(blockIdx.y) * N + n;
        *d = accumulate ? *d + t : t;
    }
    if (parts > 1) zbp::cluster_sync();  // no block leaves while its sums are read
}

// ---------------------------------------------------------------- host side
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

template <int EPI, int A_MN, int SHAPE>
zb_status launch_rows(const CUtensorMap (&mp)[5], const RowsArgs& a, long long tiles, void* stream) {
    constexpr int CG = RowsCfg<SHAPE>::CG;
    auto kern = zb_moe_rows_kernel<EPI, A_MN, SHAPE>;
    static std::atomic<int> cache[64];
    int ctas = 0;
    zb_status s = full_grid(kern, cache, rows_smem<EPI>(), NUM_THREADS, CG, &ctas);
    if (s != ZB_OK) return s;
    const int grid = static_cast<int>(std::min<long long>(tiles * CG, ctas));
    LaunchCfg lc(grid, NUM_THREADS, rows_smem<EPI>(), CG, stream);
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, kern, mp[0], mp[1], mp[2], mp[3], mp[4], a);
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string("grouped product launch: ") + cudaGetErrorString(e));
    return launched("grouped product");
}

template <int EPI, int A_MN>
zb_status launch_rows_of(Shape shape, const CUtensorMap (&mp)[5], const RowsArgs& a, long long tiles, void* stream) {
    if (shape == FEW) return launch_rows<EPI, A_MN, FEW>(mp, a, tiles, stream);
    return shape == PAIRS ? launch_rows<EPI, A_MN, PAIRS>(mp, a, tiles, stream)
                          : launch_rows<EPI, A_MN, ONE>(mp, a, tiles, stream);
}

// D[row, n] = sum_k A[row, k] W[e](k, n): W[e] is [K, N] or, transposed, [N, K].
zb_status rows_product(const zb_moe& m, const int32_t* offsets, const void* A, const void* W, bool transposed,
                       int64_t N, int64_t K, const void* bias, const void* aux, int epi, void* out0, void* out1,
                       void* stream) {
    // Pairs take tiles of 256 columns x up to 256 rows, single CTAs 128 x 128 or,
    // with few rows an expert, 128 or 64 x 32.  A pair halves the weights' copies
    // a row, so it is taken once its tiles fill the SMs; with fewer rows the time
    // is reading the weights, and twice as many tiles spread them more evenly (3000
    // rows, 16 experts, h 1024, f 4096: 89 us with pairs against 83).  The
    // smallest tiles read an expert's weights again after 32 rows: from L2, but
    // with 32 rows an expert, unevenly spread, already 2 us in 47 slower than
    // tiles of 128; with 2 rows an expert they are 119 against 127 us (64
    // experts, h 2048, f 1536), with 2 rows each of 8 experts 39 against 43.
    // The number of row tiles depends on counts that only the device knows;
    // this is their number when the rows are spread evenly over the experts.
    const int64_t used = std::min<int64_t>(m.experts, m.rows);
    const int64_t each = (m.rows + used - 1) / used;
    const long long pair_tiles = used * ((each + 255) / 256) * ((N + 255) / 256);
    const bool pair = each > 64 && pair_tiles >= sm_count() / 2;
    const Shape shape = pair ? PAIRS : each <= 16 ? FEW : ONE;
    const bool narrow = shape == FEW && used * ((N + 127) / 128) <= sm_count() / 2;
    const int tt = pair ? 256 : shape == FEW ? 32 : 128, tf = pair ? 256 : narrow ? 64 : 128;
    // no launch has more tiles than this
    const long long most = (m.rows / tt + used) * ((N + tf - 1) / tf);

    constexpr CUtensorMapDataType BF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    std::string why;
    CUtensorMap mp[5];
    const uint64_t rows = static_cast<uint64_t>(m.rows);
    bool ok = transposed ? make_map3(&mp[0], W, BF16, 2, K, N, m.experts, BK, std::min(tf, 128), &why)
                         : make_map3(&mp[0], W, BF16, 2, N, K, m.experts, 64, BK, &why);
    ok = ok && make_map(&mp[1], A, false, K, rows, K, BK, 128, &why);
    ok = ok && make_map(&mp[2], A, false, K, rows, K, BK, 32, &why);
    ok = ok && make_map(&mp[3], out0, false, N, rows, N, 32, 32, &why, CU_TENSOR_MAP_SWIZZLE_64B);
    const void* second = epi == zb::EPI_GELU_DUAL ? out1 : epi == zb::EPI_GELU_BWD ? aux : out0;
    ok = ok && make_map(&mp[4], second, false, N, rows, N, 32, 32, &why, CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return zb::fail(ZB_ERR_CUDA, why);
    unsigned int* err = zb::device_error_word();
    if (!err) return ZB_ERR_CUDA;
    RowsArgs a;
    a.offsets = offsets;
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.out0 = static_cast<__nv_bfloat16*>(out0);
    a.out1 = static_cast<__nv_bfloat16*>(out1);
    a.rows = static_cast<int>(m.rows);
    a.experts = m.experts;
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.act = m.act;
    a.tile_f = tf;
    a.err = err;
    if (epi == zb::EPI_GELU_DUAL) return launch_rows_of<zb::EPI_GELU_DUAL, 1>(shape, mp, a, most, stream);
    if (epi == zb::EPI_GELU_BWD) return launch_rows_of<zb::EPI_GELU_BWD, 0>(shape, mp, a, most, stream);
    if (transposed) return launch_rows_of<zb::EPI_STORE_BF16, 0>(shape, mp, a, most, stream);
    return launch_rows_of<zb::EPI_STORE_BF16, 1>(shape, mp, a, most, stream);
}

struct WProduct {
    const void *A, *B;  // [rows, M], [rows, N]
    float* dW;          // [E, M, N]
    int64_t M, N;
};

template <int CG>
zb_status launch_wgrad(const CUtensorMap (&mi)[4], const CUtensorMap (&mo)[2], const WArgs& a, long long tiles, void* stream) {
    auto kern = zb_moe_wgrad_kernel<CG>;
    static std::atomic<int> cache[64];
    int ctas = 0;
    zb_status s = full_grid(kern, cache, w_smem<CG>(), W_THREADS, CG, &ctas);
    if (s != ZB_OK) return s;
    LaunchCfg lc(static_cast<int>(std::min<long long>(tiles * CG, ctas)), W_THREADS, w_smem<CG>(), CG, stream);
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, kern, mi[0], mi[1], mi[2], mi[3], mo[0], mo[1], a);
    if (e != cudaSuccess)
        return zb::fail(ZB_ERR_CUDA, std::string("grouped weight gradient launch: ") + cudaGetErrorString(e));
    return launched("grouped weight gradient");
}

zb_status wgrad(const zb_moe& m, const int32_t* offsets, const WProduct* p, int products, int accumulate,
                void* stream) {
    std::string why;
    CUtensorMap mi[4], mo[2];
    WArgs a;
    const uint64_t rows = static_cast<uint64_t>(std::max<int64_t>(m.rows, 1));
    bool ok = true;
    long long tiles2 = 0, tiles1 = 0;
    for (int i = 0; i < 2; ++i) {
        const WProduct& w = p[i < products ? i : 0];
        a.M[i] = static_cast<int>(w.M);
        a.N[i] = static_cast<int>(w.N);
        ok = ok && make_map3(&mo[i], w.dW, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, w.N, w.M, m.experts, 32, 32, &why);
        if (m.rows) {
            ok = ok && make_map(&mi[2 * i], w.A, false, w.M, rows, w.M, 64, BK, &why);
            ok = ok && make_map(&mi[2 * i + 1], w.B, false, w.N, rows, w.N, 64, BK, &why);
        } else {
            mi[2 * i] = mi[2 * i + 1] = mo[i];
        }
        if (i < products) {
            tiles2 += ((w.M + 255) / 256) * ((w.N + 255) / 256);
            tiles1 += ((w.M + 127) / 128) * ((w.N + 255) / 256);
        }
    }
    if (!ok) return zb::fail(ZB_ERR_CUDA, why);
    unsigned int* err = zb::device_error_word();
    if (!err) return ZB_ERR_CUDA;
    a.offsets = offsets;
    a.rows = static_cast<int>(m.rows);
    a.experts = m.experts;
    a.products = products;
    a.accumulate = accumulate;
    a.err = err;
    tiles1 *= m.experts;
    tiles2 *= m.experts;
    // CTA pairs copy half as many bytes of B a row.  With at least as many tiles as
    // pairs of SMs they are faster: 96 tiles (16384 rows, 3 experts, h = f = 1024) 68 us
    // against 89 with single CTAs, 512 tiles (16 experts, f 4096) 226 against 261, the
    // same with narrow matrices (8 experts, 512 x 1024: 23).  They are with 64 tiles
    // too (4096 rows, 2 experts, 1024 x 1024: 25 against 30); fewer were not measured.
    return tiles2 >= sm_count() / 2 ? launch_wgrad<2>(mi, mo, a, tiles2, stream)
                                     : launch_wgrad<1>(mi, mo, a, tiles1, stream);
}

zb_status column_sums(const uint4* X, float* db, const int* offsets, int experts, int rows, int N, int accumulate,
                      cudaStream_t st) {
    // Parts of an expert's rows until 8 blocks an SM are there, while a part has
    // some 256 rows (16384 rows, 1 expert, N 1024: W with bias gradients 175 us in
    // 8 parts, 371 in one).
    const long long blocks = static_cast<long long>((N + 63) / 64) * experts;
    int parts = 1;
    while (parts < 8 && blocks * parts < 8 * sm_count() && rows / experts >= 512 * parts) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((N + 63) / 64, experts, parts);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = static_cast<unsigned>(parts);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, zb_moe_colsum_kernel, X, db, offsets, rows, N, accumulate);
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string("grouped column sums launch: ") + cudaGetErrorString(e));
    return launched("grouped column sums");
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
    if (off4(offsets) || off16(X) || off16(W1) || off16(W2) || off16(b1) || off16(b2) || off16(H_save) ||
        off16(A_save) || off16(Y))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_forward: pointers must be 16-byte aligned (offsets: 4)");
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
    if (off4(offsets) || off16(dY) || off16(W1) || off16(W2) || off16(H_save) || off16(dH_out) || off16(dX))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_backward_input: pointers must be 16-byte aligned (offsets: 4)");
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
    return static_cast<size_t>(m->experts) * 4 * 128;  // part of the interface; the kernels keep nothing in it
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
    if (off4(offsets) || off16(X) || off16(A_save) || off16(dH) || off16(dY) || off16(dW1) || off16(dW2) ||
        off16(db1) || off16(db2))
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_backward_weight: pointers must be 16-byte aligned (offsets: 4)");
    if (!workspace || ws_bytes < zb_moe_workspace_bytes(m))
        return zb::fail(ZB_ERR_WORKSPACE, "zb_moe_backward_weight: workspace missing or too small: need " +
                                              std::to_string(zb_moe_workspace_bytes(m)) + " bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return zb::fail(ZB_ERR_ALIGN, "zb_moe_backward_weight: workspace must be 256-byte aligned");
    const int rows = static_cast<int>(m->rows), h = static_cast<int>(m->h), f = static_cast<int>(m->f);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto colsum = [&](const void* A, float* db, int N) {
        return column_sums(static_cast<const uint4*>(A), db, offsets, m->experts, rows, N, accumulate ? 1 : 0, st);
    };
    if (mlp) {
        const WProduct p[2] = {{A_save, dY, dW2, f, h}, {X, dH, dW1, h, f}};
        s = wgrad(*m, offsets, p, 2, accumulate ? 1 : 0, stream);
    } else {
        const WProduct p[1] = {{X, dY, dW1, h, f}};
        s = wgrad(*m, offsets, p, 1, accumulate ? 1 : 0, stream);
    }
    if (s == ZB_OK && m->has_bias) s = colsum(mlp ? dH : dY, db1, f);
    if (s == ZB_OK && m->has_bias && mlp) s = colsum(dY, db2, h);
    if (s == ZB_OK) zb::clear_error();
    return s;
}
