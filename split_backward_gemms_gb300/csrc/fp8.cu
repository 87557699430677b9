// fp8.cu — products in 8-bit floating point (e4m3) with an fp32 scale for each
// block of 128, dense or grouped by expert, and the quantisers that make their
// operands.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <string>

#include "grouped.cuh"

namespace {

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

// Two values rounded to e4m3 (to nearest, ties to even), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// HBM-bound: 3 bytes a value.  16 lanes share a 1 x 128 block (16 bytes each,
// read once and kept), a warp Q_ILP pairs of neighbouring blocks, all loads in
// flight before the first is used (two or eight pairs: the same within 3 %, but
// 8190 x 1040 takes 10.5 us with eight, 8.4 with four).  16384 x 8192: 70 us, 5.8
// TB/s; 4096 x 4096: 10.7 us.
constexpr int Q_ILP = 4;
__global__ void __launch_bounds__(256)
    zb_fp8_quantize_rows_kernel(const uint4* __restrict__ X, uint2* __restrict__ Q, float* __restrict__ S,
                                long long total, int cols8, int blocks) {
    zbp::allow_dependent_launch();
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const long long item0 = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 2 * Q_ILP + half;
    uint4 v[Q_ILP];
    long long at[Q_ILP], item[Q_ILP];
    const bool whole = cols8 == blocks * 16;  // no partial blocks: a block's place needs no division
#pragma unroll
    for (int u = 0; u < Q_ILP; ++u) {
        item[u] = item0 + 2 * u;
        at[u] = item[u] * 16 + l;
        if (!whole) {
            const long long r = total <= 0xffffffffll
                                    ? static_cast<uint32_t>(item[u]) / static_cast<uint32_t>(blocks)
                                    : item[u] / blocks;
            const int c = static_cast<int>(item[u] - r * blocks) * 16 + l;
            at[u] = c < cols8 ? r * cols8 + c : -1;
        }
        if (item[u] >= total) at[u] = -1;
        v[u] = at[u] >= 0 ? __ldg(X + at[u]) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < Q_ILP; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t top = 0;  // the largest |x| as its bits: NaN above infinity above numbers
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        float s, inv;
        block_scale(__uint_as_float(top << 16), s, inv);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_bf16x2(w[i]);
            q[i] = e4m3x2(f.x * inv, f.y * inv);
        }
        if (at[u] >= 0) Q[at[u]] = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        if (l == 0 && item[u] < total) S[item[u]] = s;
    }
}

// HBM-bound: W read once (a block of threads holds its 128 x 128 block in
// registers while the maximum is found), each result written once.  The
// transposed copy goes through shared memory as words of four columns: word w of
// row r lies at w + 4 (r / 16) mod 32, so that the 16-byte rows of the transpose
// (a thread: 16 rows of 4 columns, transposed 4 x 4 bytes at a time) are read
// without bank conflicts and leave 128 bytes together.
// 4096 x 16384, both copies: 51 us, 5.2 TB/s (542 us with one thread a value and
// scattered stores of bytes).
__global__ void __launch_bounds__(256)
    zb_fp8_quantize_weight_kernel(const uint4* __restrict__ W, uint2* __restrict__ Q, float* S, uint8_t* QT, float* ST,
                                  int rows, int cols) {
    __shared__ uint32_t top[8];
    __shared__ __align__(16) uint32_t tile[128][32];
    const int rb = blockIdx.y, cb = blockIdx.x, e = blockIdx.z, tid = threadIdx.x;
    const int r0 = rb * BLK + tid / 16, c0 = cb * BLK + (tid & 15) * 8;  // this thread: rows r0 + 16 i, 8 columns
    const long long cols8 = cols / 8, base = static_cast<long long>(e) * rows * cols8 + c0 / 8;
    uint4 v[8];
    uint32_t m = 0;  // the largest |value|'s bits: NaN above infinity above the rest
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (c0 < cols && r0 + 16 * i < rows) v[i] = __ldg(W + base + (r0 + 16 * i) * cols8);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max((w[j] & 0x7fffu) << 16, w[j] & 0x7fff0000u));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) top[tid / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, top[i]);
    float s, inv;
    block_scale(__uint_as_float(m), s, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            q[j] = e4m3x2(__uint_as_float(w[j] << 16) * inv, __uint_as_float(w[j] & 0xffff0000u) * inv);
        const uint2 o = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        if (Q && c0 < cols && r0 + 16 * i < rows) Q[base + (r0 + 16 * i) * cols8] = o;
        if (QT) *reinterpret_cast<uint2*>(&tile[tid / 16 + 16 * i][((tid & 15) * 2 + 4 * i) & 31]) = o;
    }
    if (tid == 0) {
        const long long RB = gridDim.y, CB = gridDim.x;
        if (Q) S[(e * RB + rb) * CB + cb] = s;
        if (QT) ST[(e * CB + cb) * RB + rb] = s;
    }
    if (!QT) return;
    __syncthreads();
    const int g = tid & 7, cw = tid / 8;  // rows 16 g .. 16 g + 15, columns 4 cw .. 4 cw + 3
    uint32_t t[4][4];                     // [column][four rows]
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = tile[16 * g + 4 * k + j][(cw + 4 * g) & 31];
        const uint32_t a = __byte_perm(x[0], x[1], 0x5140), b = __byte_perm(x[2], x[3], 0x5140);
        const uint32_t c = __byte_perm(x[0], x[1], 0x7362), d = __byte_perm(x[2], x[3], 0x7362);
        t[0][k] = __byte_perm(a, b, 0x5410);
        t[1][k] = __byte_perm(a, b, 0x7632);
        t[2][k] = __byte_perm(c, d, 0x5410);
        t[3][k] = __byte_perm(c, d, 0x7632);
    }
    const int row = rb * BLK + 16 * g, col = cb * BLK + 4 * cw;
    if (row >= rows || col >= cols) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(QT + (static_cast<long long>(e) * cols + col + j) * rows + row) =
            make_uint4(t[j][0], t[j][1], t[j][2], t[j][3]);
}

// ---------------------------------------------------------------- product
// D[r, n] = sum_b xs[r, b] ws[n/128, b] P_b[r, n], P_b the product over the
// b-th block of 128 of K (4 MMAs of K = 32).  A tile's M side is rows, so that a
// thread of the epilogue (one TMEM lane) has one row.  Warp 0 copies; the scales
// are applied in one of two ways:
//
// Powers of two (MX; what the quantisers make).  The tensor core's block-scaled
// form multiplies by 2^(xs exponent + ws exponent) itself: a factor for each row
// and 32 of K, here the same for a block's four.  Warp 1 issues the MMAs over the
// whole of K into one accumulator of 256 columns, warps 2 and 3 feed it the
// exponents.  The epilogue takes the accumulator into registers at once and
// gives it back, so that the next tile's MMAs run beside the rest of it.  Bound
// by the MMAs where K is long: [4096, 4096] x [4096, 16384] 155 us, 3.55 PFLOP/s
// (the tensor pipe active 83 % of the time); with K 1040 and GeLU' by the epilogue
// and the number of tiles a CTA pair (16 experts, 8190 rows, N 4104: 79 us).
//
// Any other scales.  The accumulator holds one P_b only, and the 8 epilogue
// warps add xs ws P_b to fp32 sums in registers (a packed FMA for two elements)
// while the next is computed: two accumulators of 256 columns fill TMEM.  A
// block's MMAs take 512 cycles, but the way round an accumulator (commit, wake,
// read, arrive, wake) over 1000 on a pair, which bounds it: [4096, 4096] x
// [4096, 16384] 217 us.  Warps 1 and 2 issue a block each in turn, since a block's
// waits, MMAs and commits take one thread longer than 512 cycles.
template <int CG>
struct Fp8Cfg {
    static constexpr int TILE_T = 128 * CG;                       // rows of D per tile
    static constexpr int B_ROWS = 256 / CG;                       // columns of D held per CTA
    static constexpr uint32_t A_BYTES8 = 128 * 128;               // 128 rows x 128 k
    static constexpr uint32_t STAGE = A_BYTES8 + B_ROWS * 128;
};
// Warps 0-3 give registers to the epilogue warps behind them.  MX: 16 of these,
// with 64 columns each, four to a scheduler to hide the latency of GeLU's special
// functions, of H and of the stores (with 8: GeLU' of 16 experts, 8190 rows, K
// 1040, N 4104 92 us against 79); else 8, whose threads hold 128 sums and 32
// loaded values.  640 threads leave 96 registers each at launch, which the scale
// and epilogue roles' code overruns: 24 bytes a thread are spilled in the plain
// form, 36 to 44 with GeLU, 60 with GeLU' (none without MX).
// GeLU' keeps a warp's values of H in its staging boxes (copied while the product
// runs) and stores from them; the others store through one box, or two.
constexpr uint32_t FP8_BOX = 32 * 64;  // 32 rows x 32 columns of bf16
template <int EPI, int CG, int MX>
struct Fp8Epi {
    static constexpr int WARPS = MX ? 16 : 8;
    static constexpr int THREADS = 128 + 32 * WARPS;
    static constexpr int REGS_LOW = MX ? 64 : 72, REGS_HIGH = MX ? 104 : 216;
    static constexpr int COLS = 1024 / WARPS;  // columns of a warp (four warps have the tile's rows)
    static constexpr int BOXES = EPI == ZB_FP8_GELU_GRAD ? COLS / 32 : MX ? 1 : 2;
    static constexpr int STAGES = CG == 1 ? 3 : EPI == ZB_FP8_GELU_GRAD ? 4 : 5;
};
static_assert(128 * 64 + 512 * 104 <= 640 * 96 && 128 * 72 + 256 * 216 <= 384 * 168, "register split");
// Scales that are powers of two (MX) are applied by the tensor core itself.
// Warps 2 and 3 write a group of four K blocks' exponents into shared memory as
// the MMA reads them: 32 rows of 16 bytes for 128 rows of an operand, byte 4 r + k
// of row i the scale of operand row i + 32 r in block k.  Four groups are loaded
// and handed over at once: with one, the loads' latency and the cluster-scope
// release (about 2000 cycles) took longer than the group's MMAs.
// A batch's slot is released by the commit after its last block.  The columns in
// TMEM, eight groups in turn, need no release.  A group is copied in for block n
// (counted over all tiles) after the wait for block n - 1's stage; that stage was
// filled once the MMAs of block n - 1 - STAGES were complete, n - 6 at the earliest.
// The group it replaces, eight before, was last read by block n - 8 or an earlier one.
constexpr int MX_GROUPS = 4;      // groups in a batch
constexpr int MX_SLOTS = 2;       // batches in shared memory
constexpr uint32_t MX_TMEM = 256;  // first TMEM column of the scales, 16 a group
struct __align__(128) MxGroup {
    uint4 a[32];     // the CTA's 128 rows
    uint4 b[2][32];  // the tile's 256 columns
};
struct Fp8Ctl {
    MxGroup scale[MX_SLOTS][MX_GROUPS];
    uint64_t full[6], empty[6], tfull[2], tempty[2], drain[2];
    uint64_t hbar[16];
    uint64_t sfull[MX_SLOTS], sempty[MX_SLOTS];
    uint32_t tmem_base;
    int abort_flag;
    int off[MAX_EXPERTS + 1];
};
template <int EPI, int CG, int MX>
constexpr size_t fp8_smem() {
    using E = Fp8Epi<EPI, CG, MX>;
    return 1024 + E::STAGES * Fp8Cfg<CG>::STAGE + E::WARPS * E::BOXES * FP8_BOX + sizeof(Fp8Ctl);
}
template <int EPI>
constexpr bool fp8_fits() {
    return fp8_smem<EPI, 1, 0>() <= 232448 && fp8_smem<EPI, 2, 0>() <= 232448 && fp8_smem<EPI, 1, 1>() <= 232448 &&
           fp8_smem<EPI, 2, 1>() <= 232448;
}
static_assert(fp8_fits<ZB_FP8_STORE>() && fp8_fits<ZB_FP8_GELU>() && fp8_fits<ZB_FP8_GELU_GRAD>(), "shared memory");

struct Fp8Args {
    const int* offsets;  // nullptr: one expert with every row
    const float *xs, *ws;
    const __nv_bfloat16* bias;
    __nv_bfloat16 *out0, *out1;
    int rows, experts, N, K, act;
    unsigned int* err;
};

template <int EPI, int CG, int MX>
__global__ void __launch_bounds__(Fp8Epi<EPI, CG, MX>::THREADS, 1)
    zb_fp8_matmul_kernel(const __grid_constant__ CUtensorMap tmA128, const __grid_constant__ CUtensorMap tmA32,
                         const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmO0,
                         const __grid_constant__ CUtensorMap tmO1, const Fp8Args args) {
    using C = Fp8Cfg<CG>;
    constexpr bool PAIR = CG == 2;
    using E = Fp8Epi<EPI, CG, MX>;
    constexpr int STAGES = E::STAGES, BOXES = E::BOXES;
    constexpr int CHUNKS = E::COLS / 32;  // a warp's columns, 32 at a time
    constexpr bool GRAD = EPI == ZB_FP8_GELU_GRAD;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + STAGES * C::STAGE;
    Fp8Ctl* ctl = reinterpret_cast<Fp8Ctl*>(staging + E::WARPS * BOXES * FP8_BOX);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? zbp::cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
    const int tiles_n = (args.N + 255) / 256;
    const int num_kb = (args.K + BLK - 1) / BLK;
    const int n_blocks = (args.N + BLK - 1) / BLK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            zbp::mbar_init(zbp::smem_u32(&ctl->full[s]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            zbp::mbar_init(zbp::smem_u32(&ctl->tfull[b]), 1);
            zbp::mbar_init(zbp::smem_u32(&ctl->tempty[b]), E::WARPS * CG);
            zbp::mbar_init(zbp::smem_u32(&ctl->drain[b]), 1);
        }
        for (int g = 0; g < MX_SLOTS; ++g) {
            zbp::mbar_init(zbp::smem_u32(&ctl->sfull[g]), 2 * CG);
            zbp::mbar_init(zbp::smem_u32(&ctl->sempty[g]), 1);
        }
        if (GRAD)
            for (int w = 0; w < E::WARPS; ++w) zbp::mbar_init(zbp::smem_u32(&ctl->hbar[w]), 1);
        ctl->abort_flag = 0;
        zbp::fence_mbar_init();
        zbp::tma_prefetch_desc(&tmA128);
        zbp::tma_prefetch_desc(&tmA32);
        zbp::tma_prefetch_desc(&tmB);
        zbp::tma_prefetch_desc(&tmO0);
        if (EPI != ZB_FP8_STORE) zbp::tma_prefetch_desc(&tmO1);
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
    if (args.offsets) {
        load_offsets(ctl->off, args.offsets, args.experts, args.rows);
    } else {
        if (threadIdx.x == 0) {
            ctl->off[0] = 0;
            ctl->off[1] = args.rows;
        }
        __syncthreads();
    }

    Walk<C::TILE_T, false> walk(ctl->off, args.experts, tiles_n);
    int row0 = 0, nrows = 0, nb = 0;
    if (warp < 4) {
        zbp::regs_dec<E::REGS_LOW>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
            const uint32_t full0_lead = PAIR ? zbp::mapa_shared(full0, 0) : full0;
            const uint32_t sa0 = zbp::smem_u32(smem);
            uint32_t s = 0, sp = 1, it = 0;  // stage and the phase of its last release; stages filled
            bool ok = true;
            for (int tile = cluster; ok && walk.to(tile, row0, nrows, nb); tile += clusters) {
                // 32-row boxes of rows in this CTA, and in both
                auto boxes_of = [&](int r) { return max(0, min(4, (nrows - r * 128 + 31) / 32)); };
                const int boxes = boxes_of(static_cast<int>(rank));
                const int r0 = row0 + static_cast<int>(rank) * 128;
                const int all = boxes_of(0) + (PAIR ? boxes_of(1) : 0);
                const uint32_t bytes = static_cast<uint32_t>(all) * 32u * 128u + 256u * 128u;
                const int n0 = nb * 256 + static_cast<int>(rank) * C::B_ROWS;
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    if (!wait_bar<false>(empty0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_PRODUCER, WAIT_LIMIT_NS,
                                         true)) {
                        ok = false;
                        break;
                    }
                    if (zbp::elect_one()) {
                        const uint32_t full = full0_lead + s * 8u;
                        const uint32_t sa = sa0 + s * C::STAGE, sb = sa + C::A_BYTES8;
                        const int k0 = kb * BLK;
                        if (leader) zbp::mbar_arrive_expect_tx(full0 + s * 8u, bytes);
                        auto load_a = [&](uint32_t dst, const CUtensorMap* tm, int y) {
                            if (PAIR)
                                zbp::tma_load_2d_pair(dst, tm, full, k0, y);
                            else
                                zbp::tma_load_2d(dst, tm, full, k0, y);
                        };
                        if (boxes == 4) {
                            load_a(sa, &tmA128, r0);
                        } else {
#pragma unroll
                            for (int b = 0; b < 3; ++b)
                                if (b < boxes) load_a(sa + static_cast<uint32_t>(b) * 32u * 128u, &tmA32, r0 + 32 * b);
                        }
                        if (PAIR)
                            zbp::tma_load_3d_pair(sb, &tmB, full, k0, n0, walk.e);
                        else
                            zbp::tma_load_3d(sb, &tmB, full, k0, n0, walk.e);
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
        } else if (MX && warp == 1 && leader) {
            // ------------------------------------------------ MMA issuer (MX)
            // One accumulator of 256 columns for the whole of K: the epilogue
            // takes it into registers before it does anything else.
            constexpr uint32_t idesc = zbp::idesc_mx_e4m3(128 * CG, 256, 0);
            constexpr uint32_t hi = zbp::desc_hi(1024);
            const uint32_t lo0 = zbp::desc_lo(zbp::smem_u32(smem), 16);
            const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
            const uint32_t sfull0 = zbp::smem_u32(&ctl->sfull[0]), sempty0 = zbp::smem_u32(&ctl->sempty[0]);
            uint32_t s = 0, sp = 0, g = 0, batch = 0, done = 0;  // stage and phase; scale groups and batches; tiles
            bool ok = true;
            for (int tile = cluster; ok && walk.to(tile, row0, nrows, nb); tile += clusters, ++done) {
                if (!wait_bar<false>(zbp::smem_u32(&ctl->tempty[0]), (done & 1u) ^ 1u, abort_flag, args.err, ERR_WAIT_MMA,
                                     WAIT_LIMIT_NS, true))
                    break;
                zbp::tc_fence_after();
                for (int kb = 0; kb < num_kb; ++kb) {
                    const uint32_t slot = batch % MX_SLOTS, sf = tmem_base + MX_TMEM + (g & 7u) * 16u;
                    if ((kb & 15) == 0) {
                        if (!wait_bar<true>(sfull0 + slot * 8u, (batch / MX_SLOTS) & 1u, abort_flag, args.err,
                                            ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                            ok = false;
                            break;
                        }
                        zbp::tc_fence_after();
                    }
                    if ((kb & 3) == 0) {
                        if (zbp::elect_one()) {
                            const uint32_t src = zbp::smem_u32(&ctl->scale[slot][(kb >> 2) & 3]);
#pragma unroll
                            for (uint32_t i = 0; i < 3; ++i) {
                                if (PAIR)
                                    zbp::tc_copy_32x128b_pair(sf + 4 * i, zbp::smem_desc_rows16(src + 512 * i));
                                else
                                    zbp::tc_copy_32x128b(sf + 4 * i, zbp::smem_desc_rows16(src + 512 * i));
                            }
                        }
                        __syncwarp();
                    }
                    if (!wait_bar<false>(full0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        break;
                    }
                    zbp::tc_fence_after();
                    const bool last = kb + 1 == num_kb, batch_end = last || (kb & 15) == 15;
                    if (zbp::elect_one()) {
                        const uint32_t a = lo0 + s * (C::STAGE >> 4), b = a + (C::A_BYTES8 >> 4);
                        const uint32_t id = static_cast<uint32_t>(kb & 3), dsc = idesc | (id << 4) | (id << 29);
                        if (PAIR) {
                            zbp::mma4_mx_pair(tmem_base, a, b, hi, dsc, sf, sf + 4, kb != 0);
                            zbp::tc_commit_pair_multicast(empty0 + s * 8u, 0x3);
                            if (batch_end) zbp::tc_commit_pair_multicast(sempty0 + slot * 8u, 0x3);
                            if (last) zbp::tc_commit_pair_multicast(zbp::smem_u32(&ctl->tfull[0]), 0x3);
                        } else {
                            zbp::mma4_mx(tmem_base, a, b, hi, dsc, sf, sf + 4, kb != 0);
                            zbp::tc_commit(empty0 + s * 8u);
                            if (batch_end) zbp::tc_commit(sempty0 + slot * 8u);
                            if (last) zbp::tc_commit(zbp::smem_u32(&ctl->tfull[0]));
                        }
                    }
                    __syncwarp();
                    if (last || (kb & 3) == 3) ++g;
                    if (batch_end) ++batch;
                    if (++s == STAGES) {
                        s = 0;
                        sp ^= 1u;
                    }
                }
            }
            // every MMA issued here completes before TMEM is released
            const uint32_t drain = zbp::smem_u32(&ctl->drain[0]);
            if (zbp::elect_one()) {
                if (PAIR)
                    zbp::tc_commit_pair(drain);
                else
                    zbp::tc_commit(drain);
            }
            __syncwarp();
            wait_bar<false>(drain, 0, abort_flag, args.err, ERR_WAIT_MMA, DRAIN_LIMIT_NS, false);
        } else if (MX && warp >= 2) {
            // ------------------------------------------------ scales (MX)
            // Warp 2 has the CTA's rows 0-63 and the tile's first 128 columns,
            // warp 3 the others; a lane has two rows.
            const int hw = warp - 2;
            const bool vec = (num_kb & 3) == 0 && (reinterpret_cast<uintptr_t>(args.xs) & 15u) == 0;
            uint32_t batch = 0;
            bool ok = true;
            for (int tile = cluster; ok && walk.to(tile, row0, nrows, nb); tile += clusters) {
                const int row = row0 + static_cast<int>(rank) * 128 + hw * 64 + lane, end = row0 + nrows;
                const float* x0 = args.xs + static_cast<long long>(min(row, end - 1)) * num_kb;
                const float* x1 = args.xs + static_cast<long long>(min(row + 32, end - 1)) * num_kb;
                const float* w =
                    args.ws + (static_cast<long long>(walk.e) * n_blocks + min(nb * 2 + hw, n_blocks - 1)) * num_kb;
                for (int k16 = 0; k16 < num_kb; k16 += 16, ++batch) {
                    float a[16], b[16];
                    if (vec) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            if (k16 + i >= num_kb) break;
                            const float4 u = __ldg(reinterpret_cast<const float4*>(x0 + k16 + i));
                            const float4 v = __ldg(reinterpret_cast<const float4*>(x1 + k16 + i));
                            a[i] = u.x, a[i + 1] = u.y, a[i + 2] = u.z, a[i + 3] = u.w;
                            b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            a[i] = b[i] = 1.0f;
                            if (k16 + i < num_kb) {
                                a[i] = __ldg(x0 + k16 + i);
                                b[i] = __ldg(x1 + k16 + i);
                            }
                        }
                    }
                    // a scale's exponent; lane i has that of the columns' block i
                    auto exponent = [](float f) { return (__float_as_uint(f) >> 23) & 0xffu; };
                    const uint32_t c = exponent(__ldg(w + min(k16 + (lane & 15), num_kb - 1)));
                    const uint32_t slot = batch % MX_SLOTS;
                    if (!wait_bar<false>(zbp::smem_u32(&ctl->sempty[slot]), ((batch / MX_SLOTS) & 1u) ^ 1u, abort_flag,
                                         args.err, ERR_WAIT_PRODUCER, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        if (k16 + j >= num_kb) break;
                        uint32_t wa = 0, wb = 0, wc = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            wa |= exponent(a[j + i]) << (8 * i);
                            wb |= exponent(b[j + i]) << (8 * i);
                            wc |= __shfl_sync(0xffffffffu, c, j + i) << (8 * i);
                        }
                        MxGroup& m = ctl->scale[slot][j / 4];
                        reinterpret_cast<uint2*>(&m.a[lane])[hw] = make_uint2(wa, wb);
                        m.b[hw][lane] = make_uint4(wc, wc, wc, wc);
                    }
                    zbp::fence_proxy_async_smem();  // read by the tensor core's copies next
                    __syncwarp();
                    if (lane == 0) {
                        const uint32_t bar = zbp::smem_u32(&ctl->sfull[slot]);
                        if (PAIR)
                            zbp::mbar_arrive_cluster(zbp::mapa_shared(bar, 0));
                        else
                            zbp::mbar_arrive(bar);
                    }
                }
            }
        } else if (!MX && (warp == 1 || warp == 2) && leader) {
            // ------------------------------------------------ MMA issuers
            // Warp 1 issues the even blocks of K (into accumulator 0), warp 2
            // the odd ones: a block's two waits, four MMAs and two commits take
            // one thread longer than the 512 cycles of its MMAs.
            constexpr uint32_t idesc = zbp::idesc_e4m3_f32(128 * CG, 256);
            constexpr uint32_t hi = zbp::desc_hi(1024);
            const uint32_t buf = static_cast<uint32_t>(warp - 1);
            const uint32_t d_tmem = tmem_base + buf * ACC_COLS;
            const uint32_t lo0 = zbp::desc_lo(zbp::smem_u32(smem), 16);
            const uint32_t full0 = zbp::smem_u32(&ctl->full[0]), empty0 = zbp::smem_u32(&ctl->empty[0]);
            const uint32_t tfull = zbp::smem_u32(&ctl->tfull[buf]), tempty = zbp::smem_u32(&ctl->tempty[buf]);
            uint32_t s = buf, sp = 0;  // stage and its phase
            uint32_t tp = 1;           // phase of the accumulator's last release
            int k = static_cast<int>(buf);  // next block, counted from the tile's first
            bool ok = true;
            for (int tile = cluster; ok && walk.to(tile, row0, nrows, nb); tile += clusters) {
                for (; k < num_kb; k += 2) {
                    if (!wait_bar<false>(tempty, tp, abort_flag, args.err, ERR_WAIT_MMA, WAIT_LIMIT_NS, true) ||
                        !wait_bar<false>(full0 + s * 8u, sp, abort_flag, args.err, ERR_WAIT_MMA, WAIT_LIMIT_NS, true)) {
                        ok = false;
                        break;
                    }
                    tp ^= 1u;
                    zbp::tc_fence_after();
                    if (zbp::elect_one()) {
                        const uint32_t a = lo0 + s * (C::STAGE >> 4), b = a + (C::A_BYTES8 >> 4);
                        if (PAIR) {
                            zbp::mma4_f8_pair<2, 2>(d_tmem, a, hi, b, hi, idesc, 0);
                            zbp::tc_commit_pair_multicast(tfull, 0x3);
                            zbp::tc_commit_pair_multicast(empty0 + s * 8u, 0x3);
                        } else {
                            zbp::mma4_f8<2, 2>(d_tmem, a, hi, b, hi, idesc, 0);
                            zbp::tc_commit(tfull);
                            zbp::tc_commit(empty0 + s * 8u);
                        }
                    }
                    __syncwarp();
                    s += 2;
                    if (s >= STAGES) {
                        s -= STAGES;
                        sp ^= 1u;
                    }
                }
                k -= num_kb;
            }
            // every MMA issued here completes before TMEM is released
            const uint32_t drain = zbp::smem_u32(&ctl->drain[buf]);
            if (zbp::elect_one()) {
                if (PAIR)
                    zbp::tc_commit_pair(drain);
                else
                    zbp::tc_commit(drain);
            }
            __syncwarp();
            wait_bar<false>(drain, 0, abort_flag, args.err, ERR_WAIT_MMA, DRAIN_LIMIT_NS, false);
        }
    } else {
        // ---------------------------------------------------- epilogue
        zbp::regs_inc<E::REGS_HIGH>();
        const int ew = warp - 4, q = warp & 3;
        const int c_lo = (ew >> 2) * E::COLS;  // this warp's part of the tile's columns
        const uint32_t stg0 = zbp::smem_u32(staging + ew * BOXES * FP8_BOX);
        uint32_t it = 0, flip = 0;
        uint32_t asked = 0, taken = 0;  // tiles whose H was asked for and read
        bool ok = true;
        for (int tile = cluster; ok && walk.to(tile, row0, nrows, nb); tile += clusters) {
            const int first = row0 + static_cast<int>(rank) * 128 + q * 32;  // the warp's first row
            const int live = row0 + nrows - first;                           // its live rows
            const int n0 = nb * 256 + c_lo;
            if (GRAD && live > 0 && n0 < args.N) {
                // this warp's values of H, into the boxes of its last tile
                zbp::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    zbp::bulk_wait_read<0>();
                    const uint32_t bar = zbp::smem_u32(&ctl->hbar[ew]);
                    zbp::mbar_arrive_expect_tx(bar, BOXES * FP8_BOX);  // columns past the edge: zeros
                    for (int c = 0; c < BOXES; ++c)
                        zbp::tma_load_2d(stg0 + static_cast<uint32_t>(c) * FP8_BOX, &tmO1, bar, n0 + 32 * c, first);
                }
                ++asked;
            }
            f32x2 sum[E::COLS / 2];
            if (MX) {
                if (!wait_bar<false>(zbp::smem_u32(&ctl->tfull[0]), it & 1u, abort_flag, args.err, ERR_WAIT_EPI, WAIT_LIMIT_NS,
                                     true)) {
                    ok = false;
                    break;
                }
                ++it;
                zbp::tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c_lo;
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c) {
                    uint32_t v[32];
                    zbp::tmem_ld_32x32b_x32(taddr + c * 32, v);
                    zbp::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sum[c * 16 + i] = pk2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                }
                zbp::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t te = zbp::smem_u32(&ctl->tempty[0]);
                    if (PAIR)
                        zbp::mbar_arrive_remote(zbp::mapa_shared(te, 0));
                    else
                        zbp::mbar_arrive(te);
                }
            } else {
            const bool scaled = lane < live && n0 < args.N;
            const float* xs = args.xs + static_cast<long long>(scaled ? first + lane : 0) * num_kb;
            const float* ws = args.ws + (static_cast<long long>(walk.e) * n_blocks + (scaled ? n0 / BLK : 0)) * num_kb;
#pragma unroll
            for (int i = 0; i < E::COLS / 2; ++i) sum[i] = 0ull;
            float xn = scaled ? __ldg(xs) : 0.0f, wn = scaled ? __ldg(ws) : 0.0f;
#pragma unroll 1
            for (int kb = 0; kb < num_kb; ++kb, ++it) {
                const float f = xn * wn;
                if (scaled && kb + 1 < num_kb) {
                    xn = __ldg(xs + kb + 1);
                    wn = __ldg(ws + kb + 1);
                }
                const uint32_t buf = it & 1u;
                if (!wait_bar<false>(zbp::smem_u32(&ctl->tfull[buf]), (it >> 1) & 1u, abort_flag, args.err, ERR_WAIT_EPI,
                                     WAIT_LIMIT_NS, true)) {
                    ok = false;
                    break;
                }
                zbp::tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * ACC_COLS + c_lo;
                const f32x2 ff = pk2(f, f);
#pragma unroll
                for (int c = 0; c < 2 * CHUNKS; ++c) {
                    uint32_t v[16];
                    zbp::tmem_ld_32x32b_x16(taddr + c * 16, v);
                    zbp::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum[c * 8 + i] =
                            fma2(pk2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), ff, sum[c * 8 + i]);
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
            }
            if (!ok) break;
            if (live <= 0 || n0 >= args.N) continue;
            if (GRAD) {
                if (!wait_bar<false>(zbp::smem_u32(&ctl->hbar[ew]), taken & 1u, abort_flag, args.err, ERR_WAIT_EPI,
                                     WAIT_LIMIT_NS, true))
                    break;
                ++taken;
            }
            const long long at = static_cast<long long>(first + lane) * args.N;
            // a box of 32 rows by TMA, fewer by each row's thread
            auto store = [&](const CUtensorMap* tm, __nv_bfloat16* out, int c, const uint32_t (&w)[16]) {
                const int col0 = n0 + c * 32;
                if (live >= 32) {
                    const uint32_t stg = stg0 + (GRAD ? static_cast<uint32_t>(c) : flip) * FP8_BOX;
                    if (BOXES == 2) flip ^= 1u;
                    if (!GRAD) {  // GeLU': a lane replaces its own row of H
                        if (lane == 0) zbp::bulk_wait_read<BOXES - 1>();
                        __syncwarp();
                    }
                    stage_row64(stg, lane, w);
                    zbp::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        zbp::tma_store_2d(tm, stg, col0, first);
                        zbp::bulk_commit();
                    }
                } else if (lane < live) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (col0 + 8 * k < args.N)
                            *reinterpret_cast<uint4*>(out + at + col0 + 8 * k) =
                                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                }
            };
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                const int col0 = n0 + c * 32;
                if (col0 >= args.N) continue;
                float x[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) up2(sum[c * 16 + i], x[2 * i], x[2 * i + 1]);
                if (EPI != ZB_FP8_GELU_GRAD && args.bias) {
                    const __nv_bfloat16* bp = args.bias + static_cast<long long>(walk.e) * args.N + col0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (col0 + 8 * k >= args.N) break;
                        const uint4 b = *reinterpret_cast<const uint4*>(bp + 8 * k);
                        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f2 = unpack_bf16x2(bw[i]);
                            x[8 * k + 2 * i] += f2.x;
                            x[8 * k + 2 * i + 1] += f2.y;
                        }
                    }
                }
                if (EPI == ZB_FP8_GELU_GRAD) {
                    uint32_t h[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 v = zbp::ld_shared_v4(stg0 + static_cast<uint32_t>(c) * FP8_BOX +
                                                           static_cast<uint32_t>(lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)));
                        h[4 * k] = __float_as_uint(v.x);
                        h[4 * k + 1] = __float_as_uint(v.y);
                        h[4 * k + 2] = __float_as_uint(v.z);
                        h[4 * k + 3] = __float_as_uint(v.w);
                    }
                    if (args.act == ZB_ACT_GELU_TANH)
                        gelu_grad_mul<true, 32>(x, h);
                    else
                        gelu_grad_mul<false, 32>(x, h);
                }
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                store(&tmO0, args.out0, c, w);
                if (EPI == ZB_FP8_GELU) {
                    if (args.act == ZB_ACT_GELU_TANH)
                        gelu_pack<true, 32>(x, w);
                    else
                        gelu_pack<false, 32>(x, w);
                    store(&tmO1, args.out1, c, w);
                }
            }
        }
        if (GRAD && asked != taken)  // H asked for and not read (after an abort)
            wait_bar<false>(zbp::smem_u32(&ctl->hbar[ew]), taken & 1u, abort_flag, args.err, ERR_WAIT_EPI, DRAIN_LIMIT_NS,
                            false);
        if (lane == 0) zbp::bulk_wait<0>();
        __syncwarp();
    }

    __syncthreads();
    if (PAIR) zbp::cluster_sync();  // no remote arrivals or copies remain
    if (warp == 1) {
        zbp::tc_fence_after();
        if (PAIR)
            zbp::tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else
            zbp::tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------- host side
zb_status launched(const char* who) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string(who) + " launch: " + cudaGetErrorString(e));
    zb::clear_error();
    return ZB_OK;
}

template <int EPI, int CG, int MX>
zb_status launch_fp8(const CUtensorMap (&mp)[5], const Fp8Args& a, long long tiles, void* stream) {
    using E = Fp8Epi<EPI, CG, MX>;
    auto kern = zb_fp8_matmul_kernel<EPI, CG, MX>;
    static std::atomic<int> cache[64];
    int ctas = 0;
    zb_status s = full_grid(kern, cache, fp8_smem<EPI, CG, MX>(), E::THREADS, CG, &ctas);
    if (s != ZB_OK) return s;
    LaunchCfg lc(static_cast<int>(std::min<long long>(tiles * CG, ctas)), E::THREADS, fp8_smem<EPI, CG, MX>(),
                 CG, stream);
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, kern, mp[0], mp[1], mp[2], mp[3], mp[4], a);
    if (e != cudaSuccess) return zb::fail(ZB_ERR_CUDA, std::string("zb_fp8_matmul launch: ") + cudaGetErrorString(e));
    return launched("zb_fp8_matmul");
}

template <int EPI>
zb_status launch_fp8_by(bool pair, bool mx, const CUtensorMap (&mp)[5], const Fp8Args& a, long long tiles, void* stream) {
    if (mx) return pair ? launch_fp8<EPI, 2, 1>(mp, a, tiles, stream) : launch_fp8<EPI, 1, 1>(mp, a, tiles, stream);
    return pair ? launch_fp8<EPI, 2, 0>(mp, a, tiles, stream) : launch_fp8<EPI, 1, 0>(mp, a, tiles, stream);
}

// 2-D map of e4m3 rows, 128 bytes wide boxes, 128-byte swizzle.
bool make_map8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_outer, std::string* why) {
    EncodeTiledFn fn = encode_fn(why);
    if (!fn) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {inner};
    cuuint32_t box[2] = {BLK, box_outer};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        if (why) *why = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string(static_cast<int>(r));
        return false;
    }
    return true;
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
    const long long per = 8 * 2 * Q_ILP;  // blocks of 128 in a thread block
    const long long grid = (rows * blocks + per - 1) / per;
    if (grid > 0x7fffffffLL) return zb::fail(ZB_ERR_SHAPE, "zb_fp8_quantize_rows: too many elements");
    zb_fp8_quantize_rows_kernel<<<static_cast<unsigned>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(X), static_cast<uint2*>(Q), S, rows * blocks, static_cast<int>(cols / 8), blocks);
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
        static_cast<const uint4*>(W), static_cast<uint2*>(Q), S, static_cast<uint8_t*>(QT), ST, static_cast<int>(rows),
        static_cast<int>(cols));
    return launched("zb_fp8_quantize_weight");
}

extern "C" zb_status zb_fp8_matmul(const zb_fp8_gemm* g, const int32_t* offsets, const void* Xq, const float* xs,
                                   const void* Wq, const float* ws, const void* bias, const void* H, void* out0,
                                   void* out1, void* stream) {
    if (!g) return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: descriptor is NULL");
    if (g->scales != ZB_FP8_SCALE_POW2 && g->scales != ZB_FP8_SCALE_ANY)
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_fp8_matmul: unknown kind of scales");
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
    if (off4(offsets) || off16(Xq) || off4(xs) || off16(Wq) || off4(ws) || off16(bias) || off16(H) || off16(out0) ||
        off16(out1))
        return zb::fail(ZB_ERR_ALIGN, "zb_fp8_matmul: pointers must be 16-byte aligned (offsets, scales: 4)");
    // tiles of 256 rows on pairs when they fill the SMs, else 128 (counts as if
    // the rows were spread evenly)
    const int64_t used = std::min<int64_t>(g->experts, g->M);
    const int64_t each = (g->M + used - 1) / used;
    const long long cols = (g->N + 255) / 256;
    const bool pair = used * ((each + 255) / 256) * cols >= sm_count() / 2;
    const int tt = pair ? 256 : 128;
    const long long most = (g->M / tt + used) * cols;  // no launch has more tiles
    std::string why;
    CUtensorMap mp[5];
    const uint64_t rows = static_cast<uint64_t>(g->M);
    bool ok = make_map8(&mp[0], Xq, g->K, rows, 128, &why) && make_map8(&mp[1], Xq, g->K, rows, 32, &why) &&
              make_map3(&mp[2], Wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g->K, g->N, g->experts, BLK, pair ? 128 : 256, &why) &&
              make_map(&mp[3], out0, false, g->N, rows, g->N, 32, 32, &why, CU_TENSOR_MAP_SWIZZLE_64B) &&
              make_map(&mp[4], g->epilogue == ZB_FP8_GELU ? out1 : g->epilogue == ZB_FP8_GELU_GRAD ? H : out0, false, g->N, rows, g->N, 32, 32, &why,
                       CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return zb::fail(ZB_ERR_CUDA, why);
    unsigned int* err = zb::device_error_word();
    if (!err) return ZB_ERR_CUDA;
    Fp8Args a;
    a.offsets = offsets;
    a.xs = xs;
    a.ws = ws;
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.out0 = static_cast<__nv_bfloat16*>(out0);
    a.out1 = static_cast<__nv_bfloat16*>(out1);
    a.rows = static_cast<int>(g->M);
    a.experts = g->experts;
    a.N = static_cast<int>(g->N);
    a.K = static_cast<int>(g->K);
    a.act = g->act;
    a.err = err;
    const bool mx = g->scales == ZB_FP8_SCALE_POW2;
    switch (g->epilogue) {
        case ZB_FP8_STORE: return launch_fp8_by<ZB_FP8_STORE>(pair, mx, mp, a, most, stream);
        case ZB_FP8_GELU: return launch_fp8_by<ZB_FP8_GELU>(pair, mx, mp, a, most, stream);
        default: return launch_fp8_by<ZB_FP8_GELU_GRAD>(pair, mx, mp, a, most, stream);
    }
}
