// embedding.cu — rows of a table by id: the lookup (F of a pipeline's first
// stage) and the table's gradient (its W; there is no B) from the tokens in the
// order of their ids.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <string>

#include "launch.cuh"
#include "ptx.cuh"

namespace {

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// ---------------------------------------------------------------- lookup
// A warp copies up to 32 x LOOK_U pieces of 8 values of one token's row.  HBM bounds
// it (8192 tokens of 50000 ids, width 4096: 17 us, 7.7 TB/s with the repeated ids' rows
// from L2).
constexpr int LOOK_U = 4;

template <typename T>
__global__ void __launch_bounds__(256)
    zb_embedding_forward_kernel(const int* __restrict__ ids, const uint4* __restrict__ E, T* __restrict__ Y,
                                long long tokens, long long vocab, int w8, int segs, float scale) {
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const long long t = item / segs;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    if (t >= tokens) return;
    const int at = static_cast<int>(item - t * segs) * 32 * LOOK_U + (threadIdx.x & 31);
    const int id = ids[t];
    const bool on = id >= 0 && id < vocab;
    const uint4* src = E + static_cast<long long>(on ? id : 0) * w8;
    uint4 q[LOOK_U];
#pragma unroll
    for (int u = 0; u < LOOK_U; ++u) {
        q[u] = make_uint4(0, 0, 0, 0);
        if (on && at + 32 * u < w8) q[u] = src[at + 32 * u];
    }
#pragma unroll
    for (int u = 0; u < LOOK_U; ++u) {
        const int k = at + 32 * u;
        if (k >= w8) break;
        const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = on ? __uint_as_float(w[i] << 16) * scale : 0.0f;
            v[2 * i + 1] = on ? __uint_as_float(w[i] & 0xffff0000u) * scale : 0.0f;
        }
        T* y = Y + (t * w8 + k) * 8;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(y) =
                make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        } else {
            reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

// ---------------------------------------------------------------- sort
// Keys are ids, `vocab` standing for every id outside the table.
__device__ __forceinline__ uint32_t key_of(int id, uint32_t vocab) {
    return static_cast<uint32_t>(id) < vocab ? static_cast<uint32_t>(id) : vocab;
}
__device__ __forceinline__ int id_of(uint32_t key, uint32_t vocab) { return key < vocab ? static_cast<int>(key) : -1; }

// A stable radix sort by one cluster of 8 or 16 blocks, digits from the lowest up.
// A block owns its part of the tokens and a warp a contiguous part of that, so that a
// digit's tokens are placed in the order (block, warp, token): each warp
// counts its digits, the counts are summed over warps and blocks (through
// distributed shared memory) into the first place of each warp's tokens of each
// digit, and the warp places its tokens by them.
// Latency bounds it up to some 10000 tokens (a pass is 3 to 4 us: one read of the
// tokens, two cluster barriers, one placing), then the placing: us of 8 and 16 blocks, 32000
// ids: 1025 tokens 8.5 and 9.5, 8192 10.7 and 10.8, 16384 13.8 and 11.8, 262144 104
// and 57.  One block alone: 10.0 at 1025, 27.7 at 8192.
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_BITS = 10;  // of a digit, at most
constexpr int SORT_LONG = 8192;  // tokens from which on 16 blocks sort
constexpr int SORT_HELD = 8;   // tokens a lane holds in registers from counting to placing
constexpr size_t sort_smem(int bits) { return (static_cast<size_t>(SORT_WARPS + 2) << bits) * 4; }

struct SortArgs {
    const int* ids;
    int tokens, bits, passes;  // bits of a digit
    uint32_t vocab;
    uint2* pairs[2];  // (key, token), placed by one pass and read by the next
    int *order, *sorted_id;
};

template <int BLOCKS>
__global__ void __cluster_dims__(BLOCKS, 1, 1) __launch_bounds__(SORT_THREADS)
    zb_embedding_sort_kernel(const SortArgs a) {
    extern __shared__ uint32_t sort_shared[];
    __shared__ uint32_t warp_total[SORT_WARPS];
    const int digits = 1 << a.bits;
    uint32_t* hist = sort_shared;                        // [warp][digit]
    uint32_t* total = sort_shared + SORT_WARPS * digits;  // [digit]: the block's
    uint32_t* base = total + digits;                      // [digit]: place of the block's first such token
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = threadIdx.x;
    const uint32_t rank = zbp::cluster_ctarank();
    const long long n = a.tokens;
    const int part = static_cast<int>(rank) * SORT_WARPS + warp;
    const int lo = static_cast<int>(n * part / (BLOCKS * SORT_WARPS));
    const int hi = static_cast<int>(n * (part + 1) / (BLOCKS * SORT_WARPS));
    uint32_t* mine = hist + warp * digits;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    constexpr int STEP = 32 * SORT_HELD;
    for (int pass = 0; pass < a.passes; ++pass) {
        const uint2* src = a.pairs[(pass + 1) & 1];
        const int shift = pass * a.bits;
        uint2 held[SORT_HELD];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int k = 0; k < SORT_HELD; ++k) {
                const int i = i0 + k * 32 + lane;
                if (i < hi)
                    held[k] = pass == 0 ? make_uint2(key_of(a.ids[i], a.vocab), static_cast<uint32_t>(i)) : __ldcg(src + i);
            }
        };
        auto digit_of = [&](uint32_t k) { return (k >> shift) & static_cast<uint32_t>(digits - 1); };
        fetch(lo);
        for (int d = lane; d < digits; d += 32) mine[d] = 0;
        __syncwarp();
        for (int i0 = lo; i0 < hi; i0 += STEP) {
            if (i0 > lo) fetch(i0);
#pragma unroll
            for (int k = 0; k < SORT_HELD; ++k)
                if (i0 + k * 32 + lane < hi) atomicAdd(&mine[digit_of(held[k].x)], 1u);
        }
        __syncthreads();
        // each warp's count becomes the number of such tokens in the warps before it
        uint32_t here = 0;
        if (t < digits) {
#pragma unroll 1
            for (int w0 = 0; w0 < SORT_WARPS; w0 += 8) {
                uint32_t c[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) c[w] = hist[(w0 + w) * digits + t];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    hist[(w0 + w) * digits + t] = here;
                    here += c[w];
                }
            }
            total[t] = here;
        }
        zbp::cluster_sync();
        // the digit's tokens in the blocks before this one, and in all
        uint32_t before = 0, all = 0;
        if (t < digits) {
            const uint32_t at = zbp::smem_u32(&total[t]);
            uint32_t c[BLOCKS];
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b)
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c[b]) : "r"(zbp::mapa_shared(at, b)) : "memory");
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                if (b < static_cast<int>(rank)) before += c[b];
                all += c[b];
            }
        }
        uint32_t sum = all;  // over the digits up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        if (lane == 31) warp_total[warp] = sum;
        __syncthreads();
        uint32_t left = lane < warp ? warp_total[lane] : 0u;
        left = __reduce_add_sync(0xffffffffu, left);
        if (t < digits) base[t] = sum + left - all + before;
        __syncthreads();
        const bool last = pass + 1 == a.passes;
        for (int i0 = lo; i0 < hi; i0 += STEP) {
            if (hi - lo > STEP) fetch(i0);
#pragma unroll
            for (int k = 0; k < SORT_HELD; ++k) {
                if (i0 + k * 32 >= hi) break;
                const bool on = i0 + k * 32 + lane < hi;
                const uint32_t d = on ? digit_of(held[k].x) : ~0u;
                const uint32_t peers = __match_any_sync(0xffffffffu, d);
                const int before_me = __popc(peers & ((1u << lane) - 1u));
                uint32_t place = 0;
                if (on) place = base[d] + mine[d] + static_cast<uint32_t>(before_me);
                __syncwarp();
                if (on && before_me == 0) mine[d] += static_cast<uint32_t>(__popc(peers));
                __syncwarp();
                if (on) {
                    if (last) {
                        a.order[place] = static_cast<int>(held[k].y);
                        a.sorted_id[place] = id_of(held[k].x, a.vocab);
                    } else {
                        a.pairs[pass & 1][place] = held[k];
                    }
                }
            }
        }
        zbp::cluster_sync();  // the next pass reads what the others placed; no one's totals are read any more
    }
}

// Few tokens: a token's place is the number of tokens that go before it.  One
// block, every key in shared memory.  us of this and of the radix sort: 128 tokens
// 2.5 and 8.4, 256 tokens 4.1 and 8.4 (of 32000 ids).
constexpr int RANK_TOKENS = 256;
constexpr int RANK_THREADS = 1024;

__global__ void __launch_bounds__(RANK_THREADS)
    zb_embedding_rank_kernel(const int* __restrict__ ids, int tokens, int lanes, uint32_t vocab, int* __restrict__ order,
                             int* __restrict__ sorted_id) {
    // `lanes` (a power of two, neighbours in a warp) share the keys of a token
    __shared__ __align__(16) uint32_t keys[RANK_TOKENS];
    const int t = threadIdx.x / lanes, s = threadIdx.x & (lanes - 1);
    const int n4 = (tokens + 3) / 4;
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    if (threadIdx.x < 4 * n4)
        keys[threadIdx.x] = static_cast<int>(threadIdx.x) < tokens ? key_of(ids[threadIdx.x], vocab) : ~0u;  // behind every key
    __syncthreads();
    const uint32_t key = keys[min(t, tokens - 1)];
    int place = 0;
#pragma unroll 4
    for (int j = s; j < n4; j += lanes) {
        const uint4 k = reinterpret_cast<const uint4*>(keys)[j];
        const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) place += v[i] < key + (4 * j + i < t ? 1u : 0u);
    }
    for (int o = 1; o < lanes; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (s == 0 && t < tokens) {
        order[place] = t;
        sorted_id[place] = id_of(key, vocab);
    }
}

// ---------------------------------------------------------------- gradient
// The sorted tokens are cut into pieces of PIECE.  A block sums a piece's runs of
// equal ids, a thread 4 columns.  A run that lies within its piece goes straight
// to the table's gradient; what a run has in a piece that it shares with another
// piece goes to the workspace (a row for the run that came in from the left, one
// for the run that goes on to the right), and a second kernel adds such a run's
// parts in order.  Without accumulation blocks of their own write zeros to the
// rows of the ids that do not occur, which warps find by searching the sorted ids.
//
// 16384 tokens of 32000 ids, width 2048, bf16: 60 us of sums and zeros (329 MB, 5.4
// TB/s; zeros alone run at 6.1) and 8 of joining; accumulating 28 and 8.  One row at a
// time instead of 8: 66 accumulating in all.  Zeros in blocks before the others: 76
// overwriting for 66 in all.
constexpr int PIECE = 32;
constexpr int GRAD_THREADS = 256;
constexpr int ZERO_ROWS = 8;  // of a warp

struct GradArgs {
    const int* order;
    const int* sorted_id;
    const void* dY;
    float* dE;
    float4* part;  // [pieces][2][w4]
    int tokens, pieces, w4, col_blocks;
    long long piece_blocks, zero_blocks;
    uint32_t vocab;
    int accumulate;
    float scale;
};

// 4 consecutive values as they lie in memory.
template <typename T>
struct Four;
template <>
struct Four<float> {
    float4 q;
    __device__ __forceinline__ void load(const float* p) { q = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ float4 get() const { return q; }
};
template <>
struct Four<__nv_bfloat16> {
    uint2 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ float4 get() const {
        return make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u), __uint_as_float(q.y << 16),
                           __uint_as_float(q.y & 0xffff0000u));
    }
};
__device__ __forceinline__ void add4(float4& a, const float4& b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}
__device__ __forceinline__ float4* row_of(const GradArgs& a, int id, int c) {
    return reinterpret_cast<float4*>(a.dE) + static_cast<long long>(id) * a.w4 + c;
}
__device__ __forceinline__ float4 scaled(const GradArgs& a, const float4& s, const float4& old) {
    return make_float4(fmaf(a.scale, s.x, old.x), fmaf(a.scale, s.y, old.y), fmaf(a.scale, s.z, old.z),
                       fmaf(a.scale, s.w, old.w));
}

// The warp's searches for the first sorted id (as unsigned: -1 is the last) at
// least `a`, and at least `b`, 32 probes a step.
__device__ __forceinline__ void lower_bounds(const int* sorted_id, int n, uint32_t a, uint32_t b, int& at_a, int& at_b) {
    const int lane = threadIdx.x & 31;
    int lo[2] = {0, 0}, len[2] = {n, n};  // the place lies in [lo, lo + len]
    const uint32_t want[2] = {a, b};
    while (len[0] > 0 || len[1] > 0) {
        uint32_t v[2];
        int step[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            step[k] = (len[k] + 31) / 32;
            const int at = lo[k] + (lane + 1) * step[k] - 1;
            v[k] = len[k] > 0 && at < lo[k] + len[k] ? static_cast<uint32_t>(sorted_id[at]) : ~0u;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (len[k] <= 0) continue;
            const int end = lo[k] + len[k];
            lo[k] = min(end, lo[k] + __popc(__ballot_sync(0xffffffffu, v[k] < want[k])) * step[k]);
            len[k] = min(step[k] - 1, end - lo[k]);
        }
    }
    at_a = lo[0];
    at_b = lo[1];
}

// Zeros for those of a warp's ZERO_ROWS rows whose ids do not occur.
__device__ void zero_rows(const GradArgs& a, long long chunk) {
    const int lane = threadIdx.x & 31;
    const long long row0 = chunk * ZERO_ROWS;
    if (row0 >= a.vocab) return;
    const uint32_t first = static_cast<uint32_t>(row0), rows = min(static_cast<uint32_t>(ZERO_ROWS), a.vocab - first);
    int lo, hi;
    lower_bounds(a.sorted_id, a.tokens, first, first + rows, lo, hi);
    uint32_t occurs = 0;  // a bit a row
    if (hi - lo <= 64) {
        for (int i = lo; i < hi; i += 32) {
            uint32_t bit = 0;
            if (i + lane < hi) {
                const uint32_t r = static_cast<uint32_t>(a.sorted_id[i + lane]) - first;
                if (r < rows) bit = 1u << r;
            }
            occurs |= __reduce_or_sync(0xffffffffu, bit);
        }
    } else {
        // some ids are frequent: each row's own first place
        int at = lo;
        for (uint32_t r = 0; r < rows; ++r) {
            int next, unused;
            lower_bounds(a.sorted_id, a.tokens, first + r + 1, 0, next, unused);
            if (next > at) occurs |= 1u << r;
            at = next;
        }
    }
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (uint32_t r = 0; r < rows; ++r) {
        if ((occurs >> r) & 1u) continue;
        float4* out = reinterpret_cast<float4*>(a.dE) + (row0 + r) * a.w4;
        for (int c = lane; c < a.w4; c += 32) out[c] = zero;
    }
}

// ADD: the sums are added to what dE holds (`accumulate`).
template <typename T, bool ADD>
__global__ void __launch_bounds__(GRAD_THREADS) zb_embedding_backward_kernel(const GradArgs a) {
    zbp::grid_dependency_wait();
    zbp::allow_dependent_launch();
    // blocks that write zeros are spread evenly among the others, whose reads they overlap
    const long long all = a.piece_blocks + a.zero_blocks, zeros = blockIdx.x * a.zero_blocks / all;
    if ((blockIdx.x + 1) * a.zero_blocks / all > zeros) {
        zero_rows(a, zeros * (GRAD_THREADS / 32) + (threadIdx.x >> 5));
        return;
    }
    __shared__ int id_s[PIECE + 2], tok_s[PIECE];
    const int block = static_cast<int>(blockIdx.x - zeros), piece = block / a.col_blocks;
    const int c = (block - piece * a.col_blocks) * GRAD_THREADS + threadIdx.x;
    const int first = piece * PIECE, n = min(PIECE, a.tokens - first);
    if (threadIdx.x < PIECE + 2) {
        const int i = first - 1 + static_cast<int>(threadIdx.x);
        id_s[threadIdx.x] = i >= 0 && i < a.tokens ? a.sorted_id[i] : -1;
        if (threadIdx.x < PIECE) {
            const int tok = static_cast<int>(threadIdx.x) < n ? a.order[first + threadIdx.x] : 0;
            tok_s[threadIdx.x] = tok >= 0 && tok < a.tokens ? tok : 0;
        }
    }
    __syncthreads();
    if (c >= a.w4) return;
    const T* dY = static_cast<const T*>(a.dY) + 4 * c;
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 sum = none;
    // the run at hand came in from the left
    bool from_left = id_s[0] == id_s[1];
    // U rows at a time: all of them, and what dE holds for the runs that end among
    // them, are asked for before the first is added
    constexpr int U = 8;
    for (int i0 = 0; i0 < n; i0 += U) {
        Four<T> v[U];
        float4 old[ADD ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < n) v[u].load(dY + static_cast<long long>(tok_s[i0 + u]) * (4 * a.w4));
        if (ADD) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int id = i0 + u < n ? id_s[i0 + u + 1] : -1;
                old[ADD ? u : 0] = none;
                if (static_cast<uint32_t>(id) < a.vocab && id_s[i0 + u + 2] != id) old[ADD ? u : 0] = *row_of(a, id, c);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= n) break;
            const int id = id_s[i + 1];
            add4(sum, v[u].get());
            const bool more = id_s[i + 2] == id;  // the run goes on
            if (more && i + 1 < n) continue;
            if (static_cast<uint32_t>(id) < a.vocab) {
                if (from_left)
                    a.part[(2LL * piece) * a.w4 + c] = sum;
                else if (more)
                    a.part[(2LL * piece + 1) * a.w4 + c] = sum;
                else
                    *row_of(a, id, c) = scaled(a, sum, ADD ? old[ADD ? u : 0] : none);
            }
            sum = none;
            from_left = false;
        }
    }
}

// Adds the parts of the runs that start in a piece and go on after it.  A block has
// JOIN_PIECES pieces, of which each group of JOIN_COLS threads (4 columns each) joins
// the run of one, if it has up to JOIN_SHORT parts to add; longer ones are joined by
// the whole block, a quarter of the parts each, the quarters' sums in order.  (A
// block for each piece, most of which have nothing to do: 17 us for 16384 tokens of
// 32000 ids, width 2048, where this takes 8.5.)
constexpr int JOIN_COLS = 64, JOIN_PIECES = 4, JOIN_SHORT = 8;

__global__ void __launch_bounds__(JOIN_COLS * JOIN_PIECES) zb_embedding_join_kernel(const GradArgs a, int col_blocks) {
    __shared__ int last_s[JOIN_PIECES];  // a run's last piece; 0: no run to join
    __shared__ float4 quarters[JOIN_PIECES][JOIN_COLS];
    zbp::grid_dependency_wait();
    const int group = threadIdx.x / JOIN_COLS, lane = threadIdx.x & 31;
    const int piece0 = static_cast<int>(blockIdx.x / col_blocks) * JOIN_PIECES;
    const int col = threadIdx.x % JOIN_COLS, c = static_cast<int>(blockIdx.x % col_blocks) * JOIN_COLS + col;
    const bool on = c < a.w4;
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // parts of pieces [lo, hi), 8 at a time
    auto add_parts = [&](float4& sum, int lo, int hi) {
        for (int p0 = lo; p0 < hi; p0 += 8) {
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p0 + u < hi) v[u] = a.part[2LL * (p0 + u) * a.w4 + c];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p0 + u < hi) add4(sum, v[u]);
        }
    };
    auto put = [&](int id, const float4& sum) {
        float4* out = row_of(a, id, c);
        *out = scaled(a, sum, a.accumulate ? *out : none);
    };
    const int piece = piece0 + group;
    int last = 0, id = -1;
    if (piece + 1 < a.pieces) {
        const int first = piece * PIECE, end = first + PIECE;
        id = a.sorted_id[end - 1];
        const int next = a.sorted_id[end], here = a.sorted_id[first], prev = first > 0 ? a.sorted_id[first - 1] : -1;
        // (a run that came in from the left and fills the piece is joined at its start)
        if (static_cast<uint32_t>(id) < a.vocab && next == id && !(here == id && prev == id)) {
            // pieces that the run fills and leaves, then the one that it ends in
            for (last = piece + 1;; last += 32) {
                const int p = last + lane, n = (p + 1) * PIECE;
                const bool through = p + 1 < a.pieces && a.sorted_id[n - 1] == id && a.sorted_id[n] == id;
                const uint32_t stop = ~__ballot_sync(0xffffffffu, through);
                if (stop) {
                    last += __ffs(static_cast<int>(stop)) - 1;
                    break;
                }
            }
            if (on && last - piece <= JOIN_SHORT) {
                float4 sum = a.part[(2LL * piece + 1) * a.w4 + c];
                add_parts(sum, piece + 1, last + 1);
                put(id, sum);
            }
        }
    }
    if (col == 0) last_s[group] = last;
    __syncthreads();
    for (int k = 0; k < JOIN_PIECES; ++k) {
        const int p = piece0 + k, parts = last_s[k] - p;
        if (last_s[k] == 0 || parts <= JOIN_SHORT) continue;
        float4 sum = none;
        if (on) {
            if (group == 0) sum = a.part[(2LL * p + 1) * a.w4 + c];
            add_parts(sum, p + 1 + static_cast<int>(static_cast<long long>(parts) * group / JOIN_PIECES),
                      p + 1 + static_cast<int>(static_cast<long long>(parts) * (group + 1) / JOIN_PIECES));
        }
        quarters[group][col] = sum;
        __syncthreads();
        if (group == 0 && on) {
#pragma unroll
            for (int q = 1; q < JOIN_PIECES; ++q) add4(sum, quarters[q][col]);
            put(a.sorted_id[(p + 1) * PIECE - 1], sum);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host side
zb_status check_embedding(const char* who, const zb_embedding* e) {
    const std::string w = who;
    if (!e) return zb::fail(ZB_ERR_INVALID_ARG, w + ": descriptor is NULL");
    if (e->tokens < 0 || e->tokens > (1LL << 30)) return zb::fail(ZB_ERR_SHAPE, w + ": tokens must be in [0, 2^30]");
    if (e->vocab < 1 || e->vocab > (1LL << 30)) return zb::fail(ZB_ERR_SHAPE, w + ": vocab must be in [1, 2^30]");
    if (e->width < 1 || e->width > (1LL << 20)) return zb::fail(ZB_ERR_SHAPE, w + ": width must be in [1, 2^20]");
    if (e->width % 8) return zb::fail(ZB_ERR_ALIGN, w + ": width must be a multiple of 8");
    if (e->dtype != ZB_DT_BF16 && e->dtype != ZB_DT_F32) return zb::fail(ZB_ERR_DTYPE, w + ": unknown dtype");
    return ZB_OK;
}

// Blocks of the sort's cluster: 16 from SORT_LONG tokens on where the device can hold a
// cluster of 16 (more than the 8 that any device can), which is asked once a device.
int sort_blocks(int tokens) {
    static std::atomic<int> long_ok[64];  // 1: yes, -1: no
    int dev = 0;
    if (tokens <= SORT_LONG || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8;
    int ok = long_ok[dev].load(std::memory_order_relaxed);
    if (!ok) {
        auto kern = zb_embedding_sort_kernel<16>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(SORT_THREADS);
        cfg.dynamicSmemBytes = sort_smem(SORT_BITS);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        const bool fits = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sort_smem(SORT_BITS))) == cudaSuccess &&
                          cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                          cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0;
        if (!fits) cudaGetLastError();
        ok = fits ? 1 : -1;
        long_ok[dev].store(ok, std::memory_order_relaxed);
    }
    return ok > 0 ? 16 : 8;
}

size_t sort_bytes(const zb_embedding& e) { return e.tokens > RANK_TOKENS ? 16 * static_cast<size_t>(e.tokens) : 0; }
size_t pieces_of(const zb_embedding& e) { return (static_cast<size_t>(e.tokens) + PIECE - 1) / PIECE; }

zb_status check_workspace(const char* who, const zb_embedding* e, const void* workspace, size_t ws_bytes) {
    const size_t need = zb_embedding_workspace_bytes(e);
    if (need && (!workspace || ws_bytes < need))
        return zb::fail(ZB_ERR_WORKSPACE, std::string(who) + ": workspace missing or too small: need " +
                                              std::to_string(need) + " bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return zb::fail(ZB_ERR_ALIGN, std::string(who) + ": workspace must be 256-byte aligned");
    return ZB_OK;
}

}  // namespace

extern "C" zb_status zb_embedding_forward(const zb_embedding* e, const int32_t* ids, const void* E, void* Y,
                                          void* stream) {
    zb_status s = check_embedding("zb_embedding_forward", e);
    if (s != ZB_OK) return s;
    if (e->tokens == 0) return done();
    if (!ids || !E || !Y) return zb::fail(ZB_ERR_INVALID_ARG, "zb_embedding_forward: required pointer is NULL");
    if (off4(ids) || off16(E) || off16(Y))
        return zb::fail(ZB_ERR_ALIGN, "zb_embedding_forward: pointers must be 16-byte aligned (ids: 4)");
    const int w8 = static_cast<int>(e->width / 8);
    const int segs = (w8 + 32 * LOOK_U - 1) / (32 * LOOK_U);
    const long long blocks = (e->tokens * segs + 7) / 8;
    if (blocks > 0x7fffffffLL) return zb::fail(ZB_ERR_SHAPE, "zb_embedding_forward: too many elements");
    auto go = [&](auto kern, auto* y) {
        return launch_after(kern, blocks, 256, 0, stream, ids, static_cast<const uint4*>(E), y,
                            static_cast<long long>(e->tokens), static_cast<long long>(e->vocab), w8, segs, e->scale);
    };
    return launched("zb_embedding_forward",
                    e->dtype == ZB_DT_BF16
                        ? go(zb_embedding_forward_kernel<__nv_bfloat16>, static_cast<__nv_bfloat16*>(Y))
                        : go(zb_embedding_forward_kernel<float>, static_cast<float*>(Y)));
}

extern "C" size_t zb_embedding_workspace_bytes(const zb_embedding* e) {
    if (check_embedding("zb_embedding_workspace_bytes", e) != ZB_OK) return 0;
    // the sort's two copies of keys and tokens, or the gradient's parts of runs
    const size_t parts = pieces_of(*e) > 1 ? pieces_of(*e) * 2 * static_cast<size_t>(e->width) * 4 : 0;
    const size_t need = std::max(sort_bytes(*e), parts);
    zb::clear_error();
    return (need + 255) / 256 * 256;
}

extern "C" zb_status zb_embedding_sort(const zb_embedding* e, const int32_t* ids, int32_t* order, int32_t* sorted_id,
                                       void* workspace, size_t ws_bytes, void* stream) {
    zb_status s = check_embedding("zb_embedding_sort", e);
    if (s != ZB_OK) return s;
    if (e->tokens == 0) return done();
    if (!ids || !order || !sorted_id) return zb::fail(ZB_ERR_INVALID_ARG, "zb_embedding_sort: required pointer is NULL");
    if (off4(ids) || off4(order) || off4(sorted_id))
        return zb::fail(ZB_ERR_ALIGN, "zb_embedding_sort: pointers must be 4-byte aligned");
    s = check_workspace("zb_embedding_sort", e, workspace, ws_bytes);
    if (s != ZB_OK) return s;
    const int n = static_cast<int>(e->tokens);
    const uint32_t vocab = static_cast<uint32_t>(e->vocab);
    if (n <= RANK_TOKENS) {
        int lanes = 1;
        while (lanes < 32 && 2 * lanes * n <= RANK_THREADS) lanes *= 2;
        return launched("zb_embedding_sort", launch_after(zb_embedding_rank_kernel, 1, (n * lanes + 31) / 32 * 32, 0, stream,
                                                          ids, n, lanes, vocab, order, sorted_id));
    }
    int bits = 1;
    while (vocab >> bits) ++bits;
    SortArgs a;
    a.ids = ids;
    a.tokens = n;
    a.passes = (bits + SORT_BITS - 1) / SORT_BITS;
    a.bits = (bits + a.passes - 1) / a.passes;
    a.vocab = vocab;
    for (int i = 0; i < 2; ++i) a.pairs[i] = static_cast<uint2*>(workspace) + static_cast<size_t>(i) * n;
    a.order = order;
    a.sorted_id = sorted_id;
    const int blocks = sort_blocks(n);
    auto go = [&](auto kern) {
        // (a cluster of 16 has got its attributes from sort_blocks)
        const cudaError_t err = blocks > 8 ? cudaSuccess
                                           : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                  static_cast<int>(sort_smem(SORT_BITS)));
        if (err != cudaSuccess)
            return zb::fail(ZB_ERR_CUDA, std::string("zb_embedding_sort: cudaFuncSetAttribute: ") + cudaGetErrorString(err));
        return launched("zb_embedding_sort", launch_after(kern, blocks, SORT_THREADS, sort_smem(a.bits), stream, a));
    };
    return blocks > 8 ? go(zb_embedding_sort_kernel<16>) : go(zb_embedding_sort_kernel<8>);
}

extern "C" zb_status zb_embedding_backward(const zb_embedding* e, const int32_t* order, const int32_t* sorted_id,
                                           const void* dY, float* dE, int accumulate, void* workspace, size_t ws_bytes,
                                           void* stream) {
    zb_status s = check_embedding("zb_embedding_backward", e);
    if (s != ZB_OK) return s;
    if (!dE || (e->tokens > 0 && (!order || !sorted_id || !dY)))
        return zb::fail(ZB_ERR_INVALID_ARG, "zb_embedding_backward: required pointer is NULL");
    if (off4(order) || off4(sorted_id) || off16(dY) || off16(dE))
        return zb::fail(ZB_ERR_ALIGN, "zb_embedding_backward: dY and dE must be 16-byte aligned (indices: 4)");
    s = check_workspace("zb_embedding_backward", e, workspace, ws_bytes);
    if (s != ZB_OK) return s;
    GradArgs a;
    a.order = order;
    a.sorted_id = sorted_id;
    a.dY = dY;
    a.dE = dE;
    a.part = static_cast<float4*>(workspace);
    a.tokens = static_cast<int>(e->tokens);
    a.pieces = static_cast<int>(pieces_of(*e));
    a.w4 = static_cast<int>(e->width / 4);
    a.col_blocks = (a.w4 + GRAD_THREADS - 1) / GRAD_THREADS;
    a.vocab = static_cast<uint32_t>(e->vocab);
    a.accumulate = accumulate != 0;
    a.scale = e->scale;
    constexpr int per = ZERO_ROWS * (GRAD_THREADS / 32);
    a.zero_blocks = accumulate ? 0 : (e->vocab + per - 1) / per;
    a.piece_blocks = static_cast<long long>(a.pieces) * a.col_blocks;
    const long long blocks = a.piece_blocks + a.zero_blocks;
    const int join_cols = (a.w4 + JOIN_COLS - 1) / JOIN_COLS;
    const long long joins = (static_cast<long long>(std::max(a.pieces - 1, 0)) + JOIN_PIECES - 1) / JOIN_PIECES * join_cols;
    if (blocks > 0x7fffffffLL || joins > 0x7fffffffLL)
        return zb::fail(ZB_ERR_SHAPE, "zb_embedding_backward: too many elements");
    if (blocks == 0) return done();
    auto go = [&](auto kern) { return launch_after(kern, blocks, GRAD_THREADS, 0, stream, a); };
    cudaError_t err;
    if (e->dtype == ZB_DT_BF16)
        err = accumulate ? go(zb_embedding_backward_kernel<__nv_bfloat16, true>)
                         : go(zb_embedding_backward_kernel<__nv_bfloat16, false>);
    else
        err = accumulate ? go(zb_embedding_backward_kernel<float, true>) : go(zb_embedding_backward_kernel<float, false>);
    if (err == cudaSuccess && joins > 0)
        err = launch_after(zb_embedding_join_kernel, joins, JOIN_COLS * JOIN_PIECES, 0, stream, a, join_cols);
    return launched("zb_embedding_backward", err);
}
