// Causal grouped-query attention over whole prompts, packed one behind the
// other, bf16 on the 5th-generation tensor cores:
//   out[i,h] = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   within each prompt.
//
// A persistent block per SM works on items of two query tiles of 128 rows that
// share their keys: two heads of one group over the same rows (even groups),
// or two neighbouring row tiles of one head (odd groups).  Per 128 keys:
//   S_t = Q_t K^T      tcgen05, [128 x 128 x D] into tensor memory
//   P_t = softmax part one thread per row: the row's 128 scores are read into
//                      registers, brought to base 2 and rounded to bf16 over the
//                      scores' own place in tensor memory
//   O_t += P_t V       tcgen05 with P from tensor memory
// The products alternate between the tiles (O_0, S_0', O_1, S_1'), so that
// one tile's exponentials run under the other tile's products.  The running
// maximum is lazy: it moves, and O is rescaled by the row's own thread, only
// when a row's maximum grows by more than 2^8; S's arrival means that all
// earlier products have finished (products complete in order).  P is announced
// in two parts, so that its first products run under the last exponentials.
//
// What bounds it (32 / 8 heads of 128, 8K-token prompts, cycles per 128 keys
// of both tiles): 2048 are tensor work at its nominal rate; with the softmax
// replaced by nothing 2590 remain (the scores' product reads both operands
// from shared memory at its full bandwidth, and the loads write there too);
// with it 3250, a tile's softmax (1800: 128 exponentials a row at 16 a clock
// and SM, half overlapped with the other tile's) behind its products.  Tried
// and slower: two threads per row (3860), steps of 64 keys with two score
// buffers per tile (3560: scores 64 wide read shared memory 1.5 times as much).
// 16,384 tokens in 5 such prompts: 600 us, 1.18 PFLOP/s, in a short run and 700 back
// to back, where the clock falls under the power limit; with heads of 64, half the
// products for the same exponentials, 517 us.  All four variants spill, by 4 to 60
// bytes a thread, at the 168 registers of their launch.
//
// Warps 0-3 / 4-7: softmax and epilogue of tile 0 / 1; 8: products, tensor
// memory; 9: TMA loads; 10: zeroes the rows of a last V tile that lie behind
// the prompt (they belong to other prompts, and 0 times their infinities
// would not be 0).  Items are taken longest first.
//
// Few heads and long prompts (a model's heads dealt to several GPUs) leave fewer
// items than the longest one's time lets hide: there the keys of an item are cut
// into up to four parts, whose unnormalised fp32 sums a second kernel joins.
#include "common.cuh"
#include "gqa_prompt.cuh"
#include "launchers.h"
#include "sm100.cuh"
#include "tensor_map.h"

namespace dsa {

using namespace sm100;

namespace {

constexpr int BM = 128, BN = 128;
constexpr int MMA_WARP = 8, LOAD_WARP = 9, ZERO_WARP = 10;
constexpr int THREADS = 384;
// registers: launched at 168 x 384; the softmax warps take what the others give back
constexpr int REGS_SOFTMAX = 216, REGS_REST = 72;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_REST <= 168 * THREADS, "register split exceeds launch");
constexpr int TMEM_COLS = 512;
constexpr float RESCALE_LOG2 = 8.f;
constexpr int MAX_CHUNKS = 4;       // parts of an item's keys
// Of 16 exponentials, how many run on the multiply-add pipe, and how many of
// a tile's four 32-key pieces of P are announced together first.  Cycles per
// 128 keys of both tiles: 0 -> 3440, 2 -> 3280, 3 -> 3256, 4 -> 3370 (three
// pieces first); 2 with two pieces first 3249.
constexpr int FMA_EXP = 3, FIRST_PIECES = 2;
constexpr float LN2 = 0.6931471805599453f;

constexpr int OUT_STAGE = 4096;         // per softmax warp: 32 output rows x 64 dims
template <int D> struct Cfg {
    static constexpr int TILE = 128 * D * 2;                // bytes of a Q, K or V tile
    static constexpr int STAGES = D == 128 ? 4 : 8;         // K / V ring
    static constexpr int SMEM = 2 * TILE + STAGES * TILE + 8 * OUT_STAGE + 1024 + 1024;
    static constexpr int O_COL = 256;                       // S_0, S_1 at 0, 128; O_0, O_1 behind
};

template <int STAGES> struct Bars {
    uint64_t q_full, q_empty, kv_full[STAGES], kv_empty[STAGES];
    uint64_t s_full[2], p_ready[2][2], o_final[2], to_zero, zeroed;
    uint32_t tmem;
    int abort;
};

struct Entry {
    int seq, block;
};

struct Sched {                      // where the items come from
    const Entry* list;              // NULL: scheduled by the warp itself
    const int* count;
    int pairs;                      // items per row block: head pairs (even groups) or heads
    int rows_per_block;             // 128 (even groups) or 256
    bool two_heads;
    // split items: key tiles of one, their largest number, and what they leave:
    // [part, row, head] sums of p v and (maximum in base 2, sum of p)
    int chunk, chunks;
    float* part_o;
    float2* part_ml;
};

// One warp's view of the items, longest first.
template <bool SPLIT> struct Items {
    PromptLanes lanes;              // without a list
    int entries;

    // row blocks that reach into part c of their keys
    __device__ __forceinline__ int reaching(const Sched& s, int c) const {
        return lanes.at_least(c * (s.chunk * BN / s.rows_per_block) + 1);
    }
    __device__ __forceinline__ void init(const PromptArgs& a, const Sched& s) {
        if (!SPLIT && s.list) {
            entries = *s.count;
        } else {
            lanes.init(a, s.rows_per_block);
            entries = lanes.at_least(1);
            if (SPLIT)
                for (int c = 1; c < s.chunks; ++c) entries += reaching(s, c);
        }
    }
    // Entry e: blocks in falling order of their number (their work), part by
    // part of their keys; false past the end.
    __device__ __forceinline__ bool get(const PromptArgs& a, const Sched& s, int e, int& first, int& n, int& row0,
                                        int& part) const {
        if (e >= entries) return false;
        int block;
        part = 0;
        if (SPLIT)
            for (int left = reaching(s, 0); e >= left; left = reaching(s, ++part)) e -= left;
        if (!SPLIT && s.list) {
            const Entry x = s.list[e];
            first = a.cu_seqlens[x.seq];
            n = a.cu_seqlens[x.seq + 1] - first;
            block = x.block;
        } else {
            lanes.get(e, first, n, block);
        }
        row0 = block * s.rows_per_block;
        return true;
    }
};

struct Item {
    int first, len;                 // the prompt's first packed row, and its length
    int head[2], row0[2], n[2];     // per tile: query head, first row in the prompt, key tiles (0: no tile)
    int kvh, n_max;
    int part, tile0;                // split items: number, first key tile
    bool diagonal[2], whole[2];     // split items: whether the last tile is the diagonal one; whether this is all
};

// The block's r-th item; odd rounds run backwards over the blocks, so that
// neither end of the grid collects the longer ones.
template <bool SPLIT>
__device__ __forceinline__ bool get_item(const PromptArgs& a, const Sched& s, const Items<SPLIT>& items, int round, Item& w) {
    const int g = gridDim.x, b = blockIdx.x;
    const int64_t i = (int64_t)round * g + ((round & 1) ? g - 1 - b : b);
    const int64_t e = i / s.pairs;
    const int p = (int)(i - e * s.pairs);
    int row0;
    if (e > 0x7fffffff || !items.get(a, s, (int)e, w.first, w.len, row0, w.part)) return false;
    w.tile0 = SPLIT ? w.part * s.chunk : 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        w.head[t] = s.two_heads ? 2 * p + t : p;
        w.row0[t] = s.two_heads ? row0 : row0 + t * BM;
        w.n[t] = w.row0[t] < w.len ? w.row0[t] / BN + 1 : 0;
        w.diagonal[t] = w.whole[t] = true;
        if (SPLIT) {
            w.whole[t] = w.n[t] <= s.chunk;
            w.diagonal[t] = w.n[t] - w.tile0 <= s.chunk;
            w.n[t] = max(0, min(w.n[t] - w.tile0, s.chunk));
        }
    }
    w.kvh = w.head[0] / (a.n_heads / a.n_kv_heads);
    w.n_max = max(w.n[0], w.n[1]);
    return true;
}

// 2^x on the MUFU unit: relative error ~2^-22, -inf -> +0.
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of three; NaN where one is NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x of two numbers on the multiply-add pipe, for x <= 100: x = n + f with n
// whole (rounded by adding 1.5 * 2^23) and |f| <= 1/2, 2^f by a polynomial of
// degree 4 fitted here for the least largest relative error with its constant
// term held at 1 (2.9e-6, a thousandth of the bf16 rounding that follows), n
// added to the exponent.  x <= -127 gives +0: there f = 0, and 1 with its
// exponent lowered by 127 is +0.
__device__ __forceinline__ float2 exp2_fma(float2 x) {
    const float2 magic = make_float2(12582912.f, 12582912.f);
    x.x = fmaxf(x.x, -127.f);
    x.y = fmaxf(x.y, -127.f);
    const float2 t = add2(x, magic);
    const float2 f = fma2(add2(t, make_float2(-12582912.f, -12582912.f)), make_float2(-1.f, -1.f), x);
    float2 p = fma2(make_float2(0.009585382416844368f, 0.009585382416844368f), f,
                    make_float2(0.05590662732720375f, 0.05590662732720375f));
    p = fma2(p, f, make_float2(0.24024038016796112f, 0.24024038016796112f));
    p = fma2(p, f, make_float2(0.6931241750717163f, 0.6931241750717163f));
    p = fma2(p, f, make_float2(1.f, 1.f));
    return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                       __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace

// The items' list for more prompts than a warp holds: row blocks sorted by
// their number within their prompt, falling (a counting sort in one block).
constexpr int LIST_BINS = 4096;
__global__ void __launch_bounds__(1024) gqa_prompt_list_kernel(const PromptArgs a, int rows_per_block, Entry* list,
                                                               int* count, int max_entries) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int bins[LIST_BINS];
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < LIST_BINS; i += 1024) bins[i] = 0;
    __syncthreads();
    // bin 0 holds the largest numbers
    auto bin_of = [](int block) { return LIST_BINS - 1 - min(block, LIST_BINS - 1); };
    for (int s = warp; s < a.n_seqs; s += 32) {
        int start, len;
        prompt_bounds(a, s, start, len);
        const int blocks = (len + rows_per_block - 1) / rows_per_block;
        for (int b = lane; b < blocks; b += 32) atomicAdd(&bins[bin_of(b)], 1);
    }
    __syncthreads();
    // exclusive prefix sum over the bins, four per thread
    int v[LIST_BINS / 1024], sum = 0;
#pragma unroll
    for (int i = 0; i < LIST_BINS / 1024; ++i) {
        v[i] = bins[tid * (LIST_BINS / 1024) + i];
        sum += v[i];
    }
    int x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = x - sum;
    for (int i = 0; i < warp; ++i) before += warp_sum[i];
#pragma unroll
    for (int i = 0; i < LIST_BINS / 1024; ++i) {
        bins[tid * (LIST_BINS / 1024) + i] = before;
        before += v[i];
    }
    if (tid == 1023) *count = min(before, max_entries);
    __syncthreads();
    for (int s = warp; s < a.n_seqs; s += 32) {
        int start, len;
        prompt_bounds(a, s, start, len);
        const int blocks = (len + rows_per_block - 1) / rows_per_block;
        for (int b = lane; b < blocks; b += 32) {
            const int at = atomicAdd(&bins[bin_of(b)], 1);
            if (at < max_entries) list[at] = Entry{s, b};   // (more only when prompts overlap)
        }
    }
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) gqa_prompt_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                   const __grid_constant__ CUtensorMap k_map,
                                                                   const __grid_constant__ CUtensorMap v_map,
                                                                   const PromptArgs a, const Sched sched) {
    using C = Cfg<D>;
    constexpr int NS = C::STAGES, TILE = C::TILE, KBLK = D / 64, BLK = 128 * 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* qbuf = smem;                               // two Q tiles: [D / 64][128 rows x 128 B], swizzled
    uint8_t* kvbuf = smem + 2 * TILE;                   // ring of K and V tiles, same layout
    uint8_t* obuf = smem + (2 + NS) * TILE;             // output rows on their way to memory
    auto* bars = (Bars<NS>*)(obuf + 8 * OUT_STAGE);
    volatile int* abort_flag = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_ready[t][0], 4);
            mbar_init(&bars->p_ready[t][1], 4);
            mbar_init(&bars->o_final[t], 1);
        }
        mbar_init(&bars->to_zero, 1);
        mbar_init(&bars->zeroed, 1);
        bars->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&q_map);
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    if (warp == MMA_WARP) {
        tmem_alloc(&bars->tmem, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    pdl_wait();
    pdl_launch_dependents();
    Items<SPLIT> items;
    Item w;
    items.init(a, sched);

    if (warp < 8) {
        regs_inc<REGS_SOFTMAX>();
        // ------------------------------------------- softmax and epilogue ----
        const int t = warp >> 2, r = (warp & 3) * 32 + lane;        // tile; row = tensor-memory lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_col = lane_base + t * 128, o_col = lane_base + C::O_COL + t * D;
        uint32_t n_s = 0, n_o = 0;                                  // phases used so far
        bool ok = true;
        for (int round = 0; ok && get_item(a, sched, items, round, w); ++round) {
            const int n = w.n[t];
            if (n == 0) continue;
            float m = -INFINITY, l = 0.f;                           // maximum in use (base 2), sum
            for (int j = 0; j < n; ++j) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&bars->s_full[t], n_s & 1, a.err, DEV_ERR_TIMEOUT_MMA, abort_flag));
                if (!ok) break;
                ++n_s;
                tc_fence_after();
                float s[4][32];
                tmem_ld32(s_col, s[0]);
                tmem_ld32(s_col + 32, s[1]);
                tmem_ld_wait();
                tmem_ld32(s_col + 64, s[2]);                        // (these arrive under the first half's weights)
                tmem_ld32(s_col + 96, s[3]);
                if (j == n - 1 && (!SPLIT || w.diagonal[t])) {      // the diagonal tile: keys up to the row's own
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c * 32 + e > r) s[c][e] = -INFINITY;
                }
                // The tile's largest score.  Where it is NaN or +inf, so is the row's sum from here on: the
                // weights alone would not show it, as exp2_fma gives 0 for a NaN.
                auto largest = [&]() {
                    float mx[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) mx[c] = max3(s[c][0], s[c][1], s[c][2]);
#pragma unroll
                    for (int e = 3; e < 31; e += 2)
#pragma unroll
                        for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], s[c][e], s[c][e + 1]);
                    const float top = max3(max3(mx[0], mx[1], s[0][31]), max3(mx[2], mx[3], s[1][31]),
                                           max3(s[2][31], s[3][31], mx[0])) * a.scale_log2;
                    if (!(top < INFINITY)) l = __uint_as_float(0x7fffffffu);
                    return top;
                };
                const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
                float2 sum[2], neg;
                auto weights = [&](int c) {                         // P of 32 keys
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 x = fma2(make_float2(s[c][2 * e], s[c][2 * e + 1]), sc2, neg);
                        if ((e * FMA_EXP) % 16 < FMA_EXP) {
                            x = exp2_fma(x);
                        } else {
                            x.x = fast_exp2(x.x);
                            x.y = fast_exp2(x.y);
                        }
                        sum[e & 1] = add2(sum[e & 1], x);
                        pk[e] = bf16x2_bits(x.x, x.y);
                    }
                    tmem_st16(s_col + c * 16, pk);
                };
                auto announce = [&](int part) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->p_ready[t][part]);
                };
                if (j == 0) {
                    tmem_ld_wait();
                    m = largest();
                }
                // The weights are formed with the maximum in use while the
                // tile's own is still being found: it seldom moves.  Where it
                // does, O and the sum are rescaled and the weights formed again,
                // before any of them is announced.
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    const float base = m == -INFINITY ? 0.f : m;
                    neg = make_float2(-base, -base);
                    sum[0] = sum[1] = make_float2(0.f, 0.f);
                    weights(0);
                    weights(1);
                    if (pass == 0) tmem_ld_wait();
#pragma unroll
                    for (int c = 2; c < FIRST_PIECES; ++c) weights(c);
                    if (pass > 0 || j == 0) break;
                    const float top = largest();
                    const bool move = top > m + RESCALE_LOG2 || (m == -INFINITY && top > m);
                    if (!__any_sync(0xffffffffu, move)) break;
                    const float f = move ? fast_exp2(m - top) : 1.f;
                    if (move) m = top;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float v[32];
                        tmem_ld32(o_col + c * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] *= f;
                        tmem_st32(o_col + c * 32, v);
                    }
                }
                announce(0);
#pragma unroll
                for (int c = FIRST_PIECES; c < 4; ++c) weights(c);
                announce(1);
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_final[t], n_o & 1, a.err, DEV_ERR_TIMEOUT_MMA, abort_flag));
            if (!ok) break;
            ++n_o;
            tc_fence_after();
            // Rows of 64 dims through shared memory, so that a store covers four
            // whole 128-byte pieces instead of 32 lanes' own rows.
            const int rows = w.len - w.row0[t] - (warp & 3) * 32;   // of this warp's 32, those inside the prompt
            const int64_t row0 = (int64_t)w.first + w.row0[t] + (warp & 3) * 32;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint8_t* stage = obuf + warp * OUT_STAGE;
            if (SPLIT && !w.whole[t]) {
                // a part of the keys: the sums as they are, in fp32, 32 dims at a time
                const int64_t part_row = (int64_t)w.part * a.total + row0;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    tmem_ld32(o_col + c * 32, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        st_shared_v4(stage + lane * 128 + ((e ^ (lane & 7)) << 4), __float_as_uint(v[4 * e]),
                                     __float_as_uint(v[4 * e + 1]), __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3]));
                    __syncwarp();
                    float* out = sched.part_o + (part_row * a.n_heads + w.head[t]) * D + c * 32 + (lane & 7) * 4;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = i * 4 + (lane >> 3);
                        const uint4 x = ld_shared_v4(stage + k * 128 + (((lane & 7) ^ (k & 7)) << 4));
                        if (k < rows) *(uint4*)(out + (int64_t)k * a.n_heads * D) = x;
                    }
                    __syncwarp();
                }
                if (lane < rows) sched.part_ml[(part_row + lane) * a.n_heads + w.head[t]] = make_float2(m, l);
                tc_fence_before();
                continue;
            }
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    tmem_ld32(o_col + c * 64 + h * 32, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        st_shared_v4(stage + lane * 128 + (((4 * h + e) ^ (lane & 7)) << 4),
                                     bf16x2_bits(v[8 * e] * inv, v[8 * e + 1] * inv),
                                     bf16x2_bits(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                     bf16x2_bits(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                     bf16x2_bits(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                }
                __syncwarp();
                __nv_bfloat16* out = (__nv_bfloat16*)a.out + (row0 * a.n_heads + w.head[t]) * D + c * 64 + (lane & 7) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int k = i * 4 + (lane >> 3);
                    const uint4 x = ld_shared_v4(stage + k * 128 + (((lane & 7) ^ (k & 7)) << 4));
                    if (k < rows) *(uint4*)(out + (int64_t)k * a.n_heads * D) = x;
                }
                __syncwarp();
            }
            if (lane < rows) a.lse[(row0 + lane) * a.n_heads + w.head[t]] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
            tc_fence_before();          // O has been read before this tile's next P is announced
        }
    } else {
        regs_dec<REGS_REST>();
        if (warp == MMA_WARP) {
            // ------------------------------------------------- products ----
            constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, 0, 0), idesc_o = idesc_bf16_f32(BM, D, 0, 1);
            const uint32_t qb = smem_u32(qbuf), kvb = smem_u32(kvbuf);
            const bool leader = elect_one();
            uint32_t slot = 0, n_p[2] = {0, 0}, n_z = 0;    // first ring slot of the item; phases used
            bool ok = true;
            auto wait_kv = [&](uint32_t i) {
                return mbar_wait(&bars->kv_full[i % NS], (i / NS) & 1, a.err, DEV_ERR_TIMEOUT_TMA, abort_flag);
            };
            // low halves of the first descriptors of Q, K (K-major) and V (MN-major)
            constexpr uint32_t hi = desc_sw128_hi(1024);
            const uint32_t q_lo = desc_lo(qb, 1), k_lo = desc_lo(kvb, 1), v_lo = desc_lo(kvb, BLK >> 4);
            auto product_s = [&](int t, uint32_t kslot) {
                const uint32_t ql = q_lo + t * (TILE >> 4), kl = k_lo + (kslot % NS) * (TILE >> 4), d = tmem + t * 128;
                mma_ss_halves<false>(d, ql, kl, hi, idesc_s);
#pragma unroll
                for (int kk = 1; kk < D / 16; ++kk) {
                    const uint32_t off = (uint32_t)((kk >> 2) * BLK + (kk & 3) * 32) >> 4;
                    mma_ss_halves<true>(d, ql + off, kl + off, hi, idesc_s);
                }
                mma_commit(&bars->s_full[t]);
            };
            for (int round = 0; get_item(a, sched, items, round, w); ++round) {
                if (leader && ok) {
                    ok = mbar_wait(&bars->q_full, round & 1, a.err, DEV_ERR_TIMEOUT_TMA, abort_flag) && wait_kv(slot);
                    if (ok) {
                        tc_fence_after();
                        for (int t = 0; t < 2; ++t)
                            if (w.n[t] > 0) product_s(t, slot);
                        mma_commit(&bars->kv_empty[slot % NS]);
                        if (w.n_max == 1) mma_commit(&bars->q_empty);
                    }
                    for (int j = 0; j < w.n_max && ok; ++j) {
                        const uint32_t vslot = slot + 2 * j + 1, kslot = vslot + 1;
                        ok = wait_kv(vslot);
                        if (ok && (w.tile0 + j + 1) * BN > w.len) {
                            mbar_arrive(&bars->to_zero);        // the tile has landed
                            ok = mbar_wait(&bars->zeroed, n_z & 1, a.err, DEV_ERR_TIMEOUT_PEER, abort_flag);
                            ++n_z;
                        }
                        const int last_now = w.n[1] > j ? 1 : 0, last_next = w.n[1] > j + 1 ? 1 : 0;
                        bool have_k = false;
                        for (int t = 0; t < 2 && ok; ++t) {
                            if (j >= w.n[t]) continue;
                            const uint32_t vl = v_lo + (vslot % NS) * (TILE >> 4), d = tmem + C::O_COL + t * D;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                ok = ok && mbar_wait(&bars->p_ready[t][half], n_p[t] & 1, a.err, DEV_ERR_TIMEOUT_PEER, abort_flag);
                                if (!ok) break;
                                tc_fence_after();
#pragma unroll
                                for (int kk = half ? 2 * FIRST_PIECES : 0; kk < (half ? BN / 16 : 2 * FIRST_PIECES); ++kk)
                                    mma_ts_halves(d, tmem + t * 128 + kk * 8, vl + kk * (16 * 128 >> 4), hi, idesc_o,
                                                  kk > 0 ? 1u : j > 0);
                            }
                            if (!ok) break;
                            ++n_p[t];
                            if (j == w.n[t] - 1) mma_commit(&bars->o_final[t]);
                            if (t == last_now) mma_commit(&bars->kv_empty[vslot % NS]);
                            if (j + 1 < w.n[t]) {
                                if (!have_k) ok = wait_kv(kslot);
                                if (!ok) break;
                                have_k = true;
                                tc_fence_after();
                                product_s(t, kslot);
                                if (t == last_next) {
                                    mma_commit(&bars->kv_empty[kslot % NS]);
                                    if (j + 1 == w.n_max - 1) mma_commit(&bars->q_empty);
                                }
                            }
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, __ffs(__ballot_sync(0xffffffffu, leader)) - 1) != 0;
                if (!ok) break;
                slot += 2 * w.n_max;
            }
        } else if (warp == LOAD_WARP) {
            // ---------------------------------------------------- loads ----
            const bool leader = elect_one();
            uint32_t slot = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap* map, int col, int row) {
                const uint32_t st = slot % NS;
                if (!mbar_wait(&bars->kv_empty[st], ((slot / NS) & 1) ^ 1, a.err, DEV_ERR_TIMEOUT_MMA, abort_flag)) return false;
                mbar_arrive_expect_tx(&bars->kv_full[st], TILE);
#pragma unroll
                for (int b = 0; b < KBLK; ++b)
                    tma_load_2d(kvbuf + st * TILE + b * BLK, map, col + b * 64, row, &bars->kv_full[st]);
                ++slot;
                return true;
            };
            int q_loads = 0;
            for (int round = 0; get_item(a, sched, items, round, w); ++round) {
                if (leader && ok) {
                    ok = mbar_wait(&bars->q_empty, (round & 1) ^ 1, a.err, DEV_ERR_TIMEOUT_MMA, abort_flag);
                    if (ok) {
                        const int tiles = (w.n[0] > 0) + (w.n[1] > 0);
                        mbar_arrive_expect_tx(&bars->q_full, tiles * TILE);
                        for (int t = 0; t < 2; ++t)
                            if (w.n[t] > 0)
                                for (int b = 0; b < KBLK; ++b)
                                    tma_load_2d(qbuf + t * TILE + b * BLK, &q_map, w.head[t] * D + b * 64,
                                                w.first + w.row0[t], &bars->q_full);
                        ++q_loads;
                    }
                    for (int j = 0; j < w.n_max && ok; ++j)
                        ok = load(&k_map, w.kvh * D, w.first + (w.tile0 + j) * BN) &&
                             load(&v_map, w.kvh * D, w.first + (w.tile0 + j) * BN);
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, __ffs(__ballot_sync(0xffffffffu, leader)) - 1) != 0;
                if (!ok) break;
            }
            if (leader && *abort_flag) {
                // after an abort, tiles already requested land before the block exits
                for (uint32_t i = slot > NS ? slot - NS : 0; i < slot; ++i)
                    mbar_wait(&bars->kv_full[i % NS], (i / NS) & 1, a.err, DEV_ERR_TIMEOUT_TMA, nullptr);
                if (q_loads > 0) mbar_wait(&bars->q_full, (q_loads - 1) & 1, a.err, DEV_ERR_TIMEOUT_TMA, nullptr);
            }
        } else if (warp == ZERO_WARP) {
            // ----------------------------- rows of V behind a prompt's end ----
            uint32_t slot = 0, n_z = 0;
            for (int round = 0; get_item(a, sched, items, round, w); ++round) {
                const int left = w.len - (w.tile0 + w.n_max - 1) * BN;  // rows of the last key tile
                if (left < BN) {
                    const uint32_t i = slot + 2 * (w.n_max - 1) + 1;
                    const bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->to_zero, n_z & 1, a.err, DEV_ERR_TIMEOUT_PEER,
                                                                      abort_flag));
                    if (!ok) break;
                    ++n_z;
                    for (int b = 0; b < KBLK; ++b) {
                        uint8_t* rows = kvbuf + (i % NS) * TILE + b * BLK;
                        for (int o = left * 128 + lane * 16; o < BN * 128; o += 32 * 16) st_shared_v4(rows + o, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->zeroed);
                }
                slot += 2 * w.n_max;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// The parts of split items joined: a warp per (row, head).
template <int D>
__global__ void __launch_bounds__(128) gqa_prompt_join_kernel(const PromptArgs a, const Sched s) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t item = blockIdx.x * 4ll + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= (int64_t)a.total * a.n_heads) return;
    const int row = (int)(item / a.n_heads);
    int start = 0, len = 0;
    if (lane < a.n_seqs) prompt_bounds(a, lane, start, len);
    const unsigned mine = __ballot_sync(0xffffffffu, row >= start && row - start < len);
    if (!mine) return;                                      // outside every prompt
    const int tiles = (row - __shfl_sync(0xffffffffu, start, __ffs(mine) - 1)) / BN + 1;
    if (tiles <= s.chunk) return;                           // written whole
    const int parts = (tiles - 1) / s.chunk + 1;
    float2 ml[MAX_CHUNKS], o[MAX_CHUNKS][D / 64];
#pragma unroll
    for (int c = 0; c < MAX_CHUNKS; ++c) {
        const int64_t at = (int64_t)min(c, parts - 1) * a.total * a.n_heads + item;
        ml[c] = s.part_ml[at];
#pragma unroll
        for (int k = 0; k < D / 64; ++k) o[c][k] = *(const float2*)(s.part_o + at * D + k * 64 + 2 * lane);
        if (c >= parts) ml[c] = make_float2(-INFINITY, 0.f);
    }
    float top = ml[0].x, l = 0.f;
#pragma unroll
    for (int c = 1; c < MAX_CHUNKS; ++c) top = fmaxf(top, ml[c].x);
    const float base = top > -INFINITY ? top : 0.f;
    float2 sum[D / 64] = {};
#pragma unroll
    for (int c = 0; c < MAX_CHUNKS; ++c) {
        if (c >= parts) break;
        const float f = fast_exp2(ml[c].x - base);
        l = fmaf(f, ml[c].y, l);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) sum[k] = fma2(make_float2(f, f), o[c][k], sum[k]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
        *(uint32_t*)((__nv_bfloat16*)a.out + item * D + k * 64 + 2 * lane) = bf16x2_bits(sum[k].x * inv, sum[k].y * inv);
    if (lane == 0) a.lse[item] = l == 0.f ? -INFINITY : (top + log2f(l)) * LN2;
}

namespace {

int max_entries(int total, int n_seqs) { return total / BM + (n_seqs < total ? n_seqs : total); }

// Key tiles of a split item, or 0: items stay whole.  `pairs` items share a
// block of rows.  A block's time is its longest item, so items are cut where
// the longest (taking prompts to differ by up to twice their average) is well
// above a block's share of all work; cutting costs the parts' way through
// memory and a second kernel, which three tiles saved must pay for.  One prompt,
// heads of 128, whole / cut: 8192 tokens, 4 heads 115 / 87 us, 1 head 110 / 41;
// 4096 tokens, 4 heads 60 / 44, 8 heads 62 / 60; 2048 tokens, 4 heads 33 / 21.
int chunk_of(int total, int n_seqs, int pairs, int rows_per_block, int sms) {
    if (n_seqs > LANE_SEQS) return 0;
    const int64_t longest = total < 2 * ((int64_t)total / n_seqs + 1) ? total : 2 * ((int64_t)total / n_seqs + 1);
    const int64_t tiles = (longest + BN - 1) / BN, blocks = ((int64_t)total + rows_per_block - 1) / rows_per_block;
    const int64_t share = pairs * blocks * tiles / (2 * sms);
    const int64_t all = ((int64_t)total + BN - 1) / BN;
    int64_t chunk = share * 7 / 10 > 4 ? share * 7 / 10 : 4;        // (less than a share: blocks take unequal numbers of items)
    if (chunk * MAX_CHUNKS < all) chunk = (all + MAX_CHUNKS - 1) / MAX_CHUNKS;
    chunk += chunk & 1;
    return tiles >= chunk + 3 && 2 * tiles > 3 * share ? (int)chunk : 0;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t parts_bytes(int total, int n_heads, int head_dim) {
    const size_t rows = (size_t)MAX_CHUNKS * total * n_heads;
    return up256(rows * 8) + rows * head_dim * 4;
}

template <int D>
cudaError_t launch(const Launch& L, const PromptArgs& a, void* workspace) {
    using C = Cfg<D>;
    CUtensorMap q_map, k_map, v_map;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!make_map_sw128_ld(&q_map, bf, 2, a.q, (uint64_t)a.n_heads * D, a.total, (uint64_t)a.ld_q * 2, 64, BM) ||
        !make_map_sw128_ld(&k_map, bf, 2, a.k, (uint64_t)a.n_kv_heads * D, a.total, (uint64_t)a.ld_k * 2, 64, BN) ||
        !make_map_sw128_ld(&v_map, bf, 2, a.v, (uint64_t)a.n_kv_heads * D, a.total, (uint64_t)a.ld_v * 2, 64, BN))
        return cudaErrorInvalidValue;
    const int group = a.n_heads / a.n_kv_heads;
    Sched s;
    s.two_heads = group % 2 == 0;
    s.pairs = s.two_heads ? a.n_heads / 2 : a.n_heads;
    s.rows_per_block = s.two_heads ? BM : 2 * BM;
    s.list = nullptr;
    s.count = nullptr;
    s.chunk = chunk_of(a.total, a.n_seqs, s.pairs, s.rows_per_block, L.num_sms);
    s.chunks = s.chunk ? ceil_div(ceil_div(a.total, BN), s.chunk) : 1;
    s.part_ml = (float2*)workspace;
    s.part_o = (float*)((char*)workspace + up256((size_t)MAX_CHUNKS * a.total * a.n_heads * 8));
    static std::atomic<int> done[2][kMaxDevices];
    const auto kern = s.chunk ? gqa_prompt_tc_kernel<D, true> : gqa_prompt_tc_kernel<D, false>;
    cudaError_t e = allow_smem(done[s.chunk != 0], kern, C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.stream = L.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int most = max_entries(a.total, a.n_seqs);
    if (a.n_seqs > LANE_SEQS) {
        s.count = (const int*)workspace;
        s.list = (const Entry*)((char*)workspace + 256);
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(1024);
        e = cudaLaunchKernelEx(&cfg, gqa_prompt_list_kernel, a, s.rows_per_block, (Entry*)s.list, (int*)s.count, most);
        count_launch();
        if (e != cudaSuccess) return e;
    }
    const int64_t items = (int64_t)most * s.pairs * s.chunks;
    cfg.gridDim = dim3((unsigned)(items < L.num_sms ? items : L.num_sms));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    e = cudaLaunchKernelEx(&cfg, kern, q_map, k_map, v_map, a, s);
    count_launch();
    if (e != cudaSuccess || !s.chunk) return e;
    cfg.gridDim = dim3((unsigned)(((int64_t)a.total * a.n_heads + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, gqa_prompt_join_kernel<D>, a, s);
    count_launch();
    return e;
}

}  // namespace

// (The number of kv heads is not asked for: enough for either kind of item.)
size_t gqa_prompt_workspace_bytes(int total, int n_seqs, int n_heads, int head_dim, dsa_dtype_t dtype, int sms) {
    if (dtype != DSA_BF16) return 0;
    if (n_seqs > LANE_SEQS) return 256 + (size_t)max_entries(total, n_seqs) * sizeof(Entry);
    return chunk_of(total, n_seqs, n_heads / 2, BM, sms) || chunk_of(total, n_seqs, n_heads, 2 * BM, sms)
               ? parts_bytes(total, n_heads, head_dim)
               : 0;
}

cudaError_t launch_gqa_prompt_tc(const Launch& L, const PromptArgs& a, int head_dim, void* workspace) {
    return head_dim == 64 ? launch<64>(L, a, workspace) : launch<128>(L, a, workspace);
}

}  // namespace dsa
