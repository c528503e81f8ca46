// Causal grouped-query attention over whole prompts, packed one behind the
// other, in fp32:
//   out[i,h] = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   within each prompt.
//
// Every factor is split into two tf32 numbers, x = hi + lo (11 + 11 bits), and a
// product is three tensor products hi hi + hi lo + lo hi; what is left out or
// rounded is at most 4.5 x 2^-22 of |x y| a term, no more than a dot product of a
// few fp32 terms.  1800 tokens in 3 prompts, 8 / 4 heads of 64: 54 us (fp32
// multiply-adds on the CUDA cores: 121 us); 4000 in 8 prompts, 16 / 4 heads: 146 us.
// Spills: 60 bytes a thread with heads of 128, 12 with heads of 64.
//
// A tile is 64 query rows of one head.  A block's two groups of 4 warps, 16 rows a
// warp, and those of up to three more blocks of its cluster walk the tile's keys
// 32 at a time in turn, with an online softmax each, and are joined at the end
// through the cluster's shared memory, so that the longest rows of a short batch
// take half or a quarter as long.  K and V are split on their way into shared
// memory, in the order in which mma.m16n8k8's lanes read them: 16-byte pieces
// (hi, lo, hi, lo) of two neighbouring dims of a key (K) or of one dim of two
// neighbouring keys (V); which dims or keys a k-step takes is free as long as
// both factors agree.  Two blocks an SM hide each
// other's loads (head dim 128, one block: the next keys' rows are requested
// before the present ones' products).  Bound by latencies and barriers between
// the splitting of a tile and its products, at about half of the issue slots.
#include "common.cuh"
#include "gqa_prompt.cuh"
#include "launchers.h"
#include "sm100.cuh"

namespace dsa {

using namespace sm100;

namespace {

constexpr int BM = 64, GROUPS = 2, GROUP = 128, THREADS = GROUPS * GROUP;
constexpr float LN2 = 0.6931471805599453f;

// Index -> (prompt, tile of query rows), the longest work first (more prompts
// than a warp's lanes: prompt by prompt, the last tile of each first).  False
// past the last tile.
struct Tile {
    int first, len, row0;           // the prompt's first packed row and length; the tile's first row in it
};
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int t, Tile& w, int* sh) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32 && a.n_seqs <= LANE_SEQS) {
        PromptLanes lanes;
        lanes.init(a, BM);
        const bool found = t < lanes.at_least(1);
        int first, n, block;
        if (found) lanes.get(t, first, n, block);
        if (lane == 0) {
            if (found) {
                sh[0] = first;
                sh[1] = n;
                sh[2] = block * BM;
            }
            sh[3] = found ? 1 : -1;
        }
    } else if (threadIdx.x < 32) {
        int base = 0, found = -1;
        for (int s0 = 0; s0 < a.n_seqs && found < 0; s0 += 32) {
            const int s = s0 + lane;
            int b = 0, n = 0;
            if (s < a.n_seqs) prompt_bounds(a, s, b, n);
            const int tiles = (n + BM - 1) / BM;
            int x = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (t >= base + x - tiles && t < base + x) {
                sh[0] = b;
                sh[1] = n;
                sh[2] = (tiles - 1 - (t - (base + x - tiles))) * BM;
                found = 1;
            }
            found = __any_sync(0xffffffffu, found > 0) ? 1 : -1;
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) sh[3] = found;
    }
    __syncthreads();
    w.first = sh[0];
    w.len = sh[1];
    w.row0 = sh[2];
    return sh[3] > 0;
}


// The tf32 parts of two numbers: (hi, lo, hi, lo).
__device__ __forceinline__ uint4 split2(float x, float y) {
    uint4 r;
    tf32_split(x, r.x, r.y);
    tf32_split(y, r.z, r.w);
    return r;
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// C[t] += A B[t], A's parts in hi / lo, B's as pieces (hi, lo, hi, lo) of k = c4
// and c4 + 4; the products with a lo part go to `small` (which may be C).  A
// product's three parts follow one another at a distance of N.
template <int N>
__device__ __forceinline__ void mma_split(float (*c)[4], float (*small)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                          const uint4 (&b)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) mma1688(small[t], lo, b[t].x, b[t].z);
#pragma unroll
    for (int t = 0; t < N; ++t) mma1688(small[t], hi, b[t].y, b[t].w);
#pragma unroll
    for (int t = 0; t < N; ++t) mma1688(c[t], hi, b[t].x, b[t].z);
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D> struct Cfg {
    static constexpr int BN = 32;                                    // keys of a tile
    static constexpr int BLOCKS = D == 64 ? 2 : 1;                  // per SM
    static constexpr int NB = D == 64 ? 4 : 8;                      // tiles of 8 dims of an output step
    static constexpr int KV = BN * D * 8;                           // bytes of a split K (or V) tile
    static constexpr int Q = BM * D * 8;
    static constexpr int SMEM = Q + GROUPS * 2 * KV;
    static_assert(2 * KV >= BM * (D + 2) * 4, "a group's output is handed over in its tiles");
};

template <int D, int CLUSTER>
__global__ void __launch_bounds__(THREADS, Cfg<D>::BLOCKS) gqa_prompt_f32_kernel(const PromptArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    using C = Cfg<D>;
    constexpr int WALKERS = CLUSTER * GROUPS;           // groups that share the tile's keys
    constexpr int BN = C::BN, NT = D / 8, ST = BN / 8, NB = C::NB, HALF = D / 2;
    constexpr int LOADS = BN * HALF / GROUP;          // (key, two dims) or (two keys, dim) pieces of a tile per thread
    extern __shared__ __align__(128) uint8_t smem[];
    uint4* sq = (uint4*)smem;                           // [BM][D / 2] pieces, swizzled by row
    const int grp = threadIdx.x / GROUP, rank = (int)cluster_ctarank(), walker = rank * GROUPS + grp;
    uint4* sk = sq + BM * HALF + grp * 2 * BN * HALF;   // the group's tile: [BN][D / 2]
    uint4* sv = sk + BN * HALF;                         // [BN / 2][D], swizzled by key pair
    __shared__ int sh[4];
    Tile w;
    const int pair = blockIdx.x / CLUSTER, tile = pair / a.n_heads;
    if (!find_tile(a, tile, w, sh)) return;             // (the whole cluster)
    const int head = pair - tile * a.n_heads, kvh = head / (a.n_heads / a.n_kv_heads);
    const int tid = threadIdx.x % GROUP, lane = tid & 31, warp = tid >> 5, r4 = lane >> 2, c4 = lane & 3;
    const int rows = min(BM, w.len - w.row0);
    const float* q = (const float*)a.q + (int64_t)(w.first + w.row0) * a.ld_q + head * D;
    const float* kb = (const float*)a.k + (int64_t)w.first * a.ld_k + kvh * D;
    const float* vb = (const float*)a.v + (int64_t)w.first * a.ld_v + kvh * D;
    const int keys = w.row0 + rows;                     // the tile's last row sees this many

    float2 kx[LOADS], vx[LOADS];                        // the next tile's rows, on their way
    // piece i of a thread: key KI i + tid / HALF, dims 2 (tid % HALF) and + 1 of K;
    // keys KI i + 2 (tid / D) and + 1, dim tid % D of V
    constexpr int KI = GROUP / HALF;
    const int kr = tid / HALF, vr = tid / D, vd = tid % D;
    const float* const k_from = kb + (int64_t)kr * a.ld_k + 2 * (tid % HALF);
    const float* const v_from = vb + 2 * (int64_t)vr * a.ld_v + vd;
    auto request = [&](int k0) {
        const float *kp = k_from + (int64_t)k0 * a.ld_k, *vp = v_from + (int64_t)k0 * a.ld_v;
        const bool whole = k0 + BN <= keys;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int left = keys - k0 - i * KI;            // keys from the piece's first on
            kx[i] = whole || kr < left ? __ldg((const float2*)kp) : make_float2(0.f, 0.f);
            vx[i].x = whole || 2 * vr < left ? __ldg(vp) : 0.f;
            vx[i].y = whole || 2 * vr + 1 < left ? __ldg(vp + a.ld_v) : 0.f;
            kp += KI * a.ld_k;
            vp += KI * a.ld_v;
        }
    };
    uint4* const k_to = sk + kr * HALF + ((tid % HALF) ^ ((kr & 1) << 2));     // (KI is even)
    auto store = [&]() {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            k_to[i * KI * HALF] = split2(kx[i].x, kx[i].y);
            const int pair = i * (KI / 2) + vr;
            sv[pair * D + (vd ^ ((pair & 3) << 1))] = split2(vx[i].x, vx[i].y);
        }
    };
    constexpr bool AHEAD = C::BLOCKS == 1;              // (two blocks an SM hide each other's loads)
    if (AHEAD) request(walker * BN);
    for (int p = threadIdx.x; p < BM * HALF; p += THREADS) {
        const int r = p / HALF, d2 = p % HALF;
        const float2 x = r < rows ? __ldg((const float2*)(q + (int64_t)r * a.ld_q) + d2) : make_float2(0.f, 0.f);
        sq[r * HALF + (d2 ^ ((r & 1) << 2))] = split2(x.x * a.scale_log2, x.y * a.scale_log2);
    }
    float o[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int row = warp * 16 + r4;                     // this lane's rows of the tile: row, row + 8
    const int odd = (r4 & 1) << 2;
    const uint4 *const q_from = sq + row * HALF + c4, *const k_at = sk + r4 * HALF + c4;
    const uint4* const v_at = sv + c4 * D + (r4 ^ (c4 << 1));
    const int last = w.row0 + min(rows, warp * 16 + 16) - 1;    // the warp's last row
    __syncthreads();                                    // the queries stand
    for (int k0 = walker * BN; k0 < keys; k0 += WALKERS * BN) {
        if (!AHEAD) request(k0);
        named_bar_sync(1 + grp, GROUP);                 // the tile before has been read
        store();
        named_bar_sync(1 + grp, GROUP);
        if (AHEAD && k0 + WALKERS * BN < keys) request(k0 + WALKERS * BN);
        if (k0 > last) continue;                        // all of it lies behind this warp's rows
        // (the tensor core's sums round toward zero: the small products are
        // summed apart, which takes two thirds of the steps off the scores' sums)
        float s[ST][4], small[ST][4];
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = small[t][e] = 0.f;
        // k-step kk: dims 8 kk + 2 c4 (k = c4) and 8 kk + 2 c4 + 1 (k = c4 + 4)
#pragma unroll 4
        for (int kk = 0; kk < D / 8; ++kk) {
            const int at = 4 * (kk & ~1) + ((kk & 1) ? 4 - odd : odd);      // (4 kk + c4) ^ 4 (row & 1), less c4
            const uint4 x = q_from[at], y = q_from[8 * HALF + at];
            const uint32_t hi[4] = {x.x, y.x, x.z, y.z}, lo[4] = {x.y, y.y, x.w, y.w};
            uint4 b[ST];
#pragma unroll
            for (int t = 0; t < ST; ++t) b[t] = k_at[8 * t * HALF + at];
            mma_split<ST>(s, small, hi, lo, b);
        }
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] += small[t][e];
        // lane: rows row, row + 8; keys k0 + 8 t + 2 c4 + {0, 1}
        if (k0 + BN - 1 > w.row0 + warp * 16) {             // some keys lie behind some rows
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int t = 0; t < ST; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (k0 + 8 * t + 2 * c4 + e > w.row0 + row + 8 * half) s[t][2 * half + e] = -INFINITY;
        }
        float f[2];
        bool moved = false;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) top = fmaxf(top, s[t][2 * half + e]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            f[half] = 1.f;
            if (top > m[half]) {
                f[half] = fast_exp2(m[half] - top);
                m[half] = top;
                l[half] *= f[half];
                moved = true;
            }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                o[t][0] *= f[0]; o[t][1] *= f[0]; o[t][2] *= f[1]; o[t][3] *= f[1];
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float base = m[half] > -INFINITY ? m[half] : 0.f;
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p = fast_exp2(s[t][2 * half + e] - base);
                    l[half] += p;
                    s[t][2 * half + e] = p;
                }
        }
        // k-step t: keys 8 t + 2 c4 (k = c4) and 8 t + 2 c4 + 1 (k = c4 + 4), the
        // lane's own scores.  The tensor core's sums round toward zero, so a
        // tile's output is summed from zero and added to the running one here.
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += NB) {
            float step[NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) step[n][e] = 0.f;
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                const uint4 x = split2(s[t][0], s[t][1]), y = split2(s[t][2], s[t][3]);
                const uint32_t hi[4] = {x.x, y.x, x.z, y.z}, lo[4] = {x.y, y.y, x.w, y.w};
                uint4 b[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) b[n] = v_at[4 * t * D + 8 * (n0 + n)];
                mma_split<NB>(step, step, hi, lo, b);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n0 + n][e] += step[n][e];
        }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    }
    // Every group lays its (maximum, sum, output) into its own tiles, a row of
    // D + 2 floats each; each block of the cluster joins half of the rows.
    named_bar_sync(1 + grp, GROUP);                     // the last tile has been read
    float* hand = (float*)sk;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float* h = hand + (row + 8 * half) * (D + 2);
        if (c4 == 0) *(float2*)h = make_float2(m[half], l[half]);
#pragma unroll
        for (int n = 0; n < NT; ++n) *(float2*)(h + 2 + 8 * n + 2 * c4) = make_float2(o[n][2 * half], o[n][2 * half + 1]);
    }
    cluster_sync_all();
    const uint32_t hand0 = smem_u32(sq + BM * HALF);
    uint32_t part[WALKERS];
#pragma unroll
    for (int i = 0; i < WALKERS; ++i) part[i] = mapa_shared(hand0 + (i % GROUPS) * 2 * C::KV, i / GROUPS);
    for (int r = rank * (BM / CLUSTER) + threadIdx.x / 32; r < min(rows, (rank + 1) * (BM / CLUSTER)); r += THREADS / 32) {
        float2 ml[WALKERS], x[WALKERS][D / 64];
#pragma unroll
        for (int i = 0; i < WALKERS; ++i) {
            const uint32_t h = part[i] + r * (D + 2) * 4;
            ml[i] = ld_cluster_f2(h);
#pragma unroll
            for (int k = 0; k < D / 64; ++k) x[i][k] = ld_cluster_f2(h + 8 + (k * 64 + 2 * lane) * 4);
        }
        float top = ml[0].x, sum = 0.f;
#pragma unroll
        for (int i = 1; i < WALKERS; ++i) top = fmaxf(top, ml[i].x);
        const float base = top > -INFINITY ? top : 0.f;
        float2 y[D / 64] = {};
#pragma unroll
        for (int i = 0; i < WALKERS; ++i) {
            const float f = fast_exp2(ml[i].x - base);
            sum = fmaf(f, ml[i].y, sum);
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                y[k].x = fmaf(f, x[i][k].x, y[k].x);
                y[k].y = fmaf(f, x[i][k].y, y[k].y);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t at = ((int64_t)w.first + w.row0 + r) * a.n_heads + head;
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
            *(float2*)((float*)a.out + at * D + k * 64 + 2 * lane) = make_float2(y[k].x * inv, y[k].y * inv);
        if (lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * LN2;
    }
    cluster_sync_relaxed();                             // no block leaves while the other reads its part
}

// Blocks that share a tile.  A tile's time is its keys', so where there are few
// tiles each is cut among more blocks, whose own start and end count otherwise.
// us with 1 / 2 / 4 blocks: 16 tiles of head dim 128 65 / 37 / 24, 188 of them
// 170 / 153 / 200, 264 of them 87 / 105 / 176; 76 tiles of head dim 64 56 / 38 / 28,
// 112 of them 27 / 24 / 31, 232 of them 83 / 54 / 68, 564 of them 100 / 111 / 151.
template <int D> int cluster_of(int64_t tiles, int sms) {
    return tiles * 3 <= 2 * sms ? 4 : tiles * 5 <= 7 * Cfg<D>::BLOCKS * sms ? 2 : 1;
}

template <int D, int CLUSTER>
cudaError_t launch_cluster(const Launch& L, const PromptArgs& a) {
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = allow_smem(done, gqa_prompt_f32_kernel<D, CLUSTER>, Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2] = {pdl_attr(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CLUSTER;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    // as many tiles as any split of `total` rows over the prompts can have
    const unsigned most = (unsigned)(a.total / BM + (a.n_seqs < a.total ? a.n_seqs : a.total));
    cfg.gridDim = dim3((unsigned)CLUSTER * (unsigned)a.n_heads * most);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Cfg<D>::SMEM;
    cfg.stream = L.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, gqa_prompt_f32_kernel<D, CLUSTER>, a);
    count_launch();
    return e;
}

template <int D> cudaError_t launch(const Launch& L, const PromptArgs& a) {
    switch (cluster_of<D>((int64_t)ceil_div(a.total, BM) * a.n_heads, L.num_sms)) {
        case 4: return launch_cluster<D, 4>(L, a);
        case 2: return launch_cluster<D, 2>(L, a);
        default: return launch_cluster<D, 1>(L, a);
    }
}

}  // namespace

cudaError_t launch_gqa_prompt_f32(const Launch& L, const PromptArgs& a, int head_dim) {
    return head_dim == 64 ? launch<64>(L, a) : launch<128>(L, a);
}

}  // namespace dsa
