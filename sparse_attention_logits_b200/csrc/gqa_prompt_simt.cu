// Causal grouped-query attention over whole prompts, packed one behind the
// other, on CUDA cores in fp32:
//   out[i,h] = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   within each prompt.
//
// One block takes 64 query rows of one head and walks the keys in tiles of
// 64 with an online softmax.  Thread (ty, tx) of 16 x 16 holds a 4 x 4 patch
// of the score tile (rows 4 ty + i, keys tx + 16 j) and of the output (rows
// 4 ty + i, D/16 dims); operands come from shared memory as 16-byte vectors.
// Bound by the fp32 pipe: 4 D n (n + 1) / 2 flop per head and prompt.
#include "common.cuh"
#include "launchers.h"

namespace dsa {

namespace {

constexpr int BM = 64, BN = 64, THREADS = 256;
constexpr float LN2 = 0.6931471805599453f;

// Block index -> (prompt, tile of query rows): the tiles of the prompts in
// order, the last tile of each first (the longest work first).  False past
// the last tile.
struct Tile {
    int first, len, row0;           // the prompt's first packed row and length; the tile's first row in it
};
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int t, Tile& w, int* sh) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        int base = 0, found = -1;
        for (int s0 = 0; s0 < a.n_seqs && found < 0; s0 += 32) {
            const int s = s0 + lane;
            int b = 0, n = 0;
            if (s < a.n_seqs) {
                b = a.cu_seqlens[s];
                n = a.cu_seqlens[s + 1] - b;
                if (b < 0 || n < 0 || (int64_t)b + n > a.total) {
                    record_error(a.err, DEV_ERR_BAD_INDEX);
                    n = 0;
                }
            }
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

template <int D>
__global__ void __launch_bounds__(THREADS) gqa_prompt_simt_kernel(const PromptArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int LD = D + 4, OV = D / 64;      // OV: float4 columns of the output per thread
    extern __shared__ float sm[];
    float* sq = sm;                             // [BM][LD], scaled
    float* sk = sq + BM * LD;                   // [BN][LD]
    float* sv = sk + BN * LD;                   // [BN][D]
    float* sp = sv + BN * D;                    // [BM][BN + 4]
    __shared__ int sh[4];
    Tile w;
    const int tile = blockIdx.x / a.n_heads;
    if (!find_tile(a, tile, w, sh)) return;
    const int head = blockIdx.x - tile * a.n_heads, kvh = head / (a.n_heads / a.n_kv_heads);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int rows = min(BM, w.len - w.row0);
    const float* q = (const float*)a.q + (int64_t)(w.first + w.row0) * a.ld_q + head * D;
    for (int i = tid; i < BM * (D / 4); i += THREADS) {
        const int r = i / (D / 4), c = i % (D / 4);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) x = __ldg((const float4*)(q + r * a.ld_q + c * 4));
        *(float4*)(sq + r * LD + c * 4) =
            make_float4(x.x * a.scale_log2, x.y * a.scale_log2, x.z * a.scale_log2, x.w * a.scale_log2);
    }
    float m[4], l[4];
    float4 o[4][OV];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int v = 0; v < OV; ++v) o[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int keys = w.row0 + rows;             // the tile's last row sees this many
    const float* kb = (const float*)a.k + (int64_t)w.first * a.ld_k + kvh * D;
    const float* vb = (const float*)a.v + (int64_t)w.first * a.ld_v + kvh * D;
    for (int k0 = 0; k0 < keys; k0 += BN) {
        __syncthreads();
        for (int i = tid; i < BN * (D / 4); i += THREADS) {
            const int r = i / (D / 4), c = i % (D / 4);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (k0 + r < keys) {
                x = __ldg((const float4*)(kb + (k0 + r) * a.ld_k + c * 4));
                y = __ldg((const float4*)(vb + (k0 + r) * a.ld_v + c * 4));
            }
            *(float4*)(sk + r * LD + c * 4) = x;
            *(float4*)(sv + r * D + c * 4) = y;
        }
        __syncthreads();
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = *(const float4*)(sq + (ty * 4 + i) * LD + d);
                y[i] = *(const float4*)(sk + (tx + 16 * i) * LD + d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                    s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                    s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                    s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = w.row0 + ty * 4 + i;
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (k0 + tx + 16 * j > row) s[i][j] = -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float base = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m[i] - base);
            m[i] = top;
            l[i] *= f;
#pragma unroll
            for (int v = 0; v < OV; ++v) {
                o[i][v].x *= f; o[i][v].y *= f; o[i][v].z *= f; o[i][v].w *= f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                l[i] += p;
                sp[(ty * 4 + i) * (BN + 4) + tx + 16 * j] = p;
            }
        }
        __syncwarp();                           // a row's 16 threads are in one warp
#pragma unroll 2
        for (int k = 0; k < BN; k += 4) {
            float4 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = *(const float4*)(sp + (ty * 4 + i) * (BN + 4) + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int v = 0; v < OV; ++v) {
                    const float4 y = *(const float4*)(sv + (k + kk) * D + v * 64 + tx * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float pk = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                        o[i][v].x = fmaf(pk, y.x, o[i][v].x);
                        o[i][v].y = fmaf(pk, y.y, o[i][v].y);
                        o[i][v].z = fmaf(pk, y.z, o[i][v].z);
                        o[i][v].w = fmaf(pk, y.w, o[i][v].w);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        float sum = l[i];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (r >= rows) continue;
        const int64_t row = w.first + w.row0 + r;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        float* out = (float*)a.out + (row * a.n_heads + head) * D;
#pragma unroll
        for (int v = 0; v < OV; ++v)
            *(float4*)(out + v * 64 + tx * 4) =
                make_float4(o[i][v].x * inv, o[i][v].y * inv, o[i][v].z * inv, o[i][v].w * inv);
        if (tx == 0) a.lse[row * a.n_heads + head] = sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * LN2;
    }
}

template <int D>
cudaError_t launch(const Launch& L, const PromptArgs& a) {
    const int smem = (BM * (D + 4) + BN * (D + 4) + BN * D + BM * (BN + 4)) * 4;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = allow_smem(done, gqa_prompt_simt_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    // as many tiles as any split of `total` rows over the prompts can have
    cfg.gridDim = dim3((unsigned)a.n_heads * (unsigned)(a.total / BM + (a.n_seqs < a.total ? a.n_seqs : a.total)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gqa_prompt_simt_kernel<D>, a);
    count_launch();
    return e;
}

}  // namespace

cudaError_t launch_gqa_prompt_simt(const Launch& L, const PromptArgs& a, int head_dim) {
    return head_dim == 64 ? launch<64>(L, a) : launch<128>(L, a);
}

}  // namespace dsa
