// Grouped-query attention of single query rows over a paged key-value cache:
//   z_s    = scale * q[t,h,:] . k_s          s <= row_pos[t], kv head h / group
//   out    = sum_s softmax_s(z) v_s,   lse = log sum_s exp(z_s)
// Every visible key and value row is read once for all heads of its group,
// so the cache's bytes at the HBM rate are the floor.
//
// Work split.  A pair is (row, kv head, tile of the group's heads); its keys
// are cut into units of 64.  All pairs' units form one line, and block i of
// the grid takes the i-th equal stretch of it, whatever the rows' lengths:
// ragged batches load every SM alike, and one long row uses the whole GPU.
// Lengths are read on the device (nothing about them is known to the host),
// so a captured call serves growing sequences.  A stretch that holds a whole
// pair writes its output; a pair cut between blocks leaves fp32 partials
// (o, max, sum) in the workspace, which gqa_combine_kernel joins in order.
#include "common.cuh"
#include "launchers.h"
#include "sm100.cuh"

namespace dsa {

using namespace sm100;

namespace {

constexpr int KT = 64;              // keys per unit
constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr int WK = KT / WARPS;      // keys of a unit that one warp takes
constexpr float LN2 = 0.6931471805599453f;

// 2^x on the MUFU unit: relative error ~2^-22, -inf -> +0.
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Partials of cut pairs.  Block b has two places: 2b for a pair that an
// earlier block began, 2b + 1 for one that it begins and does not end.
struct Parts {
    float* o;                       // [2 * grid][GT][D], relative to the maximum
    float2* ml;                     // [2 * grid][GT]: maximum (log2 units), sum
    int2* meta;                     // [pairs]: first block, number of blocks (1: written whole)
};

// Units of a row: at least one, so that empty rows are written too.
__device__ __forceinline__ int row_units(const DecodeArgs& a, int row) {
    const int pos = __ldg(a.row_pos + row);
    const int64_t room = (int64_t)a.max_pages * a.page_size;
    return pos < 0 ? 1 : pos < room ? pos / KT + 1 : (int)((room - 1) / KT) + 1;
}

// A walk along the line of units.
struct Walk {
    int row, hv, unit, units;       // place: row, pair of the row, unit of the pair; the row's units
    int batch, keys;                // the row's sequence and number of visible keys (0: nothing to read)

    __device__ __forceinline__ void enter_row(const DecodeArgs& a) {
        if (row >= a.rows) return;
        units = row_units(a, row);
        batch = __ldg(a.row_batch + row);
        const int64_t room = (int64_t)a.max_pages * a.page_size;
        const int pos = __ldg(a.row_pos + row);
        keys = pos < 0 || batch < 0 || batch >= a.batch ? 0 : (int)(pos < room ? pos + 1 : room);
    }
    __device__ __forceinline__ void next(const DecodeArgs& a, int hvs) {
        if (++unit < units) return;
        unit = 0;
        if (++hv < hvs) return;
        hv = 0;
        ++row;
        enter_row(a);
    }
};

struct LocateShared {
    int warp_sum[WARPS];
    int row, units_before;
    long long total;
};

// This block's stretch [begin, end) of the line and the walk's start.  The
// whole block takes part.  `per_block` units at least, so that short lines
// are not cut finer than is worth joining.
__device__ __forceinline__ void locate(const DecodeArgs& a, int hvs, int per_block, LocateShared& sh, Walk& w,
                                       int64_t& begin, int64_t& end, int64_t& stretch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.rows + THREADS - 1) / THREADS;
    const int r0 = min(a.rows, tid * per), r1 = min(a.rows, r0 + per);
    int sum = 0;
    for (int r = r0; r < r1; ++r) sum += row_units(a, r);
    int x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sh.warp_sum[warp] = x;
    __syncthreads();
    int before = x - sum, all = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < warp) before += sh.warp_sum[i];
        all += sh.warp_sum[i];
    }
    const int64_t line = (int64_t)all * hvs;
    stretch = (line + gridDim.x - 1) / gridDim.x;
    if (stretch < per_block) stretch = per_block;
    begin = min(line, (int64_t)blockIdx.x * stretch);
    end = min(line, begin + stretch);
    if (begin < end) {
        // the thread whose rows hold the stretch's first unit finds its row
        const int64_t lo = (int64_t)before * hvs, hi = (int64_t)(before + sum) * hvs;
        if (begin >= lo && begin < hi) {
            int r = r0, u = before;
            for (; r < r1; ++r) {
                const int n = row_units(a, r);
                if (begin < (int64_t)(u + n) * hvs) break;
                u += n;
            }
            sh.row = r;
            sh.units_before = u;
        }
    }
    __syncthreads();
    if (begin < end) {
        w.row = sh.row;
        w.enter_row(a);
        const int in_row = (int)(begin - (int64_t)sh.units_before * hvs);
        w.hv = in_row / w.units;
        w.unit = in_row - w.hv * w.units;
    }
}

// Row of the cache (in head_dim vectors) that holds key s of the walk's
// sequence, or -1: not visible, or a bad page (reported).
__device__ __forceinline__ int cache_row(const DecodeArgs& a, const Walk& w, int kvh, int s) {
    if (s >= w.keys) return -1;
    const int pi = s / a.page_size;
    const int page = __ldg(a.page_table + (int64_t)w.batch * a.max_pages + pi);
    if (page < 0 || page >= a.num_pages) {
        record_error(a.err, DEV_ERR_BAD_INDEX);
        return -1;
    }
    return (page * a.n_kv_heads + kvh) * a.page_size + (s - pi * a.page_size);
}

// ------------------------------------------------------------ CUDA cores --
//
// fp32 caches (and any type, in fp32 arithmetic).  A warp takes 4 keys at a
// time for 8 heads: every lane holds D/32 dims of the queries, keys and
// outputs, the 32 partial dot products per lane are summed over the lanes by
// one transposing butterfly (31 shuffles for 32 sums), after which lane l
// holds the score of key l / 8 and head l % 8.
template <typename T, int VEC> __device__ __forceinline__ void load_vec(const T* p, float (&x)[VEC]);
template <> __device__ __forceinline__ void load_vec<float, 4>(const float* p, float (&x)[4]) {
    const float4 v = __ldg((const float4*)p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <> __device__ __forceinline__ void load_vec<float, 2>(const float* p, float (&x)[2]) {
    const float2 v = __ldg((const float2*)p);
    x[0] = v.x; x[1] = v.y;
}
template <> __device__ __forceinline__ void load_vec<__nv_bfloat16, 4>(const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 v = __ldg((const uint2*)p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
template <> __device__ __forceinline__ void load_vec<__nv_bfloat16, 2>(const __nv_bfloat16* p, float (&x)[2]) {
    const uint32_t v = __ldg((const uint32_t*)p);
    x[0] = __uint_as_float(v << 16); x[1] = __uint_as_float(v & 0xFFFF0000u);
}
template <> __device__ __forceinline__ void load_vec<__nv_fp8_e4m3, 4>(const __nv_fp8_e4m3* p, float (&x)[4]) {
    const uint32_t v = __ldg((const uint32_t*)p);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        __nv_fp8_e4m3 c;
        c.__x = (__nv_fp8_storage_t)(v >> (8 * e));
        x[e] = (float)c;
    }
}
template <> __device__ __forceinline__ void load_vec<__nv_fp8_e4m3, 2>(const __nv_fp8_e4m3* p, float (&x)[2]) {
    const uint16_t v = __ldg((const uint16_t*)p);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        __nv_fp8_e4m3 c;
        c.__x = (__nv_fp8_storage_t)(v >> (8 * e));
        x[e] = (float)c;
    }
}

template <typename Q, typename KV, int D>
__global__ void __launch_bounds__(THREADS) gqa_decode_simt_kernel(const DecodeArgs a, const Parts parts) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int GT = 8, VEC = D / 32;
    constexpr bool SCALED = sizeof(KV) == 1;
    __shared__ LocateShared sh;
    __shared__ float s_o[WARPS][GT][D];
    __shared__ float s_m[WARPS][GT], s_l[WARPS][GT];
    const int group = a.n_heads / a.n_kv_heads, tiles = ceil_div(group, GT), hvs = a.n_kv_heads * tiles;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Walk w;
    int64_t begin, end, stretch;
    locate(a, hvs, 2, sh, w, begin, end, stretch);
    const KV* kc = (const KV*)a.k_cache;
    const KV* vc = (const KV*)a.v_cache;
    for (int64_t at = begin; at < end;) {
        const int kvh = w.hv / tiles, h0 = kvh * group + (w.hv - kvh * tiles) * GT;
        const int heads = min(GT, (kvh + 1) * group - h0);
        const int n = (int)min((int64_t)(w.units - w.unit), end - at);
        if (w.unit == 0 && w.hv == 0 && tid == 0) {
            // reported once per row, by the block that begins it
            const int b = w.batch;
            if (b < 0 || b >= a.batch || __ldg(a.row_pos + w.row) >= (int64_t)a.max_pages * a.page_size)
                record_error(a.err, DEV_ERR_BAD_INDEX);
        }
        float q[GT][VEC], acc[GT][VEC];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                q[h][v] = h < heads ? to_f32(((const Q*)a.q)[(int64_t)w.row * a.ld_q + (h0 + h) * D + lane * VEC + v]) *
                                          a.scale_log2
                                    : 0.f;
                acc[h][v] = 0.f;
            }
        }
        float m = -INFINITY, l = 0.f;       // of head lane % 8
        for (int u = w.unit; u < w.unit + n; ++u) {
            const int s0 = u * KT + warp * WK;
            const int my_row = lane < WK ? cache_row(a, w, kvh, s0 + lane) : -1;
#pragma unroll 1
            for (int k0 = 0; k0 < WK; k0 += 4) {
                float kx[4][VEC], vx[4][VEC];
                int row[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    row[k] = __shfl_sync(0xffffffffu, my_row, k0 + k);
                    if (row[k] >= 0) {
                        load_vec<KV, VEC>(kc + (int64_t)row[k] * D + lane * VEC, kx[k]);
                        load_vec<KV, VEC>(vc + (int64_t)row[k] * D + lane * VEC, vx[k]);
                    } else {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) kx[k][v] = vx[k][v] = 0.f;
                    }
                }
                if (row[0] < 0 && row[1] < 0 && row[2] < 0 && row[3] < 0) continue;
                const int mine = lane >> 3;
                const int mrow = mine == 0 ? row[0] : mine == 1 ? row[1] : mine == 2 ? row[2] : row[3];
                float ks = 1.f, vs = 1.f;
                if (SCALED && mrow >= 0) {
                    ks = __ldg(a.k_scale + mrow);
                    vs = __ldg(a.v_scale + mrow);
                }
                float s[32];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int h = 0; h < GT; ++h) {
                        float d = q[h][0] * kx[k][0];
#pragma unroll
                        for (int v = 1; v < VEC; ++v) d = fmaf(q[h][v], kx[k][v], d);
                        s[k * GT + h] = d;
                    }
#pragma unroll
                for (int half = 16; half > 0; half >>= 1) {
                    const bool up = lane & half;
#pragma unroll
                    for (int i = 0; i < half; ++i) {
                        const float give = up ? s[i] : s[i + half];
                        const float keep = up ? s[i + half] : s[i];
                        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
                    }
                }
                const float z = mrow >= 0 ? s[0] * ks : -INFINITY;
                float top = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float m_new = fmaxf(m, top);
                if (__any_sync(0xffffffffu, m_new > m)) {
                    const float f = m_new > m ? fast_exp2(m - m_new) : 1.f;
                    l *= f;
                    m = m_new;
#pragma unroll
                    for (int h = 0; h < GT; ++h) {
                        const float fh = __shfl_sync(0xffffffffu, f, h);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) acc[h][v] *= fh;
                    }
                }
                const float p = mrow >= 0 && m > -INFINITY ? fast_exp2(z - m) : 0.f;
                l += p;
                const float pv = SCALED ? p * vs : p;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int h = 0; h < GT; ++h) {
                        const float ph = __shfl_sync(0xffffffffu, pv, k * GT + h);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) acc[h][v] = fmaf(ph, vx[k][v], acc[h][v]);
                    }
            }
        }
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        // the four warps' shares of the pair
        if (lane < GT) {
            s_m[warp][lane] = m;
            s_l[warp][lane] = l;
        }
#pragma unroll
        for (int h = 0; h < GT; ++h)
#pragma unroll
            for (int v = 0; v < VEC; ++v) s_o[warp][h][lane * VEC + v] = acc[h][v];
        __syncthreads();
        const bool begins = w.unit == 0, ends = w.unit + n == w.units;
        const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
        for (int h = warp; h < heads; h += WARPS) {
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) mm = fmaxf(mm, s_m[i][h]);
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[v] = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const float f = mm == -INFINITY ? 0.f : fast_exp2(s_m[i][h] - mm);
                ll += f * s_l[i][h];
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[v] = fmaf(f, s_o[i][h][lane * VEC + v], o[v]);
            }
            if (begins && ends) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                Q* out = (Q*)a.out + ((int64_t)w.row * a.n_heads + h0 + h) * D + lane * VEC;
#pragma unroll
                for (int v = 0; v < VEC; ++v) store_out(out + v, o[v] * inv);
                if (lane == 0)
                    a.lse[(int64_t)w.row * a.n_heads + h0 + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * LN2;
            } else {
                float* po = parts.o + ((int64_t)slot * GT + h) * D + lane * VEC;
#pragma unroll
                for (int v = 0; v < VEC; ++v) po[v] = o[v];
                if (lane == 0) parts.ml[slot * GT + h] = make_float2(mm, ll);
            }
        }
        if (begins && tid == 0) {
            const int64_t last = (at + w.units - 1) / stretch;      // block of the pair's last unit
            parts.meta[(int64_t)w.row * hvs + w.hv] = make_int2(blockIdx.x, (int)(last - blockIdx.x) + 1);
        }
        __syncthreads();
        at += n;
        w.unit += n - 1;
        w.next(a, hvs);
    }
}

// ---------------------------------------------------------------- joining --

// One warp per (row, head) whose pair was cut: out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,
// over the parts in the order of their blocks.
template <typename Q, int D, int GT>
__global__ void __launch_bounds__(128) gqa_combine_kernel(const DecodeArgs a, const Parts parts) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int VEC = D / 32;
    const int64_t item = blockIdx.x * 4ll + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= (int64_t)a.rows * a.n_heads) return;
    const int row = (int)(item / a.n_heads), head = (int)(item - (int64_t)row * a.n_heads);
    const int group = a.n_heads / a.n_kv_heads, tiles = ceil_div(group, GT);
    const int kvh = head / group, in = head - kvh * group, tile = in / GT, h = in - tile * GT;
    const int2 me = parts.meta[(int64_t)row * a.n_kv_heads * tiles + kvh * tiles + tile];
    if (me.y <= 1) return;                                  // written whole
    // part 0 lies in the first block's "begins" place, the others in the
    // "continues" places of the blocks behind it
    float m = -INFINITY;
    for (int i = lane; i < me.y; i += 32) m = fmaxf(m, parts.ml[(int64_t)(2 * (me.x + i) + (i == 0)) * GT + h].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float l = 0.f, o[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = 0.f;
#pragma unroll 4
    for (int i = 0; i < me.y; ++i) {
        const int64_t at = (int64_t)(2 * (me.x + i) + (i == 0)) * GT + h;
        const float2 ml = parts.ml[at];
        const float f = m == -INFINITY ? 0.f : fast_exp2(ml.x - m);
        l = fmaf(f, ml.y, l);
        const float* po = parts.o + at * D + lane * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] = fmaf(f, po[v], o[v]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    Q* out = (Q*)a.out + item * D + lane * VEC;
#pragma unroll
    for (int v = 0; v < VEC; ++v) store_out(out + v, o[v] * inv);
    if (lane == 0) a.lse[item] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

constexpr int BLOCKS_PER_SM = 4;
constexpr int GT_SIMT = 8;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <typename Q, typename KV, int D>
cudaError_t launch_decode(const Launch& L, const DecodeArgs& a, void* workspace) {
    constexpr int GT = GT_SIMT;
    const int grid = L.num_sms * BLOCKS_PER_SM;
    Parts p;
    p.o = (float*)workspace;
    p.ml = (float2*)((char*)workspace + up256((size_t)2 * grid * GT * D * 4));
    p.meta = (int2*)((char*)p.ml + up256((size_t)2 * grid * GT * 8));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = L.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, gqa_decode_simt_kernel<Q, KV, D>, a, p);
    count_launch();
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(((int64_t)a.rows * a.n_heads + 3) / 4));
    e = cudaLaunchKernelEx(&cfg, gqa_combine_kernel<Q, D, GT>, a, p);
    count_launch();
    return e;
}

}  // namespace

size_t gqa_decode_workspace_bytes(int rows, int n_heads, int n_kv_heads, int head_dim, dsa_dtype_t kv, int num_sms) {
    const size_t grid = (size_t)num_sms * BLOCKS_PER_SM, gt = GT_SIMT;
    const size_t pairs = (size_t)rows * n_kv_heads * ceil_div(n_heads / n_kv_heads, (int)gt);
    return up256(2 * grid * gt * head_dim * 4) + up256(2 * grid * gt * 8) + pairs * 8;
}

cudaError_t launch_gqa_decode(const Launch& L, const DecodeArgs& a, dsa_dtype_t kv, int head_dim, void* workspace) {
    if (kv == DSA_FP32)
        return head_dim == 64 ? launch_decode<float, float, 64>(L, a, workspace)
                              : launch_decode<float, float, 128>(L, a, workspace);
    if (kv == DSA_BF16)
        return head_dim == 64 ? launch_decode<__nv_bfloat16, __nv_bfloat16, 64>(L, a, workspace)
                              : launch_decode<__nv_bfloat16, __nv_bfloat16, 128>(L, a, workspace);
    return head_dim == 64 ? launch_decode<__nv_bfloat16, __nv_fp8_e4m3, 64>(L, a, workspace)
                          : launch_decode<__nv_bfloat16, __nv_fp8_e4m3, 128>(L, a, workspace);
}

}  // namespace dsa
