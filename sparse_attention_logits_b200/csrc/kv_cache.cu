// The paged key-value cache of grouped-query attention: writing new tokens'
// rows (kv_cache_append) and keeping the pool of pages (kv_pages_extend,
// kv_pages_free, kv_pages_fork, kv_pages_copy, kv_pages_compact).
//
// All of it runs on the device without a host read, so that a serving loop
// that admits, branches and drops sequences can be captured in CUDA graphs.
// Every decision is deterministic: pages are handed out lowest id first, in
// the order of the caller's list.
#include "common.cuh"
#include "launchers.h"
#include "sm100.cuh"

namespace dsa {

using namespace sm100;

namespace {

// Two floats to two e4m3 codes (lo in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}

// ---------------------------------------------------------------- append --
//
// A group of D/16 lanes moves one (row, head) vector of K or V, sixteen
// elements per lane.  fp8: the group's amax by shuffles, scale = amax / 448 (1
// for an all-zero row), code = nearest even of value / scale, every operation
// in binary32 rounded on its own (the indexer key cache's rule).
//
// Bandwidth bound, but behind a chain of dependent loads (position and
// sequence, page, then the stores).  A block takes a run of rows: one thread
// per row walks the chain, while all groups already load the data of their
// first vectors, which does not depend on it.  64 rows of 8 heads of 128, bf16:
// 2 us on the GPU; the 20,996 rows of a batch of prompts into an fp8 cache: 29 us,
// 4.5 TB/s of reads and writes, into a bf16 one 36 us, 5.2 TB/s, fp32 86 us, 4.7.
constexpr int APPEND_ROWS = 32, APPEND_UNROLL = 2;

// Codes of sixteen values over their scale.  All share the divisor, so its
// reciprocal r is rounded once and each quotient is corrected twice with the
// exact remainder, q <- q + r (x - q sc): by P. Markstein's theorem
// ("Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) the second correction of a quotient within one unit gives
// the correctly rounded one.  Five multiply-adds two values against about twelve
// instructions of a division, which made the kernel issue-bound (52 us where
// the loads and stores take 20).  Bits matter here: bf16 rows hold values that
// fall exactly between two codes, about one in a hundred.  Below 2^-60 the
// remainders might not be exact: scales that small divide.
__device__ __forceinline__ uint4 e4m3_codes(const float (&x)[16], float sc) {
    float q[16];
    if (sc >= 0x1p-60f) {
        const float r = __frcp_rn(sc);
        const float2 r2 = make_float2(r, r), m2 = make_float2(-sc, -sc), zero = make_float2(-0.f, -0.f);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {                   // (two values an instruction, each rounded as one)
            const float2 v = make_float2(x[e], x[e + 1]);
            float2 y = fma2(v, r2, zero);
            y = fma2(r2, fma2(y, m2, v), y);
            y = fma2(r2, fma2(y, m2, v), y);
            q[e] = y.x;
            q[e + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) q[e] = __fdiv_rn(x[e], sc);
    }
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = e4m3x2(q[4 * e], q[4 * e + 1]) | (e4m3x2(q[4 * e + 2], q[4 * e + 3]) << 16);
    return make_uint4(c[0], c[1], c[2], c[3]);
}

template <int D, bool F32_IN, int FMT>     // FMT: DSA_FP32, DSA_BF16, DSA_FP8_E4M3
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int LANES = D / 16, GROUPS = 256 / LANES, U = APPEND_UNROLL, W = F32_IN ? 4 : 2;
    __shared__ int2 place[APPEND_ROWS];         // page (-1: not stored) and place in it
    const int sub = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const unsigned group = (LANES == 8 ? 0xffu : 0xfu) << (threadIdx.x & 31 & ~(LANES - 1));
    const int rpb = min(APPEND_ROWS, (a.n + gridDim.x - 1) / (int)gridDim.x);
    for (int r0 = blockIdx.x * rpb; r0 < a.n; r0 += gridDim.x * rpb) {
        const int rows = min(rpb, a.n - r0), tasks = rows * 2 * a.n_kv_heads;
        int pos = -1, seq = -1;
        if (threadIdx.x < rows) {
            pos = __ldg(a.row_pos + r0 + threadIdx.x);
            seq = __ldg(a.row_batch + r0 + threadIdx.x);
        }
        for (int t0 = grp; t0 - grp < tasks; t0 += U * GROUPS) {        // (every group passes the barrier below)
            // head innermost, then K / V, then row
            uint4 x[U][W];
            int rs[U], head[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * GROUPS;
                if (t >= tasks) continue;
                rs[u] = a.by_head.div(t);
                head[u] = t - rs[u] * a.n_kv_heads;
                const int64_t src = (int64_t)(r0 + (rs[u] >> 1)) * ((rs[u] & 1) ? a.ld_v : a.ld_k) + head[u] * D + sub * 16;
                const uint4* s = (const uint4*)((const char*)((rs[u] & 1) ? a.v : a.k) + src * (F32_IN ? 4 : 2));
#pragma unroll
                for (int i = 0; i < W; ++i) x[u][i] = __ldcs(s + i);
            }
            if (t0 == grp) {
                if (threadIdx.x < rows) {
                    int page = -1, slot = 0;
                    if (pos >= 0) {                                     // (< 0: not stored)
                        const int pi = a.by_page.div(pos);
                        if (seq >= 0 && seq < a.batch && pi < a.max_pages)
                            page = __ldg(a.page_table + (int64_t)seq * a.max_pages + pi);
                        slot = pos - pi * a.page_size;
                        if (page < 0 || page >= a.num_pages) {
                            record_error(a.err, DEV_ERR_BAD_INDEX);
                            page = -1;
                        }
                    }
                    place[threadIdx.x] = make_int2(page, slot);
                }
                __syncthreads();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t0 + u * GROUPS >= tasks) continue;
                const bool is_v = rs[u] & 1;
                const int2 at = place[rs[u] >> 1];
                if (at.x < 0) continue;
                const int64_t dst_row = ((int64_t)at.x * a.n_kv_heads + head[u]) * a.page_size + at.y;
                constexpr int ES = FMT == DSA_FP32 ? 4 : FMT == DSA_BF16 ? 2 : 1;
                uint4* dst = (uint4*)((char*)(is_v ? a.v_cache : a.k_cache) + (dst_row * D + sub * 16) * ES);
                if constexpr (FMT == DSA_FP32 || (FMT == DSA_BF16 && !F32_IN)) {
#pragma unroll
                    for (int i = 0; i < W; ++i) dst[i] = x[u][i];
                } else {
                    float f[16];
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (F32_IN) {
                                f[(4 * i + e) & 15] = __uint_as_float(w[e]);
                            } else {
                                f[(8 * i + 2 * e) & 15] = __uint_as_float(w[e] << 16);
                                f[(8 * i + 2 * e + 1) & 15] = __uint_as_float(w[e] & 0xFFFF0000u);
                            }
                        }
                    }
                    if (FMT == DSA_BF16) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            dst[i] = make_uint4(bf16x2_bits(f[8 * i], f[8 * i + 1]), bf16x2_bits(f[8 * i + 2], f[8 * i + 3]),
                                                bf16x2_bits(f[8 * i + 4], f[8 * i + 5]), bf16x2_bits(f[8 * i + 6], f[8 * i + 7]));
                    } else {
                        float amax = 0.f;
                        if (F32_IN) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(f[e]));
                        } else {                            // (bf16 numbers: their maximum is one of them)
                            __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
                            for (int i = 0; i < W; ++i) {
                                const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t a2 = w[e] & 0x7fff7fffu;
                                    top = __hmax2(top, *(const __nv_bfloat162*)&a2);
                                }
                            }
                            amax = fmaxf(__low2float(top), __high2float(top));
                        }
#pragma unroll
                        for (int m = LANES / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, m));
                        const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
                        *dst = e4m3_codes(f, sc);
                        if (sub == 0) (is_v ? a.v_scale : a.k_scale)[dst_row] = sc;
                    }
                }
            }
        }
        __syncthreads();            // the places are read before the next run's are written
    }
}

// ----------------------------------------------------------- page copies --

// Bytes moved by one step of a block: 256 threads x 4 x 16 B, all four loads
// of a thread in flight together.  Bound by the copy rate: compacting 898 MB in
// three caches takes 150 us, 6.0 TB/s read and written.
constexpr int COPY_CHUNK = 16384;

struct CopyList {                   // kernel parameter: up to kMaxCopyCaches caches
    char* base[kMaxCopyCaches];
    uint32_t vecs[kMaxCopyCaches];  // 16-byte vectors per page
    uint32_t chunk0[kMaxCopyCaches + 1];   // first chunk of each cache within one page pair
    int n_caches, num_pages;
};

__device__ __forceinline__ void copy_chunk(const CopyList& c, int64_t src, int64_t dst, uint32_t chunk) {
    int lo = 0, hi = c.n_caches;                            // the cache that owns this chunk
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (chunk >= c.chunk0[mid]) lo = mid;
        else hi = mid;
    }
    const uint32_t vecs = c.vecs[lo];
    const uint32_t v0 = (chunk - c.chunk0[lo]) * (COPY_CHUNK / 16) + threadIdx.x;
    const uint4* s = (const uint4*)c.base[lo] + src * vecs;
    uint4* d = (uint4*)c.base[lo] + dst * vecs;
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (v0 + u * 256 < vecs) x[u] = __ldcs(s + v0 + u * 256);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (v0 + u * 256 < vecs) __stcs(d + v0 + u * 256, x[u]);
}

// Pairs (src[i], dst[i]) of the caller (n of them), or the pairs an earlier
// kernel of the same call left in the workspace (n_dev: how many).
__global__ void __launch_bounds__(256) kv_copy_kernel(const __grid_constant__ CopyList c, const int32_t* __restrict__ src,
                                                      const int32_t* __restrict__ dst, int n, unsigned* err,
                                                      const int* n_dev) {
    pdl_wait();
    pdl_launch_dependents();
    if (n_dev) n = *n_dev;
    const uint32_t per = c.chunk0[c.n_caches];
    const int64_t total = (int64_t)n * per;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int i = (int)(u / per);
        const uint32_t chunk = (uint32_t)(u - (int64_t)i * per);
        const int s = __ldg(src + i), d = __ldg(dst + i);
        if (s == -1 || d == -1 || s == d) continue;
        if (s < 0 || s >= c.num_pages || d < 0 || d >= c.num_pages) {
            if (threadIdx.x == 0) record_error(err, DEV_ERR_BAD_INDEX);
            continue;
        }
        copy_chunk(c, s, d, chunk);
    }
}

// ------------------------------------------------------------------ books --

// Pages of a sequence of `len` tokens.
__device__ __forceinline__ int pages_of(int len, int page_size) { return len > 0 ? (len - 1) / page_size + 1 : 0; }

// Bits of word w that are pages below `limit`.
__device__ __forceinline__ uint32_t below(int limit, int w) {
    const int64_t left = (int64_t)limit - (int64_t)w * 32;
    return left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
}

// Whether entry i of a list is the first that names its sequence (all
// threads of the block take part).
__device__ __forceinline__ bool first_of_its_kind(const int32_t* list, int i) {
    const int me = list[i];
    bool seen = false;
    for (int j = threadIdx.x; j < i; j += blockDim.x) seen |= list[j] == me;
    return !__syncthreads_or(seen);
}

// One block per listed sequence: its pages' reference counts go down by one,
// its table entries to -1, its length to 0.  Latency bound: giving back 64
// sequences' pages and handing out 64 new ones' (16K pages of a pool of 102K)
// takes 17 us, both calls together.
__global__ void __launch_bounds__(256) kv_free_kernel(const BooksArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x;
    const int q = a.seqs[i];
    if (q == -1) return;
    if (q < 0 || q >= a.batch) {
        if (threadIdx.x == 0) record_error(a.err, DEV_ERR_BAD_INDEX);
        return;
    }
    if (!first_of_its_kind(a.seqs, i)) return;      // listed before: that block frees it
    const int len = a.seq_len[q];
    int pages = pages_of(len, a.page_size);
    if (len < 0 || pages > a.max_pages) {
        if (threadIdx.x == 0) record_error(a.err, DEV_ERR_BAD_INDEX);
        pages = len < 0 ? 0 : a.max_pages;
    }
    __syncthreads();                                // everyone has read the length
    int32_t* row = a.page_table + (int64_t)q * a.max_pages;
    for (int j = threadIdx.x; j < pages; j += blockDim.x) {
        const int p = row[j];
        row[j] = -1;
        if (p < 0 || p >= a.num_pages) {
            record_error(a.err, DEV_ERR_BAD_INDEX);
        } else if (atomicSub(a.ref_count + p, 1) <= 0) {    // was free already: put back, and said
            atomicAdd(a.ref_count + p, 1);
            record_error(a.err, DEV_ERR_BAD_INDEX);
        }
    }
    if (threadIdx.x == 0) a.seq_len[q] = 0;
}

// The pool's books are kept by one cluster of 8 blocks: each holds an eighth of
// the pool as one bit per page in shared memory, so that the pool's counts are
// read once, by 8 SMs, and ranks of free pages need one exchange through
// distributed shared memory.
constexpr int BOOK_CTAS = 8;
constexpr int BOOK_THREADS = 1024;
constexpr int BOOK_WARPS = BOOK_THREADS / 32;

struct BookShared {
    int warp_sum[2][BOOK_WARPS];
    int mine[3];                    // this block's counts, read by the others
};

// Exclusive prefix sum of v over the block's threads; *total = the sum.
// warp_sum is still being read when it returns.
__device__ __forceinline__ int block_scan(int v, int* warp_sum, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    const int base = warp ? warp_sum[warp - 1] : 0;
    *total = warp_sum[BOOK_WARPS - 1];
    return base + x - v;
}

__device__ __forceinline__ int ld_cluster_s32(const int* p, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
    return v;
}

// Bits of this block's words of the pool: bit set = reference count <= 0 (free).
// Word `local` holds the 32 pages from 32 place(local) on; pages past the pool
// read as used.
template <class F>
__device__ __forceinline__ void load_free_bits(const int32_t* ref_count, int num_pages, int words, uint32_t* bits, F&& place) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int w0 = warp * 8; w0 < words; w0 += BOOK_WARPS * 8) {
        int v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t p = (int64_t)place(w0 + u) * 32 + lane;
            v[u] = w0 + u < words && p < num_pages ? ref_count[p] : 1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t m = __ballot_sync(0xffffffffu, v[u] <= 0);
            if (lane == 0 && w0 + u < words) bits[w0 + u] = m;
        }
    }
}

// Exclusive prefix counts of a quantity over the words of this block's slice
// (count(w) of word w) into before[w]; the slice's total is returned.
template <class F>
__device__ __forceinline__ int word_ranks(int words, int* before, int* warp_sum, F&& count) {
    const int per = (words + BOOK_THREADS - 1) / BOOK_THREADS;
    const int w0 = min(words, (int)threadIdx.x * per), w1 = min(words, w0 + per);
    int mine = 0, total;
    for (int w = w0; w < w1; ++w) mine += count(w);
    int run = block_scan(mine, warp_sum, &total);
    for (int w = w0; w < w1; ++w) {
        before[w] = run;
        run += count(w);
    }
    return total;
}

// kv_pages_extend (FORK = false) and kv_pages_fork (FORK = true).  Items are
// the list's entries; each needs some fresh pages (extend: as many as its new
// length asks for; fork: one for a last page that is not full).  An item is
// served when the needs up to and with it fit the free pages; its r-th page
// is the free page of rank (needs before it) + r, found by the block that
// holds the page.  Nothing is written before every block has read its inputs.
//
// The pool is dealt to the blocks in runs of 128 pages, since the pages handed
// out are the lowest and would otherwise all fall to the first blocks (102K
// pages, 16K of them handed out: 10 of 15 us, in three of eight blocks).
constexpr int RUN_WORDS = 4;

template <bool FORK>
__global__ void __cluster_dims__(BOOK_CTAS, 1, 1) __launch_bounds__(BOOK_THREADS)
kv_assign_kernel(const BooksArgs a, int words_per_cta) {
    pdl_wait();
    pdl_launch_dependents();
    extern __shared__ uint32_t dyn[];
    __shared__ BookShared sh;
    const int runs = words_per_cta / RUN_WORDS;         // of this block
    uint32_t* bits = dyn;                               // [words_per_cta]
    int* run_free = (int*)(dyn + words_per_cta);        // [runs] free pages of each run, read by the others
    int* before = run_free + runs;                      // [runs] free pages of the pool before each run
    int* start = before + runs;                         // [n + 1] needs before each item
    int* len = start + a.n + 1;                         // [n] extend: new length; fork: the parent's; -1: not served
    int* what = len + a.n;                              // [n] sequence (fork: child)
    int* entry = what + a.n;                            // [n] table entry of the item's page of rank 0
    int* bad_row = entry + a.n;                         // [n] fork: whether a page of the parent is out of range, said by
                                                        // block i % 8 for item i and read by the others
    const int rank = (int)cluster_ctarank(), tid = threadIdx.x;
    auto place = [&](int w) { return (w / RUN_WORDS * BOOK_CTAS + rank) * RUN_WORDS + w % RUN_WORDS; };
    const int32_t* list = FORK ? a.children : a.seqs;
    for (int i = tid; i < a.n; i += BOOK_THREADS) what[i] = list[i];
    load_free_bits(a.ref_count, a.num_pages, words_per_cta, bits, place);
    __syncthreads();
    for (int r = tid; r < runs; r += BOOK_THREADS) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < RUN_WORDS; ++w) n += __popc(bits[r * RUN_WORDS + w]);
        run_free[r] = n;
    }

    // items: validity and needs, the same in every block
    const int per = (a.n + BOOK_THREADS - 1) / BOOK_THREADS;
    const int i0 = min(a.n, tid * per), i1 = min(a.n, i0 + per);
    const int64_t room = (int64_t)a.max_pages * a.page_size;
    int need_sum = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
        const int q = what[i];
        int need = 0, l = -1;
        if (q >= 0 && q < a.batch) {
            bool ok = true;
            for (int j = 0; j < i; ++j) ok &= what[j] != q;     // listed twice: the first counts
            const int own = a.seq_len[q];
            if (FORK) {
                const int par = a.parents[i];
                const int pl = par >= 0 && par < a.batch ? a.seq_len[par] : -1;
                if (ok && own == 0 && pl >= 0 && pl <= room) {
                    l = pl;
                    need = pl % a.page_size != 0;
                }
            } else {
                const int add = a.add[i];
                const int64_t to = (int64_t)own + add;
                if (ok && own >= 0 && add >= 0 && to <= room && to <= 0x7fffffff) {
                    l = (int)to;
                    need = pages_of(l, a.page_size) - pages_of(own, a.page_size);
                }
            }
            bad |= l < 0;
        } else if (q != -1) {
            bad = true;
        }
        len[i] = l;
        start[i] = need;
        need_sum += need;
    }
    const int lane = tid & 31;
    if (FORK) {
        // a branch shares all of its parent's pages or none: the parents' rows, dealt to the cluster's warps
        __syncthreads();
        for (int i = rank + BOOK_CTAS * (tid >> 5); i < a.n; i += BOOK_CTAS * BOOK_WARPS) {
            const int pages = pages_of(len[i], a.page_size);
            const int32_t* row = a.page_table + (pages > 0 ? (int64_t)a.parents[i] * a.max_pages : 0);
            bool out = false;
            for (int j = lane; j < pages; j += 32) out |= row[j] < 0 || row[j] >= a.num_pages;
            out = __any_sync(0xffffffffu, out);
            if (lane == 0) bad_row[i] = out;
        }
        __syncwarp();
        cluster_sync_all();
        for (int i = i0; i < i1; ++i)
            if (ld_cluster_s32(bad_row + i, i % BOOK_CTAS)) {
                bad = true;
                len[i] = -1;
                need_sum -= start[i];
                start[i] = 0;
            }
    }
    if (bad && rank == 0) record_error(a.err, DEV_ERR_BAD_INDEX);
    int total_need;
    int run = block_scan(need_sum, sh.warp_sum[0], &total_need);
    for (int i = i0; i < i1; ++i) {
        const int need = start[i];
        start[i] = run;
        run += need;
        // the item's pages end where its new length ends
        entry[i] = what[i] * a.max_pages + pages_of(len[i], a.page_size) - run;
    }
    if (tid == 0) start[a.n] = total_need;
    cluster_sync_all();             // every block has read lengths and counts, and its runs' numbers stand

    // free pages of the pool before each run of this block, and in all
    const int all_runs = runs * BOOK_CTAS, rper = (all_runs + BOOK_THREADS - 1) / BOOK_THREADS;
    const int r0 = min(all_runs, tid * rper), r1 = min(all_runs, r0 + rper);
    int mine = 0, n_free;
    for (int r = r0; r < r1; ++r) mine += ld_cluster_s32(run_free + r / BOOK_CTAS, r % BOOK_CTAS);
    int sum = block_scan(mine, sh.warp_sum[1], &n_free);
    for (int r = r0; r < r1; ++r) {
        if (r % BOOK_CTAS == rank) before[r / BOOK_CTAS] = sum;
        sum += ld_cluster_s32(run_free + r / BOOK_CTAS, r % BOOK_CTAS);
    }
    __syncthreads();

    // the free pages to the items that they fall to: a page per lane; a warp's
    // words follow one another, so that a lane's item is mostly its last one's
    const int wper = (words_per_cta + BOOK_WARPS - 1) / BOOK_WARPS;
    const int w0 = min(words_per_cta, (tid >> 5) * wper), w1 = min(words_per_cta, w0 + wper);
    int lo = 0;
    for (int w = w0; w < w1; ++w) {
        const uint32_t m = bits[w];
        int page_rank = before[w / RUN_WORDS] + __popc(m & ((1u << lane) - 1u));
        for (int v = w / RUN_WORDS * RUN_WORDS; v < w; ++v) page_rank += __popc(bits[v]);
        if (m == 0 || page_rank >= total_need) continue;    // (lanes without a free page keep their place, too)
        const int page = place(w) * 32 + lane;
        // the last item with start <= rank: one that needs pages
        if (start[lo + 1] <= page_rank) {
            int hi = a.n;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= page_rank) lo = mid;
                else hi = mid;
            }
        }
        if (((m >> lane) & 1u) && start[lo + 1] <= n_free) {
            a.page_table[entry[lo] + page_rank] = page;
            a.ref_count[page] = 1;
            if (FORK) a.pair_dst[lo] = page;
        }
    }
    // the lengths, the shared pages (fork) and reports: one warp per item
    for (int i = rank + BOOK_CTAS * (tid >> 5); i < a.n; i += BOOK_CTAS * BOOK_WARPS) {
        const int need = start[i + 1] - start[i];
        const bool fits = need == 0 || start[i + 1] <= n_free;
        const bool served = len[i] >= 0 && fits;
        if (lane == 0) {
            if (len[i] >= 0 && !fits) record_error(a.err, DEV_ERR_NO_PAGES);
            if (served) a.seq_len[what[i]] = len[i];
        }
        if (FORK) {
            // a parent that holds pages is no child of this call (children
            // are empty), so its row is not being written
            const int full = served ? len[i] / a.page_size : 0;
            const int32_t* from = a.page_table + (served ? (int64_t)a.parents[i] * a.max_pages : 0);
            int32_t* to = a.page_table + (served ? (int64_t)what[i] * a.max_pages : 0);
            for (int j = lane; j < full; j += 32) {         // (all in range)
                const int p = from[j];
                to[j] = p;
                atomicAdd(a.ref_count + p, 1);
            }
            if (lane == 0) {
                a.pair_src[i] = served && need ? from[full] : -1;
                if (!(served && need)) a.pair_dst[i] = -1;
            }
        }
    }
    cluster_sync_relaxed();         // no block leaves while another may still read its number
}

// kv_pages_compact, the plan.  With n_live pages in use, the ones at or above
// n_live move to the free places below it, both in ascending order: the
// fewest moves, no page is source and destination, and what lies in the
// places to be filled is not read.  Left in the workspace: the pairs, the
// moved pages' counts, and for every page its new place (`to`: >= 0 the page
// itself or, encoded as -2 - r, the r-th pair; -1 for a free page).
__global__ void __cluster_dims__(BOOK_CTAS, 1, 1) __launch_bounds__(BOOK_THREADS)
kv_compact_plan_kernel(const CompactArgs a, int words_per_cta) {
    pdl_wait();
    pdl_launch_dependents();
    extern __shared__ uint32_t dyn[];
    __shared__ BookShared sh;
    uint32_t* bits = dyn;                               // [words_per_cta]
    int* up = (int*)(dyn + words_per_cta);              // [words_per_cta] of the slice before each word: pages that move
    int* hole = up + words_per_cta;                     // [words_per_cta] and places to fill
    const int rank = (int)cluster_ctarank(), tid = threadIdx.x;
    const int first_word = rank * words_per_cta;
    load_free_bits(a.ref_count, a.num_pages, words_per_cta, bits, [&](int w) { return first_word + w; });
    __syncthreads();
    const int wper = (words_per_cta + BOOK_THREADS - 1) / BOOK_THREADS;
    const int w0 = min(words_per_cta, tid * wper), w1 = min(words_per_cta, w0 + wper);
    int live = 0;
    for (int w = w0; w < w1; ++w) live += __popc(~bits[w] & below(a.num_pages, first_word + w));
    int slice_live;
    block_scan(live, sh.warp_sum[0], &slice_live);
    if (tid == 0) sh.mine[0] = slice_live;
    cluster_sync_all();
    int n_live = 0;
    for (int r = 0; r < BOOK_CTAS; ++r) n_live += ld_cluster_s32(&sh.mine[0], r);

    auto movers = [&](int w) { return ~bits[w] & below(a.num_pages, first_word + w) & ~below(n_live, first_word + w); };
    auto holes = [&](int w) { return bits[w] & below(n_live, first_word + w); };
    const int slice_up = word_ranks(words_per_cta, up, sh.warp_sum[1], [&](int w) { return __popc(movers(w)); });
    __syncthreads();                // warp_sum[0] is free again
    const int slice_hole = word_ranks(words_per_cta, hole, sh.warp_sum[0], [&](int w) { return __popc(holes(w)); });
    if (tid == 0) {
        sh.mine[1] = slice_up;
        sh.mine[2] = slice_hole;
    }
    cluster_sync_all();
    int moves = 0, up0 = 0, hole0 = 0;
    for (int r = 0; r < BOOK_CTAS; ++r) {
        const int u = ld_cluster_s32(&sh.mine[1], r), h = ld_cluster_s32(&sh.mine[2], r);
        if (r < rank) {
            up0 += u;
            hole0 += h;
        }
        moves += u;
    }
    if (rank == 0 && tid == 0) {
        a.state[0] = moves;
        a.state[1] = n_live;
    }
    // one warp per word, a page per lane
    const int lane = tid & 31;
    for (int w = tid >> 5; w < words_per_cta; w += BOOK_WARPS) {
        const int page = (first_word + w) * 32 + lane;
        if (page >= a.num_pages) continue;
        const uint32_t u = movers(w), h = holes(w), under = (1u << lane) - 1u;
        int to = (bits[w] >> lane) & 1u ? -1 : page;
        if ((u >> lane) & 1u) {
            const int k = up0 + up[w] + __popc(u & under);
            a.pair_src[k] = page;
            a.moved_ref[k] = a.ref_count[page];
            to = -2 - k;
        } else if ((h >> lane) & 1u) {
            a.pair_dst[hole0 + hole[w] + __popc(h & under)] = page;
        }
        a.to[page] = to;
    }
    cluster_sync_relaxed();
}

// kv_pages_compact, the moves: table entries and counts rewritten, then the
// pages copied in every cache.
__global__ void __launch_bounds__(256) kv_compact_kernel(const __grid_constant__ CopyList c, const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int moves = a.state[0], n_live = a.state[1];
    const int64_t entries = (int64_t)a.batch * a.max_pages;
    const int64_t me = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t e = me; e < entries; e += step) {
        const int p = a.page_table[e];
        int q = p;
        if (p >= 0 && p < a.num_pages) {
            const int to = a.to[p];
            q = to >= 0 ? to : to <= -2 ? a.pair_dst[-2 - to] : p;
            if (to == -1) record_error(a.err, DEV_ERR_BAD_INDEX);       // an entry of a page that counts as free
        } else if (p != -1) {
            record_error(a.err, DEV_ERR_BAD_INDEX);
        }
        a.table_out[e] = q;
    }
    // counts: the pages below n_live keep theirs or take a moved page's, the
    // rest are free.  ref_out may be ref_count itself: nothing at or above
    // n_live is read here, and places to be filled are written by their pair.
    for (int64_t p = me; p < a.num_pages; p += step) {
        if (p >= n_live) a.ref_out[p] = 0;
        else if (a.to[p] != -1) a.ref_out[p] = a.ref_count[p];
    }
    for (int64_t k = me; k < moves; k += step) a.ref_out[a.pair_dst[k]] = a.moved_ref[k];
    const uint32_t per = c.chunk0[c.n_caches];
    const int64_t total = (int64_t)moves * per;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int i = (int)(u / per);
        copy_chunk(c, a.pair_src[i], a.pair_dst[i], (uint32_t)(u - (int64_t)i * per));
    }
}

constexpr int words_per_book_cta(int num_pages) { return ceil_div(ceil_div(num_pages, 32), BOOK_CTAS); }
// kv_assign_kernel: whole runs of pages per block
constexpr int words_per_assign_cta(int num_pages) {
    return ceil_div(words_per_book_cta(num_pages), RUN_WORDS) * RUN_WORDS;
}
constexpr int books_smem(int num_pages, int n) {
    return (words_per_assign_cta(num_pages) / RUN_WORDS * (RUN_WORDS + 2) + 5 * n + 1) * 4;
}
constexpr int BOOK_SMEM_MAX = books_smem(DSA_KV_PAGES_MAX_POOL, DSA_KV_PAGES_MAX_LIST);
constexpr int PLAN_SMEM_MAX = 3 * 4 * words_per_book_cta(DSA_KV_PAGES_MAX_POOL);
static_assert(BOOK_SMEM_MAX <= 200 * 1024 && PLAN_SMEM_MAX <= 200 * 1024, "the books' bits and lists fit in shared memory");

// Caches [c0, c0 + n) of the caller's list as a kernel parameter.
CopyList copy_list(const CacheList& l, int c0, int n) {
    CopyList c = {};
    uint32_t chunk = 0;
    for (int i = 0; i < n; ++i) {
        c.base[i] = (char*)l.caches[c0 + i];
        c.vecs[i] = (uint32_t)(l.page_bytes[c0 + i] / 16);
        c.chunk0[i] = chunk;
        chunk += (uint32_t)((l.page_bytes[c0 + i] + COPY_CHUNK - 1) / COPY_CHUNK);
    }
    c.chunk0[n] = chunk;
    c.n_caches = n;
    c.num_pages = l.num_pages;
    return c;
}

template <class... P, class... A>
cudaError_t launch(void (*kern)(P...), int grid, int block, size_t smem, const Launch& L, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    count_launch();
    return e;
}

cudaError_t launch_copies(const Launch& L, const CacheList& l, const int32_t* src, const int32_t* dst, int n) {
    for (int c0 = 0; c0 < l.n_caches; c0 += kMaxCopyCaches) {
        const CopyList c = copy_list(l, c0, l.n_caches - c0 < kMaxCopyCaches ? l.n_caches - c0 : kMaxCopyCaches);
        const int64_t total = (int64_t)n * c.chunk0[c.n_caches];
        const int grid = (int)(total < (int64_t)L.num_sms * 8 ? total : (int64_t)L.num_sms * 8);
        const cudaError_t e = launch(kv_copy_kernel, grid, 256, 0, L, c, src, dst, n, L.err, (const int*)nullptr);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_append(const Launch& L, const AppendArgs& a, dsa_dtype_t in, dsa_dtype_t fmt, int head_dim) {
    // four blocks per SM (two rounds of them for long lists), one row each while that lasts
    const int grid = a.n < L.num_sms * 8 ? a.n : L.num_sms * 8;
    const bool f32 = in == DSA_FP32;
    void (*k)(AppendArgs);
#define DSA_APPEND(D)                                                                              \
    k = fmt == DSA_FP32   ? kv_append_kernel<D, true, DSA_FP32>                                    \
        : fmt == DSA_BF16 ? (f32 ? kv_append_kernel<D, true, DSA_BF16> : kv_append_kernel<D, false, DSA_BF16>) \
                          : (f32 ? kv_append_kernel<D, true, DSA_FP8_E4M3> : kv_append_kernel<D, false, DSA_FP8_E4M3>)
    if (head_dim == 64) DSA_APPEND(64);
    else DSA_APPEND(128);
#undef DSA_APPEND
    return launch(k, grid, 256, 0, L, a);
}

cudaError_t launch_kv_copy(const Launch& L, const CacheList& l, const int32_t* src, const int32_t* dst, int n) {
    return launch_copies(L, l, src, dst, n);
}

cudaError_t launch_kv_free(const Launch& L, const BooksArgs& a) { return launch(kv_free_kernel, a.n, 256, 0, L, a); }

cudaError_t launch_kv_extend(const Launch& L, const BooksArgs& a) {
    const size_t smem = books_smem(a.num_pages, a.n);
    static std::atomic<int> done[kMaxDevices];
    const cudaError_t e = allow_smem(done, kv_assign_kernel<false>, BOOK_SMEM_MAX);
    if (e != cudaSuccess) return e;
    return launch(kv_assign_kernel<false>, BOOK_CTAS, BOOK_THREADS, smem, L, a, words_per_assign_cta(a.num_pages));
}

size_t kv_fork_workspace_bytes(int n) { return (size_t)n * 8; }

cudaError_t launch_kv_fork(const Launch& L, BooksArgs a, const CacheList& l, void* workspace) {
    a.pair_src = (int32_t*)workspace;
    a.pair_dst = a.pair_src + a.n;
    const size_t smem = books_smem(a.num_pages, a.n);
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = allow_smem(done, kv_assign_kernel<true>, BOOK_SMEM_MAX);
    if (e != cudaSuccess) return e;
    e = launch(kv_assign_kernel<true>, BOOK_CTAS, BOOK_THREADS, smem, L, a, words_per_assign_cta(a.num_pages));
    if (e != cudaSuccess) return e;
    return launch_copies(L, l, a.pair_src, a.pair_dst, a.n);
}

size_t kv_compact_workspace_bytes(int num_pages) { return (4 * (size_t)num_pages + 4) * 4; }

cudaError_t launch_kv_compact(const Launch& L, CompactArgs a, const CacheList& l, void* workspace) {
    a.state = (int*)workspace;
    a.to = a.state + 4;
    a.pair_src = a.to + a.num_pages;
    a.pair_dst = a.pair_src + a.num_pages;
    a.moved_ref = a.pair_dst + a.num_pages;
    const int words = words_per_book_cta(a.num_pages);
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = allow_smem(done, kv_compact_plan_kernel, PLAN_SMEM_MAX);
    if (e != cudaSuccess) return e;
    e = launch(kv_compact_plan_kernel, BOOK_CTAS, BOOK_THREADS, (size_t)words * 12, L, a, words);
    if (e != cudaSuccess) return e;
    const CopyList c = copy_list(l, 0, l.n_caches < kMaxCopyCaches ? l.n_caches : kMaxCopyCaches);
    e = launch(kv_compact_kernel, L.num_sms * 8, 256, 0, L, c, a);
    if (e != cudaSuccess) return e;
    for (int c0 = kMaxCopyCaches; c0 < l.n_caches; c0 += kMaxCopyCaches) {
        const CopyList more = copy_list(l, c0, l.n_caches - c0 < kMaxCopyCaches ? l.n_caches - c0 : kMaxCopyCaches);
        e = launch(kv_copy_kernel, L.num_sms * 8, 256, 0, L, more, (const int32_t*)a.pair_src, (const int32_t*)a.pair_dst, 0, L.err,
                   (const int*)a.state);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace dsa
