// Grouped-query attention of single query rows over a paged key-value cache:
//   z_s    = scale * q[t,h,:] . k_s          s <= row_pos[t], kv head h / group
//   out    = sum_s softmax_s(z) v_s,   lse = log sum_s exp(z_s)
// Every visible key and value row is read once for all heads of its group (for
// each 16 of them, in larger groups), so the cache's bytes at the HBM rate are the floor.  32 sequences of up to
// 32K tokens, 8 / 32 heads of 128, bf16: 512 us, 6.4 TB/s (a plain copy runs at
// 6.5); 64 of them, 8 / 64 heads, fp8: 530 us, 6.3 TB/s in a short run, and 562,
// 6.0 TB/s, back to back, where the clock falls under the power limit.  One row of
// 777 tokens takes 7.3 us, a chain of latencies: rows, pages, cache, joining of the parts.
//
// Rows of one sequence that stand beside each other (several tokens verified
// at once) share its reads too: a bunch is up to `merge` such rows, whose heads
// fill the 16 columns of the products together; past a row's last key its
// columns are masked.  Against a pair for every row: 8 sequences of up to 16K
// tokens, 4 rows each, 8 / 32 heads: 258 -> 80 us in bf16, 124 -> 66 in fp8; 4
// of up to 5K in fp32 90 -> 50; 16 of up to 100 tokens 10.3 -> 11.4; one of 777
// tokens 9.3 -> 10.9 us.
//
// Work split.  A pair is (bunch of rows, kv head, tile of the group's heads); its keys
// are cut into units of KT (128, in fp32 64).  All pairs' units form
// one line, and block i of the grid takes the i-th equal stretch of it,
// whatever the rows' lengths: ragged batches load every SM alike, and one long row uses the whole GPU.
// Lengths are read on the device (nothing about them is known to the host),
// so a captured call serves growing sequences.  A stretch that holds a whole
// pair writes its output; a pair cut between blocks leaves fp32 partials
// (o, max, sum) in the workspace, which gqa_combine_kernel joins in order.
#include "common.cuh"
#include "launchers.h"
#include "sm100.cuh"

#include <cfloat>
#include <type_traits>

namespace dsa {

using namespace sm100;

namespace {

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr float LN2 = 0.6931471805599453f;
// fp8: what a weight at the reference becomes; the reference's range, in which
// WEIGHT_ONE / reference is a normal number.
constexpr float WEIGHT_ONE = 8192.f, VREF_LEAST = 1e-30f, VREF_MOST = 0x1p126f;

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
    int2* meta;                     // [row, kv head, tile]: first block; blocks (1: written whole), and
                                    // above bit 16 the row's place in its bunch
};

// Units of a row whose last visible token is pos: at least one, so that empty
// rows are written too.
template <int KT> __device__ __forceinline__ int units_of(const DecodeArgs& a, int pos) {
    return pos < 0 ? 1 : min(pos, a.room - 1) / KT + 1;
}
__device__ __forceinline__ int keys_of(const DecodeArgs& a, int pos, int seq) {
    return pos < 0 || seq < 0 || seq >= a.batch ? 0 : min(pos, a.room - 1) + 1;
}

// Rows' positions and sequences, and the bunches that begin with them, in
// shared memory when there are not too many.
constexpr int ROWS_HELD = 256;
struct RowsShared {
    int2 row[ROWS_HELD];
    int4 bunch[ROWS_HELD];
};
__device__ __forceinline__ int2 row_at(const DecodeArgs& a, const RowsShared& sh, int r) {
    if (a.rows <= ROWS_HELD) return sh.row[r];
    return make_int2(__ldg(a.row_pos + r), __ldg(a.row_batch + r));
}

// The bunch that begins with row r: rows of one sequence, all empty or none,
// as (rows, sequence, least and largest position); none (0 rows) where row r
// joins the one before it.
__device__ __forceinline__ int4 bunch_at(const DecodeArgs& a, const RowsShared& sh, int r) {
    const int in_seq = r - a.by_tokens.div(r) * a.tokens, k = in_seq - a.by_merge.div(in_seq) * a.merge;
    const int2 x = row_at(a, sh, r);
    if (k > 0) {
        const int2 y = row_at(a, sh, r - 1);
        if (x.y == y.y && (x.x < 0) == (y.x < 0)) return make_int4(0, 0, 0, 0);
    }
    const int most = min(min(a.merge - k, a.tokens - in_seq), a.rows - r);
    int4 b = make_int4(1, x.y, x.x, x.x);
    for (; b.x < most; ++b.x) {
        const int2 y = row_at(a, sh, r + b.x);
        if (y.y != x.y || (y.x < 0) != (x.x < 0)) break;
        b.z = min(b.z, y.x);
        b.w = max(b.w, y.x);
    }
    return b;
}

// A walk along the line of units.  MANY: pairs of more than one row.
template <int KT, bool MANY> struct Walk {
    int row, kvh, tile, unit, units;    // place: (first) row, kv head, tile of its heads, unit; the pair's units
    int batch, keys;                    // the sequence and number of visible keys (0: nothing to read)
    int rows, least;                    // MANY: the bunch's rows, the fewest visible keys of one

    __device__ __forceinline__ void set_row(const DecodeArgs& a, int pos, int seq) {
        units = units_of<KT>(a, pos);
        batch = seq;
        keys = keys_of(a, pos, seq);
    }
    __device__ __forceinline__ void set_bunch(const DecodeArgs& a, const RowsShared& sh) {
        const int4 b = a.rows <= ROWS_HELD ? sh.bunch[row] : bunch_at(a, sh, row);
        rows = b.x;
        batch = b.y;
        least = keys_of(a, b.z, batch);
        keys = keys_of(a, b.w, batch);
        units = units_of<KT>(a, b.w);
    }
    __device__ __forceinline__ void next(const DecodeArgs& a, const RowsShared& sh, int tiles) {
        if (++unit < units) return;
        unit = 0;
        if (++tile < tiles) return;
        tile = 0;
        if (++kvh < a.n_kv_heads) return;
        kvh = 0;
        row += MANY ? rows : 1;
        if (row >= a.rows) return;
        if (MANY) set_bunch(a, sh);
        else set_row(a, __ldg(a.row_pos + row), __ldg(a.row_batch + row));
    }
};

struct LocateShared {
    int warp_sum[WARPS];
    int row, units_before, pos, seq;    // of the stretch's first unit
};

// This block's stretch [begin, end) of the line and the walk's start.  The
// whole block takes part.  `per_block` units at least, so that short lines
// are not cut finer than is worth joining.
template <int KT, bool MANY>
__device__ __forceinline__ void locate(const DecodeArgs& a, int tiles, int per_block, LocateShared& sh,
                                       RowsShared& held, Walk<KT, MANY>& w,
                                       int64_t& begin, int64_t& end, int64_t& stretch) {
    const int hvs = a.n_kv_heads * tiles;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.rows + THREADS - 1) / THREADS;
    const int r0 = min(a.rows, tid * per), r1 = min(a.rows, r0 + per);
    int sum = 0, pos = -1, seq = -1;    // (of the thread's last row)
    if (MANY) {
        if (a.rows <= ROWS_HELD)
            for (int r = tid; r < a.rows; r += THREADS) held.row[r] = make_int2(__ldg(a.row_pos + r), __ldg(a.row_batch + r));
        __syncthreads();
    }
    // units of a pair that begins with row r (MANY: a row that joins another has none of its own)
    auto units_at = [&](int r) {
        if (MANY) {
            const int4 b = bunch_at(a, held, r);
            if (a.rows <= ROWS_HELD) held.bunch[r] = b;
            return b.x ? units_of<KT>(a, b.w) : 0;
        }
        pos = __ldg(a.row_pos + r);
        return units_of<KT>(a, pos);
    };
    for (int r = r0; r < r1; ++r) {
        sum += units_at(r);
        if (!MANY) seq = __ldg(a.row_batch + r);
    }
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
    // the thread whose rows hold the stretch's first unit finds its row
    if (begin < end && begin >= (int64_t)before * hvs && begin < (int64_t)(before + sum) * hvs) {
        int r = r0, u = before;
        if (per > 1) {
            for (; r < r1; ++r) {
                const int n = units_at(r);
                if (begin < (int64_t)(u + n) * hvs) break;
                u += n;
            }
            seq = __ldg(a.row_batch + r);
        }
        sh.row = r;
        sh.units_before = u;
        sh.pos = pos;
        sh.seq = seq;
    }
    __syncthreads();
    if (begin < end) {
        w.row = sh.row;
        if (MANY) w.set_bunch(a, held);
        else w.set_row(a, sh.pos, sh.seq);
        const int in_row = (int)(begin - (int64_t)sh.units_before * hvs);
        const int hv = in_row / w.units;
        w.unit = in_row - hv * w.units;
        w.kvh = hv / tiles;
        w.tile = hv - w.kvh * tiles;
    }
}

// Where key s of the walk's sequence lies: its page, and its row (of head_dim
// numbers) relative to that of the page; -1: not visible.  The page is looked
// at later (cache_row), so that its load is not waited for here.
struct Place {
    int page, row;
};
template <int KT, bool MANY> __device__ __forceinline__ Place look_up(const DecodeArgs& a, const Walk<KT, MANY>& w, int s) {
    if (s >= w.keys) return Place{0, -1};
    const int pi = a.by_page.div(s);
    return Place{__ldg(a.page_table + (int64_t)w.batch * a.max_pages + pi), w.kvh * a.page_size + (s - pi * a.page_size)};
}
// The row of the cache, or -1: not visible, or a bad page (reported).
__device__ __forceinline__ int cache_row(const DecodeArgs& a, Place p) {
    if (p.row < 0) return -1;
    if (p.page < 0 || p.page >= a.num_pages) {
        record_error(a.err, DEV_ERR_BAD_INDEX);
        return -1;
    }
    return p.page * a.n_kv_heads * a.page_size + p.row;
}

// ------------------------------------------------------------ the kernel --
//
// The work is bound by the cache's bytes, so the kernel is built around its
// loads: each warp owns 32 (fp32: 16) keys of a unit and streams their K and V
// rows through a ring of its own (cp.async, 16 bytes per lane, rows of unused
// places zero-filled), never waiting for another warp while a pair lasts.
//
// The products are formed transposed, with the cache as the M operand of
// mma.m16n8 and eight heads as N:
//   S^T [keys x heads] = K Q^T,     O^T [dims x heads] += V^T P^T
// so that a group of up to 8 heads fills the tensor instruction (with heads
// as M, half of it would be idle and twice the registers taken); P^T goes from
// the first product's result to the second's operand by 8 x 8 transposes in
// registers.  A slice costs a warp a few dozen products and one softmax step:
// a small part of an SM's issue slots at the HBM rate, which is why the
// products need no more than the warp-level instruction (M = 128 of tcgen05
// would serve 128 keys at a time and leave the softmax across lanes).
//
// Which dims a k-step of the first product holds is free as long as Q and K
// agree, and so is which dim a row of O^T holds and which key a k-step of the
// second product holds.  bf16 uses ldmatrix and the plain order; fp8 and fp32
// choose the orders so that a lane reads its keys as 16-byte pieces.
//
// fp8: codes are widened to f16 (exact) on the way into the product.  The
// query row is first brought to [1, 2) by a power of two, so that f16 holds
// it (a value below 2^-14 of the row's largest loses bits below 2^-25 of it).
// The second product's weights are p v_scale, as f16 too, relative to the
// largest of them that the warp has met for the head: a reference of its own
// beside the running maximum, since a large scale may belong to a key of next to
// no weight.  It stands at 2^13 of f16's 2^-24 .. 2^16, so that a weight down to
// 2^-27 of the largest keeps all 11 bits, and no weight is off by more than 2^-38
// of it.  Rows of zero codes do not count: their scale says nothing about the
// others' (the writer's is 1).
//
// fp32: every factor is split into two tf32 numbers, x = hi + lo (11 + 11
// bits), and a product is three tensor products hi hi + hi lo + lo hi, the
// small ones summed apart.  What is left out or rounded is at most 4.5 x 2^-22
// of |x y| a term.  The tensor core's sums round toward zero, so each slice's
// output is summed from zero and added to the running one in fp32.
// WK: keys of a warp's slice; BLOCKS per SM, with STAGES slices in flight per
// warp; Q_BYTES: the query fragments, where the registers have no room for them.
//
// Spills: 16 bytes a thread in fp8 with head dim 128 and 8 heads, 4 in fp32 with
// head dim 128 and 16 heads; none elsewhere.
//
// More blocks of one slice a warp hide each other's products and joining better
// than fewer blocks of several slices, as far as registers allow (us, fewer blocks
// or more slices -> as here; 8 kv heads, 4 heads each, or as said):
//   bf16, 128: 128 sequences of up to 500 54.6 -> 43.4, 32 of up to 32K 511.6 -> 510.3,
//              one of 32K 31.4 -> 32.6;  64: 128 of up to 500 28.7 -> 25.7
//   fp8, 128:  64 of up to 32K, 8 heads each, 579 -> 532;  64: two slices and four
//              blocks, 32 of up to 16K 80.7 -> 78.3, with one slice 82.2; 16 heads a
//              pair: two slices, 32 of up to 16K 222 -> 202 (128), and with three blocks,
//              whose registers spill, 332
//   fp32, 128: 16 of up to 8K 179 -> 144 (6.0 TB/s);  64: two slices 68.3, one 77.1, three 68.8
template <typename KV, int D, int GT> struct MmaCfg;
template <int D, int GT> struct MmaCfg<__nv_bfloat16, D, GT> {
    static constexpr int WK = 32, STAGES = 1, BLOCKS = D == 64 ? 3 : 2, Q_BYTES = 0;
};
template <int D, int GT> struct MmaCfg<__nv_fp8_e4m3, D, GT> {
    static constexpr int WK = 32, STAGES = D == 128 && GT == 8 ? 1 : 2, BLOCKS = (D == 64 ? 4 : 3) - (GT == 16 ? 1 : 0);
    static constexpr int Q_BYTES = GT == 16 ? D / 16 * 512 : 0;
};
template <int D, int GT> struct MmaCfg<float, D, GT> {
    static constexpr int WK = 16, STAGES = D == 64 ? 2 : 1, BLOCKS = 2, Q_BYTES = GT == 16 ? D / 8 * 1024 : 0;
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// C += A B on tf32: lane (r4, c4) gives A's rows r4 and r4 + 8 at k = c4 (a[0],
// a[1]) and c4 + 4 (a[2], a[3]), and B's column r4 at k = c4 and c4 + 4.
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit numbers: lane (r4, c4) gives row r4, columns 2 c4
// and 2 c4 + 1, and gets column r4, rows 2 c4 and 2 c4 + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <bool F16> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four e4m3 codes to f16: the low two, the high two.
__device__ __forceinline__ void e4m3x4_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(v));
}
__device__ __forceinline__ void cp_async_4(void* dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Shared-memory place of 16-byte piece c of key r, within a slice of rows of RB
// bytes (swizzled so that the kernel's reads meet no bank twice).
template <int ES, int RB, bool IS_V> __device__ __forceinline__ uint32_t piece_at(int r, int c) {
    if (ES == 2) return r * RB + ((c ^ (r & 7)) << 4);
    if (ES == 4) {
        const int f = (r >> 1) & 3;             // V: a read covers four even (or odd) keys and two runs of pieces
        const int x = !IS_V ? (r & 1) << 2 : RB == 512 ? f : (f & 1) | ((f & 2) << 1);
        return r * RB + ((c ^ x) << 4);
    }
    if (IS_V) {                     // lines of 128 bytes
        const int lin = r * (RB / 16) + c;
        return (lin >> 3) * 128 + (((lin & 7) ^ (((r >> 1) & 3) << 1)) << 4);
    }
    return r * RB + ((RB == 128 ? c ^ ((r & 1) << 2) : c) << 4);
}

// Whether a word of cache values holds one that is infinite or NaN.
template <int ES> __device__ __forceinline__ bool not_finite(uint32_t x) {
    if (ES == 4) return (x & 0x7f800000u) == 0x7f800000u;
    if (ES == 2) return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
    return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u;
}

// Place (in floats) of dim d of head r in the exchange buffer of the warps'
// outputs: 16-byte pieces swizzled among the eight of a 128-byte line.
template <int D> __device__ __forceinline__ int exch_at(int r, int d) {
    return r * D + (((d >> 2) ^ (((r >> 1) & 3) << 1)) << 2) + (d & 3);
}

template <typename KV, int D, int GT>
__global__ void __launch_bounds__(THREADS, (MmaCfg<KV, D, GT>::BLOCKS)) gqa_decode_kernel(const DecodeArgs a, const Parts parts) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int ES = (int)sizeof(KV);
    constexpr bool FP8 = ES == 1, FP32 = ES == 4;
    constexpr int WK = MmaCfg<KV, D, GT>::WK, KT = WK * WARPS;  // keys of a warp's slice, and of a unit
    constexpr int RB = D * ES;                      // bytes of a row
    constexpr int PIECES = RB / 16;
    constexpr int SLICE = WK * RB;                  // K (or V) bytes of a warp's slice
    constexpr int STAGES = MmaCfg<KV, D, GT>::STAGES;
    constexpr uint32_t ALL = WK == 32 ? 0xffffffffu : 0xffffu;
    constexpr int SLOT = 2 * SLICE + (FP8 ? 2 * WK * 4 : 0) + 16;   // K, V, scales, the mask of valid keys
    constexpr int KS = D / 16, MT = WK / 16, NG = GT / 8;   // k-steps; tiles of 16 keys, of 8 heads
    constexpr bool MANY = GT == 16;                 // pairs of several rows
    constexpr bool Q_SHARED = MANY && ES != 2;      // query fragments in shared memory, for want of registers
    static_assert(!FP8 || WK == 32, "a lane per key's scales");
    static_assert(2 * SLICE >= GT * D * 4, "the outputs of a pair's heads are exchanged in a slot");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LocateShared sh;
    __shared__ RowsShared held;             // (MANY only)
    __shared__ float2 s_ml[WARPS][16];
    const int group = a.n_heads / a.n_kv_heads, tiles = ceil_div(group, GT);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r4 = lane >> 2, c4 = lane & 3;        // fragment row / column group
    uint8_t* ring = smem + warp * STAGES * SLOT;
    uint8_t* qs = smem + WARPS * STAGES * SLOT;     // fp32 of 16 heads: the query fragments
    Walk<KT, MANY> w;
    int64_t begin, end, stretch;
    locate<KT, MANY>(a, tiles, 128 / KT, sh, held, w, begin, end, stretch);
    if (begin >= end) return;
    const uint8_t* kc = (const uint8_t*)a.k_cache;
    const uint8_t* vc = (const uint8_t*)a.v_cache;

    // the loads' walk runs STAGES units ahead of the products'; the page
    // of a slice is looked up one unit before its rows are requested
    Walk<KT, MANY> lw = w;
    int64_t to_load = end - begin;
    auto look = [&]() -> Place {            // of the walk's unit, and a step on
        if (to_load <= 0) return Place{0, -1};
        const Place p = look_up(a, lw, lw.unit * KT + warp * WK + (lane & (WK - 1)));
        --to_load;
        lw.next(a, held, tiles);
        return p;
    };
    int64_t to_request = end - begin;
    auto request = [&](int st, Place place) {
        if (to_request > 0) {
            const int row = cache_row(a, place);
            uint8_t* slot = ring + st * SLOT;
#pragma unroll
            for (int i = 0; i < WK * PIECES / 32; ++i) {
                const int r = (i * 32 + lane) / PIECES, c = (i * 32 + lane) % PIECES;
                const int from = __shfl_sync(0xffffffffu, row, r);
                const int64_t off = from >= 0 ? (int64_t)from * RB + c * 16 : 0;
                const uint32_t n = from >= 0 ? 16u : 0u;
                cp_async_16(slot + piece_at<ES, RB, false>(r, c), kc + off, n);
                cp_async_16(slot + SLICE + piece_at<ES, RB, true>(r, c), vc + off, n);
            }
            if (FP8) {
                cp_async_4(slot + 2 * SLICE + lane * 4, a.k_scale + (row >= 0 ? row : 0), row >= 0 ? 4u : 0u);
                cp_async_4(slot + 2 * SLICE + WK * 4 + lane * 4, a.v_scale + (row >= 0 ? row : 0), row >= 0 ? 4u : 0u);
            }
            const uint32_t valid = __ballot_sync(0xffffffffu, row >= 0) & ALL;
            if (lane == 0) *(uint32_t*)(slot + SLOT - 16) = valid;
            --to_request;
        }
        cp_async_commit();
    };
    Place ahead[STAGES];
#pragma unroll
    for (int st = 0; st < STAGES; ++st) ahead[st] = look();
    Place place = look();
#pragma unroll
    for (int st = 0; st < STAGES; ++st) request(st, ahead[st]);
    auto request_next = [&](int st) {
        request(st, place);
        place = look();
    };

    int st = 0;
    for (int64_t at = begin; at < end;) {
        // columns of the products: the tile's heads, or all heads of all rows of the bunch
        const bool bunch = MANY && w.rows > 1;
        const int h0 = w.kvh * group + w.tile * GT, heads = bunch ? w.rows * group : min(GT, group - w.tile * GT);
        const int n = (int)min((int64_t)(w.units - w.unit), end - at);
        if (w.unit == 0 && w.kvh == 0 && w.tile == 0 && tid < (MANY ? w.rows : 1) &&
            (w.batch < 0 || w.batch >= a.batch || __ldg(a.row_pos + w.row + tid) >= (int64_t)a.max_pages * a.page_size))
            record_error(a.err, DEV_ERR_BAD_INDEX);     // reported once per row, by the block that begins it
        // Q fragments: head 8 g + r4; k-step kk holds dims
        // 16 kk + {2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9} (bf16), or
        // 64 (kk / 4) + 16 c4 + 4 (kk % 4) + {0, 1, 2, 3} (fp8), or, as two
        // k-steps of 8, 16 kk + 4 c4 + {0, 1} and {2, 3} (fp32: hi, then lo)
        uint32_t qf[KS][FP32 ? 8 : 2 * NG];         // (Q_SHARED: in shared memory; fp32: place of k-step 2 kk + i)
        auto q_at = [&](int step, int g) { return qs + ((step * (FP32 ? NG : 1) + g) * 32 + lane) * 16; };
        float zs[NG][2];                            // score scale of heads 8 g + 2 c4 + {0, 1}
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const bool on = 8 * g + r4 < heads;
            const int x = on ? 8 * g + r4 : 0, xr = bunch ? a.by_group.div(x) : 0;
            const int64_t at_q = (int64_t)(w.row + xr) * a.ld_q + (h0 + x - xr * group) * D;
            const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + at_q;
            zs[g][0] = zs[g][1] = a.scale_log2;
            if constexpr (FP32) {
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    if (Q_SHARED && kk % WARPS != warp) continue;
                    const float4 v = on ? __ldg((const float4*)((const float*)a.q + at_q + 16 * kk + 4 * c4))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                    uint32_t y[8];
                    tf32_split(v.x, y[0], y[4]);
                    tf32_split(v.y, y[1], y[5]);
                    tf32_split(v.z, y[2], y[6]);
                    tf32_split(v.w, y[3], y[7]);
                    if (Q_SHARED) {
                        st_shared_v4(q_at(2 * kk, g), y[0], y[1], y[4], y[5]);
                        st_shared_v4(q_at(2 * kk + 1, g), y[2], y[3], y[6], y[7]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) qf[kk][i] = y[i];
                    }
                }
            } else if constexpr (!FP8) {
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    qf[kk][2 * g] = on ? __ldg((const uint32_t*)(q + 16 * kk + 2 * c4)) : 0u;
                    qf[kk][2 * g + 1] = on ? __ldg((const uint32_t*)(q + 16 * kk + 2 * c4 + 8)) : 0u;
                }
            } else {
                float top = 0.f;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    const uint2 x = on ? __ldg((const uint2*)(q + 64 * (kk / 4) + 16 * c4 + 4 * (kk % 4))) : make_uint2(0u, 0u);
                    qf[kk][2 * g] = x.x;
                    qf[kk][2 * g + 1] = x.y;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[kk][2 * g + e] << 16)),
                                               fabsf(__uint_as_float(qf[kk][2 * g + e] & 0xFFFF0000u))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^e <= top < 2^(e + 1), e kept where 2^-e is a normal number
                const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 253) - 127;
                const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                // of head r4; a normal number, so that a hidden key's score (-inf times it) stays -inf
                const float up = fminf(fmaxf(a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23), FLT_MIN), FLT_MAX);
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                    for (int i = 2 * g; i < 2 * g + 2; ++i)
                        qf[kk][i] = pack2<true>(__uint_as_float(qf[kk][i] << 16) * down,
                                                __uint_as_float(qf[kk][i] & 0xFFFF0000u) * down);
                zs[g][0] = __shfl_sync(0xffffffffu, up, 8 * c4);
                zs[g][1] = __shfl_sync(0xffffffffu, up, 8 * c4 + 4);
            }
        }
        if constexpr (FP8 && Q_SHARED) {
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
                if (kk % WARPS == warp) st_shared_v4(q_at(kk, 0), qf[kk][0], qf[kk][1], qf[kk][NG], qf[kk][NG + 1]);
        }
        if (Q_SHARED) __syncthreads();
        int sees[NG][2];                            // MANY: keys that heads 8 g + 2 c4 + {0, 1} see
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int x = 8 * g + 2 * c4 + e;
                sees[g][e] = !bunch      ? w.keys
                             : x < heads ? keys_of(a, row_at(a, held, w.row + a.by_group.div(x)).x, w.batch)
                                         : w.least;
            }
        // O^T: tile t, rows (dims) r4 and r4 + 8, columns (heads) 8 g + 2 c4 + {0, 1}
        float o[KS][NG][4];
#pragma unroll
        for (int t = 0; t < KS; ++t)
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][g][e] = 0.f;
        float m[NG][2], l[NG][2], vref[NG][2];      // (vref: fp8)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[g][e] = -INFINITY;
                l[g][e] = vref[g][e] = 0.f;
            }

        for (int u = 0; u < n; ++u) {
            cp_async_wait<STAGES - 1>();
            __syncwarp();
            const uint8_t* slot = ring + st * SLOT;
            const uint32_t kb = smem_u32(slot), vb = kb + SLICE;
            const uint32_t valid = *(const uint32_t*)(slot + SLOT - 16);
            // MANY: the slice's first key; whether some of its keys are hidden from some of the rows
            const int key0 = (w.unit + u) * KT + warp * WK;
            const bool partly = MANY && bunch && key0 + WK > w.least;
            if (valid) {
                // S^T: keys 16 t + r4 (+ 8), heads 8 g + 2 c4 + {0, 1}
                float s[MT][NG][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[t][g][e] = 0.f;
                if constexpr (FP32) {
                    float small[MT][NG][4], small2[MT][NG][4];      // the products with a lo part
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e) small[t][g][e] = small2[t][g][e] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 x = ld_shared_v4(slot + piece_at<ES, RB, false>(t * 16 + r4, 4 * kk + c4));
                            const uint4 y = ld_shared_v4(slot + piece_at<ES, RB, false>(t * 16 + r4 + 8, 4 * kk + c4));
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t hi[4], lo[4];
                                tf32_split(__uint_as_float(xs[2 * i]), hi[0], lo[0]);
                                tf32_split(__uint_as_float(ys[2 * i]), hi[1], lo[1]);
                                tf32_split(__uint_as_float(xs[2 * i + 1]), hi[2], lo[2]);
                                tf32_split(__uint_as_float(ys[2 * i + 1]), hi[3], lo[3]);
#pragma unroll
                                for (int g = 0; g < NG; ++g) {
                                    uint4 y = make_uint4(qf[kk][2 * i], qf[kk][2 * i + 1], qf[kk][2 * i + 4], qf[kk][2 * i + 5]);
                                    if (Q_SHARED) y = ld_shared_v4(q_at(2 * kk + i, g));
                                    mma1688(s[t][g], hi, y.x, y.y);
                                    mma1688(small[t][g], lo, y.x, y.y);
                                    mma1688(small2[t][g], hi, y.z, y.w);
                                }
                            }
                        }
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[t][g][e] += small[t][g][e] + small2[t][g][e];
                } else if constexpr (!FP8) {
#pragma unroll
                    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            uint32_t x[4];
                            ldmatrix_x4(x, kb + piece_at<ES, RB, false>(t * 16 + (lane & 15), kk * 2 + (lane >> 4)));
#pragma unroll
                            for (int g = 0; g < NG; ++g) mma16816<FP8>(s[t][g], x, qf[kk][2 * g], qf[kk][2 * g + 1]);
                        }
                } else if constexpr (Q_SHARED) {
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 x = ld_shared_v4(slot + piece_at<ES, RB, false>(t * 16 + r4, 4 * i + c4));
                            const uint4 y = ld_shared_v4(slot + piece_at<ES, RB, false>(t * 16 + r4 + 8, 4 * i + c4));
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t k16[4];
                                e4m3x4_f16(xs[j], k16[0], k16[2]);
                                e4m3x4_f16(ys[j], k16[1], k16[3]);
                                const uint4 q = ld_shared_v4(q_at(4 * i + j, 0));
                                mma16816<FP8>(s[t][0], k16, q.x, q.y);
                                mma16816<FP8>(s[t][NG - 1], k16, q.z, q.w);
                            }
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        uint32_t x[WK / 8][4];      // (keys 8 t + r4)
#pragma unroll
                        for (int t = 0; t < WK / 8; ++t) {
                            const uint4 y = ld_shared_v4(slot + piece_at<ES, RB, false>(t * 8 + r4, 4 * i + c4));
                            x[t][0] = y.x; x[t][1] = y.y; x[t][2] = y.z; x[t][3] = y.w;
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int t = 0; t < MT; ++t) {
                                uint32_t k16[4];
                                e4m3x4_f16(x[2 * t][j], k16[0], k16[2]);
                                e4m3x4_f16(x[2 * t + 1][j], k16[1], k16[3]);
#pragma unroll
                                for (int g = 0; g < NG; ++g)
                                    mma16816<FP8>(s[t][g], k16, qf[4 * i + j][2 * g], qf[4 * i + j][2 * g + 1]);
                            }
                    }
                }
                float vs[WK / 8];                   // value scales of keys 8 t + r4
                if (FP8) {
                    const float* ks = (const float*)(slot + 2 * SLICE);
#pragma unroll
                    for (int t = 0; t < WK / 8; ++t) {
                        const float k1 = ks[t * 8 + r4];
                        vs[t] = ks[WK + t * 8 + r4];
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            s[t / 2][g][2 * (t & 1)] *= k1;
                            s[t / 2][g][2 * (t & 1) + 1] *= k1;
                        }
                    }
                }
                if (valid != ALL) {
#pragma unroll
                    for (int t = 0; t < WK / 8; ++t)
                        if (!((valid >> (t * 8 + r4)) & 1u)) {
#pragma unroll
                            for (int g = 0; g < NG; ++g) s[t / 2][g][2 * (t & 1)] = s[t / 2][g][2 * (t & 1) + 1] = -INFINITY;
                        }
                }
                if (MANY && partly) {
#pragma unroll
                    for (int t = 0; t < WK / 8; ++t)
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (key0 + 8 * t + r4 >= sees[g][e]) s[t / 2][g][2 * (t & 1) + e] = -INFINITY;
                }
                // running maximum (scores times zs; zs > 0), and the output brought to it (fp8: below)
                float f[NG][2];
                bool moved = false;
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[0][g][e], s[0][g][2 + e]);
#pragma unroll
                        for (int t = 1; t < MT; ++t) top = fmaxf(top, fmaxf(s[t][g][e], s[t][g][2 + e]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) * zs[g][e];
                        f[g][e] = 1.f;
                        if (top > m[g][e]) {
                            f[g][e] = fast_exp2(m[g][e] - top);
                            m[g][e] = top;
                            l[g][e] *= f[g][e];
                            moved = true;
                        }
                    }
                if (!FP8 && __any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int t = 0; t < KS; ++t)
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[t][g][e] *= f[g][e & 1];
                }
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float base = m[g][e] > -INFINITY ? m[g][e] : 0.f;
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float p = fast_exp2(fmaf(s[t][g][2 * i + e], zs[g][e], -base));
                                l[g][e] += p;
                                s[t][g][2 * i + e] = FP8 ? p * vs[2 * t + i] : p;
                                if (FP8 && MANY && partly && key0 + 16 * t + 8 * i + r4 >= sees[g][e]) s[t][g][2 * i + e] = 0.f;
                            }
                    }
                if constexpr (FP8) {
                    // the weights p v_scale relative to vref, which follows the largest of them at a distance of 2;
                    // vref too is relative to the running maximum, so that the output need not move with it
                    auto largest = [&](int g, int e) {
                        float top = 0.f;
#pragma unroll
                        for (int t = 0; t < MT; ++t) top = fmaxf(top, fmaxf(fabsf(s[t][g][e]), fabsf(s[t][g][2 + e])));
                        return top;
                    };
                    bool grows = false;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            vref[g][e] *= f[g][e];
                            grows = grows || largest(g, e) > 2.f * vref[g][e] || vref[g][e] < VREF_LEAST;
                        }
                    if (__any_sync(0xffffffffu, grows)) {
                        // rows whose codes are all zero weigh nothing, whatever their scale: where one of a
                        // row's pieces is zero, the rows are looked at whole
                        constexpr int READS = WK * PIECES / 32, PER = 32 / PIECES;     // rows a read covers
                        auto codes = [&](int r, int c) {
                            const uint4 x = ld_shared_v4(slot + SLICE + piece_at<ES, RB, true>(r, c));
                            return (x.x | x.y | x.z | x.w) & 0x7f7f7f7fu;
                        };
                        if (__any_sync(0xffffffffu, codes(lane, lane % PIECES) == 0u && ((valid >> lane) & 1u))) {
                            uint32_t some[READS];
#pragma unroll
                            for (int i = 0; i < READS; ++i)
                                some[i] = __ballot_sync(0xffffffffu, codes(i * PER + lane / PIECES, lane % PIECES) != 0u);
#pragma unroll
                            for (int t = 0; t < WK / 8; ++t) {
                                const uint32_t rows8 = PER == 8 ? some[t % READS] : (r4 & 4) ? some[(2 * t + 1) % READS] : some[2 * t % READS];
                                if ((rows8 >> (r4 % PER * PIECES) & ((1u << PIECES) - 1u)) == 0u) {
#pragma unroll
                                    for (int g = 0; g < NG; ++g)
#pragma unroll
                                        for (int e = 0; e < 2; ++e) s[t / 2][g][2 * (t & 1) + e] *= 0.f;    // (NaN stays)
                                }
                            }
                        }
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            float move[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float top = largest(g, e);
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                                const float was = vref[g][e];
                                if (top > 2.f * was) vref[g][e] = top;
                                vref[g][e] = fminf(fmaxf(vref[g][e], VREF_LEAST), VREF_MOST);
                                move[e] = __fdividef(was, vref[g][e]);
                            }
#pragma unroll
                            for (int t = 0; t < KS; ++t)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[t][g][e] *= move[e & 1];
                        }
                    }
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float inv = __fdividef(WEIGHT_ONE, vref[g][e]);
#pragma unroll
                            for (int t = 0; t < MT; ++t)
#pragma unroll
                                for (int i = 0; i < 2; ++i) s[t][g][2 * i + e] *= inv;
                        }
                }
                // O^T += V^T P^T.  Zero times a value that a row may not see need not be zero: where some
                // such value is infinite or NaN, the product is formed once per row (ONE: the row of `sees`
                // = n_keys) with the values behind its keys set to zero, for its columns alone.
                auto product_o = [&](auto one, int n_keys) {
                    constexpr bool ONE = decltype(one)::value;
                    auto put = [&](float (&to)[4], const float (&from)[4], int g) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (sees[g][e & 1] == n_keys) to[e] = from[e];
                    };
                    auto shown = [&](int key) { return ONE && key0 + key >= n_keys ? 0u : 0xffffffffu; };
                    if constexpr (FP32) {
                        // k-step (t, i): keys 16 t + 8 i + 2 c4 (k = c4) and + 1 (k = c4 + 4); P^T's pieces by
                        // shuffles from the lanes of those keys.  Rows r4 / r4 + 8 of tile j are dims
                        // (D / 8) r4 + 2 j and + 1.
                        constexpr int RUN = D / 8;
                        uint32_t ph[2 * MT][NG][2], pl[2 * MT][NG][2];
#pragma unroll
                        for (int ti = 0; ti < 2 * MT; ++ti)
#pragma unroll
                            for (int g = 0; g < NG; ++g)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int from = (2 * c4 + e) * 4 + (r4 >> 1);
                                    const float even = __shfl_sync(0xffffffffu, s[ti / 2][g][2 * (ti & 1)], from);
                                    const float odd = __shfl_sync(0xffffffffu, s[ti / 2][g][2 * (ti & 1) + 1], from);
                                    tf32_split((r4 & 1) ? odd : even, ph[ti][g][e], pl[ti][g][e]);
                                }
#pragma unroll
                        for (int n4 = 0; n4 < RUN / 4; ++n4) {
                            float step[2][NG][4];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int g = 0; g < NG; ++g)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) step[k][g][e] = 0.f;
#pragma unroll
                            for (int ti = 0; ti < 2 * MT; ++ti) {
                                const int key = 8 * ti + 2 * c4;
                                const uint4 x = ld_shared_v4(slot + SLICE + piece_at<ES, RB, true>(key, r4 * RUN / 4 + n4));
                                const uint4 y = ld_shared_v4(slot + SLICE + piece_at<ES, RB, true>(key + 1, r4 * RUN / 4 + n4));
                                const uint32_t mx = shown(key), my = shown(key + 1);
                                const uint32_t xs[4] = {x.x & mx, x.y & mx, x.z & mx, x.w & mx};
                                const uint32_t ys[4] = {y.x & my, y.y & my, y.z & my, y.w & my};
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    uint32_t hi[4], lo[4];
                                    tf32_split(__uint_as_float(xs[2 * k]), hi[0], lo[0]);
                                    tf32_split(__uint_as_float(xs[2 * k + 1]), hi[1], lo[1]);
                                    tf32_split(__uint_as_float(ys[2 * k]), hi[2], lo[2]);
                                    tf32_split(__uint_as_float(ys[2 * k + 1]), hi[3], lo[3]);
#pragma unroll
                                    for (int g = 0; g < NG; ++g) {
                                        mma1688(step[k][g], lo, ph[ti][g][0], ph[ti][g][1]);
                                        mma1688(step[k][g], hi, pl[ti][g][0], pl[ti][g][1]);
                                        mma1688(step[k][g], hi, ph[ti][g][0], ph[ti][g][1]);
                                    }
                                }
                            }
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int g = 0; g < NG; ++g) {
                                    float (&to)[4] = o[2 * n4 + k][g];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) step[k][g][e] += to[e];
                                    if (ONE) put(to, step[k][g], g);
                                    else
#pragma unroll
                                        for (int e = 0; e < 4; ++e) to[e] = step[k][g][e];
                                }
                        }
                    } else {
                        // keys 16 t + 2 c4 + {0, 1} lie in x[0] and x[1], + {8, 9} in x[2] and x[3]
                        auto add = [&](int t, int j, int g, const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
                            if (ONE) {
                                float sum[4];
                                uint32_t y[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    sum[e] = o[j][g][e];
                                    const int key = 16 * t + 2 * c4 + 8 * (e >> 1);
                                    y[e] = x[e] & ((shown(key) & 0xffffu) | (shown(key + 1) & 0xffff0000u));
                                }
                                mma16816<FP8>(sum, y, b0, b1);
                                put(o[j][g], sum, g);
                            } else {
                                mma16816<FP8>(o[j][g], x, b0, b1);
                            }
                        };
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            uint32_t pf[NG][2];
#pragma unroll
                            for (int g = 0; g < NG; ++g)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    pf[g][i] = transpose8(pack2<FP8>(s[t][g][2 * i], s[t][g][2 * i + 1]));
                            if constexpr (!FP8) {
                                // rows r4 / r4 + 8 of tile j are dims 16 j + r4 and + 8
#pragma unroll
                                for (int j = 0; j < KS; ++j) {
                                    uint32_t x[4];
                                    ldmatrix_x4_t(x, vb + piece_at<ES, RB, true>(t * 16 + (lane >> 4) * 8 + (lane & 7),
                                                                                 2 * j + ((lane >> 3) & 1)));
#pragma unroll
                                    for (int g = 0; g < NG; ++g) add(t, j, g, x, pf[g][0], pf[g][1]);
                                }
                            } else {
                                // rows r4 / r4 + 8 of tile j are dims (D / 8) r4 + 2 j and + 1; keys 2 c4 + {0, 1, 8, 9}
                                constexpr int RUN = D / 8;
                                uint32_t x[4][RUN / 4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int key = t * 16 + 2 * c4 + (k & 1) + 8 * (k >> 1);
                                    const uint8_t* src = slot + SLICE + piece_at<ES, RB, true>(key, r4 * RUN / 16) + (r4 * RUN) % 16;
                                    if (RUN == 16) {
                                        const uint4 v = ld_shared_v4(src);
                                        x[k][0] = v.x; x[k][1] = v.y; x[k][RUN / 4 - 2] = v.z; x[k][RUN / 4 - 1] = v.w;
                                    } else {
                                        const uint2 v = *(const uint2*)src;
                                        x[k][0] = v.x; x[k][1] = v.y;
                                    }
                                }
#pragma unroll
                                for (int j = 0; j < RUN / 4; ++j) {
                                    // the pairs' codes side by side: dims 0, 1 and 2, 3 of keys 0, 1 and of 8, 9
                                    uint32_t v0[4], v1[4];
                                    e4m3x4_f16(__byte_perm(x[0][j], x[1][j], 0x5140), v0[0], v0[1]);
                                    e4m3x4_f16(__byte_perm(x[2][j], x[3][j], 0x5140), v0[2], v0[3]);
                                    e4m3x4_f16(__byte_perm(x[0][j], x[1][j], 0x7362), v1[0], v1[1]);
                                    e4m3x4_f16(__byte_perm(x[2][j], x[3][j], 0x7362), v1[2], v1[3]);
#pragma unroll
                                    for (int g = 0; g < NG; ++g) {
                                        add(t, 2 * j, g, v0, pf[g][0], pf[g][1]);
                                        add(t, 2 * j + 1, g, v1, pf[g][0], pf[g][1]);
                                    }
                                }
                            }
                        }
                    }
                };
                bool apart = false;
                if (MANY && partly) {
                    bool odd = false;
                    for (int r = max(w.least - key0, 0) + lane / PIECES; r < WK; r += max(32 / PIECES, 1))
                        for (int c = lane % PIECES; c < PIECES; c += 32) {
                            const uint4 x = ld_shared_v4(slot + SLICE + piece_at<ES, RB, true>(r, c));
                            odd = odd || not_finite<ES>(x.x) || not_finite<ES>(x.y) || not_finite<ES>(x.z) || not_finite<ES>(x.w);
                        }
                    apart = __any_sync(0xffffffffu, odd);
                }
                if constexpr (MANY) {
                    if (!apart) product_o(std::false_type{}, 0);
                    else                                    // from row to row of different numbers of keys
                        for (int i = 0; i < w.rows; ++i) {
                            const int n_keys = keys_of(a, row_at(a, held, w.row + i).x, w.batch);
                            bool again = false;
                            for (int k = 0; k < i; ++k)
                                again = again || keys_of(a, row_at(a, held, w.row + k).x, w.batch) == n_keys;
                            if (!again) product_o(std::true_type{}, n_keys);
                        }
                } else {
                    product_o(std::false_type{}, 0);
                }
            }
            __syncwarp();
            if (u + 1 < n) {
                request_next(st);
                st = st + 1 == STAGES ? 0 : st + 1;
            }
        }
        // the four warps' shares of the pair, joined through the slots whose
        // slices were just used (their next loads are requested afterwards)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], 4);
                l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], 8);
                l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], 16);
                if (r4 == 0) s_ml[warp][8 * g + 2 * c4 + e] = make_float2(m[g][e], l[g][e]);
            }
        const bool begins = w.unit == 0, ends = w.unit + n == w.units;
        const int place = 2 * blockIdx.x + (begins ? 1 : 0);
        float* mine = (float*)(ring + st * SLOT);
#pragma unroll
        for (int half = 0; half < NG; ++half)
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float carry = FP8 ? vref[half][e] * (1.f / WEIGHT_ONE) : 1.f;
                    if (ES == 2) {
                        mine[exch_at<D>(8 * half + 2 * c4 + e, 16 * t + r4)] = o[t][half][e];
                        mine[exch_at<D>(8 * half + 2 * c4 + e, 16 * t + r4 + 8)] = o[t][half][2 + e];
                    } else if ((t & 1) == 0) {
                        *(float4*)(mine + exch_at<D>(8 * half + 2 * c4 + e, (D / 8) * r4 + 2 * t)) =
                            make_float4(o[t][half][e] * carry, o[t][half][2 + e] * carry, o[t + 1][half][e] * carry,
                                        o[t + 1][half][2 + e] * carry);
                    }
                }
        __syncthreads();
        constexpr int VEC = D / 32;
        for (int h = warp; h < heads; h += WARPS) {
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) mm = fmaxf(mm, s_ml[i][h].x);
            float acc[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const float2 ml = s_ml[i][h];
                const float g = mm == -INFINITY ? 0.f : fast_exp2(ml.x - mm);
                ll += g * ml.y;
                const float* from = (const float*)(smem + (i * STAGES + st) * SLOT) + exch_at<D>(h, lane * VEC);
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[v] = fmaf(g, from[v], acc[v]);
            }
            if (begins && ends) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const int hr = bunch ? a.by_group.div(h) : 0;
                const int64_t to_head = (int64_t)(w.row + hr) * a.n_heads + h0 + h - hr * group;
                const int64_t to = to_head * D + lane * VEC;
#pragma unroll
                for (int v = 0; v < VEC; v += 2) {
                    if (FP32) *(float2*)((float*)a.out + to + v) = make_float2(acc[v] * inv, acc[v + 1] * inv);
                    else *(uint32_t*)((__nv_bfloat16*)a.out + to + v) = pack2<false>(acc[v] * inv, acc[v + 1] * inv);
                }
                if (lane == 0)
                    a.lse[to_head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * LN2;
            } else {
                float* po = parts.o + ((int64_t)place * GT + h) * D + lane * VEC;
#pragma unroll
                for (int v = 0; v < VEC; ++v) po[v] = acc[v];
                if (lane == 0) parts.ml[place * GT + h] = make_float2(mm, ll);
            }
        }
        __syncthreads();
        if (begins && tid < (MANY ? w.rows : 1)) {
            const int64_t last = (at + w.units - 1) / stretch;      // block of the pair's last unit
            parts.meta[((int64_t)(w.row + tid) * a.n_kv_heads + w.kvh) * tiles + w.tile] =
                make_int2(blockIdx.x, (int)(last - blockIdx.x) + 1 + (tid << 16));
        }
        request_next(st);
        st = st + 1 == STAGES ? 0 : st + 1;
        at += n;
        w.unit += n - 1;
        if (at < end) w.next(a, held, tiles);
    }
    cp_async_wait<0>();
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
    const int kvh = head / group, in = head - kvh * group, tile = in / GT;
    int h = in - tile * GT;
    int2 me = parts.meta[(int64_t)row * a.n_kv_heads * tiles + kvh * tiles + tile];
    if (GT == 16) h += (me.y >> 16) * group;                // the row's columns within its bunch
    me.y &= 0xffff;
    if (me.y <= 1) return;                                  // written whole
    // part 0 lies in the first block's "begins" place, the others in the
    // "continues" places of the blocks behind it; eight parts' numbers are
    // requested together and joined like the steps of an online softmax
    constexpr int BATCH = 8;
    float m = -INFINITY, l = 0.f, o[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = 0.f;
    for (int i0 = 0; i0 < me.y; i0 += BATCH) {
        float2 ml[BATCH];
        float po[BATCH][VEC];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = min(i0 + k, me.y - 1);
            const int64_t at = (int64_t)(2 * (me.x + i) + (i == 0)) * GT + h;
            ml[k] = parts.ml[at];
            if (VEC == 4) *(float4*)po[k] = *(const float4*)(parts.o + at * D + lane * VEC);
            else *(float2*)po[k] = *(const float2*)(parts.o + at * D + lane * VEC);
            if (i0 + k >= me.y) ml[k].x = -INFINITY;
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
        // a part without a visible key has zero sums; one whose scores are all
        // NaN has no maximum either, and NaN sums, which must not be passed over
        const float base = top > -INFINITY ? top : 0.f;
        const float f = fast_exp2(m - base);
        m = top;
        l *= f;
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] *= f;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const float g = fast_exp2(ml[k].x - base);
            l = fmaf(g, ml[k].y, l);
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[v] = fmaf(g, po[k][v], o[v]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    Q* out = (Q*)a.out + item * D + lane * VEC;
#pragma unroll
    for (int v = 0; v < VEC; ++v) store_out(out + v, o[v] * inv);
    if (lane == 0) a.lse[item] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Rows of one sequence that share a pair: as many as fill the products' 16
// columns, when the sequences have one and a half rows or more on average (16
// heads a pair cost up to 1.5 times the time of 8 per byte, over fp8) and come in
// runs of about `tokens`.
int tokens_of(int rows, int batch) { return 2ll * rows < 3ll * batch ? 1 : ceil_div(rows, batch); }
int merge_of(int group, int tokens) {
    const int most = 16 / group;
    return most < 2 || tokens < 2 ? 1 : ceil_div(tokens, ceil_div(tokens, most));
}
// Heads per pair: as many columns of the products as the pair fills (16, or 8
// when half of them would be idle).
int head_tile(int group, int merge) { return group > 8 || merge > 1 ? 16 : 8; }
template <int GT> int blocks_per_sm(dsa_dtype_t kv, int d) {
    return kv == DSA_FP32   ? (d == 64 ? MmaCfg<float, 64, GT>::BLOCKS : MmaCfg<float, 128, GT>::BLOCKS)
           : kv == DSA_BF16 ? (d == 64 ? MmaCfg<__nv_bfloat16, 64, GT>::BLOCKS : MmaCfg<__nv_bfloat16, 128, GT>::BLOCKS)
           : d == 64        ? MmaCfg<__nv_fp8_e4m3, 64, GT>::BLOCKS
                            : MmaCfg<__nv_fp8_e4m3, 128, GT>::BLOCKS;
}

template <typename Q, typename KV, int D, int GT>
cudaError_t launch_tile(const Launch& L, const DecodeArgs& a, void* workspace) {
    using C = MmaCfg<KV, D, GT>;
    constexpr bool FP8 = sizeof(KV) == 1;
    constexpr int slot = 2 * C::WK * D * (int)sizeof(KV) + (FP8 ? 2 * C::WK * 4 : 0) + 16;
    constexpr int smem = WARPS * C::STAGES * slot + C::Q_BYTES;
    const auto kern = gqa_decode_kernel<KV, D, GT>;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = allow_smem(done, kern, smem);
    if (e != cudaSuccess) return e;
    const int grid = L.num_sms * C::BLOCKS;
    Parts p;
    p.o = (float*)workspace;
    p.ml = (float2*)((char*)workspace + up256((size_t)2 * grid * GT * D * 4));
    p.meta = (int2*)((char*)p.ml + up256((size_t)2 * grid * GT * 8));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, p);
    count_launch();
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(((int64_t)a.rows * a.n_heads + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, gqa_combine_kernel<Q, D, GT>, a, p);
    count_launch();
    return e;
}

template <typename Q, typename KV, int D>
cudaError_t launch_typed(const Launch& L, const DecodeArgs& a, void* workspace) {
    return head_tile(a.n_heads / a.n_kv_heads, a.merge) == 16 ? launch_tile<Q, KV, D, 16>(L, a, workspace)
                                                              : launch_tile<Q, KV, D, 8>(L, a, workspace);
}

template <int GT> size_t workspace_of(int rows, int n_heads, int n_kv_heads, int head_dim, dsa_dtype_t kv, int num_sms) {
    const size_t grid = (size_t)num_sms * blocks_per_sm<GT>(kv, head_dim);
    const size_t pairs = (size_t)rows * n_kv_heads * ceil_div(n_heads / n_kv_heads, GT);
    return up256(2 * grid * GT * head_dim * 4) + up256(2 * grid * GT * 8) + pairs * 8;
}

}  // namespace

// (The number of sequences is not asked for: enough for either head tile,
// where rows might share pairs.)
size_t gqa_decode_workspace_bytes(int rows, int n_heads, int n_kv_heads, int head_dim, dsa_dtype_t kv, int num_sms) {
    const int group = n_heads / n_kv_heads;
    const size_t one = workspace_of<8>(rows, n_heads, n_kv_heads, head_dim, kv, num_sms);
    const size_t many = workspace_of<16>(rows, n_heads, n_kv_heads, head_dim, kv, num_sms);
    return group > 8 ? many : rows == 1 || one > many ? one : many;
}

cudaError_t launch_gqa_decode(const Launch& L, const DecodeArgs& args, dsa_dtype_t kv, int head_dim, void* workspace) {
    typedef __nv_bfloat16 bf16;
    DecodeArgs a = args;
    a.tokens = tokens_of(a.rows, a.batch);
    a.merge = merge_of(a.n_heads / a.n_kv_heads, a.tokens);
    a.by_tokens = fast_div(a.tokens);
    a.by_merge = fast_div(a.merge);
    a.by_group = fast_div(a.n_heads / a.n_kv_heads);
    const int64_t room = (int64_t)a.max_pages * a.page_size;
    a.room = room < 0x7fffffff ? (int)room : 0x7fffffff;
    if (kv == DSA_FP32)
        return head_dim == 64 ? launch_typed<float, float, 64>(L, a, workspace) : launch_typed<float, float, 128>(L, a, workspace);
    if (kv == DSA_BF16)
        return head_dim == 64 ? launch_typed<bf16, bf16, 64>(L, a, workspace) : launch_typed<bf16, bf16, 128>(L, a, workspace);
    return head_dim == 64 ? launch_typed<bf16, __nv_fp8_e4m3, 64>(L, a, workspace)
                          : launch_typed<bf16, __nv_fp8_e4m3, 128>(L, a, workspace);
}

}  // namespace dsa
