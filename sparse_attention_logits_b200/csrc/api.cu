// extern "C" entry points of libdsa_b200.so: argument validation, kernel
// selection and the device error word.  Declarations and contracts are in
// include/dsa_b200.h.
#include <stdio.h>
#include <stdarg.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "launchers.h"

namespace {

thread_local char g_last_error[256] = "";
thread_local uint64_t g_launches = 0;

dsa_status_t fail(dsa_status_t st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return st;
}

dsa_status_t cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return DSA_OK;
    return fail(DSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// One error word per device; its device address is looked up once per device.
__device__ unsigned g_device_error;

constexpr int kMaxDevices = dsa::kMaxDevices;
// Filled once per device under dsa::init_mutex(): the SM count is stored
// first and the error-word address is then published with release order, so
// a thread that sees the address (acquire) also sees the SM count.
std::atomic<unsigned*> g_err_ptr[kMaxDevices] = {};
int g_num_sms[kMaxDevices] = {};

dsa_status_t make_launch(void* stream, dsa::Launch* L) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(DSA_ERR_UNSUPPORTED, "device ordinal %d too large", dev);
    unsigned* err = g_err_ptr[dev].load(std::memory_order_acquire);
    if (!err) {
        std::lock_guard<std::mutex> lock(dsa::init_mutex());
        err = g_err_ptr[dev].load(std::memory_order_relaxed);
        if (!err) {
            void* p = nullptr;
            e = cudaGetSymbolAddress(&p, g_device_error);
            if (e != cudaSuccess) return cuda_status(e, "cudaGetSymbolAddress(device error word)");
            int sms = 0;
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (e != cudaSuccess) return cuda_status(e, "cudaDeviceGetAttribute");
            g_num_sms[dev] = sms;
            err = (unsigned*)p;
            g_err_ptr[dev].store(err, std::memory_order_release);
        }
    }
    L->stream = (cudaStream_t)stream;
    L->err = err;
    L->num_sms = g_num_sms[dev];
    return DSA_OK;
}

// Fixed scratch of dsa_sparse_mla_noalloc: the bf16 partial outputs and fp32
// log-sum-exps of a key list split over several clusters.  A (row, split)
// pair takes 128 heads x (512 x 2 + 4) = 131,584 bytes, and the split count is
// chosen so that rows x splits <= SMs / 2, so 20 MiB covers every size on a
// GPU of up to 318 SMs.  No byte of it has to start at zero: each cluster
// writes its whole partial block before the merge kernel, launched after it
// on the same stream, reads it.  One copy per device: calls that overlap on
// one device (two streams, two threads) race on it.
constexpr size_t kMlaScratchBytes = DSA_MLA_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char g_mla_scratch[kMlaScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of g_mla_scratch on the current device, looked up once per
// device (cudaGetSymbolAddress may load the module, so the first call must
// not happen inside a stream capture).
dsa_status_t mla_scratch(void** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(DSA_ERR_UNSUPPORTED, "device ordinal %d too large", dev);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_mla_scratch);
        if (e != cudaSuccess) return cuda_status(e, "cudaGetSymbolAddress(sparse MLA scratch)");
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return DSA_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t dtype_size(dsa_dtype_t t) { return t == DSA_FP32 ? 4 : t == DSA_BF16 ? 2 : 1; }
bool valid_dtype(dsa_dtype_t t) { return t == DSA_FP32 || t == DSA_BF16 || t == DSA_FP8_E4M3; }
bool valid_key_dtype(dsa_dtype_t t) { return valid_dtype(t) || t == DSA_FP4_E2M1; }

}  // namespace

namespace dsa {
void count_launch(int n) { g_launches += (uint64_t)n; }
std::mutex& init_mutex() {
    static std::mutex mu;
    return mu;
}
}  // namespace dsa

extern "C" {

int dsa_version(void) { return 100; }

uint64_t dsa_launch_count(void) { return g_launches; }

const char* dsa_last_error(void) { return g_last_error; }

dsa_status_t csa_compress(const void* src, dsa_dtype_t dtype, int batch, int len, int dim, int m, void* dst,
                          void* stream) {
    if (!src || !dst) return fail(DSA_ERR_INVALID_ARG, "csa_compress: null pointer");
    if (batch < 0 || len < 0 || dim <= 0 || m < 1 || m > 1024)
        return fail(DSA_ERR_INVALID_ARG, "csa_compress: bad sizes (batch=%d len=%d dim=%d m=%d)", batch, len, dim, m);
    if (len % m) return fail(DSA_ERR_INVALID_ARG, "csa_compress: len=%d not a multiple of m=%d", len, m);
    if (dtype != DSA_BF16 && dtype != DSA_FP32) return fail(DSA_ERR_UNSUPPORTED, "csa_compress: dtype must be bf16 or fp32");
    if ((dim * dtype_size(dtype)) % 16) return fail(DSA_ERR_UNSUPPORTED, "csa_compress: dim*elem_size must be a multiple of 16 bytes");
    if (!aligned(src, 16) || !aligned(dst, 16)) return fail(DSA_ERR_INVALID_ARG, "csa_compress: pointers must be 16-byte aligned");
    const size_t bytes_in = (size_t)batch * len * dim * dtype_size(dtype);
    const size_t bytes_out = bytes_in / m;
    const char* s = (const char*)src; const char* d = (const char*)dst;
    if (bytes_in && s < d + bytes_out && d < s + bytes_in) return fail(DSA_ERR_INVALID_ARG, "csa_compress: src and dst overlap");
    dsa::Launch L;
    dsa_status_t st = make_launch(stream, &L);
    if (st != DSA_OK) return st;
    return cuda_status(dsa::launch_csa_compress(L, src, dtype, batch, len, dim, m, dst), "csa_compress launch");
}

dsa_status_t dsa_indexer_logits(const void* q, dsa_dtype_t q_dtype, const float* w, const void* k,
                                dsa_dtype_t k_dtype, const float* k_scale, const int32_t* row_batch,
                                const int32_t* row_pos, int rows, int batch, int ctx_len, int n_heads,
                                int head_dim, float* logits, int64_t ld_logits, void* stream) {
    if (rows < 0 || batch <= 0 || ctx_len < 0 || n_heads <= 0 || head_dim <= 0)
        return fail(DSA_ERR_INVALID_ARG, "dsa_indexer_logits: bad sizes");
    if (rows == 0 || ctx_len == 0) return DSA_OK;
    if (!q || !w || !k || !row_batch || !row_pos || !logits)
        return fail(DSA_ERR_INVALID_ARG, "dsa_indexer_logits: null pointer");
    if (!valid_dtype(q_dtype) || !valid_key_dtype(k_dtype)) return fail(DSA_ERR_INVALID_ARG, "dsa_indexer_logits: bad dtype");
    if (ld_logits < ctx_len) return fail(DSA_ERR_INVALID_ARG, "dsa_indexer_logits: ld_logits < ctx_len");
    if ((k_dtype == DSA_FP8_E4M3 || k_dtype == DSA_FP4_E2M1) != (k_scale != nullptr))
        return fail(DSA_ERR_INVALID_ARG, "dsa_indexer_logits: k_scale must be given exactly when k is fp8 or fp4");
    const bool combo_ok = (q_dtype == DSA_FP32 && k_dtype == DSA_FP32) || (q_dtype == DSA_BF16 && k_dtype == DSA_BF16) ||
                          (q_dtype == DSA_BF16 && k_dtype == DSA_FP8_E4M3) ||
                          (q_dtype == DSA_BF16 && k_dtype == DSA_FP4_E2M1);
    if (!combo_ok) return fail(DSA_ERR_UNSUPPORTED, "dsa_indexer_logits: unsupported q/k dtype pair");
    if (head_dim != 32 && head_dim != 64 && head_dim != 128)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_indexer_logits: head_dim must be 32, 64 or 128");
    if (n_heads > 128) return fail(DSA_ERR_UNSUPPORTED, "dsa_indexer_logits: n_heads > 128");
    if (k_dtype == DSA_FP4_E2M1 && !dsa::indexer_tc_supported(q_dtype, k_dtype, n_heads, head_dim))
        return fail(DSA_ERR_UNSUPPORTED, "dsa_indexer_logits: fp4 keys need n_heads = 64 and head_dim = 128");
    dsa::Launch L;
    dsa_status_t st = make_launch(stream, &L);
    if (st != DSA_OK) return st;
    if (dsa::indexer_tc_supported(q_dtype, k_dtype, n_heads, head_dim)) {
        if (!aligned(q, 16) || !aligned(k, 16))
            return fail(DSA_ERR_INVALID_ARG, "dsa_indexer_logits: q and k must be 16-byte aligned");
        return cuda_status(dsa::launch_indexer_tc(L, q, k_dtype, w, k, k_scale, row_batch, row_pos, rows, batch,
                                                  ctx_len, logits, ld_logits),
                           "dsa_indexer_logits (tensor-core) launch");
    }
    return cuda_status(dsa::launch_indexer_simt(L, q, q_dtype, w, k, k_dtype, k_scale, row_batch, row_pos, rows,
                                                batch, ctx_len, n_heads, head_dim, logits, ld_logits),
                       "dsa_indexer_logits launch");
}

size_t dsa_topk_workspace_size(int rows, int ctx_len, int k) { return dsa::topk_workspace_bytes(rows, ctx_len, k); }

dsa_status_t dsa_topk(const float* logits, int64_t ld, const int32_t* row_pos, int rows, int ctx_len, int k,
                      int32_t* idx, void* workspace, size_t workspace_bytes, void* stream) {
    if (rows < 0 || ctx_len < 0 || k < 1 || k > 8192) return fail(DSA_ERR_INVALID_ARG, "dsa_topk: bad sizes (k must be in [1, 8192])");
    if (rows == 0) return DSA_OK;
    if (!logits || !row_pos || !idx) return fail(DSA_ERR_INVALID_ARG, "dsa_topk: null pointer");
    if (ld < ctx_len) return fail(DSA_ERR_INVALID_ARG, "dsa_topk: ld < ctx_len");
    if (!dsa::topk_supported(ctx_len)) return fail(DSA_ERR_UNSUPPORTED, "dsa_topk: ctx_len %d above the supported maximum", ctx_len);
    const size_t need = dsa::topk_workspace_bytes(rows, ctx_len, k);
    if (need && (!workspace || workspace_bytes < need))
        return fail(DSA_ERR_INVALID_ARG, "dsa_topk: workspace of %zu bytes needed", need);
    dsa::Launch L;
    dsa_status_t st = make_launch(stream, &L);
    if (st != DSA_OK) return st;
    return cuda_status(dsa::launch_topk(L, logits, ld, row_pos, rows, ctx_len, k, idx, workspace, workspace_bytes),
                       "dsa_topk launch");
}

size_t dsa_sparse_mla_workspace_size(int rows, int k, int n_heads, int d_qk, int d_v, dsa_dtype_t dtype) {
    if (rows <= 0 || k <= 0 || !dsa::mla_tc_supported(dtype, n_heads, d_qk, d_v)) return 0;
    int dev = 0, sms = 0;
    // No device: size for a very large GPU.  The split count grows with the
    // SM count (up to one split per 64 keys), so this bounds every device.
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 1024;
    return dsa::mla_tc_workspace_bytes(rows, k, sms);
}

size_t dsa_indexer_prepare_workspace_size(int tokens, int n_heads, int d_c, int d_model) {
    if (tokens <= 0 || n_heads <= 0 || d_c <= 0 || d_model <= 0) return 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 1024;  // no device: size for a large GPU (the most splits)
    return dsa::indexer_prepare_workspace_bytes(tokens, n_heads, d_c, d_model, sms);
}

namespace {

// Checks shared by the two key-cache writers.
dsa_status_t check_key_cache(const char* name, const float* rope_cos, const float* rope_sin, int max_pos, int d_rope,
                             const int32_t* pos, const int64_t* slot, int head_dim, const void* k_cache,
                             dsa_dtype_t k_dtype, const float* k_scale, int64_t cache_rows) {
    if (head_dim != 128) return fail(DSA_ERR_UNSUPPORTED, "%s: head_dim must be 128", name);
    if (d_rope < 0 || d_rope > head_dim || (d_rope & 1))
        return fail(DSA_ERR_INVALID_ARG, "%s: d_rope must be even and in [0, head_dim]", name);
    if (d_rope > 0 && (!rope_cos || !rope_sin || !pos || max_pos < 1))
        return fail(DSA_ERR_INVALID_ARG, "%s: rotary tables, positions and max_pos >= 1 needed when d_rope > 0", name);
    if (!slot || !k_cache || cache_rows < 0) return fail(DSA_ERR_INVALID_ARG, "%s: null slot or cache pointer", name);
    if (k_dtype != DSA_BF16 && k_dtype != DSA_FP8_E4M3 && k_dtype != DSA_FP4_E2M1)
        return fail(DSA_ERR_UNSUPPORTED, "%s: the key cache must be bf16, fp8 or fp4", name);
    if ((k_dtype != DSA_BF16) != (k_scale != nullptr))
        return fail(DSA_ERR_INVALID_ARG, "%s: k_scale must be given exactly when the cache is fp8 or fp4", name);
    if (!aligned(k_cache, 16)) return fail(DSA_ERR_INVALID_ARG, "%s: k_cache must be 16-byte aligned", name);
    return DSA_OK;
}

}  // namespace

dsa_status_t dsa_indexer_prepare(const void* c_q, const float* q_norm_weight, float eps, const void* wq_b,
                                 const void* h, const void* wk, const void* w_proj, const float* rope_cos,
                                 const float* rope_sin, int max_pos, int d_rope, const int32_t* pos,
                                 const int64_t* slot, int tokens, int d_c, int d_model, int n_heads, int head_dim,
                                 void* q_out, float* w_out, void* k_cache, dsa_dtype_t k_dtype, float* k_scale,
                                 int64_t cache_rows, void* workspace, size_t workspace_bytes, void* stream) {
    const char* name = "dsa_indexer_prepare";
    if (tokens < 0 || d_c <= 0 || d_model <= 0 || n_heads <= 0 || head_dim <= 0)
        return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    if (tokens == 0) return DSA_OK;
    if (!c_q || !q_norm_weight || !wq_b || !h || !wk || !w_proj || !pos || !q_out || !w_out)
        return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!(eps >= 0.f)) return fail(DSA_ERR_INVALID_ARG, "%s: eps must be >= 0", name);
    dsa_status_t st = check_key_cache(name, rope_cos, rope_sin, max_pos, d_rope, pos, slot, head_dim, k_cache,
                                      k_dtype, k_scale, cache_rows);
    if (st != DSA_OK) return st;
    if (d_c % 64 || d_model % 64) return fail(DSA_ERR_UNSUPPORTED, "%s: d_c and d_model must be multiples of 64", name);
    if (d_c > dsa::indexer_prepare_max_dc())
        return fail(DSA_ERR_UNSUPPORTED, "%s: d_c above %d", name, dsa::indexer_prepare_max_dc());
    if (n_heads > 256) return fail(DSA_ERR_UNSUPPORTED, "%s: n_heads > 256", name);
    if (!aligned(c_q, 16) || !aligned(h, 16) || !aligned(wq_b, 16) || !aligned(wk, 16) || !aligned(w_proj, 16) ||
        !aligned(q_norm_weight, 16) || !aligned(q_out, 16))
        return fail(DSA_ERR_INVALID_ARG, "%s: c_q, h, the weights, q_norm_weight and q_out must be 16-byte aligned", name);
    dsa::Launch L;
    st = make_launch(stream, &L);
    if (st != DSA_OK) return st;
    const size_t need = dsa::indexer_prepare_workspace_bytes(tokens, n_heads, d_c, d_model, L.num_sms);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
        return fail(DSA_ERR_INVALID_ARG, "%s: a 256-byte aligned workspace of %zu bytes is needed", name, need);
    dsa::PrepareArgs a;
    a.c_q = c_q;
    a.gamma = q_norm_weight;
    a.eps = eps;
    a.wq_b = wq_b;
    a.h = h;
    a.wk = wk;
    a.w_proj = w_proj;
    a.rope_cos = rope_cos;
    a.rope_sin = rope_sin;
    a.max_pos = max_pos;
    a.d_rope = d_rope;
    a.pos = pos;
    a.slot = slot;
    a.T = tokens;
    a.d_c = d_c;
    a.d_model = d_model;
    a.n_heads = n_heads;
    a.q_out = q_out;
    a.w_out = w_out;
    a.k_cache = k_cache;
    a.k_fmt = k_dtype;
    a.k_scale = k_scale;
    a.cache_rows = cache_rows;
    return cuda_status(dsa::launch_indexer_prepare(L, a, workspace, workspace_bytes), "dsa_indexer_prepare launch");
}

dsa_status_t dsa_indexer_key_append(const void* k, dsa_dtype_t k_in_dtype, const float* rope_cos,
                                    const float* rope_sin, int max_pos, int d_rope, const int32_t* pos,
                                    const int64_t* slot, int n, int head_dim, void* k_cache, dsa_dtype_t k_dtype,
                                    float* k_scale, int64_t cache_rows, void* stream) {
    const char* name = "dsa_indexer_key_append";
    if (n < 0 || head_dim <= 0) return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    if (n == 0) return DSA_OK;
    if (!k) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    if (k_in_dtype != DSA_FP32 && k_in_dtype != DSA_BF16)
        return fail(DSA_ERR_UNSUPPORTED, "%s: keys must be fp32 or bf16", name);
    dsa_status_t st = check_key_cache(name, rope_cos, rope_sin, max_pos, d_rope, pos, slot, head_dim, k_cache,
                                      k_dtype, k_scale, cache_rows);
    if (st != DSA_OK) return st;
    if (!aligned(k, 16)) return fail(DSA_ERR_INVALID_ARG, "%s: k must be 16-byte aligned", name);
    dsa::Launch L;
    st = make_launch(stream, &L);
    if (st != DSA_OK) return st;
    return cuda_status(dsa::launch_key_append(L, k, k_in_dtype, n, pos, slot, rope_cos, rope_sin, max_pos, d_rope,
                                              k_cache, k_dtype, k_scale, cache_rows),
                       "dsa_indexer_key_append launch");
}

}  // extern "C"

namespace {

// Shared body of dsa_sparse_mla, csa_core_attention and hca_attention: the
// selected (or, with idx NULL, every visible) keys of kv, plus an optional
// window segment of raw rows (x).
dsa_status_t sparse_attention(const char* name, const void* q, const void* kv, dsa_dtype_t dtype,
                              const int32_t* page_table, int page_size, int num_pages, const int32_t* row_batch,
                              const int32_t* idx, int k, int rows, int batch, int ctx_len, int n_heads, int d_qk,
                              int d_v, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream, const dsa::KvExtra& x) {
    const int window = x.kv2 ? x.window : 0;
    const int n_sink = x.kv2 ? x.n_sink : 0;
    if (rows < 0 || batch <= 0 || ctx_len <= 0 || k < 0 || window < 0 || n_sink < 0 ||
        (int64_t)k + window + n_sink < 1 || (int64_t)k + window + n_sink > (1 << 30) || n_heads <= 0 ||
        d_qk <= 0 || d_v <= 0 || d_v > d_qk)
        return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    const bool raw = window + n_sink > 0;                   // a segment of raw rows
    if ((int64_t)batch * ctx_len >= ((int64_t)1 << 31) - 2 ||
        (raw && (int64_t)batch * x.len2 >= ((int64_t)1 << 31) - 2) ||
        (page_table && (int64_t)num_pages * page_size >= ((int64_t)1 << 31) - 2))
        return fail(DSA_ERR_UNSUPPORTED, "%s: a cache holds more than 2^31 - 2 rows", name);
    if (rows == 0) return DSA_OK;
    if (!q || !kv || !row_batch || !out || !lse || (k > 0 && !idx && !x.row_last))
        return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    if (raw && (!x.pos2 || x.len2 <= 0))
        return fail(DSA_ERR_INVALID_ARG, "%s: a window or sink needs win_pos and win_len", name);
    if (dtype != DSA_BF16 && dtype != DSA_FP32) return fail(DSA_ERR_UNSUPPORTED, "%s: dtype must be bf16 or fp32", name);
    if (page_table) {
        if (page_size <= 0 || ctx_len % page_size)
            return fail(DSA_ERR_INVALID_ARG, "%s: ctx_len must be a multiple of page_size", name);
        if (num_pages <= 0) return fail(DSA_ERR_INVALID_ARG, "%s: num_pages must be positive with a page table", name);
    }
    if (!(scale > 0.f) || !(scale < 1e30f)) return fail(DSA_ERR_INVALID_ARG, "%s: scale must be positive and finite", name);
    const bool tc = dsa::mla_tc_supported(dtype, n_heads, d_qk, d_v);
    if (!tc && !dsa::mla_simt_supported(d_qk, d_v, n_heads))
        return fail(DSA_ERR_UNSUPPORTED, "%s: no kernel for d_qk=%d d_v=%d n_heads=%d", name, d_qk, d_v, n_heads);
    dsa::Launch L;
    dsa_status_t st = make_launch(stream, &L);
    if (st != DSA_OK) return st;
    if (tc) {
        if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(out, 16) || (raw && !aligned(x.kv2, 16)))
            return fail(DSA_ERR_INVALID_ARG, "%s: q, kv, the window cache and out must be 16-byte aligned", name);
        const size_t need = dsa::mla_tc_workspace_bytes(rows, k + window + n_sink, L.num_sms);
        if (need && (!workspace || workspace_bytes < need))
            return fail(DSA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", name, need);
        return cuda_status(dsa::launch_mla_tc(L, q, kv, page_table, page_size, num_pages, row_batch, idx, k, rows,
                                              batch, ctx_len, scale, out, lse, workspace, workspace_bytes, x),
                           "sparse attention (tensor-core) launch");
    }
    return cuda_status(dsa::launch_mla_simt(L, q, kv, dtype, page_table, page_size, num_pages, row_batch, idx, k, rows,
                                            batch, ctx_len, n_heads, d_qk, d_v, scale, out, lse, x),
                       "sparse attention launch");
}

}  // namespace

extern "C" {

dsa_status_t dsa_sparse_mla(const void* q, const void* kv, dsa_dtype_t dtype, const int32_t* page_table,
                            int page_size, int num_pages, const int32_t* row_batch, const int32_t* idx, int k, int rows, int batch,
                            int ctx_len, int n_heads, int d_qk, int d_v, float scale, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
    if (k < 1) return fail(DSA_ERR_INVALID_ARG, "dsa_sparse_mla: bad sizes (k=%d)", k);
    if (rows > 0 && !idx) return fail(DSA_ERR_INVALID_ARG, "dsa_sparse_mla: null pointer");
    return sparse_attention("dsa_sparse_mla", q, kv, dtype, page_table, page_size, num_pages, row_batch, idx, k, rows,
                            batch, ctx_len, n_heads, d_qk, d_v, scale, out, lse, workspace, workspace_bytes, stream,
                            dsa::KvExtra());
}

dsa_status_t csa_core_attention(const void* q, const void* kv, dsa_dtype_t dtype, const int32_t* page_table,
                                int page_size, int num_pages, const int32_t* row_batch, const int32_t* idx, int k,
                                int rows, int batch, int ctx_len, const void* kv_win, const int32_t* win_pos,
                                int win_len, int window, int n_sink, int n_heads, int d_qk, int d_v, float scale,
                                void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (window < 0 || n_sink < 0 || (window + n_sink > 0 && !kv_win))
        return fail(DSA_ERR_INVALID_ARG, "csa_core_attention: bad window or sink");
    if (n_sink > win_len) return fail(DSA_ERR_INVALID_ARG, "csa_core_attention: n_sink above win_len");
    if (rows > 0 && k > 0 && !idx) return fail(DSA_ERR_INVALID_ARG, "csa_core_attention: null pointer");
    dsa::KvExtra x;
    x.kv2 = kv_win;
    x.pos2 = win_pos;
    x.len2 = win_len;
    x.window = window;
    x.n_sink = n_sink;
    return sparse_attention("csa_core_attention", q, kv, dtype, page_table, page_size, num_pages, row_batch, idx, k,
                            rows, batch, ctx_len, n_heads, d_qk, d_v, scale, out, lse, workspace, workspace_bytes,
                            stream, x);
}

dsa_status_t hca_attention(const void* q, const void* kv, dsa_dtype_t dtype, const int32_t* row_batch,
                           const int32_t* row_last, int rows, int batch, int ctx_len, int n_heads, int d_qk, int d_v,
                           float scale, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (rows > 0 && !row_last) return fail(DSA_ERR_INVALID_ARG, "hca_attention: null pointer");
    dsa::KvExtra x;
    x.row_last = row_last;
    return sparse_attention("hca_attention", q, kv, dtype, nullptr, 0, 0, row_batch, nullptr, ctx_len, rows, batch,
                            ctx_len, n_heads, d_qk, d_v, scale, out, lse, workspace, workspace_bytes, stream, x);
}

dsa_status_t dsa_sparse_mla_noalloc(const void* q, const void* kv, dsa_dtype_t dtype, const int32_t* page_table,
                                    int page_size, int num_pages, const int32_t* row_batch, const int32_t* idx, int k,
                                    int rows, int batch, int ctx_len, int n_heads, int d_qk, int d_v, float scale,
                                    void* out, float* lse, void* stream) {
    void* scratch = nullptr;
    if (rows > 0 && k >= 1 && dsa::mla_tc_supported(dtype, n_heads, d_qk, d_v)) {
        dsa::Launch L;
        dsa_status_t st = make_launch(stream, &L);
        if (st != DSA_OK) return st;
        const size_t need = dsa::mla_tc_workspace_bytes(rows, k, L.num_sms);
        if (need > kMlaScratchBytes)
            return fail(DSA_ERR_INVALID_ARG,
                        "dsa_sparse_mla_noalloc: %d rows x k=%d need %zu bytes of scratch, more than its fixed %zu",
                        rows, k, need, kMlaScratchBytes);
        if (need) {
            st = mla_scratch(&scratch);
            if (st != DSA_OK) return st;
        }
    }
    return dsa_sparse_mla(q, kv, dtype, page_table, page_size, num_pages, row_batch, idx, k, rows, batch, ctx_len,
                          n_heads, d_qk, d_v, scale, out, lse, scratch, scratch ? kMlaScratchBytes : 0, stream);
}

namespace {

bool kv_head_dim(int d) { return d == 64 || d == 128; }

// Cache geometry shared by kv_cache_append and gqa_decode_attention.
dsa_status_t check_paged_kv(const char* name, const int32_t* page_table, int batch, int max_pages, int page_size,
                            int num_pages, int n_kv_heads, int head_dim, const void* k_cache, const void* v_cache,
                            dsa_dtype_t kv_dtype, const float* k_scale, const float* v_scale) {
    if (batch <= 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0 || n_kv_heads <= 0 || head_dim <= 0)
        return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    if (!page_table || !k_cache || !v_cache) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    if (kv_dtype != DSA_BF16 && kv_dtype != DSA_FP32 && kv_dtype != DSA_FP8_E4M3)
        return fail(DSA_ERR_UNSUPPORTED, "%s: the cache must be bf16, fp32 or fp8", name);
    if ((kv_dtype == DSA_FP8_E4M3) != (k_scale != nullptr) || (k_scale != nullptr) != (v_scale != nullptr))
        return fail(DSA_ERR_INVALID_ARG, "%s: k_scale and v_scale must be given exactly when the cache is fp8", name);
    if (!kv_head_dim(head_dim)) return fail(DSA_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", name);
    if (n_kv_heads > 1024) return fail(DSA_ERR_UNSUPPORTED, "%s: n_kv_heads > 1024", name);
    const int64_t lim = ((int64_t)1 << 31) - 2;
    if ((int64_t)num_pages * page_size > lim || (int64_t)num_pages * page_size * n_kv_heads > lim ||
        (int64_t)batch * max_pages > lim || (int64_t)max_pages * page_size > lim)
        return fail(DSA_ERR_UNSUPPORTED, "%s: more than 2^31 - 2 cache rows, table entries or positions", name);
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16))
        return fail(DSA_ERR_INVALID_ARG, "%s: the caches must be 16-byte aligned", name);
    return DSA_OK;
}

// A [rows, heads, head_dim] operand whose rows are `ld` elements apart.
dsa_status_t check_rows(const char* name, const char* what, const void* p, int64_t ld, int heads, int head_dim,
                        dsa_dtype_t t) {
    if (!p) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer (%s)", name, what);
    if (ld < (int64_t)heads * head_dim) return fail(DSA_ERR_INVALID_ARG, "%s: rows of %s overlap", name, what);
    if (!aligned(p, 16) || (ld * dtype_size(t)) % 16)
        return fail(DSA_ERR_INVALID_ARG, "%s: %s and its row stride must be 16-byte aligned", name, what);
    return DSA_OK;
}

// The pool's books.
dsa_status_t check_books(const char* name, const int32_t* page_table, int batch, int max_pages, int page_size,
                         const int32_t* seq_len, const int32_t* ref_count, int num_pages, int n) {
    if (batch <= 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0 || n < 0)
        return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    if (n > DSA_KV_PAGES_MAX_LIST) return fail(DSA_ERR_UNSUPPORTED, "%s: more than %d list entries", name, DSA_KV_PAGES_MAX_LIST);
    if (num_pages > DSA_KV_PAGES_MAX_POOL) return fail(DSA_ERR_UNSUPPORTED, "%s: more than %d pages", name, DSA_KV_PAGES_MAX_POOL);
    const int64_t lim = ((int64_t)1 << 31) - 2;
    if ((int64_t)batch * max_pages > lim || (int64_t)n * max_pages > lim)
        return fail(DSA_ERR_UNSUPPORTED, "%s: more than 2^31 - 2 table entries", name);
    if (!page_table || !seq_len || !ref_count) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    return DSA_OK;
}

dsa_status_t check_caches(const char* name, void* const* caches, const size_t* page_bytes, int n_caches) {
    if (n_caches < 0 || (n_caches > 0 && (!caches || !page_bytes)))
        return fail(DSA_ERR_INVALID_ARG, "%s: bad cache list", name);
    for (int i = 0; i < n_caches; ++i) {
        if (!caches[i] || !aligned(caches[i], 16))
            return fail(DSA_ERR_INVALID_ARG, "%s: cache %d is null or not 16-byte aligned", name, i);
        if (page_bytes[i] == 0 || page_bytes[i] % 16 || page_bytes[i] > ((size_t)1 << 30))
            return fail(DSA_ERR_UNSUPPORTED, "%s: the page bytes of cache %d must be a multiple of 16, at most 2^30", name, i);
    }
    return DSA_OK;
}

}  // namespace

dsa_status_t kv_cache_append(const void* k, int64_t ld_k, const void* v, int64_t ld_v, dsa_dtype_t dtype,
                             const int32_t* row_batch, const int32_t* row_pos, int n, const int32_t* page_table,
                             int batch, int max_pages, int page_size, int num_pages, int n_kv_heads, int head_dim,
                             void* k_cache, void* v_cache, dsa_dtype_t kv_dtype, float* k_scale, float* v_scale,
                             void* stream) {
    const char* name = "kv_cache_append";
    if (n < 0) return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    if (n == 0) return DSA_OK;
    dsa_status_t st = check_paged_kv(name, page_table, batch, max_pages, page_size, num_pages, n_kv_heads, head_dim,
                                     k_cache, v_cache, kv_dtype, k_scale, v_scale);
    if (st != DSA_OK) return st;
    if (dtype != DSA_BF16 && dtype != DSA_FP32) return fail(DSA_ERR_UNSUPPORTED, "%s: k and v must be bf16 or fp32", name);
    if (kv_dtype == DSA_FP32 && dtype != DSA_FP32)
        return fail(DSA_ERR_UNSUPPORTED, "%s: an fp32 cache takes fp32 keys and values", name);
    if (!row_batch || !row_pos) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    if ((st = check_rows(name, "k", k, ld_k, n_kv_heads, head_dim, dtype)) != DSA_OK) return st;
    if ((st = check_rows(name, "v", v, ld_v, n_kv_heads, head_dim, dtype)) != DSA_OK) return st;
    if ((int64_t)n * 2 * n_kv_heads > ((int64_t)1 << 31) - 2) return fail(DSA_ERR_UNSUPPORTED, "%s: too many rows and heads", name);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    dsa::AppendArgs a;
    a.k = k;
    a.v = v;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.row_batch = row_batch;
    a.row_pos = row_pos;
    a.n = n;
    a.n_kv_heads = n_kv_heads;
    a.page_table = page_table;
    a.batch = batch;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.by_page = dsa::fast_div(page_size);
    a.by_head = dsa::fast_div(n_kv_heads);
    a.err = L.err;
    return cuda_status(dsa::launch_kv_append(L, a, dtype, kv_dtype, head_dim), "kv_cache_append launch");
}

size_t gqa_decode_attention_workspace_size(int rows, int n_heads, int n_kv_heads, int head_dim, dsa_dtype_t kv_dtype) {
    if (rows <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads || !kv_head_dim(head_dim)) return 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 1024;  // no device: size for a large GPU
    return dsa::gqa_decode_workspace_bytes(rows, n_heads, n_kv_heads, head_dim, kv_dtype, sms);
}

dsa_status_t gqa_decode_attention(const void* q, int64_t ld_q, dsa_dtype_t dtype, const void* k_cache,
                                  const void* v_cache, dsa_dtype_t kv_dtype, const float* k_scale,
                                  const float* v_scale, const int32_t* page_table, int batch, int max_pages,
                                  int page_size, int num_pages, const int32_t* row_batch, const int32_t* row_pos,
                                  int rows, int n_heads, int n_kv_heads, int head_dim, float scale, void* out,
                                  float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    const char* name = "gqa_decode_attention";
    if (rows < 0) return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    if (rows == 0) return DSA_OK;
    dsa_status_t st = check_paged_kv(name, page_table, batch, max_pages, page_size, num_pages, n_kv_heads, head_dim,
                                     k_cache, v_cache, kv_dtype, k_scale, v_scale);
    if (st != DSA_OK) return st;
    if (!(dtype == DSA_FP32 && kv_dtype == DSA_FP32) &&
        !(dtype == DSA_BF16 && (kv_dtype == DSA_BF16 || kv_dtype == DSA_FP8_E4M3)))
        return fail(DSA_ERR_UNSUPPORTED, "%s: unsupported query / cache type pair", name);
    if (n_heads <= 0 || n_heads % n_kv_heads)
        return fail(DSA_ERR_INVALID_ARG, "%s: n_heads must be a multiple of n_kv_heads", name);
    if (!row_batch || !row_pos || !out || !lse) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    if ((st = check_rows(name, "q", q, ld_q, n_heads, head_dim, dtype)) != DSA_OK) return st;
    if (!aligned(out, 16)) return fail(DSA_ERR_INVALID_ARG, "%s: out must be 16-byte aligned", name);
    if (!(scale > 0.f) || !(scale < 1e30f)) return fail(DSA_ERR_INVALID_ARG, "%s: scale must be positive and finite", name);
    const int64_t units = ((int64_t)max_pages * page_size - 1) / 64 + 1, lim = ((int64_t)1 << 31) - 2;
    if ((int64_t)rows * units > lim || units * n_heads > lim || (int64_t)rows * n_heads > lim)
        return fail(DSA_ERR_UNSUPPORTED, "%s: too many rows, heads or positions", name);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    const size_t need = dsa::gqa_decode_workspace_bytes(rows, n_heads, n_kv_heads, head_dim, kv_dtype, L.num_sms);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
        return fail(DSA_ERR_INVALID_ARG, "%s: a 256-byte aligned workspace of %zu bytes is needed", name, need);
    dsa::DecodeArgs a;
    a.q = q;
    a.ld_q = ld_q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.page_table = page_table;
    a.batch = batch;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.row_batch = row_batch;
    a.row_pos = row_pos;
    a.rows = rows;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.by_page = dsa::fast_div(page_size);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = out;
    a.lse = lse;
    a.err = L.err;
    return cuda_status(dsa::launch_gqa_decode(L, a, kv_dtype, head_dim, workspace), "gqa_decode_attention launch");
}

size_t gqa_prompt_attention_workspace_size(int total, int n_seqs, int n_heads, int head_dim, dsa_dtype_t dtype) {
    if (total <= 0 || n_seqs <= 0 || n_heads <= 0 || !kv_head_dim(head_dim)) return 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 1024;  // no device: size for a large GPU
    return dsa::gqa_prompt_workspace_bytes(total, n_seqs, n_heads, head_dim, dtype, sms);
}

dsa_status_t gqa_prompt_attention(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                                  int64_t ld_v, dsa_dtype_t dtype, const int32_t* cu_seqlens, int n_seqs, int total,
                                  int n_heads, int n_kv_heads, int head_dim, float scale, void* out, float* lse,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const char* name = "gqa_prompt_attention";
    if (n_seqs < 0 || total < 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0)
        return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    if (n_heads % n_kv_heads) return fail(DSA_ERR_INVALID_ARG, "%s: n_heads must be a multiple of n_kv_heads", name);
    if (n_seqs == 0 || total == 0) return DSA_OK;
    if (dtype != DSA_BF16 && dtype != DSA_FP32) return fail(DSA_ERR_UNSUPPORTED, "%s: dtype must be bf16 or fp32", name);
    if (!kv_head_dim(head_dim)) return fail(DSA_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", name);
    if (!cu_seqlens || !out || !lse) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    dsa_status_t st = check_rows(name, "q", q, ld_q, n_heads, head_dim, dtype);
    if (st != DSA_OK) return st;
    if ((st = check_rows(name, "k", k, ld_k, n_kv_heads, head_dim, dtype)) != DSA_OK) return st;
    if ((st = check_rows(name, "v", v, ld_v, n_kv_heads, head_dim, dtype)) != DSA_OK) return st;
    if (!aligned(out, 16)) return fail(DSA_ERR_INVALID_ARG, "%s: out must be 16-byte aligned", name);
    if (!(scale > 0.f) || !(scale < 1e30f)) return fail(DSA_ERR_INVALID_ARG, "%s: scale must be positive and finite", name);
    const int64_t tiles = (int64_t)total / 64 + (n_seqs < total ? n_seqs : total);
    if (tiles * n_heads > ((int64_t)1 << 31) - 2) return fail(DSA_ERR_UNSUPPORTED, "%s: too many rows and heads", name);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    const size_t need = dsa::gqa_prompt_workspace_bytes(total, n_seqs, n_heads, head_dim, dtype, L.num_sms);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(DSA_ERR_INVALID_ARG, "%s: a 256-byte aligned workspace of %zu bytes is needed", name, need);
    dsa::PromptArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.cu_seqlens = cu_seqlens;
    a.n_seqs = n_seqs;
    a.total = total;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = out;
    a.lse = lse;
    a.err = L.err;
    return cuda_status(dtype == DSA_BF16 ? dsa::launch_gqa_prompt_tc(L, a, head_dim, workspace)
                                         : dsa::launch_gqa_prompt_f32(L, a, head_dim),
                       "gqa_prompt_attention launch");
}

dsa_status_t kv_pages_copy(void* const* caches, const size_t* page_bytes, int n_caches, int num_pages,
                           const int32_t* src, const int32_t* dst, int n, void* stream) {
    const char* name = "kv_pages_copy";
    if (n < 0 || num_pages <= 0) return fail(DSA_ERR_INVALID_ARG, "%s: bad sizes", name);
    dsa_status_t st = check_caches(name, caches, page_bytes, n_caches);
    if (st != DSA_OK) return st;
    if (n == 0 || n_caches == 0) return DSA_OK;
    if (!src || !dst) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    const dsa::CacheList l = {caches, page_bytes, n_caches, num_pages};
    return cuda_status(dsa::launch_kv_copy(L, l, src, dst, n), "kv_pages_copy launch");
}

dsa_status_t kv_pages_extend(int32_t* page_table, int batch, int max_pages, int page_size, int32_t* seq_len,
                             int32_t* ref_count, int num_pages, const int32_t* seqs, const int32_t* add, int n,
                             void* stream) {
    const char* name = "kv_pages_extend";
    dsa_status_t st = check_books(name, page_table, batch, max_pages, page_size, seq_len, ref_count, num_pages, n);
    if (st != DSA_OK) return st;
    if (n == 0) return DSA_OK;
    if (!seqs || !add) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    dsa::BooksArgs a = {page_table, seq_len, ref_count, batch, max_pages, page_size, num_pages, seqs, add,
                        nullptr, nullptr, n, nullptr, nullptr, L.err};
    return cuda_status(dsa::launch_kv_extend(L, a), "kv_pages_extend launch");
}

dsa_status_t kv_pages_free(int32_t* page_table, int batch, int max_pages, int page_size, int32_t* seq_len,
                           int32_t* ref_count, int num_pages, const int32_t* seqs, int n, void* stream) {
    const char* name = "kv_pages_free";
    dsa_status_t st = check_books(name, page_table, batch, max_pages, page_size, seq_len, ref_count, num_pages, n);
    if (st != DSA_OK) return st;
    if (n == 0) return DSA_OK;
    if (!seqs) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    dsa::BooksArgs a = {page_table, seq_len, ref_count, batch, max_pages, page_size, num_pages, seqs, nullptr,
                        nullptr, nullptr, n, nullptr, nullptr, L.err};
    return cuda_status(dsa::launch_kv_free(L, a), "kv_pages_free launch");
}

size_t kv_pages_fork_workspace_size(int n) { return n > 0 ? dsa::kv_fork_workspace_bytes(n) : 0; }

dsa_status_t kv_pages_fork(int32_t* page_table, int batch, int max_pages, int page_size, int32_t* seq_len,
                           int32_t* ref_count, int num_pages, const int32_t* parents, const int32_t* children, int n,
                           void* const* caches, const size_t* page_bytes, int n_caches, void* workspace,
                           size_t workspace_bytes, void* stream) {
    const char* name = "kv_pages_fork";
    dsa_status_t st = check_books(name, page_table, batch, max_pages, page_size, seq_len, ref_count, num_pages, n);
    if (st != DSA_OK) return st;
    if ((st = check_caches(name, caches, page_bytes, n_caches)) != DSA_OK) return st;
    if (n == 0) return DSA_OK;
    if (!parents || !children) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    const size_t need = dsa::kv_fork_workspace_bytes(n);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return fail(DSA_ERR_INVALID_ARG, "%s: a 16-byte aligned workspace of %zu bytes is needed", name, need);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    dsa::BooksArgs a = {page_table, seq_len, ref_count, batch, max_pages, page_size, num_pages, nullptr, nullptr,
                        parents, children, n, nullptr, nullptr, L.err};
    const dsa::CacheList l = {caches, page_bytes, n_caches, num_pages};
    return cuda_status(dsa::launch_kv_fork(L, a, l, workspace), "kv_pages_fork launch");
}

size_t kv_pages_compact_workspace_size(int num_pages) {
    return num_pages > 0 ? dsa::kv_compact_workspace_bytes(num_pages) : 0;
}

dsa_status_t kv_pages_compact(const int32_t* page_table, int batch, int max_pages, const int32_t* ref_count,
                              int num_pages, void* const* caches, const size_t* page_bytes, int n_caches,
                              int32_t* table_out, int32_t* ref_out, void* workspace, size_t workspace_bytes,
                              void* stream) {
    const char* name = "kv_pages_compact";
    if (!table_out || !ref_out) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
    dsa_status_t st = check_books(name, page_table, batch, max_pages, 1, ref_count, ref_count, num_pages, 0);
    if (st != DSA_OK) return st;
    if ((st = check_caches(name, caches, page_bytes, n_caches)) != DSA_OK) return st;
    const size_t table_bytes = (size_t)batch * max_pages * 4, ref_bytes = (size_t)num_pages * 4;
    auto overlap = [](const void* x, const void* y, size_t n) {
        return x != y && (const char*)x < (const char*)y + n && (const char*)y < (const char*)x + n;
    };
    if (overlap(page_table, table_out, table_bytes) || overlap(ref_count, ref_out, ref_bytes))
        return fail(DSA_ERR_INVALID_ARG, "%s: an output overlaps its input without being it", name);
    const size_t need = dsa::kv_compact_workspace_bytes(num_pages);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return fail(DSA_ERR_INVALID_ARG, "%s: a 16-byte aligned workspace of %zu bytes is needed", name, need);
    dsa::Launch L;
    if ((st = make_launch(stream, &L)) != DSA_OK) return st;
    dsa::CompactArgs a = {page_table, ref_count, table_out, ref_out, batch, max_pages, num_pages,
                          nullptr, nullptr, nullptr, nullptr, nullptr, L.err};
    const dsa::CacheList l = {caches, page_bytes, n_caches, num_pages};
    return cuda_status(dsa::launch_kv_compact(L, a, l, workspace), "kv_pages_compact launch");
}

dsa_status_t dsa_get_device_error(void* stream) {
    dsa::Launch L;
    dsa_status_t st = make_launch(stream, &L);
    if (st != DSA_OK) return st;
    cudaError_t e = cudaStreamSynchronize(L.stream);
    if (e != cudaSuccess) return cuda_status(e, "dsa_get_device_error: stream synchronize");
    unsigned word = 0;
    e = cudaMemcpyFromSymbol(&word, g_device_error, sizeof word);
    if (e != cudaSuccess) return cuda_status(e, "dsa_get_device_error: read");
    if (word == 0) return DSA_OK;
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
    if (e != cudaSuccess) return cuda_status(e, "dsa_get_device_error: clear");
    if (word & (dsa::DEV_ERR_TIMEOUT_TMA | dsa::DEV_ERR_TIMEOUT_MMA | dsa::DEV_ERR_TIMEOUT_PEER))
        return fail(DSA_ERR_DEVICE_TIMEOUT, "a kernel gave up a bounded wait (device error word 0x%x)", word);
    if (word & dsa::DEV_ERR_BAD_INDEX)
        return fail(DSA_ERR_INVALID_ARG, "a kernel met an out-of-range index and skipped it (device error word 0x%x)", word);
    return fail(DSA_ERR_OUT_OF_PAGES, "a sequence found too few free pages and was left as it was (device error word 0x%x)", word);
}

}  // extern "C"
