// Python binding of the grouped-query attention and page-pool entry points:
// argument checks, outputs and workspaces, torch's current stream.  Written
// against torch's C++ interface because these calls are small (a decode step's
// append is 2 us on the GPU) and the same checks in Python took 12 to 26 us.
// The arithmetic is all behind the C entry points of include/dsa_b200.h; the
// functions here take their arguments by position and are documented in the
// package's __init__.py.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "dsa_b200.h"

namespace {

PyObject* g_error = nullptr;            // DSAError(status, where)

// Python's ValueError and TypeError (END_HANDLE_TH_ERRORS converts them).
template <class... A> [[noreturn]] void value_error(const A&... what) {
    TORCH_CHECK_VALUE(false, what...);
    std::abort();                       // (not reached)
}
template <class... A> [[noreturn]] void type_error(const A&... what) {
    TORCH_CHECK_TYPE(false, what...);
    std::abort();                       // (not reached)
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(name, " must be a tensor");
    return THPVariable_Unpack(o);
}

struct Call {
    int device = -1;
    c10::cuda::OptionalCUDAGuard guard;

    // A tensor that the library reads or writes: on the GPU, on the call's
    // device (the first tensor's, which is made current).
    void on(const at::Tensor& t) {
        if (!t.is_cuda()) value_error("all tensors must be CUDA tensors (the library takes device pointers)");
        if (device < 0) {
            device = t.get_device();
            if (c10::cuda::current_device() != device) guard.set_index(device);
        } else if (t.get_device() != device) {
            value_error("tensors on different devices");
        }
    }
    const at::Tensor& dense(PyObject* o, const char* name) {
        const at::Tensor& t = tensor(o, name);
        on(t);
        if (!t.is_contiguous()) value_error("tensors must be contiguous");
        return t;
    }
    const at::Tensor& dense_i32(PyObject* o, const char* name, int dim) {
        const at::Tensor& t = dense(o, name);
        if (t.scalar_type() != at::kInt) type_error(name, " must be int32");
        if (t.dim() != dim) value_error(name, " must have ", dim, " dimension(s)");
        return t;
    }
    // A [rows, heads, dim] operand: rows may be strided (views of a fused
    // projection), heads and dims dense.  Returns the rows' distance.
    int64_t rows(const at::Tensor& t, const char* name) {
        on(t);
        if (t.dim() != 3) value_error(name, " must be [rows, heads, dim]");
        const int64_t heads = t.size(1), dim = t.size(2);
        if ((dim > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != dim))
            value_error(name, ": the heads and dims of a row must be contiguous");
        return t.size(0) > 1 ? t.stride(0) : heads * dim;
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

// Sizes go to the library as int.
int as_int(int64_t v) {
    if (v > 0x7fffffff) value_error("a size is above 2^31 - 1");
    return (int)v;
}

dsa_dtype_t type_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return DSA_FP32;
        case at::kBFloat16: return DSA_BF16;
        case at::kByte:
        case at::kFloat8_e4m3fn: return DSA_FP8_E4M3;
        default: type_error("unsupported dtype");
    }
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v < -0x7fffffffl || v > 0x7fffffffl) value_error("an integer argument is out of range");
    return (int)v;
}

// True when the call succeeded; else DSAError(status, where) is set.
bool succeeded(dsa_status_t st, const char* where) {
    if (st == DSA_OK) return true;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return false;
}

// The cache pair and its scales.
struct Cache {
    const at::Tensor *k, *v;
    const float *k_scale = nullptr, *v_scale = nullptr;
    dsa_dtype_t type;
    int pages, heads, page, dim;

    Cache(Call& c, PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso) {
        k = &c.dense(ko, "k_cache");
        v = &c.dense(vo, "v_cache");
        if (k->dim() != 4 || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type())
            value_error("k_cache and v_cache must be [num_pages, n_kv_heads, page_size, head_dim] of one type");
        type = type_of(*k);
        pages = as_int(k->size(0));
        heads = as_int(k->size(1));
        page = as_int(k->size(2));
        dim = as_int(k->size(3));
        k_scale = scales(c, kso);
        v_scale = scales(c, vso);
    }
    const float* scales(Call& c, PyObject* o) {
        if (o == Py_None) return nullptr;
        const at::Tensor& s = c.dense(o, "scales");
        if (s.scalar_type() != at::kFloat || s.dim() != 3 || s.sizes() != k->sizes().slice(0, 3))
            value_error("scales must be fp32 [num_pages, n_kv_heads, page_size]");
        return s.const_data_ptr<float>();
    }
};

// An output given by the caller, or a fresh one.
at::Tensor output(Call& c, PyObject* o, const char* name, at::IntArrayRef shape, const at::TensorOptions& opt) {
    if (o == Py_None) return at::empty(shape, opt);
    const at::Tensor& t = c.dense(o, name);
    if (t.sizes() != shape || t.scalar_type() != c10::typeMetaToScalarType(opt.dtype()))
        value_error(name, " has another shape or type than the result");
    return t;
}

at::Tensor scratch(Call& c, PyObject* o, size_t bytes, const at::TensorOptions& opt) {
    if (o == Py_None) return at::empty({(int64_t)bytes + 1}, opt.dtype(at::kByte));
    return c.dense(o, "workspace");
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b), *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) type_error("wrong number of arguments");
}

// k, v, row_batch, row_pos, page_table, k_cache, v_cache, k_scale, v_scale
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 9);
    Call c;
    const Cache kv(c, a[5], a[6], a[7], a[8]);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int64_t ld_k = c.rows(k, "k"), ld_v = c.rows(v, "v");
    if (k.size(1) != kv.heads || k.size(2) != kv.dim || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
        value_error("k and v must be [n, n_kv_heads, head_dim] of one type");
    const int n = as_int(k.size(0));
    const at::Tensor &batch = c.dense_i32(a[2], "row_batch", 1), &pos = c.dense_i32(a[3], "row_pos", 1),
                     &table = c.dense_i32(a[4], "page_table", 2);
    if (batch.size(0) != n || pos.size(0) != n) value_error("row_batch and row_pos must be [n]");
    if (!succeeded(kv_cache_append(k.const_data_ptr(), ld_k, v.const_data_ptr(), ld_v, type_of(k),
                                   batch.const_data_ptr<int32_t>(), pos.const_data_ptr<int32_t>(), n,
                                   table.const_data_ptr<int32_t>(), as_int(table.size(0)), as_int(table.size(1)), kv.page,
                                   kv.pages, kv.heads, kv.dim, kv.k->mutable_data_ptr(), kv.v->mutable_data_ptr(), kv.type,
                                   const_cast<float*>(kv.k_scale), const_cast<float*>(kv.v_scale), c.stream()),
                   "kv_cache_append"))
        return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, page_table, row_batch, row_pos, scale, k_scale, v_scale, out, lse, workspace
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 12);
    Call c;
    const at::Tensor& q = tensor(a[0], "q");
    const int64_t ld_q = c.rows(q, "q");
    const Cache kv(c, a[1], a[2], a[7], a[8]);
    if (q.size(2) != kv.dim) value_error("q and the caches differ in head_dim");
    const int rows = as_int(q.size(0)), heads = as_int(q.size(1));
    const at::Tensor &table = c.dense_i32(a[3], "page_table", 2), &batch = c.dense_i32(a[4], "row_batch", 1),
                     &pos = c.dense_i32(a[5], "row_pos", 1);
    if (batch.size(0) != rows || pos.size(0) != rows) value_error("row_batch and row_pos must be [rows]");
    const at::Tensor out = output(c, a[9], "out", q.sizes(), q.options());
    const at::Tensor lse = output(c, a[10], "lse", {rows, heads}, q.options().dtype(at::kFloat));
    const at::Tensor ws = scratch(c, a[11], a[11] == Py_None ? gqa_decode_attention_workspace_size(rows, heads, kv.heads, kv.dim, kv.type) : 0,
                                  q.options());
    if (!succeeded(gqa_decode_attention(q.const_data_ptr(), ld_q, type_of(q), kv.k->const_data_ptr(), kv.v->const_data_ptr(),
                                        kv.type, kv.k_scale, kv.v_scale, table.const_data_ptr<int32_t>(),
                                        as_int(table.size(0)), as_int(table.size(1)), kv.page, kv.pages,
                                        batch.const_data_ptr<int32_t>(), pos.const_data_ptr<int32_t>(), rows, heads, kv.heads,
                                        kv.dim, (float)number(a[6]), out.mutable_data_ptr(), lse.mutable_data_ptr<float>(),
                                        ws.mutable_data_ptr(), ws.nbytes(), c.stream()),
                   "gqa_decode_attention"))
        return nullptr;
    return pair(out, lse);
    END_HANDLE_TH_ERRORS
}

// q, k, v, cu_seqlens, scale, out, lse, workspace
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 8);
    Call c;
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int64_t ld_q = c.rows(q, "q"), ld_k = c.rows(k, "k"), ld_v = c.rows(v, "v");
    if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || v.sizes() != k.sizes() || k.scalar_type() != q.scalar_type() ||
        v.scalar_type() != q.scalar_type())
        value_error("k and v must be [total, n_kv_heads, head_dim] of q's type");
    const at::Tensor& cu = c.dense_i32(a[3], "cu_seqlens", 1);
    if (cu.size(0) < 1) value_error("cu_seqlens must be [n_seqs + 1]");
    const int total = as_int(q.size(0)), heads = as_int(q.size(1)), dim = as_int(q.size(2)), n_seqs = as_int(cu.size(0) - 1);
    const dsa_dtype_t type = type_of(q);
    const at::Tensor out = output(c, a[5], "out", q.sizes(), q.options());
    const at::Tensor lse = output(c, a[6], "lse", {total, heads}, q.options().dtype(at::kFloat));
    at::Tensor ws;
    if (a[7] != Py_None) {
        ws = c.dense(a[7], "workspace");
    } else if (const size_t need = gqa_prompt_attention_workspace_size(total, n_seqs, heads, dim, type)) {
        ws = scratch(c, a[7], need, q.options());
    }
    if (!succeeded(gqa_prompt_attention(q.const_data_ptr(), ld_q, k.const_data_ptr(), ld_k, v.const_data_ptr(), ld_v, type,
                                        cu.const_data_ptr<int32_t>(), n_seqs, total, heads, as_int(k.size(1)), dim,
                                        (float)number(a[4]), out.mutable_data_ptr(), lse.mutable_data_ptr<float>(),
                                        ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0,
                                        c.stream()),
                   "gqa_prompt_attention"))
        return nullptr;
    return pair(out, lse);
    END_HANDLE_TH_ERRORS
}

// The pool's books.
struct Books {
    const at::Tensor *table, *len, *count;
    int batch, width, pages;

    Books(Call& c, PyObject* t, PyObject* l, PyObject* r) {
        table = &c.dense_i32(t, "page_table", 2);
        len = &c.dense_i32(l, "seq_len", 1);
        count = &c.dense_i32(r, "ref_count", 1);
        batch = as_int(table->size(0));
        width = as_int(table->size(1));
        pages = as_int(count->size(0));
        if (len->size(0) != batch) value_error("page_table [batch, max_pages] and seq_len [batch] are needed");
    }
    int32_t* t() const { return table->mutable_data_ptr<int32_t>(); }
    int32_t* l() const { return len->mutable_data_ptr<int32_t>(); }
    int32_t* r() const { return count->mutable_data_ptr<int32_t>(); }
};

// Caches [num_pages, ...] as the library's arrays.
struct CacheArrays {
    std::vector<void*> ptrs;
    std::vector<size_t> sizes;

    CacheArrays(Call& c, PyObject* list, int64_t pages) {
        PyObject* seq = PySequence_Fast(list, "caches must be a sequence of tensors");
        if (!seq) throw python_error();
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
        try {
            ptrs.reserve(n);
            sizes.reserve(n);
            for (Py_ssize_t i = 0; i < n; ++i) {
                const at::Tensor& t = c.dense(PySequence_Fast_GET_ITEM(seq, i), "a cache");
                if (t.dim() < 1 || t.size(0) != pages) value_error("caches must be [num_pages, ...]");
                ptrs.push_back(t.mutable_data_ptr());
                sizes.push_back(pages ? t.nbytes() / (size_t)pages : 0);
            }
        } catch (...) {
            Py_DECREF(seq);
            throw;
        }
        Py_DECREF(seq);
    }
    int n() const { return as_int((int64_t)ptrs.size()); }
};

int same_length(const at::Tensor& a, const at::Tensor& b) {
    if (a.size(0) != b.size(0)) value_error("lists must be [n], of one length");
    return as_int(a.size(0));
}

// page_table, seq_len, ref_count, seqs, add, page_size
PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 6);
    Call c;
    const Books b(c, a[0], a[1], a[2]);
    const at::Tensor &seqs = c.dense_i32(a[3], "seqs", 1), &add = c.dense_i32(a[4], "add", 1);
    const int n = same_length(seqs, add);
    if (!succeeded(kv_pages_extend(b.t(), b.batch, b.width, integer(a[5]), b.l(), b.r(), b.pages,
                                   seqs.const_data_ptr<int32_t>(), add.const_data_ptr<int32_t>(), n, c.stream()),
                   "kv_pages_extend"))
        return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// page_table, seq_len, ref_count, seqs, page_size
PyObject* free_(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 5);
    Call c;
    const Books b(c, a[0], a[1], a[2]);
    const at::Tensor& seqs = c.dense_i32(a[3], "seqs", 1);
    if (!succeeded(kv_pages_free(b.t(), b.batch, b.width, integer(a[4]), b.l(), b.r(), b.pages,
                                 seqs.const_data_ptr<int32_t>(), as_int(seqs.size(0)), c.stream()),
                   "kv_pages_free"))
        return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// page_table, seq_len, ref_count, parents, children, page_size, caches, workspace
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 8);
    Call c;
    const Books b(c, a[0], a[1], a[2]);
    const at::Tensor &parents = c.dense_i32(a[3], "parents", 1), &children = c.dense_i32(a[4], "children", 1);
    const int n = same_length(parents, children);
    const CacheArrays caches(c, a[6], b.pages);
    const at::Tensor ws = scratch(c, a[7], kv_pages_fork_workspace_size(n), parents.options());
    if (!succeeded(kv_pages_fork(b.t(), b.batch, b.width, integer(a[5]), b.l(), b.r(), b.pages,
                                 parents.const_data_ptr<int32_t>(), children.const_data_ptr<int32_t>(), n,
                                 caches.ptrs.data(), caches.sizes.data(), caches.n(), ws.mutable_data_ptr(), ws.nbytes(),
                                 c.stream()),
                   "kv_pages_fork"))
        return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// caches, src, dst, num_pages
PyObject* copy(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 4);
    Call c;
    const at::Tensor &src = c.dense_i32(a[1], "src", 1), &dst = c.dense_i32(a[2], "dst", 1);
    const int n = same_length(src, dst), pages = integer(a[3]);
    const CacheArrays caches(c, a[0], pages);
    if (!succeeded(kv_pages_copy(caches.ptrs.data(), caches.sizes.data(), caches.n(), pages, src.const_data_ptr<int32_t>(),
                                 dst.const_data_ptr<int32_t>(), n, c.stream()),
                   "kv_pages_copy"))
        return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// page_table, ref_count, caches, table_out, ref_out, workspace
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    arity(n_args, 6);
    Call c;
    const at::Tensor &table = c.dense_i32(a[0], "page_table", 2), &count = c.dense_i32(a[1], "ref_count", 1);
    const at::Tensor table_out = output(c, a[3], "table_out", table.sizes(), table.options());
    const at::Tensor ref_out = output(c, a[4], "ref_out", count.sizes(), count.options());
    const int pages = as_int(count.size(0));
    const CacheArrays caches(c, a[2], pages);
    const at::Tensor ws = scratch(c, a[5], kv_pages_compact_workspace_size(pages), count.options());
    if (!succeeded(kv_pages_compact(table.const_data_ptr<int32_t>(), as_int(table.size(0)), as_int(table.size(1)),
                                    count.const_data_ptr<int32_t>(), pages, caches.ptrs.data(), caches.sizes.data(),
                                    caches.n(), table_out.mutable_data_ptr<int32_t>(), ref_out.mutable_data_ptr<int32_t>(),
                                    ws.mutable_data_ptr(), ws.nbytes(), c.stream()),
                   "kv_pages_compact"))
        return nullptr;
    return pair(table_out, ref_out);
    END_HANDLE_TH_ERRORS
}

// The class of the errors to raise.
PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

#define DSA_FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DSA_FAST("append", append), DSA_FAST("decode", decode),   DSA_FAST("prompt", prompt),
                         DSA_FAST("extend", extend), DSA_FAST("free", free_),      DSA_FAST("fork", fork),
                         DSA_FAST("copy", copy),     DSA_FAST("compact", compact), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gqa", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gqa(void) { return PyModule_Create(&module); }
