// fd_binding.cpp -- the Python binding's compiled half for the prompt, shared-
// prefix, page and append calls: the checks of their tensors, the allocation of
// outputs and workspace on the stream that uses them, and the call of the C
// entry point.  The same steps in Python cost 12-15 us a call beside 2-6 us of
// GPU time (a decode step's page assignment: 18.9 us a call in Python, 6.4 us
// here; four short prompts: 19.8 and 5.2 us).  libfd.so itself stays free of
// torch: this module opens it at run time.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <dlfcn.h>

#include <climits>
#include <cmath>
#include <optional>

#include "fd.h"

namespace {

using at::Tensor;

// The entry points, from the library that bind() opened.
struct Library {
    decltype(&fd_prefill_workspace_size) prefill_workspace_size;
    decltype(&fd_prefill_packed) prefill_packed;
    decltype(&fd_prefill_paged) prefill_paged;
    decltype(&fd_shared_prefix_workspace_size) shared_workspace_size;
    decltype(&fd_decode_paged_shared_prefix) paged_shared;
    decltype(&fd_decode_dense_shared_prefix) dense_shared;
    decltype(&fd_assign_pages) assign_pages;
    decltype(&fd_append_kv_paged) append;
    decltype(&fd_append_kv_paged_fp8) append_fp8;
};
Library lib = {};
PyObject* fd_error = nullptr;  // the class FdError(status, where)

// ---- arguments ----------------------------------------------------------------

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

int integer(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, name, " is out of range");
    return (int)v;
}

int size_of(int64_t n, const char* name) {
    TORCH_CHECK_VALUE(n <= INT_MAX, name, " is too large");
    return (int)n;
}

bool truth(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw python_error();
    return r != 0;
}

float scale_of(PyObject* o, int64_t d) {
    if (o == Py_None) return (float)(1.0 / std::sqrt((double)d));
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

void on_device(const Tensor& t, const char* name, c10::Device dev) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.device() == dev, name, " is on ", t.device(), ", expected ", dev, " (the first tensor's device)");
}

// A contiguous tensor of the given type on `dev`; its shape where one is given.
const Tensor& check(const Tensor& t, const char* name, c10::Device dev, at::ScalarType type,
                    std::optional<at::IntArrayRef> shape = std::nullopt) {
    on_device(t, name, dev);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
    if (shape) TORCH_CHECK_VALUE(t.sizes() == *shape, name, " must have shape ", *shape, ", got ", t.sizes());
    return t;
}

// [T, H, d] bf16 whose tokens may lie further apart than H * d elements (a slice
// of a fused projection); H, d < 0: any.  Returns the token stride in elements.
int64_t check_tokens(const Tensor& t, const char* name, c10::Device dev, int64_t H = -1, int64_t d = -1) {
    on_device(t, name, dev);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16, name, " must be ", at::kBFloat16, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == 3 && (H < 0 || t.size(1) == H) && (d < 0 || t.size(2) == d), name,
                      " must be [tokens, heads, d] with the heads and d of the other tensors, got ", t.sizes());
    const int64_t row = t.size(1) * t.size(2);
    if (t.is_contiguous() || t.numel() == 0) return row;
    TORCH_CHECK_VALUE((t.size(2) == 1 || t.stride(2) == 1) && (t.size(1) == 1 || t.stride(1) == t.size(2)), name,
                      ": the heads of a token must be contiguous");
    if (t.size(0) == 1) return row;
    TORCH_CHECK_VALUE(t.stride(0) >= row, name, ": tokens must not overlap");
    return t.stride(0);
}

// Offsets [B + 1]: returns B.
int check_offsets(const Tensor& t, const char* name, c10::Device dev) {
    check(t, name, dev, at::kInt);
    TORCH_CHECK_VALUE(t.dim() == 1 && t.numel() >= 1, name, " must be [B + 1]");
    return size_of(t.numel() - 1, name);
}

int check_table(const Tensor& t, int B, c10::Device dev) {
    check(t, "page_table", dev, at::kInt);
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == B, "page_table must be [B, max_pages]");
    return size_of(t.size(1), "page_table");
}

void check_pool(const Tensor& k, const Tensor& v, int64_t d, c10::Device dev) {
    check(k, "k_pages", dev, at::kBFloat16);
    TORCH_CHECK_VALUE(k.dim() == 4 && k.size(3) == d, "k_pages must be [P, Hkv, page, d]");
    check(v, "v_pages", dev, at::kBFloat16, k.sizes());
}

int check_num_pages(PyObject* o, const Tensor& pool) {
    const int n = integer(o, "num_pages");
    TORCH_CHECK_VALUE(n >= 0 && n <= pool.size(0), "num_pages must be within the pool");
    return n;
}

// ---- device, stream, outputs ------------------------------------------------------

// Makes the tensors' device and the call's stream current, so that what is
// allocated belongs to that stream.
struct Place {
    c10::cuda::CUDAGuard device;
    std::optional<c10::cuda::CUDAStreamGuard> given;
    void* stream;

    Place(c10::Device dev, PyObject* o) : device(dev) {
        if (o != Py_None) {
            THPObjectPtr where(PyObject_GetAttrString(o, "device"));
            if (!where) throw python_error();
            THPObjectPtr index(PyObject_GetAttrString(where.get(), "index"));
            THPObjectPtr handle(PyObject_GetAttrString(o, "cuda_stream"));
            if (!index || !handle) throw python_error();
            const int at = integer(index.get(), "stream");
            TORCH_CHECK_VALUE(at == dev.index(), "stream is on cuda:", at, ", the tensors on ", dev);
            void* const h = PyLong_AsVoidPtr(handle.get());
            if (PyErr_Occurred()) throw python_error();
            // the default stream has handle 0, which is no external stream
            given.emplace(h ? c10::cuda::getStreamFromExternal((cudaStream_t)h, dev.index())
                            : c10::cuda::getDefaultCUDAStream(dev.index()));
        }
        stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
};

c10::Device first_device(PyObject* o, const char* call) {
    TORCH_CHECK_VALUE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), call,
                      ": the first argument must be a CUDA tensor");
    return THPVariable_Unpack(o).device();
}

// On the current stream, like at::empty, without its way through the dispatcher.
Tensor fresh_tensor(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
    return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}

struct Outputs {
    Tensor out, lse;  // lse may be undefined: none wanted
    int code;

    Outputs(int64_t T, int64_t Hq, int64_t d, PyObject* o, PyObject* l, int out_code, bool want_lse, c10::Device dev)
        : code(out_code) {
        const at::ScalarType type = out_code == FD_OUT_BF16 ? at::kBFloat16 : at::kFloat;
        if (o == Py_None) out = fresh_tensor({T, Hq, d}, type, dev);
        else out = check(tensor(o, "out"), "out", dev, type, {{T, Hq, d}});
        if (l != Py_None) lse = check(tensor(l, "lse"), "lse", dev, at::kFloat, {{T, Hq}});
        else if (want_lse) lse = fresh_tensor({T, Hq}, at::kFloat, dev);
    }
    float* lse_data() const { return lse.defined() ? lse.mutable_data_ptr<float>() : nullptr; }
};

struct Workspace {
    Tensor t;
    Workspace(size_t bytes, PyObject* o, c10::Device dev) {
        if (o != Py_None) {
            t = tensor(o, "workspace");
            on_device(t, "workspace", dev);
            TORCH_CHECK_VALUE(t.is_contiguous(), "workspace must be contiguous");
            TORCH_CHECK_VALUE((size_t)t.nbytes() >= bytes, "workspace too small");
        } else if (bytes > 0) {
            t = fresh_tensor({(int64_t)bytes}, at::kByte, dev);
        }
    }
    void* data() const { return t.defined() ? t.mutable_data_ptr() : nullptr; }
    size_t bytes() const { return t.defined() ? t.nbytes() : 0; }
};

void expect(int status, const char* call) {
    if (status == FD_OK) return;
    TORCH_CHECK_VALUE(fd_error, call, " failed");
    THPObjectPtr e(PyObject_CallFunction(fd_error, "is", status, call));
    if (e) PyErr_SetObject(fd_error, e.get());
    throw python_error();
}

PyObject* none() {
    Py_INCREF(Py_None);
    return Py_None;
}

PyObject* pair(const Outputs& o) {
    THPObjectPtr t(PyTuple_New(2));
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t.get(), 0, THPVariable_Wrap(o.out));
    PyTuple_SET_ITEM(t.get(), 1, o.lse.defined() ? THPVariable_Wrap(o.lse) : none());
    return t.release();
}

// The arguments themselves, as a tuple.
PyObject* same(std::initializer_list<PyObject*> items) {
    THPObjectPtr t(PyTuple_New((Py_ssize_t)items.size()));
    if (!t) throw python_error();
    Py_ssize_t i = 0;
    for (PyObject* o : items) {
        Py_INCREF(o);
        PyTuple_SET_ITEM(t.get(), i++, o);
    }
    return t.release();
}

void ready(Py_ssize_t got, Py_ssize_t want) {
    TORCH_CHECK(lib.prefill_packed, "libfd.so is not bound");
    TORCH_CHECK(got == want, "expected ", want, " arguments, got ", got);
}

// ---- the calls ----------------------------------------------------------------------

// (q, k, v, cu_seqlens_q, cu_seqlens_k, scale, causal, num_splits, out, lse, out_code, want_lse, workspace, stream)
PyObject* prefill_packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 14);
    const c10::Device dev = first_device(a[0], "fd_prefill_packed");
    const Place place(dev, a[13]);
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int64_t qs = check_tokens(q, "q", dev);
    const int64_t Tq = q.size(0), Hq = q.size(1), d = q.size(2);
    const int64_t ks = check_tokens(k, "k", dev, -1, d);
    const int64_t Tk = k.size(0), Hkv = k.size(1);
    const int64_t vs = check_tokens(v, "v", dev, Hkv, d);
    TORCH_CHECK_VALUE(v.size(0) == Tk, "k and v must have the same number of tokens");
    const Tensor& cq = tensor(a[3], "cu_seqlens_q");
    const int B = check_offsets(cq, "cu_seqlens_q", dev);
    const Tensor& ck = a[4] == Py_None ? cq : tensor(a[4], "cu_seqlens_k");
    if (a[4] != Py_None) check(ck, "cu_seqlens_k", dev, at::kInt, {{(int64_t)B + 1}});
    const int tq = size_of(Tq, "q"), tk = size_of(Tk, "k"), splits = integer(a[7], "num_splits");
    const Outputs o(Tq, Hq, d, a[8], a[9], integer(a[10], "out_dtype"), truth(a[11]), dev);
    const Workspace ws(lib.prefill_workspace_size(B, tq, (int)Hq, (int)Hkv, tk, (int)d, splits), a[12], dev);
    expect(lib.prefill_packed(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), qs, ks, vs,
                              cq.const_data_ptr<int>(), ck.const_data_ptr<int>(), B, tq, tk, (int)Hq, (int)Hkv, (int)d,
                              scale_of(a[5], d), truth(a[6]), splits, o.out.mutable_data_ptr(), o.code, o.lse_data(),
                              ws.data(), ws.bytes(), place.stream),
           "fd_prefill_packed");
    return pair(o);
    END_HANDLE_TH_ERRORS
}

// (q, k_pages, v_pages, page_table, num_pages, cu_seqlens_q, seq_lens, scale, causal, num_splits, out, lse, out_code,
//  want_lse, workspace, stream)
PyObject* prefill_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 16);
    const c10::Device dev = first_device(a[0], "fd_prefill_paged");
    const Place place(dev, a[15]);
    const Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
    const int64_t qs = check_tokens(q, "q", dev);
    const int64_t Tq = q.size(0), Hq = q.size(1), d = q.size(2);
    check_pool(kp, vp, d, dev);
    const int num_pages = check_num_pages(a[4], kp);
    const Tensor &cq = tensor(a[5], "cu_seqlens_q"), &table = tensor(a[3], "page_table");
    const int B = check_offsets(cq, "cu_seqlens_q", dev);
    const int max_pages = check_table(table, B, dev);
    const Tensor& lens = check(tensor(a[6], "seq_lens"), "seq_lens", dev, at::kInt, {{(int64_t)B}});
    const int tq = size_of(Tq, "q"), splits = integer(a[9], "num_splits"), Hkv = (int)kp.size(1);
    const int page = (int)kp.size(2);
    const Outputs o(Tq, Hq, d, a[10], a[11], integer(a[12], "out_dtype"), truth(a[13]), dev);
    const int64_t max_k = (int64_t)max_pages * page;
    const Workspace ws(max_k > INT_MAX ? 0 : lib.prefill_workspace_size(B, tq, (int)Hq, Hkv, (int)max_k, (int)d, splits),
                       a[14], dev);
    expect(lib.prefill_paged(q.const_data_ptr(), kp.const_data_ptr(), vp.const_data_ptr(), qs,
                             table.const_data_ptr<int>(), max_pages, num_pages, cq.const_data_ptr<int>(),
                             lens.const_data_ptr<int>(), page, B, tq, (int)Hq, Hkv, (int)d, scale_of(a[7], d),
                             truth(a[8]), splits, o.out.mutable_data_ptr(), o.code, o.lse_data(), ws.data(), ws.bytes(),
                             place.stream),
           "fd_prefill_paged");
    return pair(o);
    END_HANDLE_TH_ERRORS
}

const Tensor& check_queries(PyObject* o, c10::Device dev) {
    const Tensor& q = check(tensor(o, "q"), "q", dev, at::kBFloat16);
    TORCH_CHECK_VALUE(q.dim() == 3, "q must be [B, Hq, d]");
    size_of(q.size(0), "q");
    return q;
}

// (q, k_pages, v_pages, prefix_table, page_table, num_pages, seq_lens, scale, num_splits, out, lse, out_code, want_lse,
//  workspace, stream)
PyObject* paged_shared_prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 15);
    const c10::Device dev = first_device(a[0], "fd_decode_paged_shared_prefix");
    const Place place(dev, a[14]);
    const Tensor& q = check_queries(a[0], dev);
    const int B = (int)q.size(0), Hq = (int)q.size(1), d = (int)q.size(2);
    const Tensor &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
    check_pool(kp, vp, d, dev);
    const int num_pages = check_num_pages(a[5], kp), Hkv = (int)kp.size(1), page = (int)kp.size(2);
    const Tensor& prefix = check(tensor(a[3], "prefix_table"), "prefix_table", dev, at::kInt);
    TORCH_CHECK_VALUE(prefix.dim() == 1, "prefix_table must be [prefix_pages]");
    const Tensor& table = tensor(a[4], "page_table");
    const int max_pages = check_table(table, B, dev);
    TORCH_CHECK_VALUE(prefix.numel() <= max_pages, "prefix_table must be no longer than a row of page_table");
    const int shared = (int)prefix.numel();
    const Tensor& lens = check(tensor(a[6], "seq_lens"), "seq_lens", dev, at::kInt, {{(int64_t)B}});
    const int splits = integer(a[8], "num_splits");
    const Outputs o(B, Hq, d, a[9], a[10], integer(a[11], "out_dtype"), truth(a[12]), dev);
    const bool fits = (int64_t)max_pages * page <= INT_MAX;
    const Workspace ws(
        fits ? lib.shared_workspace_size(B, Hq, Hkv, shared * page, (max_pages - shared) * page, d, splits) : 0, a[13],
        dev);
    expect(lib.paged_shared(q.const_data_ptr(), kp.const_data_ptr(), vp.const_data_ptr(), prefix.const_data_ptr<int>(),
                            shared, table.const_data_ptr<int>(), max_pages, num_pages, lens.const_data_ptr<int>(), page,
                            B, Hq, Hkv, d, scale_of(a[7], d), splits, o.out.mutable_data_ptr(), o.code, o.lse_data(),
                            ws.data(), ws.bytes(), place.stream),
           "fd_decode_paged_shared_prefix");
    return pair(o);
    END_HANDLE_TH_ERRORS
}

// (q, k_prefix, v_prefix, k, v, seq_lens, scale, num_splits, out, lse, out_code, want_lse, workspace, stream)
PyObject* dense_shared_prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 14);
    const c10::Device dev = first_device(a[0], "fd_decode_dense_shared_prefix");
    const Place place(dev, a[13]);
    const Tensor& q = check_queries(a[0], dev);
    const int B = (int)q.size(0), Hq = (int)q.size(1), d = (int)q.size(2);
    const Tensor& kp = check(tensor(a[1], "k_prefix"), "k_prefix", dev, at::kBFloat16);
    TORCH_CHECK_VALUE(kp.dim() == 3 && kp.size(2) == d, "k_prefix must be [Hkv, P, d]");
    const Tensor& vp = check(tensor(a[2], "v_prefix"), "v_prefix", dev, at::kBFloat16, kp.sizes());
    const int Hkv = size_of(kp.size(0), "k_prefix"), P = size_of(kp.size(1), "k_prefix");
    const Tensor& k = check(tensor(a[3], "k"), "k", dev, at::kBFloat16);
    TORCH_CHECK_VALUE(k.dim() == 4 && k.size(0) == B && k.size(1) == Hkv && k.size(3) == d,
                      "k must be [B, Hkv, L_max, d]");
    const int L = size_of(k.size(2), "k");
    const Tensor& v = check(tensor(a[4], "v"), "v", dev, at::kBFloat16, k.sizes());
    const int* lens = nullptr;
    if (a[5] != Py_None)
        lens = check(tensor(a[5], "seq_lens"), "seq_lens", dev, at::kInt, {{(int64_t)B}}).const_data_ptr<int>();
    const int splits = integer(a[7], "num_splits");
    const Outputs o(B, Hq, d, a[8], a[9], integer(a[10], "out_dtype"), truth(a[11]), dev);
    const Workspace ws(lib.shared_workspace_size(B, Hq, Hkv, P, L, d, splits), a[12], dev);
    expect(lib.dense_shared(q.const_data_ptr(), kp.const_data_ptr(), vp.const_data_ptr(), P, k.const_data_ptr(),
                            v.const_data_ptr(), lens, B, Hq, Hkv, L, d, scale_of(a[6], d), splits,
                            o.out.mutable_data_ptr(), o.code, o.lse_data(), ws.data(), ws.bytes(), place.stream),
           "fd_decode_dense_shared_prefix");
    return pair(o);
    END_HANDLE_TH_ERRORS
}

Tensor ints_out(PyObject* o, const char* name, int64_t n, c10::Device dev) {
    if (o == Py_None) return fresh_tensor({n}, at::kInt, dev);
    return check(tensor(o, name), name, dev, at::kInt, {{n}});
}

// (page_table, cached_lens, new_lens, free_pages, total_new, free_head, page_size, seq_lens, cu_seqlens, slots,
//  free_head_out, stream)
PyObject* assign_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 12);
    const c10::Device dev = first_device(a[0], "fd_assign_pages");
    const Place place(dev, a[11]);
    const Tensor& table = check(tensor(a[0], "page_table"), "page_table", dev, at::kInt);
    TORCH_CHECK_VALUE(table.dim() == 2, "page_table must be [B, max_pages]");
    const int B = size_of(table.size(0), "page_table"), max_pages = size_of(table.size(1), "page_table");
    const Tensor& cached = check(tensor(a[1], "cached_lens"), "cached_lens", dev, at::kInt, {{(int64_t)B}});
    const Tensor& fresh = check(tensor(a[2], "new_lens"), "new_lens", dev, at::kInt, {{(int64_t)B}});
    const Tensor& free = check(tensor(a[3], "free_pages"), "free_pages", dev, at::kInt);
    TORCH_CHECK_VALUE(free.dim() == 1, "free_pages must be [F]");
    const int total = integer(a[4], "total_new");
    TORCH_CHECK_VALUE(total >= 0, "total_new must be >= 0");
    const int* head = nullptr;
    if (a[5] != Py_None)
        head = check(tensor(a[5], "free_head"), "free_head", dev, at::kInt, {{(int64_t)1}}).const_data_ptr<int>();
    const int page = integer(a[6], "page_size");
    const Tensor lens = ints_out(a[7], "seq_lens", B, dev), cu = ints_out(a[8], "cu_seqlens", (int64_t)B + 1, dev);
    const Tensor slots = a[9] == Py_None ? fresh_tensor({(int64_t)total}, at::kLong, dev)
                                         : check(tensor(a[9], "slots"), "slots", dev, at::kLong, {{(int64_t)total}});
    const Tensor head_out = ints_out(a[10], "free_head_out", 1, dev);
    expect(lib.assign_pages(cached.const_data_ptr<int>(), fresh.const_data_ptr<int>(), B, table.mutable_data_ptr<int>(),
                            max_pages, page, free.const_data_ptr<int>(), size_of(free.numel(), "free_pages"), head,
                            total, lens.mutable_data_ptr<int>(), cu.mutable_data_ptr<int>(),
                            slots.mutable_data_ptr<int64_t>(), head_out.mutable_data_ptr<int>(), place.stream),
           "fd_assign_pages");
    THPObjectPtr t(PyTuple_New(4));
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t.get(), 0, THPVariable_Wrap(lens));
    PyTuple_SET_ITEM(t.get(), 1, THPVariable_Wrap(cu));
    PyTuple_SET_ITEM(t.get(), 2, THPVariable_Wrap(slots));
    PyTuple_SET_ITEM(t.get(), 3, THPVariable_Wrap(head_out));
    return t.release();
    END_HANDLE_TH_ERRORS
}

struct NewRows {
    int64_t ks, vs;
    int T, Hkv, d;
    const int64_t* slots;
    NewRows(const Tensor& k, const Tensor& v, PyObject* s, c10::Device dev) {
        ks = check_tokens(k, "k", dev);
        vs = check_tokens(v, "v", dev, k.size(1), k.size(2));
        TORCH_CHECK_VALUE(v.size(0) == k.size(0), "k and v must have the same number of tokens");
        T = size_of(k.size(0), "k");
        Hkv = size_of(k.size(1), "k");
        d = size_of(k.size(2), "k");
        slots = check(tensor(s, "slots"), "slots", dev, at::kLong, {{(int64_t)T}}).const_data_ptr<int64_t>();
    }
};

// (k, v, slots, k_pages, v_pages, stream)
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 6);
    const c10::Device dev = first_device(a[0], "fd_append_kv_paged");
    const Place place(dev, a[5]);
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const NewRows r(k, v, a[2], dev);
    const Tensor &kp = tensor(a[3], "k_pages"), &vp = tensor(a[4], "v_pages");
    check_pool(kp, vp, r.d, dev);
    TORCH_CHECK_VALUE(kp.size(1) == r.Hkv, "k_pages must have the heads of k");
    expect(lib.append(k.const_data_ptr(), v.const_data_ptr(), r.ks, r.vs, r.slots, r.T, r.Hkv, r.d,
                      kp.mutable_data_ptr(), vp.mutable_data_ptr(), size_of(kp.size(0), "k_pages"), (int)kp.size(2),
                      place.stream),
           "fd_append_kv_paged");
    return same({a[3], a[4]});
    END_HANDLE_TH_ERRORS
}

// (k, v, slots, k_pages, k_page_scales, v_pages, v_page_scales, stream)
PyObject* append_kv_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 8);
    const c10::Device dev = first_device(a[0], "fd_append_kv_paged_fp8");
    const Place place(dev, a[7]);
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const NewRows r(k, v, a[2], dev);
    const Tensor& kp = check(tensor(a[3], "k_pages"), "k_pages", dev, at::kByte);
    TORCH_CHECK_VALUE(kp.dim() == 4 && kp.size(1) == r.Hkv && kp.size(3) == r.d, "k_pages must be [P, Hkv, page, d]");
    const Tensor& vp = check(tensor(a[5], "v_pages"), "v_pages", dev, at::kByte, kp.sizes());
    const at::IntArrayRef rows = kp.sizes().slice(0, 3);
    const Tensor& ks = check(tensor(a[4], "k_page_scales"), "k_page_scales", dev, at::kFloat, rows);
    const Tensor& vs = check(tensor(a[6], "v_page_scales"), "v_page_scales", dev, at::kFloat, rows);
    expect(lib.append_fp8(k.const_data_ptr(), v.const_data_ptr(), r.ks, r.vs, r.slots, r.T, r.Hkv, r.d,
                          kp.mutable_data_ptr<uint8_t>(), ks.mutable_data_ptr<float>(), vp.mutable_data_ptr<uint8_t>(),
                          vs.mutable_data_ptr<float>(), size_of(kp.size(0), "k_pages"), (int)kp.size(2), place.stream),
           "fd_append_kv_paged_fp8");
    return same({a[3], a[4], a[5], a[6]});
    END_HANDLE_TH_ERRORS
}

// bind(path of libfd.so, FdError)
PyObject* bind(PyObject*, PyObject* args) {
    const char* path;
    PyObject* error;
    if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_ImportError, dlerror());
        return nullptr;
    }
    Library l = {};
    const auto get = [&](auto& f, const char* name) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
        return f != nullptr;
    };
    if (!(get(l.prefill_workspace_size, "fd_prefill_workspace_size") && get(l.prefill_packed, "fd_prefill_packed") &&
          get(l.prefill_paged, "fd_prefill_paged") &&
          get(l.shared_workspace_size, "fd_shared_prefix_workspace_size") &&
          get(l.paged_shared, "fd_decode_paged_shared_prefix") &&
          get(l.dense_shared, "fd_decode_dense_shared_prefix") && get(l.assign_pages, "fd_assign_pages") &&
          get(l.append, "fd_append_kv_paged") && get(l.append_fp8, "fd_append_kv_paged_fp8"))) {
        PyErr_Format(PyExc_ImportError, "%s lacks an entry point of this binding", path);
        return nullptr;
    }
    lib = l;
    Py_INCREF(error);
    Py_XSETREF(fd_error, error);
    Py_RETURN_NONE;
}

#define FD_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FD_FAST(prefill_packed),
                         FD_FAST(prefill_paged),
                         FD_FAST(paged_shared_prefix),
                         FD_FAST(dense_shared_prefix),
                         FD_FAST(assign_pages),
                         FD_FAST(append_kv),
                         FD_FAST(append_kv_fp8),
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "compiled half of the binding", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
