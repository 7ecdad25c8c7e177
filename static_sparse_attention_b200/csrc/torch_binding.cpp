// torch_binding.cpp -- the tensor side of the operators around the attention:
// checks torch tensors, allocates outputs from torch's caching allocator and calls
// the library's C entry points (include/radattn.h).  A CPython extension
// (_torch_binding.so): a call of a few microseconds cannot wait for the same checks
// in Python (17 us for the norm and rotation of a small clip against 6 here).
//
// It is not linked to the library: bind() receives the entry points' addresses from
// the package, which has loaded the release or the debug build.  A function returns
// its outputs, or the C call's status where that is not RA_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "radattn.h"

namespace {

decltype(&ra_qk_norm_rope) f_qk_norm_rope;
decltype(&ra_qk_norm_rope_bwd_workspace_bytes) f_qk_norm_rope_bwd_workspace_bytes;
decltype(&ra_qk_norm_rope_bwd) f_qk_norm_rope_bwd;
decltype(&ra_cache8_append) f_cache8_append;
decltype(&ra_cache8_attention_workspace_bytes) f_cache8_attention_workspace_bytes;
decltype(&ra_cache8_attention) f_cache8_attention;
decltype(&ra_cache8_attention_check) f_cache8_attention_check;

constexpr int64_t CACHE8_BLOCK = 64;

// A tensor argument, or null for None.
const at::Tensor* tensor_or_none(PyObject* o, const char* name)
{
    if (o == Py_None)
        return nullptr;
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    const at::Tensor* t = tensor_or_none(o, name);
    TORCH_CHECK_VALUE(t, name, " must be a tensor");
    return *t;
}

int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

int int_of(PyObject* o, const char* name)
{
    const int64_t v = integer(o);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " is out of range");
    return static_cast<int>(v);
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

// A size that the C calls take as an int.
int size_of(int64_t n, const char* what)
{
    TORCH_CHECK_VALUE(n <= INT32_MAX, what, " is too large (", n, ")");
    return static_cast<int>(n);
}

// The device and stream of a call: the inputs' device, which has to be the current
// one, and the given stream's handle or the current stream; new tensors belong to it.
struct Where {
    c10::DeviceIndex dev;
    cudaStream_t stream;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
};

void where(Where& w, const at::Tensor& x, const char* name, PyObject* stream)
{
    TORCH_CHECK_VALUE(x.is_cuda() && x.get_device() == c10::cuda::current_device(), name,
                      " must be on the current CUDA device");
    w.dev = static_cast<c10::DeviceIndex>(x.get_device());
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(w.dev);
    w.stream = current.stream();
    if (stream != Py_None) {
        const cudaStream_t given = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(stream));
        if (PyErr_Occurred())
            throw python_error();
        if (given != w.stream) {
            w.guard.emplace(given ? c10::cuda::getStreamFromExternal(given, w.dev)
                                  : c10::cuda::getDefaultCUDAStream(w.dev));
            w.stream = given;
        }
    }
}

bool is(const at::Tensor& t, at::ScalarType type, const Where& w)
{
    return t.scalar_type() == type && t.is_cuda() && t.get_device() == w.dev;
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const Where& w)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::DeviceType::CUDA, w.dev));
}

// A strided [B, n, heads, d] input and its norm weight.
ra_head_rows rows_of(const at::Tensor& x, const at::Tensor* weight, const char* name, const Where& w)
{
    TORCH_CHECK_VALUE(is(x, at::kBFloat16, w) && x.stride(3) == 1, name,
                      " must be a bf16 tensor [B, n, H, d] with contiguous channels on the current CUDA device");
    ra_head_rows r{x.const_data_ptr(), x.stride(0), x.stride(1), x.stride(2), size_of(x.size(2), "H"), 0, nullptr};
    if (weight) {
        r.weight_fp32 = weight->scalar_type() == at::kFloat;
        TORCH_CHECK_VALUE((r.weight_fp32 || weight->scalar_type() == at::kBFloat16) && weight->is_cuda() &&
                              weight->get_device() == w.dev && weight->dim() == 1 && weight->size(0) == x.size(3) &&
                              weight->is_contiguous(),
                          "the weight of ", name, " must be a contiguous bf16 or fp32 tensor [d] on its device");
        r.weight = weight->const_data_ptr();
    }
    return r;
}

// The position tables; returns null for None.
const ra_rope* rope_of(ra_rope& r, PyObject* o, const Where& w)
{
    if (o == Py_None)
        return nullptr;
    TORCH_CHECK_VALUE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 3, "rope must be a tuple of the tables of three axes");
    const float* at[3];
    int length[3], pairs[3];
    for (int i = 0; i < 3; ++i) {
        const at::Tensor& t = tensor(PyTuple_GET_ITEM(o, i), "a rope table");
        TORCH_CHECK_VALUE(is(t, at::kFloat, w) && t.dim() == 3 && t.size(2) == 2 && t.is_contiguous(),
                          "rope tables must be contiguous fp32 tensors [positions, pairs, 2] on the inputs' device");
        at[i] = static_cast<const float*>(t.const_data_ptr());
        length[i] = size_of(t.size(0), "a rope table");
        pairs[i] = size_of(t.size(1), "a rope table");
    }
    r = ra_rope{at[0], at[1], at[2], length[0], length[1], length[2], pairs[0], pairs[1], pairs[2]};
    return &r;
}

// A contiguous output of that shape and type: the caller's, checked, or a new one.
at::Tensor output(const at::Tensor* given, const char* name, at::IntArrayRef sizes, at::ScalarType type, const Where& w)
{
    if (!given)
        return empty(sizes, type, w);
    TORCH_CHECK_VALUE(is(*given, type, w) && given->sizes() == sizes && given->is_contiguous(), name,
                      " must be a contiguous ", c10::toString(type), " tensor ", sizes, " on the inputs' device");
    return *given;
}

// The caller's workspace, checked, or a new one (undefined when none is needed).
at::Tensor workspace_of(const at::Tensor* given, size_t need, const Where& w)
{
    if (!given)
        return need ? empty({static_cast<int64_t>(need)}, at::kByte, w) : at::Tensor();
    TORCH_CHECK_VALUE(given->is_cuda() && given->get_device() == w.dev && given->is_contiguous() &&
                          given->nbytes() >= need,
                      "workspace must be a contiguous tensor of at least ", need, " bytes on the inputs' device");
    return *given;
}

void* address(const at::Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }

PyObject* wrap(const at::Tensor& t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* tuple_of(std::initializer_list<at::Tensor> tensors)
{
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
    if (!r)
        throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor& t : tensors)
        PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

void arguments(Py_ssize_t n, Py_ssize_t want)
{
    TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

void check_qk(const at::Tensor& q, const at::Tensor* k)
{
    TORCH_CHECK_VALUE(q.dim() == 4, "q must be a tensor [B, n, H, d]");
    TORCH_CHECK_VALUE(!k || (k->dim() == 4 && k->size(0) == q.size(0) && k->size(1) == q.size(1) &&
                             k->size(3) == q.size(3)),
                      "k must be a tensor [B, n, Hk, d] with q's B, n and d");
}

// q, k, q_weight, k_weight, rope, frame0, eps, q_out, k_out, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    arguments(n_args, 10);
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor *k = tensor_or_none(a[1], "k"), *qw = tensor_or_none(a[2], "q_weight"),
                     *kw = tensor_or_none(a[3], "k_weight"), *k_given = tensor_or_none(a[8], "k_out");
    Where w;
    where(w, q, "q", a[9]);
    check_qk(q, k);
    TORCH_CHECK_VALUE(k || (!kw && !k_given), "k_weight and k_out need k");
    const int64_t B = q.size(0), n = q.size(1), H = q.size(2), d = q.size(3);
    const ra_head_rows rows_q = rows_of(q, qw, "q", w);
    ra_head_rows rows_k;
    ra_rope table;
    const ra_rope* rope = rope_of(table, a[4], w);
    const at::Tensor q_out = output(tensor_or_none(a[7], "q_out"), "q_out", {B, H, n, d}, at::kBFloat16, w);
    at::Tensor k_out;
    if (k) {
        rows_k = rows_of(*k, kw, "k", w);
        k_out = output(k_given, "k_out", {B, k->size(2), n, d}, at::kBFloat16, w);
    }
    if (n) {
        const ra_status st =
            f_qk_norm_rope(&rows_q, k ? &rows_k : nullptr, address(q_out), address(k_out), size_of(B, "B"),
                           size_of(n, "n"), size_of(d, "d"), rope, int_of(a[5], "frame0"),
                           static_cast<float>(number(a[6])), reinterpret_cast<ra_stream>(w.stream));
        if (st != RA_OK)
            return PyLong_FromLong(st);
    }
    return tuple_of({q_out, k_out});
    END_HANDLE_TH_ERRORS
}

// One tensor's gradients: dx and dweight (the caller's or new ones) and their description.
ra_head_grads grads_of(const at::Tensor& x, const at::Tensor* weight, const at::Tensor& dy, const at::Tensor* dx_given,
                       const at::Tensor* dw_given, const char* name, const Where& w, at::Tensor& dx, at::Tensor& dw)
{
    const int64_t B = x.size(0), n = x.size(1), H = x.size(2), d = x.size(3);
    const int64_t head_major[4] = {B, H, n, d};
    TORCH_CHECK_VALUE(is(dy, at::kBFloat16, w) && dy.sizes() == at::IntArrayRef(head_major) && dy.is_contiguous(), "d",
                      name, "_out must be a contiguous bf16 tensor ", at::IntArrayRef(head_major),
                      " on the inputs' device");
    if (dx_given) {
        TORCH_CHECK_VALUE(is(*dx_given, at::kBFloat16, w) && dx_given->sizes() == x.sizes() && dx_given->stride(3) == 1,
                          "d", name, " must be a bf16 tensor ", x.sizes(),
                          " with contiguous channels on the inputs' device");
        dx = *dx_given;
    } else {
        dx = empty(x.sizes(), at::kBFloat16, w);
    }
    if (weight) {
        TORCH_CHECK_VALUE(!dw_given || (is(*dw_given, at::kFloat, w) && dw_given->dim() == 1 && dw_given->size(0) == d &&
                                        dw_given->is_contiguous()),
                          "d", name, "_weight must be a contiguous fp32 tensor [d] on the inputs' device");
        dw = dw_given ? *dw_given : empty({d}, at::kFloat, w);
    } else {
        TORCH_CHECK_VALUE(!dw_given, "d", name, "_weight needs a weight of ", name);
    }
    return ra_head_grads{dy.const_data_ptr(), address(dx), dx.stride(0), dx.stride(1), dx.stride(2),
                         static_cast<float*>(address(dw))};
}

// q, k, dq_out, dk_out, q_weight, k_weight, rope, frame0, eps, dq, dk, dq_weight, dk_weight, workspace, stream
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    arguments(n_args, 15);
    const at::Tensor &q = tensor(a[0], "q"), &dyq = tensor(a[2], "dq_out");
    const at::Tensor *k = tensor_or_none(a[1], "k"), *dyk = tensor_or_none(a[3], "dk_out"),
                     *qw = tensor_or_none(a[4], "q_weight"), *kw = tensor_or_none(a[5], "k_weight"),
                     *dk_given = tensor_or_none(a[10], "dk"), *dkw_given = tensor_or_none(a[12], "dk_weight");
    Where w;
    where(w, q, "q", a[14]);
    TORCH_CHECK_VALUE(!k == !dyk, "k and dk_out go together");
    check_qk(q, k);
    TORCH_CHECK_VALUE(k || (!kw && !dk_given && !dkw_given), "k_weight, dk and dk_weight need k");
    const int64_t B = q.size(0), n = q.size(1), d = q.size(3);
    ra_rope table;
    const ra_rope* rope = rope_of(table, a[6], w);
    at::Tensor dq, dk, dqw, dkw;
    const ra_head_rows rows_q = rows_of(q, qw, "q", w);
    const ra_head_grads grads_q = grads_of(q, qw, dyq, tensor_or_none(a[9], "dq"), tensor_or_none(a[11], "dq_weight"),
                                           "q", w, dq, dqw);
    ra_head_rows rows_k;
    ra_head_grads grads_k;
    if (k) {
        rows_k = rows_of(*k, kw, "k", w);
        grads_k = grads_of(*k, kw, *dyk, dk_given, dkw_given, "k", w, dk, dkw);
    }
    if (n) {
        const size_t need = qw || kw ? f_qk_norm_rope_bwd_workspace_bytes(size_of(d, "d")) : 0;
        const at::Tensor ws = workspace_of(tensor_or_none(a[13], "workspace"), need, w);
        const ra_status st =
            f_qk_norm_rope_bwd(&rows_q, k ? &rows_k : nullptr, &grads_q, k ? &grads_k : nullptr, size_of(B, "B"),
                               size_of(n, "n"), size_of(d, "d"), rope, int_of(a[7], "frame0"),
                               static_cast<float>(number(a[8])), address(ws), need,
                               reinterpret_cast<ra_stream>(w.stream));
        if (st != RA_OK)
            return PyLong_FromLong(st);
    } else {
        for (at::Tensor* t : {&dqw, &dkw})
            if (t->defined())
                t->zero_();
    }
    return tuple_of({dq, dk, dqw, dkw});
    END_HANDLE_TH_ERRORS
}

struct Ring {
    int64_t B, H, d, s, W;
};

Ring ring_of(const at::Tensor& k8, const at::Tensor& v8, const at::Tensor& ks, const at::Tensor& vs, const Where& w)
{
    TORCH_CHECK_VALUE(k8.dim() == 4 && ks.dim() == 4,
                      "k8 must be [B, H, W * s, d] and k_scale [B, H, W, ceil(s / 64)]");
    Ring r{k8.size(0), k8.size(1), k8.size(3), 0, ks.size(2)};
    r.s = r.W ? k8.size(2) / r.W : 0;
    TORCH_CHECK_VALUE(r.s >= 1 && r.s * r.W == k8.size(2) && ks.size(0) == r.B && ks.size(1) == r.H &&
                          ks.size(3) == (r.s + CACHE8_BLOCK - 1) / CACHE8_BLOCK,
                      "k_scale must be [B, H, W, ceil(s / 64)] for k8 [B, H, W * s, d]");
    for (const at::Tensor* t : {&k8, &v8})
        TORCH_CHECK_VALUE(is(*t, at::kFloat8_e4m3fn, w) && t->sizes() == k8.sizes() && t->is_contiguous(),
                          "k8 and v8 must be contiguous float8_e4m3fn tensors ", k8.sizes(), " on the inputs' device");
    for (const at::Tensor* t : {&ks, &vs})
        TORCH_CHECK_VALUE(is(*t, at::kFloat, w) && t->sizes() == ks.sizes() && t->is_contiguous(),
                          "k_scale and v_scale must be contiguous fp32 tensors ", ks.sizes(), " on the inputs' device");
    return r;
}

// k, v, k8, v8, k_scale, v_scale, frame, k_weight, rope, eps, stream
PyObject* cache8_append(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    arguments(n_args, 11);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &k8 = tensor(a[2], "k8"), &v8 = tensor(a[3], "v8"),
                     &ks = tensor(a[4], "k_scale"), &vs = tensor(a[5], "v_scale");
    Where w;
    where(w, k, "k", a[10]);
    const Ring r = ring_of(k8, v8, ks, vs, w);
    TORCH_CHECK_VALUE(k.dim() == 4 && v.sizes() == k.sizes() && k.size(0) == r.B && k.size(2) == r.H &&
                          k.size(3) == r.d && k.size(1) % r.s == 0,
                      "k and v must have shape [", r.B, ", frames * ", r.s, ", ", r.H, ", ", r.d, "]");
    ra_rope table;
    const ra_rope* rope = rope_of(table, a[8], w);
    const ra_head_rows rows_k = rows_of(k, tensor_or_none(a[7], "k_weight"), "k", w), rows_v = rows_of(v, nullptr, "v", w);
    const ra_status st = f_cache8_append(
        &rows_k, &rows_v, size_of(r.B, "B"), size_of(k.size(1) / r.s, "frames"), size_of(r.d, "d"), size_of(r.s, "s"),
        size_of(r.W, "W"), integer(a[6]), rope, static_cast<float>(number(a[9])), address(k8), address(v8),
        static_cast<float*>(address(ks)), static_cast<float*>(address(vs)), reinterpret_cast<ra_stream>(w.stream));
    return PyLong_FromLong(st);
    END_HANDLE_TH_ERRORS
}

// The attention, or (launch false) all of its checks and allocations: returns out, or (out, workspace).
PyObject* cache8_attention_of(PyObject* const* a, bool launch)
{
    const at::Tensor &q = tensor(a[0], "q"), &k8 = tensor(a[1], "k8"), &v8 = tensor(a[2], "v8"),
                     &ks = tensor(a[3], "k_scale"), &vs = tensor(a[4], "v_scale");
    const at::Tensor *counts = tensor_or_none(a[6], "key_counts"), *lse = tensor_or_none(a[9], "lse");
    Where w;
    where(w, q, "q", a[11]);
    const Ring r = ring_of(k8, v8, ks, vs, w);
    TORCH_CHECK_VALUE(is(q, at::kBFloat16, w) && q.dim() == 4 && q.size(0) == r.B && q.size(1) == r.H &&
                          q.size(3) == r.d && q.is_contiguous(),
                      "q must be a contiguous bf16 tensor [", r.B, ", ", r.H, ", nq, ", r.d, "]");
    const int64_t nq = q.size(2);
    TORCH_CHECK_VALUE(!counts || (is(*counts, at::kInt, w) && counts->dim() == 1 && counts->size(0) == r.B &&
                                  counts->is_contiguous()),
                      "key_counts must be a contiguous int32 tensor [", r.B, "] on the inputs' device");
    TORCH_CHECK_VALUE(!lse || (is(*lse, at::kFloat, w) && lse->dim() == 3 && lse->size(0) == r.B &&
                               lse->size(1) == r.H && lse->size(2) == nq && lse->is_contiguous()),
                      "lse must be a contiguous fp32 tensor [B, H, nq] on the inputs' device");
    const at::Tensor out = output(tensor_or_none(a[8], "out"), "out", {r.B, r.H, nq, r.d}, at::kBFloat16, w);
    at::Tensor ws;
    if (nq) {
        const int B = size_of(r.B, "B"), H = size_of(r.H, "H"), d = size_of(r.d, "d"), s = size_of(r.s, "s"),
                  W = size_of(r.W, "W"), n = size_of(nq, "nq"), held = int_of(a[5], "held");
        size_t need = 0;
        ra_status st = f_cache8_attention_workspace_bytes(B, H, d, n, s, W, held, &need);
        if (st != RA_OK)
            return PyLong_FromLong(st);
        ws = workspace_of(tensor_or_none(a[10], "workspace"), need, w);
        const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(r.d)) : number(a[7]);
        const void *Q = q.const_data_ptr(), *K = k8.const_data_ptr(), *V = v8.const_data_ptr();
        const float *k_scale = static_cast<const float*>(ks.const_data_ptr()),
                    *v_scale = static_cast<const float*>(vs.const_data_ptr());
        const int* key_counts = counts ? static_cast<const int*>(counts->const_data_ptr()) : nullptr;
        float* lse_at = lse ? static_cast<float*>(lse->mutable_data_ptr()) : nullptr;
        st = launch ? f_cache8_attention(Q, K, V, k_scale, v_scale, address(out), B, H, d, n, s, W, held, key_counts,
                                         static_cast<float>(scale), lse_at, address(ws), need,
                                         reinterpret_cast<ra_stream>(w.stream))
                    : f_cache8_attention_check(Q, K, V, k_scale, v_scale, address(out), B, H, d, n, s, W, held,
                                               key_counts, static_cast<float>(scale), lse_at, address(ws), need);
        if (st != RA_OK)
            return PyLong_FromLong(st);
    }
    return launch ? wrap(out) : tuple_of({out, ws});
}

// q, k8, v8, k_scale, v_scale, held, key_counts, scale, out, lse, workspace, stream
PyObject* cache8_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    arguments(n_args, 12);
    return cache8_attention_of(a, true);
    END_HANDLE_TH_ERRORS
}

// The same arguments: (out, workspace) for a call that will not be refused
PyObject* cache8_attention_prepare(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    arguments(n_args, 12);
    return cache8_attention_of(a, false);
    END_HANDLE_TH_ERRORS
}

// The addresses of the library's entry points, in the order of the functions below.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    constexpr int N = 7;
    arguments(n_args, N);
    void* at[N];
    for (int i = 0; i < N; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        TORCH_CHECK_VALUE(at[i] && !PyErr_Occurred(), "an entry point's address is missing");
    }
    f_qk_norm_rope = reinterpret_cast<decltype(f_qk_norm_rope)>(at[0]);
    f_qk_norm_rope_bwd_workspace_bytes = reinterpret_cast<decltype(f_qk_norm_rope_bwd_workspace_bytes)>(at[1]);
    f_qk_norm_rope_bwd = reinterpret_cast<decltype(f_qk_norm_rope_bwd)>(at[2]);
    f_cache8_append = reinterpret_cast<decltype(f_cache8_append)>(at[3]);
    f_cache8_attention_workspace_bytes = reinterpret_cast<decltype(f_cache8_attention_workspace_bytes)>(at[4]);
    f_cache8_attention = reinterpret_cast<decltype(f_cache8_attention)>(at[5]);
    f_cache8_attention_check = reinterpret_cast<decltype(f_cache8_attention_check)>(at[6]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),
                         METHOD(qk_norm_rope),
                         METHOD(qk_norm_rope_bwd),
                         METHOD(cache8_append),
                         METHOD(cache8_attention),
                         METHOD(cache8_attention_prepare),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
