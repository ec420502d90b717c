// The attention and cache calls for torch tensors: checks of the arguments,
// allocation of what is not given, and the C call (include/compfp32.h).
//
// In C++ because a single token's attention runs in some 15 microseconds on
// the device, which the same checks written in Python exceed.  Nothing is
// computed here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <string>

#include "compfp32.h"

namespace {

struct Refusal {
    PyObject* type;
    std::string what;
};

[[noreturn]] void refuse(std::string what)
{
    throw Refusal{PyExc_ValueError, std::move(what)};
}

struct Failure {
    comp_status_t status;
    const char* call;
};

void check(comp_status_t status, const char* call)
{
    if (status != COMP_OK)
        throw Failure{status, call};
}

struct PythonError {};  // already set

// Runs f; refusals, errors of the library and of torch become Python exceptions.
template <typename F>
PyObject* guarded(F f)
{
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const PythonError&) {
    } catch (const Failure& e) {
        PyObject* const native = PyImport_ImportModule("compensated_fp32_projection_gb300._native");
        PyObject* const type = native ? PyObject_GetAttrString(native, "CompError") : nullptr;
        PyObject* const error = type ? PyObject_CallFunction(type, "is", static_cast<int>(e.status), e.call) : nullptr;
        if (error)
            PyErr_SetObject(type, error);
        Py_XDECREF(error);
        Py_XDECREF(type);
        Py_XDECREF(native);
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

void arguments(Py_ssize_t given, Py_ssize_t wanted)
{
    if (given != wanted)
        throw Refusal{PyExc_TypeError, "wrong number of arguments"};
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o))
        throw Refusal{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
    return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t)
{
    return t == at::kFloat ? "torch.float32" : t == at::kHalf ? "torch.float16" : "torch.int32";
}

// A CUDA tensor of this type, on the call's device (-1: the first one says).
const at::Tensor& typed(PyObject* o, at::ScalarType type, const char* name, int& device)
{
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
        refuse(std::string(name) + " must be " + type_name(type));
    if (!t.is_cuda())
        refuse(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
    if (t.is_neg())  // its memory holds the values before the negation
        refuse(std::string(name) + " must not be a lazily negated view (see Tensor.resolve_neg)");
    if (device < 0)
        device = t.get_device();
    else if (t.get_device() != device)
        refuse(std::string(name) + " is on another device");
    return t;
}

// A dense tensor of this type and shape.
const at::Tensor& dense(PyObject* o, at::ScalarType type, const char* name, int& device, at::IntArrayRef shape)
{
    const at::Tensor& t = typed(o, type, name, device);
    if (t.sizes() != shape) {
        std::string s;
        for (const int64_t n : shape)
            s += (s.empty() ? "" : ", ") + std::to_string(n);
        refuse(std::string(name) + " must be of shape (" + s + ")");
    }
    if (!t.is_contiguous())
        refuse(std::string(name) + " must be contiguous");
    return t;
}

// A [tokens, heads, head_dim] tensor with any token and head strides.
const at::Tensor& heads(PyObject* o, at::ScalarType type, const char* name, int& device)
{
    const at::Tensor& t = typed(o, type, name, device);
    if (t.dim() != 3)
        refuse(std::string(name) + " must be [tokens, heads, head_dim]");
    if (t.size(2) > 1 && t.stride(2) != 1 && t.numel() > 0)
        refuse(std::string(name) + " must be contiguous in its last dimension");
    return t;
}

// An int32 list.
const at::Tensor& list(PyObject* o, const char* name, int& device)
{
    const at::Tensor& t = typed(o, at::kInt, name, device);
    if (t.dim() != 1)
        refuse(std::string(name) + " must be one-dimensional");
    if (!t.is_contiguous())
        refuse(std::string(name) + " must be contiguous");
    return t;
}

const at::Tensor& table_of(PyObject* o, int& device)
{
    const at::Tensor& t = typed(o, at::kInt, "table", device);
    if (t.dim() != 2)
        refuse("table must be [rows, width]");
    if (!t.is_contiguous())
        refuse("table must be contiguous");
    return t;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int device)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
}

// An output: the given tensor, or a new one.
at::Tensor output(PyObject* o, at::ScalarType type, const char* name, int device, at::IntArrayRef shape)
{
    return o == Py_None ? fresh(shape, type, device) : dense(o, type, name, device, shape);
}

// The address of an optional tensor.
template <typename T>
T* optional(PyObject* o, at::ScalarType type, const char* name, int& device, at::IntArrayRef shape)
{
    return o == Py_None ? nullptr : static_cast<T*>(dense(o, type, name, device, shape).data_ptr());
}

const int32_t* ints(const at::Tensor& t)
{
    return static_cast<const int32_t*>(t.data_ptr());
}

int32_t* ints_out(const at::Tensor& t)
{
    return static_cast<int32_t*>(t.data_ptr());
}

// The stream of a call.  While this lives the tensors' device is the current one,
// which the library launches on, and the stream its current one, so that what
// the call allocates belongs to it: a workspace of another stream could be
// given away before this one has used it, and an output could still be in use
// there.
struct Stream {
    comp_stream_t at;
    c10::cuda::CUDAGuard on_device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;

    Stream(PyObject* o, int device) : on_device(static_cast<c10::DeviceIndex>(device))
    {
        const auto on = static_cast<c10::DeviceIndex>(device);
        at = c10::cuda::getCurrentCUDAStream(on).stream();
        if (o == Py_None)
            return;
        PyObject* const number = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!number)
            throw PythonError{};
        void* const given = PyLong_AsVoidPtr(number);
        Py_DECREF(number);
        if (PyErr_Occurred())
            throw PythonError{};
        if (given != at) {
            at = given;
            guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(given), on));
        }
    }
};

int64_t integer(PyObject* o)
{
    const int64_t n = PyLong_AsLongLong(o);
    if (n == -1 && PyErr_Occurred())
        throw PythonError{};
    return n;
}

bool truth(PyObject* o)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0)
        throw PythonError{};
    return t != 0;
}

float scale_of(PyObject* o, int64_t dim)
{
    if (o == Py_None)
        return static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim > 0 ? dim : 1)));
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred())
        throw PythonError{};
    return static_cast<float>(x);
}

// A workspace of `need` bytes at least is the library's to ask for.
struct Workspace {
    at::Tensor held;
    void* at = nullptr;
    int64_t bytes = 0;

    Workspace(PyObject* given, int64_t need, int device)
    {
        if (given != Py_None) {
            const at::Tensor& t = tensor(given, "workspace");
            if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
                refuse("workspace must be a contiguous tensor on the inputs' device");
            at = t.data_ptr();
            bytes = static_cast<int64_t>(t.nbytes());
        } else if (need > 0) {
            held = fresh({need}, at::kByte, device);
            at = held.data_ptr();
            bytes = need;
        }
    }
};

struct Cache {
    comp_kv_cache_t c;
    int device = -1;

    Cache(PyObject* k, PyObject* v)
    {
        const at::Tensor& a = typed(k, at::kHalf, "k_pages", device);
        if (a.dim() != 4)
            refuse("k_pages must be [pages, kv_heads, page_size, head_dim]");
        if (!a.is_contiguous())
            refuse("k_pages must be contiguous");
        const at::Tensor& b = dense(v, at::kHalf, "v_pages", device, a.sizes());
        c.k = static_cast<uint16_t*>(a.data_ptr());
        c.v = static_cast<uint16_t*>(b.data_ptr());
        c.pages = a.size(0);
        c.kv_heads = static_cast<int32_t>(a.size(1));
        c.page_size = static_cast<int32_t>(a.size(2));
        c.head_dim = static_cast<int32_t>(a.size(3));
    }
};

// attn(f32, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 12);
        const bool f32 = a[0] == Py_True;
        const at::ScalarType kv = f32 ? at::kFloat : at::kHalf;
        int device = -1;
        const at::Tensor& q = heads(a[1], at::kFloat, "q", device);
        const at::Tensor& k = heads(a[2], kv, "k", device);
        const at::Tensor& v = heads(a[3], kv, "v", device);
        const int64_t tokens = q.size(0), h = q.size(1), dim = q.size(2);
        if (k.sizes() != v.sizes() || k.size(2) != dim)
            refuse("k and v must be [keys, kv_heads, head_dim] with q's head_dim");
        if (h == 0 || k.size(1) == 0 || h % k.size(1) != 0)
            refuse("q's heads must be a multiple of the key/value heads");
        int64_t n_seq = 1;
        const int32_t *cu_q = nullptr, *cu_k = nullptr;
        if (a[4] != Py_None || a[5] != Py_None) {
            if (a[4] == Py_None || a[5] == Py_None)
                refuse("cu_q and cu_k go together");
            const at::Tensor& c = list(a[4], "cu_q", device);
            if (c.size(0) < 1)
                refuse("cu_q and cu_k must be [sequences + 1]");
            n_seq = c.size(0) - 1;
            cu_q = ints(c);
            cu_k = ints(dense(a[5], at::kInt, "cu_k", device, c.sizes()));
        }
        const Stream on(a[11], device);
        at::Tensor out;
        if (a[8] == Py_None) {
            out = fresh(q.sizes(), at::kFloat, device);
        } else {
            out = heads(a[8], at::kFloat, "out", device);
            if (out.sizes() != q.sizes())
                refuse("out must have the shape of q");
        }
        float* const lse = optional<float>(a[9], at::kFloat, "lse", device, {tokens, h});
        comp_attn_t d{};
        d.n_seq = n_seq;
        d.total_q = tokens;
        d.total_k = k.size(0);
        d.heads = static_cast<int32_t>(h);
        d.kv_heads = static_cast<int32_t>(k.size(1));
        d.head_dim = static_cast<int32_t>(dim);
        d.causal = truth(a[7]) ? 1 : 0;
        d.scale = scale_of(a[6], dim);
        d.q_token = q.stride(0);
        d.q_head = q.stride(1);
        d.k_token = k.stride(0);
        d.k_head = k.stride(1);
        d.v_token = v.stride(0);
        d.v_head = v.stride(1);
        d.out_token = out.stride(0);
        d.out_head = out.stride(1);
        const void *kp = k.data_ptr(), *vp = v.data_ptr();
        const Workspace ws(a[10], comp_attn_workspace_bytes(&d, f32 ? 4 : 2, kp, vp), device);
        const float* const qp = static_cast<const float*>(q.data_ptr());
        float* const op = static_cast<float*>(out.data_ptr());
        if (f32)
            check(comp_attn_f32(&d, qp, static_cast<const float*>(kp), static_cast<const float*>(vp), cu_q, cu_k, op,
                                lse, ws.at, ws.bytes, on.at),
                  "comp_attn_f32");
        else
            check(comp_attn_f32x16(&d, qp, static_cast<const uint16_t*>(kp), static_cast<const uint16_t*>(vp), cu_q,
                                   cu_k, op, lse, ws.at, ws.bytes, on.at),
                  "comp_attn_f32x16");
        return a[8] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[8]);
    });
}

// append(k, v, k_pages, v_pages, table, start, cu, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 8);
        Cache c(a[2], a[3]);
        const at::Tensor& table = table_of(a[4], c.device);
        const at::Tensor& k = heads(a[0], at::kFloat, "k", c.device);
        const at::Tensor& v = heads(a[1], at::kFloat, "v", c.device);
        const int64_t rows = table.size(0), tokens = k.size(0);
        if (k.sizes() != v.sizes() || k.size(1) != c.c.kv_heads || k.size(2) != c.c.head_dim)
            refuse("k and v must be [tokens, kv_heads, head_dim] as the cache has them");
        const at::Tensor& start = dense(a[5], at::kInt, "start", c.device, {rows});
        const int32_t* const cu = optional<const int32_t>(a[6], at::kInt, "cu", c.device, {rows + 1});
        if (!cu && tokens != rows)
            refuse("without cu there must be one token for each row of table");
        const Stream on(a[7], c.device);
        check(comp_kv_append_f32(&c.c, static_cast<const float*>(k.data_ptr()),
                                 static_cast<const float*>(v.data_ptr()), k.stride(0), k.stride(1), v.stride(0),
                                 v.stride(1), tokens, ints(table), rows, table.size(1), cu, ints(start),
                                 on.at),
              "comp_kv_append_f32");
        return Py_NewRef(Py_None);
    });
}

// decode(q, k_pages, v_pages, table, lengths, shared, scale, out, lse, workspace, stream)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 11);
        Cache c(a[1], a[2]);
        const at::Tensor& table = table_of(a[3], c.device);
        const at::Tensor& q = heads(a[0], at::kFloat, "q", c.device);
        const int64_t batch = table.size(0), width = table.size(1), h = q.size(1), dim = q.size(2);
        if (q.size(0) != batch || dim != c.c.head_dim || c.c.kv_heads == 0 || h == 0 || h % c.c.kv_heads != 0)
            refuse("q must be [rows of table, a multiple of kv_heads, head_dim]");
        const at::Tensor& lengths = dense(a[4], at::kInt, "lengths", c.device, {batch});
        const int64_t shared = integer(a[5]);
        const Stream on(a[10], c.device);
        at::Tensor out = output(a[7], at::kFloat, "out", c.device, q.sizes());
        float* const lse = optional<float>(a[8], at::kFloat, "lse", c.device, {batch, h});
        const Workspace ws(a[9],
                           comp_attn_decode_workspace_bytes(&c.c, batch, static_cast<int32_t>(h), width, shared),
                           c.device);
        check(comp_attn_decode_f32x16(&c.c, static_cast<const float*>(q.data_ptr()), q.stride(0), q.stride(1),
                                      static_cast<int32_t>(h), scale_of(a[6], dim), ints(table), batch, width,
                                      ints(lengths), shared, static_cast<float*>(out.data_ptr()), lse, ws.at,
                                      ws.bytes, on.at),
              "comp_attn_decode_f32x16");
        return a[7] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[7]);
    });
}

// The outputs as a tuple: what was given itself, what was not as new tensors.
template <size_t N>
PyObject* results(PyObject* const (&given)[N], at::Tensor (&made)[N])
{
    PyObject* const r = PyTuple_New(N);
    if (!r)
        throw PythonError{};
    for (size_t i = 0; i < N; ++i)
        PyTuple_SET_ITEM(r, i, given[i] == Py_None ? THPVariable_Wrap(std::move(made[i])) : Py_NewRef(given[i]));
    return r;
}

// reserve(table, want, refs, page_size, table_out, refs_out, left, stream)
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 8);
        int device = -1;
        const at::Tensor& table = table_of(a[0], device);
        const int64_t rows = table.size(0);
        const at::Tensor& want = dense(a[1], at::kInt, "want", device, {rows});
        const at::Tensor& refs = list(a[2], "refs", device);
        const int64_t page_size = integer(a[3]);
        if (page_size < 0 || page_size > INT32_MAX)
            refuse("page_size must be 16, 32, 64 or 128");
        const Stream on(a[7], device);
        PyObject* const given[] = {a[4], a[5], a[6]};
        at::Tensor out[] = {output(a[4], at::kInt, "table_out", device, table.sizes()),
                            output(a[5], at::kInt, "refs_out", device, refs.sizes()),
                            output(a[6], at::kInt, "left", device, {1})};
        check(comp_kv_reserve(refs.size(0), static_cast<int32_t>(page_size), ints(table), ints(refs), rows,
                              table.size(1), ints(want), ints_out(out[0]), ints_out(out[1]), ints_out(out[2]),
                              on.at),
              "comp_kv_reserve");
        return results(given, out);
    });
}

// fork(k_pages, v_pages, table, lengths, refs, parents, children, table_out, lengths_out, refs_out, left, stream)
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 12);
        Cache c(a[0], a[1]);
        const at::Tensor& table = table_of(a[2], c.device);
        const int64_t rows = table.size(0);
        const at::Tensor& lengths = dense(a[3], at::kInt, "lengths", c.device, {rows});
        const at::Tensor& refs = dense(a[4], at::kInt, "refs", c.device, {c.c.pages});
        const at::Tensor& parents = list(a[5], "parents", c.device);
        const at::Tensor& children = dense(a[6], at::kInt, "children", c.device, parents.sizes());
        const Stream on(a[11], c.device);
        PyObject* const given[] = {a[7], a[8], a[9], a[10]};
        at::Tensor out[] = {output(a[7], at::kInt, "table_out", c.device, table.sizes()),
                            output(a[8], at::kInt, "lengths_out", c.device, lengths.sizes()),
                            output(a[9], at::kInt, "refs_out", c.device, refs.sizes()),
                            output(a[10], at::kInt, "left", c.device, {1})};
        check(comp_kv_fork(&c.c, ints(table), ints(lengths), ints(refs), rows, table.size(1), ints(parents),
                           ints(children), parents.size(0), ints_out(out[0]), ints_out(out[1]), ints_out(out[2]),
                           ints_out(out[3]), on.at),
              "comp_kv_fork");
        return results(given, out);
    });
}

// free(table, lengths, refs, seqs, table_out, lengths_out, refs_out, stream)
PyObject* free_(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 8);
        int device = -1;
        const at::Tensor& table = table_of(a[0], device);
        const int64_t rows = table.size(0);
        const at::Tensor& lengths = dense(a[1], at::kInt, "lengths", device, {rows});
        const at::Tensor& refs = list(a[2], "refs", device);
        const at::Tensor& seqs = list(a[3], "seqs", device);
        const Stream on(a[7], device);
        PyObject* const given[] = {a[4], a[5], a[6]};
        at::Tensor out[] = {output(a[4], at::kInt, "table_out", device, table.sizes()),
                            output(a[5], at::kInt, "lengths_out", device, lengths.sizes()),
                            output(a[6], at::kInt, "refs_out", device, refs.sizes())};
        check(comp_kv_free(refs.size(0), ints(table), ints(lengths), ints(refs), rows, table.size(1), ints(seqs),
                           seqs.size(0), ints_out(out[0]), ints_out(out[1]), ints_out(out[2]),
                           on.at),
              "comp_kv_free");
        return results(given, out);
    });
}

// compact(k_pages, v_pages, table, refs, table_out, refs_out, remap, live, stream)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 9);
        Cache c(a[0], a[1]);
        const at::Tensor& table = table_of(a[2], c.device);
        const at::Tensor& refs = dense(a[3], at::kInt, "refs", c.device, {c.c.pages});
        const Stream on(a[8], c.device);
        PyObject* const given[] = {a[4], a[5], a[6], a[7]};
        at::Tensor out[] = {output(a[4], at::kInt, "table_out", c.device, table.sizes()),
                            output(a[5], at::kInt, "refs_out", c.device, refs.sizes()),
                            output(a[6], at::kInt, "remap", c.device, refs.sizes()),
                            output(a[7], at::kInt, "live", c.device, {1})};
        check(comp_kv_compact(&c.c, ints(table), ints(refs), table.size(0), table.size(1), ints_out(out[0]),
                              ints_out(out[1]), ints_out(out[2]), ints_out(out[3]), on.at),
              "comp_kv_compact");
        return results(given, out);
    });
}

// copy_pages(k_pages, v_pages, src, dst, stream)
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 5);
        Cache c(a[0], a[1]);
        const at::Tensor& src = list(a[2], "src", c.device);
        const at::Tensor& dst = dense(a[3], at::kInt, "dst", c.device, src.sizes());
        const Stream on(a[4], c.device);
        check(comp_kv_copy_pages(&c.c, ints(src), ints(dst), src.size(0), on.at), "comp_kv_copy_pages");
        return Py_NewRef(Py_None);
    });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);

PyMethodDef method(const char* name, Fast f)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method("attn", attn),       method("append", append),   method("decode", decode),
                         method("reserve", reserve), method("fork", fork),       method("free", free_),
                         method("compact", compact), method("copy_pages", copy_pages),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding()
{
    return PyModule_Create(&module);
}
