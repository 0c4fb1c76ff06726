// launch_ext.cpp -- the argument checks and launches of the prompt and 8-bit
// cache entry points, as a CPython module.
//
// These calls are small (a decode step's append runs 3 us on the GPU), and
// checking eight tensors through Python attributes costs 5 to 15 us of host
// time a call.  Here the same checks read the tensors directly: 1 to 2 us
// beside the launch.  Errors are the binding's: TypeError, ValueError, and
// MlraError for a status the library returns.  The functions take fixed
// positional arguments; binding.py documents and calls them.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>
#include <initializer_list>

#include "mlra.h"

namespace {

PyObject* g_error = nullptr;       // binding.MlraError
PyObject* g_workspaces = nullptr;  // binding._ws_cache
PyObject* g_workspace_fn = nullptr;  // binding._new_workspace

// the library's entries, bound from the one libmlra.so that binding.py loads
decltype(&mlra_prefill) f_prefill = nullptr;
decltype(&mlra_append_fp8) f_append_fp8 = nullptr;
decltype(&mlra_decode_fp8) f_decode_fp8 = nullptr;
decltype(&mlra_decode_workspace_bytes) f_workspace_bytes = nullptr;

struct Refused {};  // a Python error is set

// A reference that is given up with its scope unless it is returned.
struct Ref {
    PyObject* p;
    explicit Ref(PyObject* owned) : p(owned) {}
    Ref(const Ref&) = delete;
    ~Ref() { Py_XDECREF(p); }
    PyObject* release() {
        PyObject* out = p;
        p = nullptr;
        return out;
    }
};

PyObject* new_ref(PyObject* o) {
    Py_INCREF(o);
    return o;
}

[[noreturn]] void refuse(PyObject* type, const char* format, ...) {
    va_list ap;
    va_start(ap, format);
    PyErr_FormatV(type, format, ap);
    va_end(ap);
    throw Refused{};
}

std::string text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

// The first look at a tensor whose shape the call's sizes are taken from.
const at::Tensor& sized(PyObject* o, const char* name, int64_t ndim, const char* where) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != ndim) refuse(PyExc_ValueError, "%s must have %d dimensions, got shape %s", name, (int)ndim, text(t.sizes()).c_str());
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s runs on CUDA tensors only", where);
    return t;
}

// The data pointer of a contiguous tensor of this type, shape and device.
void* pointer(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, at::Device device) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
        refuse(PyExc_ValueError, "%s must have shape %s, got %s", name, text(at::IntArrayRef(shape.begin(), shape.size())).c_str(), text(t.sizes()).c_str());
    if (t.device() != device) refuse(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), device.str().c_str());
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) refuse(PyExc_TypeError, "%s must be a number", name);
    return v;
}

int32_t size32(int64_t v, const char* what) {
    if (v > INT32_MAX) refuse(PyExc_ValueError, "%s is too large", what);
    return (int32_t)v;
}

// The stream of the call: a torch stream's handle, or the current one (None).
void* stream_of(PyObject* o, at::Device device) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device.index()).stream();
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) throw Refused{};
    void* s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Refused{};
    return s;
}

// The call's output like q, when the caller gives none (a new reference).  On
// a stream of the caller's the memory is that stream's, so that nothing still
// queued on the current one uses it, and is not given away before the current
// stream is done with it either.
PyObject* output_like(const at::Tensor& q, PyObject* stream_obj, void* stream) {
    if (stream_obj == Py_None) return THPVariable_Wrap(at::empty_like(q));
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(q.device().index());
    if (current.stream() == stream) return THPVariable_Wrap(at::empty_like(q));
    at::Tensor out;
    {
        const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), q.device().index()));
        out = at::empty_like(q);
    }
    out.record_stream(current);
    return THPVariable_Wrap(out);
}

void check(mlra_status st, const char* where) {
    if (st == MLRA_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, where);
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

// Runs f with C++ errors turned into Python ones.
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool expects(Py_ssize_t n, Py_ssize_t want, const char* where) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %d arguments, got %d", where, (int)want, (int)n);
    return false;
}

constexpr at::ScalarType kBf16 = at::ScalarType::BFloat16, kI32 = at::ScalarType::Int, kF32 = at::ScalarType::Float,
                         kE4m3 = at::ScalarType::Float8_e4m3fn;

// (q_lat, q_rope, latent_cache, rope_cache, block_table, seqlens, cu_seqlens, scale, out_scale, out, device_status, stream)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expects(n, 12, "mlra_prefill")) return nullptr;
    return guarded([&]() -> PyObject* {
        const char* where = "mlra_prefill";
        const at::Tensor &q = sized(a[0], "q_lat", 4, where), &qr = sized(a[1], "q_rope", 3, where), &cache = sized(a[2], "latent_cache", 4, where),
                         &bt = sized(a[4], "block_table", 2, where);
        const at::Device dev = q.device();
        const int64_t T = q.size(0), H = q.size(1), B = q.size(2), dc = q.size(3), dr = qr.size(2), pages = cache.size(0), P = cache.size(1),
                      N = bt.size(0), mp = bt.size(1);
        const c10::cuda::OptionalCUDAGuard guard(dev);
        const void* p[7] = {pointer(a[0], "q_lat", kBf16, {T, H, B, dc}, dev), pointer(a[1], "q_rope", kBf16, {T, H, dr}, dev),
                            pointer(a[2], "latent_cache", kBf16, {pages, P, B, dc}, dev), pointer(a[3], "rope_cache", kBf16, {pages, P, dr}, dev),
                            pointer(a[4], "block_table", kI32, {N, mp}, dev), pointer(a[5], "seqlens", kI32, {N}, dev),
                            pointer(a[6], "cu_seqlens", kI32, {N + 1}, dev)};
        void* stream = stream_of(a[11], dev);
        Ref out(a[9] == Py_None ? output_like(q, a[11], stream) : new_ref(a[9]));
        void* po = pointer(out.p, "out", kBf16, {T, H, B, dc}, dev);
        void* ps = a[10] == Py_None ? nullptr : pointer(a[10], "device_status", kI32, {1}, dev);
        const mlra_dims d = {size32(N, "the batch"), size32(H, "heads"), size32(B, "branches"), size32(dc, "d_c"), size32(dr, "d_r"),
                             size32(P, "the page size"), size32(mp, "block_table"), size32(pages, "the pool")};
        check(f_prefill(&d, size32(T, "the packed rows"), p[0], p[1], p[2], p[3], (const int32_t*)p[4], (const int32_t*)p[5],
                        (const int32_t*)p[6], (float)number(a[7], "scale"), (float)number(a[8], "out_scale"), po, (int32_t*)ps, stream),
              where);
        return out.release();
    });
}

// (c_new, kr_new, cu_seqlens, seqlens, block_table, latent_cache, latent_scale, rope_cache, rope_base, device_status, stream)
PyObject* append_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expects(n, 11, "mlra_append_fp8")) return nullptr;
    return guarded([&]() -> PyObject* {
        const char* where = "mlra_append_fp8";
        const at::Tensor &c = sized(a[0], "c_new", 3, where), &kr = sized(a[1], "kr_new", 2, where), &bt = sized(a[4], "block_table", 2, where),
                         &cache = sized(a[5], "latent_cache", 4, where);
        const at::Device dev = c.device();
        const int64_t T = c.size(0), B = c.size(1), dc = c.size(2), dr = kr.size(1), N = bt.size(0), mp = bt.size(1), pages = cache.size(0),
                      P = cache.size(1);
        const c10::cuda::OptionalCUDAGuard guard(dev);
        const void* p[5] = {pointer(a[0], "c_new", kBf16, {T, B, dc}, dev), pointer(a[1], "kr_new", kBf16, {T, dr}, dev),
                            pointer(a[2], "cu_seqlens", kI32, {N + 1}, dev), pointer(a[3], "seqlens", kI32, {N}, dev),
                            pointer(a[4], "block_table", kI32, {N, mp}, dev)};
        void* lat = pointer(a[5], "latent_cache", kE4m3, {pages, P, B, dc}, dev);
        void* sc = pointer(a[6], "latent_scale", kF32, {pages, P / MLRA_FP8_BLOCK, B}, dev);
        void* rope = pointer(a[7], "rope_cache", kBf16, {pages, P, dr}, dev);
        void* ps = a[9] == Py_None ? nullptr : pointer(a[9], "device_status", kI32, {1}, dev);
        const mlra_dims d = {size32(N, "the batch"), 1, size32(B, "branches"), size32(dc, "d_c"), size32(dr, "d_r"), size32(P, "the page size"),
                             size32(mp, "block_table"), size32(pages, "the pool")};
        check(f_append_fp8(&d, size32(T, "the new rows"), p[0], p[1], (const int32_t*)p[2], (const int32_t*)p[3], (const int32_t*)p[4],
                              (float)number(a[8], "rope_base"), lat, sc, rope, (int32_t*)ps, stream_of(a[10], dev)),
              where);
        Py_RETURN_NONE;
    });
}

// The default workspace of a call on `stream` that needs `need` bytes: the one
// kept for (device, stream, capture id or 0), or a first or larger one that
// binding.py makes.  A new reference.
PyObject* default_workspace(size_t need, at::Device dev, void* stream, PyObject* stream_obj) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    C10_CUDA_CHECK(cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &id));
    if (status == cudaStreamCaptureStatusNone) id = 0;
    Ref key(Py_BuildValue("iNK", (int)dev.index(), PyLong_FromVoidPtr(stream), id));
    if (key.p == nullptr) throw Refused{};
    PyObject* kept = PyDict_GetItemWithError(g_workspaces, key.p);  // borrowed
    if (kept == nullptr && PyErr_Occurred()) throw Refused{};
    if (kept != nullptr && THPVariable_Check(kept) && THPVariable_Unpack(kept).nbytes() >= need) return new_ref(kept);
    PyObject* ws = PyObject_CallFunction(g_workspace_fn, "nOO", (Py_ssize_t)need, key.p, stream_obj);
    if (ws == nullptr) throw Refused{};
    return ws;
}

// (bytes, device index, stream): the default workspace of a call on that stream
PyObject* workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expects(n, 3, "workspace")) return nullptr;
    return guarded([&]() -> PyObject* {
        const size_t need = PyLong_AsSize_t(a[0]);
        const long index = PyLong_AsLong(a[1]);
        if (PyErr_Occurred()) throw Refused{};
        const at::Device dev(at::kCUDA, (at::DeviceIndex)index);
        const c10::cuda::OptionalCUDAGuard guard(dev);
        return default_workspace(need, dev, stream_of(a[2], dev), a[2]);
    });
}

// (q_lat, q_rope, latent_cache, latent_scale, rope_cache, block_table, seqlens, scale, out_scale, out, workspace, stream)
PyObject* decode_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expects(n, 12, "mlra_decode_fp8")) return nullptr;
    return guarded([&]() -> PyObject* {
        const char* where = "mlra_decode_fp8";
        const at::Tensor &q = sized(a[0], "q_lat", 4, where), &qr = sized(a[1], "q_rope", 3, where), &cache = sized(a[2], "latent_cache", 4, where),
                         &bt = sized(a[5], "block_table", 2, where);
        const at::Device dev = q.device();
        const int64_t N = q.size(0), H = q.size(1), B = q.size(2), dc = q.size(3), dr = qr.size(2), pages = cache.size(0), P = cache.size(1),
                      mp = bt.size(1);
        const c10::cuda::OptionalCUDAGuard guard(dev);
        const void* p[7] = {pointer(a[0], "q_lat", kBf16, {N, H, B, dc}, dev), pointer(a[1], "q_rope", kBf16, {N, H, dr}, dev),
                            pointer(a[2], "latent_cache", kE4m3, {pages, P, B, dc}, dev),
                            pointer(a[3], "latent_scale", kF32, {pages, P / MLRA_FP8_BLOCK, B}, dev),
                            pointer(a[4], "rope_cache", kBf16, {pages, P, dr}, dev), pointer(a[5], "block_table", kI32, {N, mp}, dev),
                            pointer(a[6], "seqlens", kI32, {N}, dev)};
        const mlra_dims d = {size32(N, "the batch"), size32(H, "heads"), size32(B, "branches"), size32(dc, "d_c"), size32(dr, "d_r"),
                             size32(P, "the page size"), size32(mp, "block_table"), size32(pages, "the pool")};
        void* stream = stream_of(a[11], dev);
        if (a[10] != Py_None) {
            const at::Tensor& w = tensor(a[10], "workspace");
            if (w.device() != dev || !w.is_contiguous()) refuse(PyExc_ValueError, "workspace must be a contiguous tensor on %s", dev.str().c_str());
        }
        const size_t need = a[10] == Py_None ? f_workspace_bytes(&d, 0) : 1;
        if (need == 0) check(MLRA_ERR_INVALID_ARG, "mlra_decode_workspace_bytes");
        Ref ws(a[10] == Py_None ? default_workspace(need, dev, stream, a[11]) : new_ref(a[10]));
        Ref out(a[9] == Py_None ? output_like(q, a[11], stream) : new_ref(a[9]));
        void* po = pointer(out.p, "out", kBf16, {N, H, B, dc}, dev);
        const at::Tensor& w = THPVariable_Unpack(ws.p);
        check(f_decode_fp8(&d, p[0], p[1], p[2], p[3], p[4], (const int32_t*)p[5], (const int32_t*)p[6], (float)number(a[7], "scale"),
                           (float)number(a[8], "out_scale"), po, w.data_ptr(), w.nbytes(), stream),
              where);
        return out.release();
    });
}

template <class F>
bool bind_entry(F& f, PyObject* address) {
    f = reinterpret_cast<F>(PyLong_AsVoidPtr(address));
    return !PyErr_Occurred();
}

// (MlraError, _ws_cache, _new_workspace, addresses of the four entries)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expects(n, 7, "bind")) return nullptr;
    if (!bind_entry(f_prefill, a[3]) || !bind_entry(f_append_fp8, a[4]) || !bind_entry(f_decode_fp8, a[5]) || !bind_entry(f_workspace_bytes, a[6]))
        return nullptr;
    for (Py_ssize_t i = 0; i < 3; ++i) Py_INCREF(a[i]);
    g_error = a[0], g_workspaces = a[1], g_workspace_fn = a[2];
    Py_RETURN_NONE;
}

#define MLRA_FAST(name) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL
PyMethodDef methods[] = {{"prefill", MLRA_FAST(prefill), nullptr},
                         {"append_fp8", MLRA_FAST(append_fp8), nullptr},
                         {"decode_fp8", MLRA_FAST(decode_fp8), nullptr},
                         {"workspace", MLRA_FAST(workspace), nullptr},
                         {"bind", MLRA_FAST(bind), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_launch", "Checked launches of the prompt and 8-bit cache entry points.", -1, methods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__launch() { return PyModule_Create(&module); }
