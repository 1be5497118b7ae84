// kv8_binding.cpp -- the Python calls of the paged 8-bit cache, compiled.
//
// One audio frame's append or attention takes a few microseconds on the GPU; checked and marshalled in Python, a call
// took 12 on the host.  This module reads the tensors' properties in C++, refuses what the Python classes refuse, and
// calls the C ABI through the function pointers that the package hands over at import.  It computes nothing.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <Python.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/hra.h"

namespace {

PyObject* g_error = nullptr;                            // HraError
decltype(&hra_kv8_append) f_append = nullptr;
decltype(&hra_kv8_attention) f_attend = nullptr;
decltype(&hra_kv8_attention_workspace_size) f_attend_size = nullptr;
decltype(&hra_kv8_update) f_update = nullptr;
decltype(&hra_kv8_compact) f_compact = nullptr;
decltype(&hra_status_string) f_status = nullptr;

struct Refused {   // becomes an HraError
    std::string text;
};
[[noreturn]] void refuse(const std::string& text) { throw Refused{text}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
void on_device(const at::Tensor& t, int index, const char* name) {
    if (!t.is_cuda() || t.get_device() != index) refuse(std::string(name) + " must be on the device of the cache");
}
// contiguous int32 of `n` elements in `dim` dimensions
int32_t* ints(const at::Tensor& t, int64_t n, int64_t dim, int index, const char* name) {
    on_device(t, index, name);
    if (t.scalar_type() != at::kInt || t.dim() != dim || t.numel() != n || !t.is_contiguous())
        refuse(std::string(name) + " must be contiguous int32 with " + std::to_string(n) + " elements");
    return static_cast<int32_t*>(t.data_ptr());
}
// bf16 [rows][heads][head_dim] with contiguous heads (heads 0: any number): its row stride
int64_t row_stride(const at::Tensor& t, int64_t heads, int64_t head_dim, int index, const char* name) {
    on_device(t, index, name);
    if (t.scalar_type() != at::kBFloat16) refuse(std::string(name) + " must be torch.bfloat16");
    if (t.dim() != 3 || t.size(2) != head_dim || (heads && t.size(1) != heads) ||
        (t.size(0) && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != head_dim))))
        refuse(std::string(name) + " must be [rows, " + (heads ? std::to_string(heads) : "heads") + ", " +
               std::to_string(head_dim) + "] with contiguous heads");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * head_dim;
}
const hra_kv8_cache* cache(PyObject* o) { return static_cast<const hra_kv8_cache*>(PyLong_AsVoidPtr(o)); }
int integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (PyErr_Occurred()) throw std::nullopt;
    if (v != static_cast<int>(v)) refuse("an integer argument is out of range");
    return static_cast<int>(v);
}
// The stream of a call, the device's current one (None) or any object's cuda_stream: as launches take it, and as the allocator
// does, which does not know CUDA's special handles (1: the default stream, 2: the thread's default stream).
struct Stream {
    void* raw;
    c10::cuda::CUDAStream memory;
};
Stream stream_of(PyObject* o, int index) {
    const auto device = static_cast<c10::DeviceIndex>(index);
    if (o == Py_None) {
        const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(device);
        return {now.stream(), now};
    }
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) throw std::nullopt;
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw std::nullopt;
    if (reinterpret_cast<uintptr_t>(p) <= 2) return {p, c10::cuda::getDefaultCUDAStream(device)};
    return {p, c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), device)};
}
// The allocator must not hand out t's memory before `st` is done with it, whichever stream it was allocated for.
void used_on(const at::Tensor& t, c10::cuda::CUDAStream st) {
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), st);
}
// Whether a call on `st` uses memory of another stream.
bool away(PyObject* home, const Stream& st) {
    void* h = PyLong_AsVoidPtr(home);
    if (PyErr_Occurred()) throw std::nullopt;
    return h != st.raw;
}
void check(int rc, const char* what) {
    if (rc != HRA_OK) refuse(std::string(what) + " failed: " + f_status(rc) + " (" + std::to_string(rc) + ")");
}
// The launches go to the cache's device, whichever is current, and without the interpreter's lock: a launch may wait
// for room in the stream's queue, and what the stream waits for may need Python.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
int on(int index, F&& f) {
    const Unlocked unlocked;
    if (c10::cuda::current_device() == index) return f();
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    return f();
}
// No C++ exception leaves a Python entry.
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused& r) {
        PyErr_SetString(g_error, r.text.c_str());
    } catch (const std::nullopt_t&) {   // a Python error is set
    } catch (const std::exception& e) {
        PyErr_SetString(g_error, e.what());
    } catch (...) {
        PyErr_SetString(g_error, "unknown error");
    }
    return nullptr;
}
bool counted(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return n == want;
}

// append(cache, device, layer, k, v, cu, start, max_new, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 9)) return nullptr;
    return guarded([&]() -> PyObject* {
        const hra_kv8_cache* c = cache(a[0]);
        const int index = integer(a[1]);
        const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v"), &cu = tensor(a[5], "cu"), &start = tensor(a[6], "start");
        const int64_t stride = row_stride(k, c->n_kv_heads, c->head_dim, index, "k");
        if (row_stride(v, c->n_kv_heads, c->head_dim, index, "v") != stride || v.size(0) != k.size(0))
            refuse("k and v must have the same rows and row stride");
        const int64_t batch = start.dim() == 1 ? start.size(0) : 0;
        const int32_t* pcu = ints(cu, batch + 1, 1, index, "cu");
        const int32_t* ps = ints(start, batch, 1, index, "start");
        if (batch > INT32_MAX || k.size(0) > INT32_MAX) refuse("too many rows");
        void* st = stream_of(a[8], index).raw;
        const int layer = integer(a[2]), most = integer(a[7]);
        check(on(index, [&] {
                  return f_append(c, layer, k.data_ptr(), v.data_ptr(), stride, pcu, ps, static_cast<int32_t>(batch),
                                  static_cast<int32_t>(k.size(0)), most, st);
              }), "hra_kv8_append");
        Py_RETURN_NONE;
    });
}

// attend(cache, device, layer, q, cu, kv_len, max_new, max_len, scale, out or None, workspace or None, home, stream) -> out.
// home: None for a workspace of the caller's; of the cache's own one the stream whose memory it is, and where that workspace is
// too small, the answer is the size it has to have
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 13)) return nullptr;
    return guarded([&]() -> PyObject* {
        const hra_kv8_cache* c = cache(a[0]);
        const int index = integer(a[1]);
        const at::Tensor &q = tensor(a[3], "q"), &cu = tensor(a[4], "cu"), &len = tensor(a[5], "kv_len");
        const int64_t stride = row_stride(q, 0, c->head_dim, index, "q");
        const int64_t batch = len.dim() == 1 ? len.size(0) : 0, rows = q.size(0), heads = q.size(1);
        const int32_t* pcu = ints(cu, batch + 1, 1, index, "cu");
        const int32_t* pl = ints(len, batch, 1, index, "kv_len");
        if (batch > INT32_MAX || rows > INT32_MAX || heads > INT32_MAX) refuse("too many rows");
        const int layer = integer(a[2]), max_new = integer(a[6]), max_len = integer(a[7]);
        const double scale = PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred()) throw std::nullopt;
        if (scale != 0.0 && static_cast<float>(scale) == 0.f) refuse("scale is below float32's smallest");   // 0: the default
        const bool own = a[11] != Py_None;
        const Stream st = stream_of(a[12], index);
        void* ws = nullptr;
        size_t bytes = 0;
        if (a[10] != Py_None) {
            const at::Tensor& w = tensor(a[10], "workspace");
            on_device(w, index, "workspace");
            if (!w.is_contiguous()) refuse("workspace must be contiguous");
            ws = w.data_ptr();
            bytes = w.nbytes();
            if (own && away(a[11], st)) used_on(w, st.memory);
        }
        size_t need = 0;
        if (own) {
            on(index, [&] {
                need = f_attend_size(c, static_cast<int32_t>(batch), static_cast<int32_t>(rows), static_cast<int32_t>(heads), max_new, max_len);
                return 0;
            });
            // (0: the call below refuses the arguments)
            if (bytes < need || ws == nullptr) return PyLong_FromSize_t(need > 256 ? need : 256);
        }
        at::Tensor out;
        if (a[9] == Py_None) {
            const Unlocked unlocked;
            const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index));
            const bool other = st.memory.stream() != now.stream();
            c10::cuda::OptionalCUDAStreamGuard guard;
            if (other) guard.reset_stream(st.memory);
            out = at::empty(q.sizes(), q.options());   // memory of the stream that writes it ...
            if (other) used_on(out, now);              // ... kept for the caller's, too
        } else {
            out = tensor(a[9], "out");
            on_device(out, index, "out");
            if (out.scalar_type() != at::kBFloat16 || !out.sizes().equals(q.sizes()) || !out.is_contiguous())
                refuse("out must be contiguous bf16 [T, n_q_heads, head_dim] on the device of the cache");
        }
        check(on(index, [&] {
                  return f_attend(c, layer, q.data_ptr(), stride, static_cast<int32_t>(heads), static_cast<float>(scale), pcu, pl,
                                  static_cast<int32_t>(batch), static_cast<int32_t>(rows), max_new, max_len, out.data_ptr(),
                                  ws, bytes, st.raw);
              }), "hra_kv8_attention");
        if (a[9] != Py_None) {
            Py_INCREF(a[9]);
            return a[9];
        }
        return THPVariable_Wrap(std::move(out));
    });
}

// pages(cache, device, update, parents or None, room or None, table, lens, refs, workspace, home (see attend), stream)
PyObject* pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 11)) return nullptr;
    return guarded([&]() -> PyObject* {
        const hra_kv8_cache* c = cache(a[0]);
        const int index = integer(a[1]);
        const bool update = a[2] == Py_True;
        const int32_t* parents = a[3] == Py_None ? nullptr : ints(tensor(a[3], "parents"), c->rows, 1, index, "parents");
        const int32_t* room = a[4] == Py_None ? nullptr : ints(tensor(a[4], "room"), c->rows, 1, index, "room");
        const at::Tensor& t = tensor(a[5], "page table");
        int32_t* table = ints(t, static_cast<int64_t>(c->rows) * c->max_pages, 2, index, "page table");
        if (t.size(1) != c->max_pages) refuse("page table must be [rows, max_pages]");
        int32_t* lens = ints(tensor(a[6], "lens"), c->rows, 1, index, "lens");
        int32_t* refs = ints(tensor(a[7], "refs"), c->n_pages, 1, index, "refs");
        const at::Tensor& w = tensor(a[8], "workspace");
        on_device(w, index, "workspace");
        if (!w.is_contiguous()) refuse("workspace must be contiguous");
        const Stream st = stream_of(a[10], index);
        if (a[9] != Py_None && away(a[9], st)) used_on(w, st.memory);
        check(on(index, [&] {
                  return update ? f_update(c, parents, room, table, lens, refs, w.data_ptr(), w.nbytes(), st.raw)
                                : f_compact(c, table, lens, refs, w.data_ptr(), w.nbytes(), st.raw);
              }), update ? "hra_kv8_update" : "hra_kv8_compact");
        Py_RETURN_NONE;
    });
}

// connect(HraError, append, attention, attention_workspace_size, update, compact, status_string): the library's entry points
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 7)) return nullptr;
    void* p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (PyErr_Occurred()) return nullptr;
    }
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    f_append = reinterpret_cast<decltype(f_append)>(p[0]);
    f_attend = reinterpret_cast<decltype(f_attend)>(p[1]);
    f_attend_size = reinterpret_cast<decltype(f_attend_size)>(p[2]);
    f_update = reinterpret_cast<decltype(f_update)>(p[3]);
    f_compact = reinterpret_cast<decltype(f_compact)>(p[4]);
    f_status = reinterpret_cast<decltype(f_status)>(p[5]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pages)), METH_FASTCALL, nullptr},
    {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(connect)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv8_binding", "Calls of the paged 8-bit cache", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv8_binding() { return PyModule_Create(&module); }
