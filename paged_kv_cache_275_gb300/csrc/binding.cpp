// Python entry of the rotary append, the windowed and the shared-prefix attention: checks of the tensors, the
// current stream and the workspace, then the C ABI call.  The smallest of these calls take the GPU two microseconds,
// less than the interpreter needs to look at their tensors (measured on the same host, rope_append of eight tokens,
// microseconds a call: checks in Python and a ctypes call 11.5, this 2.7).  _capi.py holds the signatures and their
// documentation; every function here takes its arguments by position, None where they were not given.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <memory>
#include <string>
#include <vector>

#include "pagedkv.h"

namespace {

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// The tensor's type, number of dims and device (-1: any GPU, which is returned through `device`).
const at::Tensor& on_device(PyObject* o, const char* name, at::ScalarType type, int64_t dims, int& device) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
  if (t.dim() != dims)
    raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dims) + " dims, got shape " + shape_of(t.sizes()));
  if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
  if (device >= 0 && t.get_device() != device)
    raise(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" +
                                std::to_string(device));
  device = t.get_device();
  return t;
}
const at::Tensor& contiguous(PyObject* o, const char* name, at::ScalarType type, int64_t dims, int& device) {
  const at::Tensor& t = on_device(o, name, type, dims, device);
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t;
}

int32_t int32(PyObject* o, const char* name) {
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (overflow || v < INT32_MIN || v > INT32_MAX)
    raise(PyExc_ValueError, std::string(name) + " does not fit in 32 bits");
  return static_cast<int32_t>(v);
}
// A size of a tensor as the C ABI takes it.
int32_t extent(int64_t v, const char* name) {
  if (v > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is too large");
  return static_cast<int32_t>(v);
}

// What _capi.py registered: raises PagedKVError of a status.
PyObject* g_check = nullptr;

void check(int status) {
  if (status == PKV_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", status);
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, "the library reported an error");
  throw Raised{};
}

// The tensors' device current while it lives.
class OnDevice {
 public:
  explicit OnDevice(int device) : before_(c10::cuda::current_device()), changed_(before_ != device) {
    if (changed_) c10::cuda::set_device(static_cast<c10::DeviceIndex>(device));
  }
  ~OnDevice() {
    if (changed_) (void)cudaSetDevice(before_);  // (nothing may be thrown here; the call's own status says what failed)
  }
  OnDevice(const OnDevice&) = delete;

 private:
  int before_;
  bool changed_;
};

pkv_stream_t stream_of(PyObject* stream, int device) {
  if (stream == Py_None)
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* handle = PyObject_GetAttrString(stream, "cuda_stream");
  if (!handle) throw Raised{};
  void* p = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (PyErr_Occurred()) throw Raised{};
  PyObject* index = PyObject_GetAttrString(stream, "device_index");
  if (!index) throw Raised{};
  const long of = PyLong_AsLong(index);
  Py_DECREF(index);
  if (PyErr_Occurred()) throw Raised{};
  if (of != device)
    raise(PyExc_ValueError, "stream is on cuda:" + std::to_string(of) + ", the tensors on cuda:" + std::to_string(device));
  return static_cast<pkv_stream_t>(p);
}

// Device memory of torch's allocator, for use on one stream.
struct Release {
  void operator()(void* p) const noexcept {
    try {
      c10::cuda::CUDACachingAllocator::raw_delete(p);
    } catch (...) {  // (the allocator is gone: the process is ending)
    }
  }
};
using Buffer = std::unique_ptr<void, Release>;
Buffer allocate(size_t bytes, pkv_stream_t stream) {  // on the current device
  return Buffer(c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, static_cast<cudaStream_t>(stream)));
}

// This OS thread's workspaces, one per device and stream, for calls that were given none: calls that share a buffer run in
// order (two threads' calls on one stream could interleave their launches).  The buffers are owned here and live as long as
// the thread does.  Nothing of Python's may own them: a thread that Python did not start gets new thread-local storage each
// time it enters the interpreter.
struct Scratch {
  int device;
  pkv_stream_t stream;
  size_t bytes;
  Buffer data;
};
thread_local std::vector<Scratch> t_scratch;

// The caller's workspace (kept alive by `owner`), or one of this thread, device and stream.
struct Workspace {
  PyObject* owner = nullptr;
  Buffer own;
  void* data = nullptr;
  size_t bytes = 0;
  Workspace() = default;
  Workspace(const Workspace&) = delete;
  ~Workspace() { Py_XDECREF(owner); }
  void take(PyObject* given, int device, pkv_stream_t handle, size_t need) {  // `device` is the current one
    if (given != Py_None) {
      Py_INCREF(given);
      owner = given;
      const at::Tensor& t = contiguous(given, "workspace", at::kByte, 1, device);
      data = t.data_ptr();
      bytes = static_cast<size_t>(t.numel());
      if (bytes < need)
        raise(PyExc_ValueError, "workspace must hold " + std::to_string(need) + " bytes (got " + std::to_string(bytes) + ")");
      return;
    }
    bytes = std::max<size_t>(need, 256);
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(handle, &capture) != cudaSuccess) {
      (void)cudaGetLastError();
      capture = cudaStreamCaptureStatusActive;
    }
    // A call that is being captured takes a buffer of its own: the allocator gives it from the memory that torch reserves for
    // the graph, for as long as the graph lives, and what the graph's later calls are given there comes behind this call.
    if (capture != cudaStreamCaptureStatusNone) {
      own = allocate(bytes, handle);
      data = own.get();
      return;
    }
    Scratch* mine = nullptr;
    for (Scratch& x : t_scratch)
      if (x.device == device && x.stream == handle) mine = &x;
    if (!mine) {
      t_scratch.push_back({device, handle, 0, nullptr});
      mine = &t_scratch.back();
    }
    if (mine->bytes < need) {  // (the old buffer goes back first, to what runs behind it on its stream)
      mine->bytes = 0;
      mine->data.reset();
      mine->data = allocate(bytes, handle);
      mine->bytes = bytes;
    }
    data = mine->data.get();
    bytes = mine->bytes;
  }
};

// The call without the interpreter's lock.
template <typename F>
void run(F&& f) {
  pkv_status status;
  Py_BEGIN_ALLOW_THREADS status = f();
  Py_END_ALLOW_THREADS check(status);
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception&) {
    torch::translate_exception_to_python(std::current_exception());  // (no memory is torch.OutOfMemoryError)
  }
  return nullptr;
}

// Elements between the token rows of a [tokens, heads, head_dim] tensor whose rows are contiguous.
int64_t token_stride(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads, int64_t head_dim) {
  if (t.size(0) != tokens || t.size(1) != heads || t.size(2) != head_dim)
    raise(PyExc_ValueError, std::string(name) + " must be " + shape_of({tokens, heads, head_dim}) + ", got " + shape_of(t.sizes()));
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != head_dim))
    raise(PyExc_ValueError, std::string(name) + "[token] must be contiguous (got strides " + shape_of(t.strides()) + ")");
  return tokens > 1 ? t.stride(0) : heads * head_dim;
}

PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    int dev = -1;
    const at::Tensor& kc = contiguous(a[6], "k_cache", at::kBFloat16, 4, dev);
    const at::Tensor& vc = contiguous(a[7], "v_cache", at::kBFloat16, 4, dev);
    const at::Tensor& slots = contiguous(a[4], "slot_mapping", at::kLong, 1, dev);
    const at::Tensor& table = contiguous(a[5], "cos_sin", at::kFloat, 2, dev);
    const at::Tensor& q = on_device(a[0], "q", at::kBFloat16, 3, dev);
    const at::Tensor& k = on_device(a[1], "k", at::kBFloat16, 3, dev);
    const at::Tensor& v = on_device(a[2], "v", at::kBFloat16, 3, dev);
    const at::Tensor& out = on_device(a[8], "q_out", at::kBFloat16, 3, dev);
    const int64_t n = slots.size(0), hkv = kc.size(1), d = kc.size(3), hq = q.size(1);
    if (vc.sizes() != kc.sizes()) raise(PyExc_ValueError, "k_cache and v_cache shapes differ");
    if (table.size(1) != d) raise(PyExc_ValueError, "cos_sin must be [max_position, head_dim]");
    const int64_t qs = token_stride(q, "q", n, hq, d), ks = token_stride(k, "k", n, hkv, d);
    const int64_t vs = token_stride(v, "v", n, hkv, d), os = token_stride(out, "q_out", n, hq, d);
    const at::Tensor& pos = tensor(a[3], "positions");
    if (pos.scalar_type() != at::kLong || !pos.is_cuda() || pos.get_device() != dev || pos.dim() < 1 || pos.dim() > 2 ||
        pos.size(-1) != n || (n > 1 && pos.stride(-1) != 1))
      raise(PyExc_ValueError, "positions must be int64 [" + std::to_string(n) + "] or [axes, " + std::to_string(n) +
                                  "] on cuda:" + std::to_string(dev) + ", with contiguous rows");
    const int64_t axes = pos.dim() == 1 ? 1 : pos.size(0), axis_stride = pos.dim() == 1 ? 0 : pos.stride(0);
    PyObject* held = nullptr;  // the axes as bytes
    struct Release {
      PyObject*& o;
      ~Release() { Py_XDECREF(o); }
    } release{held};
    const uint8_t* axis_of = nullptr;
    if (axes > 1) {
      if (a[9] == Py_None) raise(PyExc_ValueError, "positions of several axes need freq_axes");
      held = PyBytes_FromObject(a[9]);
      if (!held) throw Raised{};
      if (PyBytes_GET_SIZE(held) != d / 2)
        raise(PyExc_ValueError, "freq_axes must hold head_dim / 2 = " + std::to_string(d / 2) + " axes (got " +
                                    std::to_string(PyBytes_GET_SIZE(held)) + ")");
      axis_of = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(held));
    }
    const pkv_stream_t stream = stream_of(a[10], dev);
    const int32_t num_axes = extent(axes, "positions"), num_q = extent(hq, "q"), num_kv = extent(hkv, "k_cache");
    const int32_t head_dim = extent(d, "head_dim"), block = extent(kc.size(2), "block size");
    const OnDevice guard(dev);
    run([&] {
      return pkv_rope_append(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                             static_cast<const int64_t*>(pos.data_ptr()), num_axes, axis_stride, axis_of,
                             static_cast<const float*>(table.data_ptr()), table.size(0),
                             static_cast<const int64_t*>(slots.data_ptr()), n, num_q, num_kv, head_dim, out.data_ptr(),
                             os, kc.data_ptr(), vc.data_ptr(), kc.size(0), block, stream);
    });
    Py_INCREF(a[8]);
    return a[8];
  });
}

// The tensors that every paged attention call takes: q, k_cache, v_cache, block_tables, context_lens, out.
struct Attention {
  int dev = -1;
  const void *q, *kc, *vc;
  const int32_t *table, *lens;
  void* out;
  int32_t rows, hq, hkv, d, width, batch, block;
  int64_t blocks;
  Attention(PyObject* q_, PyObject* kc_, PyObject* vc_, PyObject* table_, PyObject* lens_, PyObject* out_) {
    const at::Tensor& tq = contiguous(q_, "q", at::kBFloat16, 3, dev);
    const at::Tensor& tk = contiguous(kc_, "k_cache", at::kBFloat16, 4, dev);
    const at::Tensor& tv = contiguous(vc_, "v_cache", at::kBFloat16, 4, dev);
    const at::Tensor& tt = contiguous(table_, "block_tables", at::kInt, 2, dev);
    const at::Tensor& tl = contiguous(lens_, "context_lens", at::kInt, 1, dev);
    const at::Tensor& to = contiguous(out_, "out", at::kBFloat16, 3, dev);
    if (tv.sizes() != tk.sizes() || tk.size(3) != tq.size(2)) raise(PyExc_ValueError, "cache shapes do not match q");
    if (to.sizes() != tq.sizes()) raise(PyExc_ValueError, "out must have the shape of q");
    if (tt.size(0) != tl.size(0)) raise(PyExc_ValueError, "block_tables / context_lens batch mismatch");
    q = tq.data_ptr();
    kc = tk.data_ptr();
    vc = tv.data_ptr();
    table = static_cast<const int32_t*>(tt.data_ptr());
    lens = static_cast<const int32_t*>(tl.data_ptr());
    out = to.data_ptr();
    rows = extent(tq.size(0), "q");
    hq = extent(tq.size(1), "q");
    d = extent(tq.size(2), "q");
    blocks = tk.size(0);
    hkv = extent(tk.size(1), "k_cache");
    block = extent(tk.size(2), "k_cache");
    width = extent(tt.size(1), "block_tables");
    batch = extent(tl.size(0), "context_lens");
  }
  void one_row_a_sequence() const {
    if (batch != rows) raise(PyExc_ValueError, "block_tables / context_lens batch mismatch");
  }
};

PyObject* window_decode(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    const Attention t(a[0], a[1], a[2], a[3], a[4], a[6]);
    t.one_row_a_sequence();
    const double scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) throw Raised{};
    const int32_t window = int32(a[7], "window"), sinks = int32(a[8], "num_sink_tokens");
    const int32_t parts = int32(a[9], "num_partitions");
    if (t.rows > 0) {
      const pkv_stream_t stream = stream_of(a[11], t.dev);
      const OnDevice guard(t.dev);
      size_t need = 0;
      check(pkv_window_decode_workspace_size(t.rows, t.hq, t.hkv, t.d, t.width, window, sinks, parts, &need));
      Workspace ws;
      if (need > 0) ws.take(a[10], t.dev, stream, need);
      run([&] {
        return pkv_paged_window_decode_attention(t.q, t.kc, t.vc, t.table, t.width, t.lens, t.rows, t.hq, t.hkv, t.d,
                                                 t.blocks, t.block, static_cast<float>(scale), window, sinks, t.out,
                                                 ws.data, ws.bytes, parts, stream);
      });
    }
    Py_INCREF(a[6]);
    return a[6];
  });
}

PyObject* window_prefill(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Attention t(a[0], a[1], a[2], a[3], a[4], a[8]);
    const at::Tensor& start = contiguous(a[5], "query_start", at::kInt, 1, t.dev);
    if (start.size(0) != static_cast<int64_t>(t.batch) + 1)
      raise(PyExc_ValueError, "query_start must hold " + std::to_string(static_cast<int64_t>(t.batch) + 1) + " rows' starts");
    const int32_t most = int32(a[6], "max_query_len");
    const double scale = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) throw Raised{};
    const int32_t window = int32(a[9], "window"), sinks = int32(a[10], "num_sink_tokens");
    int32_t splits = int32(a[11], "num_splits");
    const pkv_stream_t stream = stream_of(a[13], t.dev);
    const OnDevice guard(t.dev);
    if (splits == 0) check(pkv_window_prefill_default_splits(t.batch, most, t.hq, t.hkv, window, sinks, &splits));
    if (splits != 1) check(pkv_window_prefill_splits(t.rows, most, t.batch, t.hq, t.hkv, splits, &splits));
    Workspace ws;
    if (splits > 1) {
      size_t need = 0;
      check(pkv_window_prefill_workspace_size(t.d, splits, &need));
      ws.take(a[12], t.dev, stream, need);
    }
    run([&] {
      return pkv_paged_window_prefill_attention(t.q, t.kc, t.vc, t.table, t.width, t.lens,
                                                static_cast<const int32_t*>(start.data_ptr()), t.rows, most, t.batch, t.hq,
                                                t.hkv, t.d, t.blocks, t.block, static_cast<float>(scale), window, sinks,
                                                t.out, splits, ws.data, ws.bytes, stream);
    });
    Py_INCREF(a[8]);
    return a[8];
  });
}

PyObject* prefix_decode(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    Attention t(a[0], a[1], a[2], a[3], a[4], a[8]);
    t.one_row_a_sequence();
    const at::Tensor& start = contiguous(a[5], "group_start", at::kInt, 1, t.dev);
    const at::Tensor& prefix = contiguous(a[6], "prefix_lens", at::kInt, 1, t.dev);
    const int32_t groups = extent(prefix.size(0), "prefix_lens");
    if (start.size(0) != static_cast<int64_t>(groups) + 1)
      raise(PyExc_ValueError, "group_start must hold " + std::to_string(static_cast<int64_t>(groups) + 1) + " rows' starts");
    const double scale = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) throw Raised{};
    if (t.rows > 0) {
      const pkv_stream_t stream = stream_of(a[10], t.dev);
      const OnDevice guard(t.dev);
      size_t need = 0;
      check(pkv_prefix_decode_workspace_size(t.rows, t.hq, t.hkv, t.d, t.width, groups, &need));
      Workspace ws;
      if (need > 0) ws.take(a[9], t.dev, stream, need);
      run([&] {
        return pkv_paged_prefix_decode_attention(t.q, t.kc, t.vc, t.table, t.width, t.lens,
                                                 static_cast<const int32_t*>(start.data_ptr()),
                                                 static_cast<const int32_t*>(prefix.data_ptr()), groups, t.rows, t.hq,
                                                 t.hkv, t.d, t.blocks, t.block, static_cast<float>(scale), t.out, ws.data,
                                                 ws.bytes, stream);
      });
    }
    Py_INCREF(a[8]);
    return a[8];
  });
}

// register(check): the Python side's helper.
PyObject* register_helpers(PyObject*, PyObject* const* a, Py_ssize_t) {
  Py_INCREF(a[0]);
  Py_XDECREF(g_check);
  g_check = a[0];
  Py_RETURN_NONE;
}

// A function of exactly kCount positional arguments.
template <int kCount, PyObject* (*kFunction)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != kCount) {
    PyErr_Format(PyExc_TypeError, "%d arguments wanted, got %zd", kCount, n);
    return nullptr;
  }
  return kFunction(self, a, n);
}

template <int kCount, PyObject* (*kFunction)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&counted<kCount, kFunction>)), METH_FASTCALL,
          nullptr};
}

PyMethodDef g_methods[] = {
    method<1, register_helpers>("register"), method<11, rope_append>("rope_append"),
    method<12, window_decode>("window_decode"), method<14, window_prefill>("window_prefill"),
    method<11, prefix_decode>("prefix_decode"), {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
