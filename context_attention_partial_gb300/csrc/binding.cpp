// binding.cpp -- the PyTorch side of the rotary and cross-attention calls:
// tensors to cpattn_tensor descriptors, outputs and workspace from PyTorch's
// allocator, the current stream, one call of the C ABI.  Argument marshalling
// only, like the ctypes binding beside it, which spends 20 to 40 us of host
// time on a call of six to twelve tensors; this one 5.5 (rotary, forward) to 11
// (gradient), launches included.
//
// Every function takes the address of its C entry point first, so the same
// module serves any build of the library, and returns (status, results...).
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>

#include "../../include/cpattn.h"

namespace {

using at::Tensor;

// Tensors of one call: all on one CUDA device.
struct Call {
  int device = -1;
  bool ok = true;   // false: a Python error is set
  // while the call allocates and launches: its device, and its stream where that
  // is not the device's current one (then `caller`)
  std::optional<c10::cuda::CUDAGuard> device_guard;
  std::optional<c10::cuda::CUDAStreamGuard> stream_guard;
  std::optional<c10::cuda::CUDAStream> caller;
  void* stream = nullptr;

  // Makes the given stream (None: the device's current one) the current one, so
  // that what the call allocates is that stream's memory: a block that the caller's
  // stream has freed may still be read there by work not yet done.
  void enter(PyObject* given) {
    const auto index = static_cast<c10::DeviceIndex>(device);
    device_guard.emplace(index);
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(index);
    stream = given == Py_None ? static_cast<void*>(current.stream()) : PyLong_AsVoidPtr(given);
    if (stream == static_cast<void*>(current.stream())) return;
    caller = current;
    stream_guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), index));
  }

  // A result that this call allocated: not given out again, once it is released,
  // before what the caller's stream does with it is done.
  Tensor made(Tensor t) const {
    if (caller) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *caller);
    return t;
  }

  const Tensor* tensor(PyObject* o) {
    if (!ok) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "a tensor is expected, not %s", Py_TYPE(o)->tp_name);
      ok = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
      PyErr_SetString(PyExc_ValueError, "cpattn runs on CUDA tensors only (no CPU path)");
      ok = false;
    } else if (device >= 0 && t.get_device() != device) {
      PyErr_Format(PyExc_ValueError, "tensors on cuda:%d and cuda:%d in one call", device, static_cast<int>(t.get_device()));
      ok = false;
    } else {
      device = static_cast<int>(t.get_device());
    }
    return ok ? &t : nullptr;
  }

  // An input.  No autograd graph is recorded, so one that asks for a gradient is
  // worth a warning where graphs are recorded (not inside no_grad(), nor in the
  // forward or backward of an autograd.Function that calls this).
  const Tensor* input(PyObject* o) {
    const Tensor* t = tensor(o);
    if (t && t->requires_grad() && at::GradMode::is_enabled() &&
        PyErr_WarnEx(PyExc_UserWarning,
                     "cpattn records no autograd graph: the result is detached from an input that requires a gradient "
                     "(call the gradient entry points, under torch.no_grad() or in a torch.autograd.Function)",
                     2) < 0)
      ok = false;
    return ok ? t : nullptr;
  }

  // An input for kernels that read each element from a place of its own: a
  // broadcast view (the gradient that out.sum() sends back, a prompt expanded over a
  // guided pair) is copied into one, on the call's stream (so after enter()).
  const Tensor* dense(const Tensor* t) {
    bool broadcast = false;
    for (int64_t i = 0; i < t->dim(); ++i) broadcast = broadcast || (t->size(i) > 1 && t->stride(i) == 0);
    return broadcast ? copy(*t) : t;
  }
  // For kernels that read broadcast rows, heads and batches where they are.
  const Tensor* dense_rows(const Tensor* t) {
    const int64_t n = t->dim();
    return n > 0 && t->size(n - 1) > 1 && t->stride(n - 1) == 0 ? copy(*t) : t;
  }
  const Tensor* copy(const Tensor& t) {
    const at::NoGradGuard no_grad;
    copies[n_copies] = t.contiguous();
    return &copies[n_copies++];
  }
  Tensor copies[7];   // of the at most seven inputs of a call
  int n_copies = 0;

  void describe(const Tensor& t, cpattn_tensor* d, bool lengths = false) {
    if (!ok) return;
    const auto type = t.scalar_type();
    if (lengths ? type != at::kInt : type != at::kFloat && type != at::kBFloat16) {
      PyErr_Format(PyExc_TypeError, "dtype %s is not supported (%s)", at::toString(type),
                   lengths ? "kv_lengths are int32" : "float32 or bfloat16");
      ok = false;
      return;
    }
    if (t.dim() > CPATTN_MAX_DIMS) {
      PyErr_Format(PyExc_IndexError, "%d dimensions: at most %d", static_cast<int>(t.dim()), CPATTN_MAX_DIMS);
      ok = false;
      return;
    }
    d->data = t.numel() > 0 ? t.data_ptr() : nullptr;
    d->dtype = lengths ? CPATTN_I32 : type == at::kFloat ? CPATTN_F32 : CPATTN_BF16;
    d->ndim = static_cast<int32_t>(t.dim());
    for (int i = 0; i < CPATTN_MAX_DIMS; ++i) {
      d->shape[i] = i < d->ndim ? t.size(i) : 0;
      d->stride[i] = i < d->ndim ? t.stride(i) : 0;
    }
  }

  // A given output, or a new one like `like` (keeping a [B, S, H, D] tensor's order).
  Tensor output(PyObject* o, const Tensor& like) {
    if (!ok) return Tensor();
    if (o != Py_None) {
      const Tensor* t = tensor(o);
      return t ? *t : Tensor();
    }
    // (like empty_like, without its two passes through the dispatcher)
    if (like.is_non_overlapping_and_dense())
      return made(Tensor(at::detail::empty_strided_cuda(like.sizes(), like.strides(), like.scalar_type(), like.device())));
    return made(at::empty_like(like));
  }

  Tensor fresh(at::IntArrayRef sizes, at::ScalarType type) const {
    const at::Device on(at::kCUDA, static_cast<c10::DeviceIndex>(device));
    return Tensor(at::detail::empty_cuda(sizes, type, on, std::nullopt));
  }

  // A given workspace, or a new one of `need` bytes (none if 0).
  Tensor workspace(PyObject* o, size_t need) {
    if (!ok) return Tensor();
    if (o != Py_None) {
      const Tensor* t = tensor(o);
      if (t && !t->is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "a workspace is contiguous");
        ok = false;
      }
      return ok ? *t : Tensor();
    }
    return need > 0 ? fresh({static_cast<int64_t>(need)}, at::kByte) : Tensor();
  }
};

// A reference of this scope's own.
class Owned {
 public:
  explicit Owned(PyObject* o) : o_(o) {}
  ~Owned() { Py_XDECREF(o_); }
  Owned(const Owned&) = delete;
  Owned& operator=(const Owned&) = delete;
  explicit operator bool() const { return o_ != nullptr; }
  PyObject* get() const { return o_; }
  PyObject* release() {
    PyObject* o = o_;
    o_ = nullptr;
    return o;
  }

 private:
  PyObject* o_;
};

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

bool arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  return false;
}

typedef size_t (*WorkspaceFn)(const cpattn_tensor*, const cpattn_tensor*);

// rotary(entry, xs, positions, axes_dims, theta, interleaved, inverse, outs | None, stream | None)
//   -> (status, [outs])
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (!arguments(count, 9)) return nullptr;
  typedef cpattn_status (*Fn)(int, const cpattn_tensor*, const cpattn_tensor*, int, const int32_t*, double, int, int,
                              cpattn_tensor*, void*);
  const Fn fn = reinterpret_cast<Fn>(PyLong_AsVoidPtr(a[0]));
  Owned xs(PySequence_Fast(a[1], "xs is a sequence of tensors"));
  if (!xs) return nullptr;
  Owned axes(PySequence_Fast(a[3], "axes_dims is a sequence of whole numbers"));
  if (!axes) return nullptr;
  Owned outs(a[7] != Py_None ? PySequence_Fast(a[7], "outs is a sequence of tensors") : nullptr);
  if (a[7] != Py_None && !outs) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(xs.get());
  const Py_ssize_t n_axes = PySequence_Fast_GET_SIZE(axes.get());
  if (outs && PySequence_Fast_GET_SIZE(outs.get()) != n) {
    PyErr_Format(PyExc_ValueError, "%zd tensors but %zd outputs", n, PySequence_Fast_GET_SIZE(outs.get()));
    return nullptr;
  }
  if (n < 1 || n > CPATTN_MAX_PERMUTE_BATCH || n_axes > CPATTN_MAX_ROTARY_AXES)
    return Py_BuildValue("iO", static_cast<int>(CPATTN_ERR_SHAPE), Py_None);
  int32_t dims[CPATTN_MAX_ROTARY_AXES + 1] = {};
  for (Py_ssize_t i = 0; i < n_axes; ++i) {
    int overflow = 0;
    const long d = PyLong_AsLongAndOverflow(PySequence_Fast_GET_ITEM(axes.get(), i), &overflow);
    if (d == -1 && PyErr_Occurred()) return nullptr;
    dims[i] = overflow != 0 || d > (1 << 30) || d < 0 ? -1 : static_cast<int32_t>(d);   // (refused by the library)
  }
  const double theta = PyFloat_AsDouble(a[4]);
  const int interleaved = PyObject_IsTrue(a[5]), inverse = PyObject_IsTrue(a[6]);
  if (PyErr_Occurred()) return nullptr;
  Call call;
  cpattn_tensor x[CPATTN_MAX_PERMUTE_BATCH], y[CPATTN_MAX_PERMUTE_BATCH], pos;
  const Tensor* in[CPATTN_MAX_PERMUTE_BATCH];
  for (Py_ssize_t i = 0; i < n; ++i) in[i] = call.input(PySequence_Fast_GET_ITEM(xs.get(), i));
  const Tensor* positions = call.input(a[2]);
  if (!call.ok) return nullptr;
  call.enter(a[8]);
  for (Py_ssize_t i = 0; i < n; ++i) call.describe(*call.dense_rows(in[i]), &x[i]);
  call.describe(*positions, &pos);
  if (!call.ok) return nullptr;
  Owned list(PyList_New(n));
  if (!list) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor out = call.output(outs ? PySequence_Fast_GET_ITEM(outs.get(), i) : Py_None, *in[i]);
    if (call.ok) call.describe(out, &y[i]);
    if (!call.ok) return nullptr;
    PyObject* o = wrap(out);
    if (!o) return nullptr;
    PyList_SET_ITEM(list.get(), i, o);
  }
  cpattn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = fn(static_cast<int>(n), x, &pos, static_cast<int>(n_axes), dims, theta, interleaved, inverse, y, call.stream);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("iN", static_cast<int>(st), list.release());
  END_HANDLE_TH_ERRORS
}

// cross(entry, workspace_bytes entry, q, k, v, kv_lengths | None, scale, out | None, lse | None,
//       workspace | None, stream | None) -> (status, out, lse)
PyObject* cross(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (!arguments(count, 11)) return nullptr;
  typedef cpattn_status (*Fn)(const cpattn_tensor*, const cpattn_tensor*, const cpattn_tensor*, const cpattn_tensor*,
                              float, cpattn_tensor*, cpattn_tensor*, void*, size_t, void*);
  const Fn fn = reinterpret_cast<Fn>(PyLong_AsVoidPtr(a[0]));
  const WorkspaceFn bytes = reinterpret_cast<WorkspaceFn>(PyLong_AsVoidPtr(a[1]));
  const float scale = static_cast<float>(PyFloat_AsDouble(a[6]));
  if (PyErr_Occurred()) return nullptr;
  Call call;
  cpattn_tensor q, k, v, n, o, l;
  const Tensor* tq = call.input(a[2]);
  const Tensor* tk = call.input(a[3]);
  const Tensor* tv = call.input(a[4]);
  const Tensor* tn = a[5] != Py_None ? call.tensor(a[5]) : nullptr;
  if (!call.ok) return nullptr;
  call.enter(a[10]);
  call.describe(*call.dense(tq), &q);
  call.describe(*call.dense(tk), &k);
  call.describe(*call.dense(tv), &v);
  if (tn) call.describe(*call.dense(tn), &n, true);
  if (!call.ok) return nullptr;
  const Tensor out = call.output(a[7], *tq);
  if (call.ok) call.describe(out, &o);
  Tensor lse;
  if (call.ok) {
    if (a[8] != Py_None) {
      const Tensor* t = call.tensor(a[8]);
      if (t) lse = *t;
    } else {
      const auto sizes = tq->sizes();
      lse = call.made(call.fresh(sizes.slice(0, sizes.size() < 3 ? sizes.size() : 3), at::kFloat));
    }
  }
  if (call.ok) call.describe(lse, &l);
  const Tensor ws = call.workspace(a[9], call.ok && a[9] == Py_None ? bytes(&q, &k) : 0);
  if (!call.ok) return nullptr;
  void* ws_ptr = ws.defined() ? ws.data_ptr() : nullptr;
  const size_t ws_bytes = ws.defined() ? static_cast<size_t>(ws.nbytes()) : 0;
  cpattn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = fn(&q, &k, &v, tn ? &n : nullptr, scale, &o, &l, ws_ptr, ws_bytes, call.stream);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("iNN", static_cast<int>(st), wrap(out), wrap(lse));
  END_HANDLE_TH_ERRORS
}

// cross_backward(entry, workspace_bytes entry, q, k, v, out, lse, dout, kv_lengths | None, scale,
//                dq | None, dk | None, dv | None, workspace | None, stream | None)
//   -> (status, dq, dk, dv)
PyObject* cross_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (!arguments(count, 15)) return nullptr;
  typedef cpattn_status (*Fn)(const cpattn_tensor*, const cpattn_tensor*, const cpattn_tensor*, const cpattn_tensor*,
                              const cpattn_tensor*, const cpattn_tensor*, const cpattn_tensor*, float, cpattn_tensor*,
                              cpattn_tensor*, cpattn_tensor*, void*, size_t, void*);
  const Fn fn = reinterpret_cast<Fn>(PyLong_AsVoidPtr(a[0]));
  const WorkspaceFn bytes = reinterpret_cast<WorkspaceFn>(PyLong_AsVoidPtr(a[1]));
  const float scale = static_cast<float>(PyFloat_AsDouble(a[9]));
  if (PyErr_Occurred()) return nullptr;
  Call call;
  cpattn_tensor in[6], n, grad[3];
  const Tensor* t[6];
  for (int i = 0; i < 6; ++i) t[i] = call.input(a[2 + i]);
  const Tensor* tn = a[8] != Py_None ? call.tensor(a[8]) : nullptr;
  if (!call.ok) return nullptr;
  call.enter(a[14]);
  for (int i = 0; i < 6; ++i) call.describe(*call.dense(t[i]), &in[i]);
  if (tn) call.describe(*call.dense(tn), &n, true);
  if (!call.ok) return nullptr;
  Tensor out[3];
  for (int i = 0; i < 3 && call.ok; ++i) {
    out[i] = call.output(a[10 + i], *t[i]);
    if (call.ok) call.describe(out[i], &grad[i]);
  }
  const Tensor ws = call.workspace(a[13], call.ok && a[13] == Py_None ? bytes(&in[0], &in[1]) : 0);
  if (!call.ok) return nullptr;
  void* ws_ptr = ws.defined() ? ws.data_ptr() : nullptr;
  const size_t ws_bytes = ws.defined() ? static_cast<size_t>(ws.nbytes()) : 0;
  cpattn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = fn(&in[0], &in[1], &in[2], &in[3], &in[4], &in[5], tn ? &n : nullptr, scale, &grad[0], &grad[1],
          &grad[2], ws_ptr, ws_bytes, call.stream);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("iNNN", static_cast<int>(st), wrap(out[0]), wrap(out[1]), wrap(out[2]));
  END_HANDLE_TH_ERRORS
}

#define CPATTN_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CPATTN_METHOD(rotary), CPATTN_METHOD(cross), CPATTN_METHOD(cross_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
