// calls.h: what the compiled Python calls of train.py and tune.py share: their checks of
// arguments, the tensors that they allocate, their errors.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <initializer_list>
#include <string>

#include "../../include/lp_train.h"

namespace {

PyObject* lp_error = nullptr;  // the LpError class

// A Python error that has been set, or is to be.
struct Refused {
  PyObject* type = nullptr;
  std::string message;
};
[[noreturn]] void value_error(const std::string& m) { throw Refused{PyExc_ValueError, m}; }
[[noreturn]] void type_error(const std::string& m) { throw Refused{PyExc_TypeError, m}; }

void check_status(const char* entry, lp_status status) {
  if (status == LP_OK) return;
  PyObject* error = PyObject_CallFunction(lp_error, "si", entry, int(status));
  if (error != nullptr) {
    PyErr_SetObject(lp_error, error);
    Py_DECREF(error);
  }
  throw Refused{};
}

// An argument: a tensor, or null for None.
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& required(PyObject* o, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (t == nullptr) type_error(std::string(what) + " must be a tensor");
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

void* data(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
void* data(const at::Tensor& t) { return t.data_ptr(); }
float* floats(const at::Tensor* t) { return static_cast<float*>(data(t)); }
float* floats(const at::Tensor& t) { return static_cast<float*>(data(t)); }

int dtype_code(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return LP_BFLOAT16;
  if (t.scalar_type() == at::kFloat) return LP_FLOAT32;
  type_error(std::string(what) + " must be float32 or bfloat16");
}
const char* name_of(at::ScalarType s) {
  switch (s) {
    case at::kFloat: return "float32";
    case at::kBFloat16: return "bfloat16";
    case at::kLong: return "int64";
    case at::kByte: return "uint8";
    default: return "bool";
  }
}
void same_dtype(const at::Tensor* t, at::ScalarType s, const char* what) {
  if (t != nullptr && t->scalar_type() != s)
    type_error(std::string(what) + " must be " + name_of(s));
}
void vector(const at::Tensor* t, int64_t n, const char* what, at::ScalarType s = at::kFloat) {
  if (t == nullptr) return;
  same_dtype(t, s, what);
  if (t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    value_error(std::string(what) + " must be a contiguous vector of " + std::to_string(n));
}
// The bytes of a workspace that the caller gives: all that its elements span, each once.
size_t workspace_bytes(const at::Tensor& t) {
  if (!t.is_contiguous()) value_error("workspace must be contiguous");
  return t.nbytes();
}
// Row stride of a 2-D operand; a single row may have any.
int64_t row_stride(const at::Tensor* t, int64_t T, int64_t d, const char* what) {
  if (t == nullptr) return 0;
  if (t->dim() != 2 || t->size(0) != T || t->size(1) != d)
    value_error(std::string(what) + " must have the shape (" + std::to_string(T) + ", " +
                std::to_string(d) + ")");
  if (d > 1 && t->stride(1) != 1) value_error(std::string(what) + " must have contiguous rows");
  return T > 1 ? t->stride(0) : d;
}
// All on one CUDA device: that of the first.
c10::Device device_of(const at::Tensor& first, std::initializer_list<const at::Tensor*> others) {
  if (!first.is_cuda()) value_error("expected CUDA tensors");
  for (const at::Tensor* t : others)
    if (t != nullptr && (!t->is_cuda() || t->get_device() != first.get_device()))
      value_error("expected CUDA tensors of one device");
  return first.device();
}
void* current_stream(c10::Device device) {
  return c10::cuda::getCurrentCUDAStream(device.index()).stream();
}
// The memory of a tensor that the caller cannot see or may drop is not handed out again before the
// call on this stream is done.  (On the stream that it was allocated on this changes nothing.)
void used_on(c10::cuda::CUDAStream stream, const at::Tensor* t) {
  if (t != nullptr) c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), stream);
}
// Tells autograd that a call has written a tensor of the caller's: a graph that saved the old values
// refuses to go back through the new ones.
void written_in_place(const at::Tensor* t) {
  if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType s, c10::Device device) {
  return at::empty(sizes, at::TensorOptions().dtype(s).device(device));
}

// The tensors that a call allocates.  An allocation takes 1 us on the host, half of what a launch
// does, so the small ones of one dtype, and all of one dtype of a small call's, are parts of one;
// large ones are allocated each, so that none keeps another's memory.  Tensors of two dtypes share
// none: torch.save refuses them.
class Tensors {
 public:
  explicit Tensors(c10::Device device) : device_(device) {}
  // A tensor to be allocated, contiguous; `out` is set by allocate().
  void add(at::Tensor* out, std::initializer_list<int64_t> sizes, at::ScalarType type) {
    Item& item = items_[count_++];
    item = {out, {1, 1}, int(sizes.size()), type, type, int64_t(c10::elementSize(type))};
    int i = 0;
    for (int64_t n : sizes) item.bytes *= item.sizes[i++] = n;
    item.bytes = (item.bytes + 255) / 256 * 256;
    all_ += item.bytes;
  }
  // Scratch of so many bytes.  It is a part of the float32 tensors' allocation if it is next to
  // nothing, and is not kept by what the call returns otherwise.
  void scratch(at::Tensor* out, size_t bytes) {
    const int64_t n = std::max<int64_t>(int64_t(bytes), 256);
    if (n > 256) {
      *out = empty({n}, at::kByte, device_);
      return;
    }
    add(out, {n}, at::kByte);
    items_[count_ - 1].with = at::kFloat;
  }
  void allocate() {
    const int64_t part = all_ <= kSmallCall ? kSmallCall : kSmallTensor;  // the largest part
    for (at::ScalarType type : {at::kFloat, at::kBFloat16}) {
      int64_t together = 0, at = 0;
      for (int i = 0; i < count_; ++i)
        if (items_[i].with == type && items_[i].bytes <= part) together += items_[i].bytes;
      at::Tensor whole;
      for (int i = 0; i < count_; ++i) {
        const Item& item = items_[i];
        if (item.with != type) continue;
        const at::IntArrayRef sizes(item.sizes, size_t(item.dims));
        if (item.bytes > part) {
          *item.out = empty(sizes, item.type, device_);
          continue;
        }
        if (!whole.defined()) whole = empty({together}, at::kByte, device_);
        *item.out = at::detail::make_tensor<c10::TensorImpl>(
            c10::Storage(whole.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
            c10::scalarTypeToTypeMeta(item.type));
        c10::TensorImpl* impl = item.out->unsafeGetTensorImpl();
        impl->set_storage_offset(at / int64_t(c10::elementSize(item.type)));
        impl->set_sizes_contiguous(sizes);
        at += item.bytes;
      }
    }
  }

 private:
  static constexpr int64_t kSmallTensor = 64 << 10, kSmallCall = 256 << 10;
  struct Item {
    at::Tensor* out;
    int64_t sizes[2];
    int dims;
    at::ScalarType type;
    at::ScalarType with;  // the dtype whose allocation it is a part of
    int64_t bytes;
  };
  c10::Device device_;
  Item items_[8];
  int count_ = 0;
  int64_t all_ = 0;
};

// A tuple of tensors, None for undefined ones.
PyObject* tuple_of(std::initializer_list<const at::Tensor*> tensors) {
  PyObject* out = PyTuple_New(Py_ssize_t(tensors.size()));
  if (out == nullptr) throw Refused{};
  Py_ssize_t i = 0;
  for (const at::Tensor* t : tensors) {
    PyObject* o = Py_None;
    if (t->defined())
      o = THPVariable_Wrap(*t);
    else
      Py_INCREF(o);
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// Keeps what an optimizer's step reads and writes until it is done, wherever it runs: the plan and
// the moments, and the tensors that the optimizer was given where the step is on a stream that is not
// in `streams`: those that have it on record (which lasts as long as the tensor), and the one that
// the plan was laid out on.  A captured step reads its plan and gradients at every replay:
// `captured` keeps them.
void keep_for_step(c10::cuda::CUDAStream stream, PyObject* plan,
                   std::initializer_list<const at::Tensor*> moments, PyObject* written, PyObject* grads,
                   PyObject* streams, PyObject* captured) {
  if (!PyTuple_Check(written) || !PyTuple_Check(grads) || !PyList_Check(streams) || !PyList_Check(captured))
    type_error("expected tuples of tensors and lists");
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
    const Py_ssize_t last = PyList_GET_SIZE(captured) - 1;
    if (last >= 0 && PyTuple_GET_ITEM(PyList_GET_ITEM(captured, last), 0) == plan) return;
    PyObject* both = PyTuple_Pack(2, plan, grads);
    const int failed = both == nullptr ? -1 : PyList_Append(captured, both);
    Py_XDECREF(both);
    if (failed) throw Refused{};
    return;
  }
  used_on(stream, tensor(plan, "plan"));
  for (const at::Tensor* t : moments) used_on(stream, t);
  const int64_t handle = int64_t(reinterpret_cast<intptr_t>(stream.stream()));
  for (Py_ssize_t i = 0; i < PyList_GET_SIZE(streams); ++i)
    if (integer(PyList_GET_ITEM(streams, i)) == handle) return;
  for (PyObject* tensors : {written, grads})
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tensors); ++i)
      used_on(stream, &required(PyTuple_GET_ITEM(tensors, i), "a tensor of the step"));
  PyObject* seen = PyLong_FromLongLong(handle);
  const int failed = seen == nullptr ? -1 : PyList_Append(streams, seen);
  Py_XDECREF(seen);
  if (failed) throw Refused{};
}

template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t expected, F&& f) {
  HANDLE_TH_ERRORS
  if (given != expected) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, given);
    return nullptr;
  }
  if (lp_error == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    if (r.type != nullptr) PyErr_SetString(r.type, r.message.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(LpError, addresses): the entry points in the order of a module's table, of `kSlots` pointers.
PyObject* bind_table(void** slots, Py_ssize_t kSlots, PyObject* const* v, Py_ssize_t n) {
  if (n != 2 || !PyTuple_Check(v[1]) || PyTuple_GET_SIZE(v[1]) != kSlots) {
    PyErr_SetString(PyExc_TypeError, "bind(LpError, addresses)");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < kSlots; ++i) {
    slots[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(v[1], i));
    if (slots[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  Py_INCREF(v[0]);
  Py_XDECREF(lp_error);
  lp_error = v[0];
  Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

}  // namespace
