// PyTorch binding of the training operators (the calls that a training step
// makes most often, on tensors that may be small): argument checks, output
// allocation and the C ABI call of include/fp8opt.h in one native call.  The
// same steps taken in Python cost more than a small operator's kernel.
//
// It holds no arithmetic: everything goes through the C ABI, whose functions
// ops.py hands over by address from the library it has loaded (bind()).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>
#include <vector>

namespace {

using at::Tensor;
using at::ScalarType;

// The C entry points, in the order of ops.py's list (the last one gives the text
// of a call's error).
enum { kActSave, kActLoad, kGelu, kGeluBackward, kNorm, kNormBackward, kXent, kXentBackward,
       kEmbedding, kEmbeddingBackward, kPolicy, kPolicyBackward, kDistill, kDistillBackward,
       kLastError, kEntries };
void* g_fn[kEntries];
PyObject* g_fail = nullptr;   // ops.py's function that raises for a status

constexpr int64_t kGroup = 128;

// Reported as a Python exception of the given type.
struct Refusal {
  PyObject* type;
  std::string what;
};

[[noreturn]] void refuse(PyObject* type, const std::string& what) { throw Refusal{type, what}; }

int code(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return 0;
    case ScalarType::BFloat16: return 1;
    case ScalarType::Half: return 2;
    default: return -1;
  }
}

int dtype_of(const Tensor& t, const char* name) {
  const int c = code(t.scalar_type());
  if (c < 0)
    refuse(PyExc_TypeError, std::string(name) + ": unsupported dtype " + c10::toString(t.scalar_type()));
  return c;
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// A contiguous CUDA tensor on the first one's device.
struct Args {
  int device = -1;
  const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    if (t.layout() != at::kStrided || !t.is_contiguous())
      refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    if (device < 0) device = t.get_device();
    else if (t.get_device() != device) refuse(PyExc_ValueError, std::string(name) + " is on another device");
    return t;
  }
  const Tensor& tensor(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) {
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
      refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", not " +
                                  c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
      refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) +
                                   ", not " + shape_text(t.sizes()));
    return t;
  }
};

// Makes a stream (its handle, or None for the current one of the tensors'
// device) and its device current while outputs are allocated and the call is
// made.
class OnStream {
 public:
  OnStream(PyObject* stream, int device) : device_(device) {
    before_ = c10::cuda::current_device();
    if (before_ != device) c10::cuda::set_device(device);
    try {
      use(stream);
    } catch (...) {
      if (before_ != device_) c10::cuda::set_device(before_);
      throw;
    }
  }
  ~OnStream() {
    if (swapped_) c10::cuda::setCurrentCUDAStream(old_);
    if (before_ != device_) c10::cuda::set_device(before_);
  }
  void* handle = nullptr;

 private:
  void use(PyObject* stream) {
    old_ = c10::cuda::getCurrentCUDAStream(device_);
    if (stream != Py_None) {
      // torch.cuda.Stream's identity: (stream_id, device_index, device_type)
      PyObject* id = PyObject_GetAttrString(stream, "stream_id");
      PyObject* dev = id ? PyObject_GetAttrString(stream, "device_index") : nullptr;
      PyObject* kind = dev ? PyObject_GetAttrString(stream, "device_type") : nullptr;
      const bool ok = kind != nullptr;
      const long long i = ok ? PyLong_AsLongLong(id) : 0, d = ok ? PyLong_AsLongLong(dev) : 0,
                      k = ok ? PyLong_AsLongLong(kind) : 0;
      Py_XDECREF(id);
      Py_XDECREF(dev);
      Py_XDECREF(kind);
      if (!ok || PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "stream must be a torch.cuda.Stream");
      }
      if (d != device_) refuse(PyExc_ValueError, "stream is on another device than the tensors");
      c10::cuda::setCurrentCUDAStream(c10::cuda::CUDAStream::unpack3(
          i, (c10::DeviceIndex)d, (c10::DeviceType)k));
      swapped_ = true;
    }
    handle = c10::cuda::getCurrentCUDAStream(device_).stream();
  }
  int device_, before_ = 0;
  bool swapped_ = false;
  c10::cuda::CUDAStream old_ = c10::cuda::getDefaultCUDAStream();
};

Tensor fresh(at::IntArrayRef shape, ScalarType type, int device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
}

// The interpreter's lock, given up for a scope: taken back also where something
// in it throws.
struct Unlocked {
  Unlocked() : state(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state); }
  Unlocked(const Unlocked&) = delete;
  PyThreadState* state;
};

bool out_of_memory() {
  const char* text = reinterpret_cast<const char* (*)()>(g_fn[kLastError])();
  return std::strstr(text, "cudaErrorMemoryAllocation") != nullptr;
}

// Calls C entry point i without the interpreter's lock; raises for a status.
// The library's scratch is not torch's memory: where there is no room for it,
// torch gives back what it caches, as for an allocation of its own.
template <class... T>
void call(int i, T... a) {
  int status = 0;
  {
    Unlocked scope;
    const auto fn = reinterpret_cast<int (*)(T...)>(g_fn[i]);
    status = fn(a...);
    if (status != 0 && out_of_memory()) {
      c10::cuda::CUDACachingAllocator::emptyCache();
      status = fn(a...);
    }
  }
  if (status == 0) return;
  PyObject* r = PyObject_CallFunction(g_fail, "i", status);   // raises
  Py_XDECREF(r);
  throw python_error();
}

template <class... T>
PyObject* give(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(T));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  const auto put = [&](const Tensor& x) {
    PyObject* o = x.defined() ? THPVariable_Wrap(x) : (Py_INCREF(Py_None), Py_None);
    PyTuple_SET_ITEM(r, i++, o);
    if (o == nullptr) {
      Py_DECREF(r);
      throw python_error();
    }
  };
  (put(t), ...);
  return r;
}

template <class F>
PyObject* entry(Py_ssize_t got, Py_ssize_t want, F f) {
  HANDLE_TH_ERRORS
  if (got != want) refuse(PyExc_TypeError, "wrong number of arguments");
  return f();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  END_HANDLE_TH_ERRORS
}

int64_t groups(const Tensor& t) { return (t.numel() + kGroup - 1) / kGroup; }

int form_of(PyObject* o) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "none") == 0) return 0;
    if (PyUnicode_CompareWithASCIIString(o, "tanh") == 0) return 1;
  }
  refuse(PyExc_ValueError, "approximate must be 'none' or 'tanh'");
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be a number");
  }
  return (float)v;
}

int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be a 64-bit integer");
  }
  return v;
}

// act_save(x, stream) -> codes, scales
PyObject* act_save(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 2, [&] {
    Args args;
    const Tensor& x = args.tensor(a[0], "x");
    const int dt = dtype_of(x, "x");
    OnStream on(a[1], args.device);
    const Tensor codes = fresh(x.sizes(), ScalarType::Byte, args.device);
    const Tensor scales = fresh({groups(x)}, ScalarType::Float, args.device);
    call(kActSave, x.data_ptr(), x.numel(), dt, codes.data_ptr(), scales.data_ptr(), on.handle);
    return give(codes, scales);
  });
}

void checkpoint(Args& args, PyObject* codes, PyObject* scales, const Tensor** c,
                const Tensor** s) {
  *c = &args.tensor(codes, "codes");
  if ((*c)->scalar_type() != ScalarType::Byte) refuse(PyExc_TypeError, "codes must be uint8");
  *s = &args.tensor(scales, "scales", ScalarType::Float, {groups(**c)});
}

// act_load(codes, scales, dtype code, stream) -> (x,)
PyObject* act_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 4, [&] {
    Args args;
    const Tensor *c, *s;
    checkpoint(args, a[0], a[1], &c, &s);
    const int dt = (int)whole(a[2], "dtype");
    const ScalarType type = dt == 0 ? ScalarType::Float : dt == 1 ? ScalarType::BFloat16
                                                                  : ScalarType::Half;
    OnStream on(a[3], args.device);
    const Tensor x = fresh(c->sizes(), type, args.device);
    call(kActLoad, c->data_ptr(), s->data_ptr(), c->numel(), dt, x.data_ptr(), on.handle);
    return give(x);
  });
}

// gelu(x, approximate, stream) -> y, codes, scales
PyObject* gelu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 3, [&] {
    Args args;
    const Tensor& x = args.tensor(a[0], "x");
    const int dt = dtype_of(x, "x"), form = form_of(a[1]);
    OnStream on(a[2], args.device);
    const Tensor y = fresh(x.sizes(), x.scalar_type(), args.device);
    const Tensor codes = fresh(x.sizes(), ScalarType::Byte, args.device);
    const Tensor scales = fresh({groups(x)}, ScalarType::Float, args.device);
    call(kGelu, x.data_ptr(), x.numel(), dt, form, y.data_ptr(), codes.data_ptr(), scales.data_ptr(),
        on.handle);
    return give(y, codes, scales);
  });
}

// gelu_backward(dy, codes, scales, approximate, stream) -> (dx,)
PyObject* gelu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 5, [&] {
    Args args;
    const Tensor& dy = args.tensor(a[0], "dy");
    const int dt = dtype_of(dy, "dy"), form = form_of(a[3]);
    const Tensor *c, *s;
    checkpoint(args, a[1], a[2], &c, &s);
    args.tensor(a[1], "codes", ScalarType::Byte, dy.sizes());
    OnStream on(a[4], args.device);
    const Tensor dx = fresh(dy.sizes(), dy.scalar_type(), args.device);
    call(kGeluBackward, dy.data_ptr(), c->data_ptr(), s->data_ptr(), dy.numel(), dt, form,
                       dx.data_ptr(), on.handle);
    return give(dx);
  });
}

int64_t columns(const Tensor& t, const char* name) {
  if (t.dim() < 1 || t.size(-1) < 1)
    refuse(PyExc_ValueError, std::string(name) + " needs a last dimension of at least 1");
  return t.size(-1);
}

// A parameter vector of the row's length.
const Tensor& parameter(Args& args, PyObject* o, const char* name, int64_t cols) {
  const Tensor& t = args.tensor(o, name);
  if (t.dim() != 1 || t.size(0) != cols)
    refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text({cols}) +
                                 ", not " + shape_text(t.sizes()));
  return t;
}

// layer_norm(x, weight, bias or None, eps, fp8, stream)
//   -> y, mean, rstd, or y, codes, scales, rstd with fp8
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 6, [&] {
    Args args;
    const Tensor& x = args.tensor(a[0], "x");
    const int dt = dtype_of(x, "x");
    const int64_t cols = columns(x, "x");
    const Tensor& w = parameter(args, a[1], "weight", cols);
    const int wdt = dtype_of(w, "weight");
    const void* b = a[2] == Py_None
                        ? nullptr : args.tensor(a[2], "bias", w.scalar_type(), {cols}).data_ptr();
    const float eps = number(a[3], "eps");
    const bool fp8 = a[4] == Py_True;
    const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
    OnStream on(a[5], args.device);
    const Tensor y = fresh(x.sizes(), x.scalar_type(), args.device);
    const Tensor rstd = fresh(lead, ScalarType::Float, args.device);
    const Tensor codes = fp8 ? fresh(x.sizes(), ScalarType::Byte, args.device) : Tensor();
    const Tensor other = fresh(lead, ScalarType::Float, args.device);   // scales, or mean
    call(kNorm, x.data_ptr(), w.data_ptr(), b, x.numel() / cols, cols, dt, wdt, eps, y.data_ptr(),
        fp8 ? nullptr : other.data_ptr(), rstd.data_ptr(), fp8 ? codes.data_ptr() : nullptr,
        fp8 ? other.data_ptr() : nullptr, on.handle);
    return fp8 ? give(y, codes, other, rstd) : give(y, other, rstd);
  });
}

// layer_norm_backward(dy, weight, rstd, x, mean, codes, scales, need_bias,
// stream) -> dx, dweight, dbias (None without need_bias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 9, [&] {
    Args args;
    const Tensor& dy = args.tensor(a[0], "dy");
    const int dt = dtype_of(dy, "dy");
    const int64_t cols = columns(dy, "dy");
    const at::IntArrayRef lead = dy.sizes().slice(0, dy.dim() - 1);
    const Tensor& w = parameter(args, a[1], "weight", cols);
    const int wdt = dtype_of(w, "weight");
    const Tensor& rstd = args.tensor(a[2], "rstd", ScalarType::Float, lead);
    const bool whole_x = a[3] != Py_None && a[4] != Py_None && a[5] == Py_None && a[6] == Py_None;
    const bool fp8 = a[3] == Py_None && a[4] == Py_None && a[5] != Py_None && a[6] != Py_None;
    if (!whole_x && !fp8) refuse(PyExc_ValueError, "give x and mean, or codes and scales");
    const void *x = nullptr, *mean = nullptr, *codes = nullptr, *scales = nullptr;
    if (fp8) {
      codes = args.tensor(a[5], "codes", ScalarType::Byte, dy.sizes()).data_ptr();
      scales = args.tensor(a[6], "scales", ScalarType::Float, lead).data_ptr();
    } else {
      x = args.tensor(a[3], "x", dy.scalar_type(), dy.sizes()).data_ptr();
      mean = args.tensor(a[4], "mean", ScalarType::Float, lead).data_ptr();
    }
    const bool need_bias = a[7] == Py_True;
    OnStream on(a[8], args.device);
    const Tensor dx = fresh(dy.sizes(), dy.scalar_type(), args.device);
    const Tensor dw = fresh({cols}, w.scalar_type(), args.device);
    const Tensor db = need_bias ? fresh({cols}, w.scalar_type(), args.device) : Tensor();
    call(kNormBackward, dy.data_ptr(), x, mean, codes, scales, rstd.data_ptr(), w.data_ptr(),
                       dy.numel() / cols, cols, dt, wdt, dx.data_ptr(), dw.data_ptr(),
                       need_bias ? db.data_ptr() : nullptr, on.handle);
    return give(dx, dw, db);
  });
}

// The linear layer of the cross entropy and of distillation.
struct Linear {
  const Tensor *x, *w, *target;
  int64_t rows, dim, vocab, ignore;
  int dt;
};

Linear linear_layer(Args& args, PyObject* x, PyObject* w) {
  Linear l = {};
  l.x = &args.tensor(x, "x");
  l.dt = dtype_of(*l.x, "x");
  if (l.dt == 0) refuse(PyExc_TypeError, "x must be bfloat16 or float16");
  if (l.x->dim() != 2 || l.x->size(1) < 1)
    refuse(PyExc_ValueError, "x must have shape (tokens, dim)");
  l.w = &args.tensor(w, "w");
  if (l.w->scalar_type() != l.x->scalar_type())
    refuse(PyExc_TypeError, std::string("w must be ") + c10::toString(l.x->scalar_type()) +
                                ", not " + c10::toString(l.w->scalar_type()));
  if (l.w->dim() != 2 || l.w->size(0) < 1 || l.w->size(1) != l.x->size(1))
    refuse(PyExc_ValueError, "w must have shape (vocabulary, " + std::to_string(l.x->size(1)) +
                                 "), not " + shape_text(l.w->sizes()));
  l.rows = l.x->size(0);
  l.dim = l.x->size(1);
  l.vocab = l.w->size(0);
  return l;
}

Linear linear(Args& args, PyObject* x, PyObject* w, PyObject* target, PyObject* ignore) {
  Linear l = linear_layer(args, x, w);
  l.target = &args.tensor(target, "target", ScalarType::Long, {l.rows});
  l.ignore = whole(ignore, "ignore_index");
  return l;
}

// linear_cross_entropy(x, w, target, ignore_index, stream) -> loss, lse
PyObject* xent(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 5, [&] {
    Args args;
    const Linear l = linear(args, a[0], a[1], a[2], a[3]);
    OnStream on(a[4], args.device);
    const Tensor loss = fresh({l.rows}, ScalarType::Float, args.device);
    const Tensor lse = fresh({l.rows}, ScalarType::Float, args.device);
    call(kXent, l.x->data_ptr(), l.w->data_ptr(), l.target->data_ptr(), l.rows, l.dim, l.vocab, l.dt,
        l.ignore, loss.data_ptr(), lse.data_ptr(), on.handle);
    return give(loss, lse);
  });
}

// linear_cross_entropy_backward(dloss, x, w, target, lse, ignore_index, stream)
//   -> dx, dw
PyObject* xent_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&] {
    Args args;
    const Linear l = linear(args, a[1], a[2], a[3], a[5]);
    const Tensor& dloss = args.tensor(a[0], "dloss", ScalarType::Float, {l.rows});
    const Tensor& lse = args.tensor(a[4], "lse", ScalarType::Float, {l.rows});
    OnStream on(a[6], args.device);
    const Tensor dx = fresh(l.x->sizes(), l.x->scalar_type(), args.device);
    const Tensor dw = fresh(l.w->sizes(), l.w->scalar_type(), args.device);
    call(kXentBackward, dloss.data_ptr(), l.x->data_ptr(), l.w->data_ptr(), l.target->data_ptr(), lse.data_ptr(),
        l.rows, l.dim, l.vocab, l.dt, l.ignore, dx.data_ptr(), dw.data_ptr(), on.handle);
    return give(dx, dw);
  });
}

// embedding(ids, w, scale, stream) -> (y,)
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 4, [&] {
    Args args;
    const Tensor& ids = args.tensor(a[0], "ids");
    if (ids.scalar_type() != ScalarType::Long)
      refuse(PyExc_TypeError, std::string("ids must be Long, not ") + c10::toString(ids.scalar_type()));
    const Tensor& w = args.tensor(a[1], "w");
    const int dt = dtype_of(w, "w");
    if (w.dim() != 2 || w.size(0) < 1 || w.size(1) < 1)
      refuse(PyExc_ValueError, "w must have shape (vocabulary, dim), not " + shape_text(w.sizes()));
    const float scale = number(a[2], "scale");
    std::vector<int64_t> shape(ids.sizes().begin(), ids.sizes().end());
    shape.push_back(w.size(1));
    OnStream on(a[3], args.device);
    const Tensor y = fresh(shape, w.scalar_type(), args.device);
    call(kEmbedding, ids.data_ptr(), w.data_ptr(), ids.numel(), w.size(1), w.size(0), dt, scale,
         y.data_ptr(), on.handle);
    return give(y);
  });
}

// embedding_backward(dy, ids, vocab, scale, padding_idx or None, stream) -> (dw,)
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 6, [&] {
    Args args;
    const Tensor& dy = args.tensor(a[0], "dy");
    const int dt = dtype_of(dy, "dy");
    const int64_t dim = columns(dy, "dy");
    const Tensor& ids = args.tensor(a[1], "ids", ScalarType::Long,
                                    dy.sizes().slice(0, dy.dim() - 1));
    const int64_t vocab = whole(a[2], "vocab");
    if (vocab < 1) refuse(PyExc_ValueError, "vocab must be at least 1");
    const float scale = number(a[3], "scale");
    const int64_t padding = a[4] == Py_None ? -1 : whole(a[4], "padding_idx");
    if (a[4] != Py_None && (padding < 0 || padding >= vocab))
      refuse(PyExc_ValueError, "padding_idx must be in [0, vocab)");
    OnStream on(a[5], args.device);
    const Tensor dw = fresh({vocab, dim}, dy.scalar_type(), args.device);
    call(kEmbeddingBackward, dy.data_ptr(), ids.data_ptr(), ids.numel(), dim, vocab, dt, scale,
         padding, dw.data_ptr(), on.handle);
    return give(dw);
  });
}

// What both directions of the policy loss take.
struct Policy {
  const Tensor* logp;
  const void *old_logp, *advantage, *mask = nullptr, *ref = nullptr;
  int64_t batch, length;
  int per_token;
  double low, high, kl;
};

double real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be a number");
  }
  return v;
}

// a: logp, old_logp, advantage, mask or None, ref_logp or None, clip_low,
// clip_high, kl_coef
Policy policy(Args& args, PyObject* const* a) {
  Policy p;
  p.logp = &args.tensor(a[0], "logp");
  if (p.logp->scalar_type() != ScalarType::Float)
    refuse(PyExc_TypeError, std::string("logp must be Float, not ") +
                                c10::toString(p.logp->scalar_type()));
  if (p.logp->dim() != 2)
    refuse(PyExc_ValueError, "logp must have shape (batch, length), not " +
                                 shape_text(p.logp->sizes()));
  const at::IntArrayRef shape = p.logp->sizes();
  p.batch = shape[0];
  p.length = shape[1];
  p.old_logp = args.tensor(a[1], "old_logp", ScalarType::Float, shape).data_ptr();
  const Tensor& adv = args.tensor(a[2], "advantage");
  p.per_token = adv.dim() == 2;
  p.advantage = args.tensor(a[2], "advantage", ScalarType::Float,
                            p.per_token ? shape : shape.slice(0, 1)).data_ptr();
  if (a[3] != Py_None) p.mask = args.tensor(a[3], "mask", ScalarType::Bool, shape).data_ptr();
  if (a[4] != Py_None) p.ref = args.tensor(a[4], "ref_logp", ScalarType::Float, shape).data_ptr();
  p.low = real(a[5], "clip_low");
  p.high = real(a[6], "clip_high");
  p.kl = real(a[7], "kl_coef");
  return p;
}

// policy_loss(logp, old_logp, advantage, mask, ref_logp, clip_low, clip_high,
// kl_coef, reduction code, stream) -> stats, weight
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&] {
    Args args;
    const Policy p = policy(args, a);
    const int reduction = (int)whole(a[8], "reduction");
    OnStream on(a[9], args.device);
    const Tensor stats = fresh({4}, ScalarType::Float, args.device);
    const Tensor weight = fresh({p.batch}, ScalarType::Float, args.device);
    call(kPolicy, p.logp->data_ptr(), p.old_logp, p.advantage, p.mask, p.ref, p.batch, p.length,
         p.per_token, p.low, p.high, p.kl, reduction, stats.data_ptr(), weight.data_ptr(),
         on.handle);
    return give(stats, weight);
  });
}

// policy_loss_backward(dloss, weight, logp, old_logp, advantage, mask, ref_logp,
// clip_low, clip_high, kl_coef, stream) -> (dlogp,)
PyObject* policy_loss_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 11, [&] {
    Args args;
    const Policy p = policy(args, a + 2);
    const Tensor& dloss = args.tensor(a[0], "dloss");
    if (dloss.scalar_type() != ScalarType::Float)
      refuse(PyExc_TypeError, std::string("dloss must be Float, not ") +
                                  c10::toString(dloss.scalar_type()));
    if (dloss.numel() != 1) refuse(PyExc_ValueError, "dloss must have one element");
    const Tensor& weight = args.tensor(a[1], "weight", ScalarType::Float, {p.batch});
    OnStream on(a[10], args.device);
    const Tensor dlogp = fresh(p.logp->sizes(), ScalarType::Float, args.device);
    call(kPolicyBackward, dloss.data_ptr(), p.logp->data_ptr(), p.old_logp, p.advantage,
         weight.data_ptr(), p.mask, p.ref, p.batch, p.length, p.per_token, p.low, p.high, p.kl,
         dlogp.data_ptr(), on.handle);
    return give(dlogp);
  });
}

// The teacher's top logits of a linear layer's tokens.
struct Top {
  const Tensor *ids, *logits;
  int k, dt;
  float temperature;
};

Top teacher(Args& args, const Linear& l, PyObject* ids, PyObject* logits, PyObject* temperature) {
  Top t;
  t.ids = &args.tensor(ids, "ids");
  if (t.ids->scalar_type() != ScalarType::Long)
    refuse(PyExc_TypeError, std::string("ids must be Long, not ") +
                                c10::toString(t.ids->scalar_type()));
  if (t.ids->dim() != 2 || t.ids->size(0) != l.rows || t.ids->size(1) < 1 || t.ids->size(1) > 256)
    refuse(PyExc_ValueError, "ids must have shape (" + std::to_string(l.rows) +
                                 ", 1 to 256), not " + shape_text(t.ids->sizes()));
  t.logits = &args.tensor(logits, "logits");
  t.dt = dtype_of(*t.logits, "logits");
  args.tensor(logits, "logits", t.logits->scalar_type(), t.ids->sizes());
  t.k = (int)t.ids->size(1);
  t.temperature = number(temperature, "temperature");
  return t;
}

// linear_distillation(x, w, ids, logits, temperature, stream) -> loss, lse
PyObject* distill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 6, [&] {
    Args args;
    const Linear l = linear_layer(args, a[0], a[1]);
    const Top t = teacher(args, l, a[2], a[3], a[4]);
    OnStream on(a[5], args.device);
    const Tensor loss = fresh({l.rows}, ScalarType::Float, args.device);
    const Tensor lse = fresh({l.rows}, ScalarType::Float, args.device);
    call(kDistill, l.x->data_ptr(), l.w->data_ptr(), t.ids->data_ptr(), t.logits->data_ptr(),
         l.rows, l.dim, l.vocab, t.k, l.dt, t.dt, t.temperature, loss.data_ptr(), lse.data_ptr(),
         on.handle);
    return give(loss, lse);
  });
}

// linear_distillation_backward(dloss, x, w, ids, logits, lse, temperature, stream)
//   -> dx, dw
PyObject* distill_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 8, [&] {
    Args args;
    const Linear l = linear_layer(args, a[1], a[2]);
    const Top t = teacher(args, l, a[3], a[4], a[6]);
    const Tensor& dloss = args.tensor(a[0], "dloss", ScalarType::Float, {l.rows});
    const Tensor& lse = args.tensor(a[5], "lse", ScalarType::Float, {l.rows});
    OnStream on(a[7], args.device);
    const Tensor dx = fresh(l.x->sizes(), l.x->scalar_type(), args.device);
    const Tensor dw = fresh(l.w->sizes(), l.w->scalar_type(), args.device);
    call(kDistillBackward, dloss.data_ptr(), l.x->data_ptr(), l.w->data_ptr(), t.ids->data_ptr(),
         t.logits->data_ptr(), lse.data_ptr(), l.rows, l.dim, l.vocab, t.k, l.dt, t.dt,
         t.temperature, dx.data_ptr(), dw.data_ptr(), on.handle);
    return give(dx, dw);
  });
}

// bind(addresses of the C entry points, function that raises for a status)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, kEntries + 1, [&]() -> PyObject* {
    for (int i = 0; i < kEntries; ++i) {
      g_fn[i] = PyLong_AsVoidPtr(a[i]);
      if (PyErr_Occurred()) throw python_error();
    }
    Py_INCREF(a[kEntries]);
    Py_XSETREF(g_fail, a[kEntries]);
    Py_RETURN_NONE;
  });
}

#define METHOD(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    METHOD("bind", bind), METHOD("act_save", act_save), METHOD("act_load", act_load),
    METHOD("gelu", gelu), METHOD("gelu_backward", gelu_backward),
    METHOD("layer_norm", layer_norm), METHOD("layer_norm_backward", layer_norm_backward),
    METHOD("linear_cross_entropy", xent),
    METHOD("linear_cross_entropy_backward", xent_backward), METHOD("embedding", embedding),
    METHOD("embedding_backward", embedding_backward), METHOD("policy_loss", policy_loss),
    METHOD("policy_loss_backward", policy_loss_backward),
    METHOD("linear_distillation", distill),
    METHOD("linear_distillation_backward", distill_backward), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fp8opt_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fp8opt_binding() { return PyModule_Create(&g_module); }
