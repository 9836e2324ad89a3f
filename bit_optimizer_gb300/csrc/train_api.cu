// The C entry points of the training operators (include/fp8opt.h): argument
// checks, scratch, and the launches under the library lock.  Nothing is
// launched and no output touched on an argument error; no exception leaves an
// entry point.
#include <cmath>
#include <exception>
#include <string>

#include "../../include/fp8opt.h"
#include "ops_internal.cuh"

using namespace fp8opt;

namespace fp8opt {
namespace {

static_assert(kActGroup == FP8OPT_ACT_GROUP, "one group size");

// Most elements of one tensor: byte offsets of every type stay far from 2^63.
constexpr int64_t kMaxElems = (int64_t)1 << 40;

int bad(const char* fn, const char* what) {
  return record_error(FP8OPT_ERR_ARG, (std::string(fn) + ": " + what).c_str());
}

int unsupported(const char* fn, const char* what) {
  return record_error(FP8OPT_ERR_UNSUPPORTED, (std::string(fn) + ": " + what).c_str());
}

template <class F>
int entry(F f) {
  try {
    return f();
  } catch (const std::exception&) {
    try {
      return record_error(FP8OPT_ERR_LIMIT, "out of host memory");
    } catch (...) {
      return FP8OPT_ERR_LIMIT;
    }
  }
}

bool known(int dtype) {
  return dtype == FP8OPT_F32 || dtype == FP8OPT_BF16 || dtype == FP8OPT_F16;
}

template <class... P>
bool aligned_all(const P*... p) {
  return (((reinterpret_cast<uintptr_t>(p) & 15u) == 0) && ...);
}

int act_call(const char* fn, int act, bool fwd, const ActArgs& args, bool null,
             void* stream_ptr) {
  if (args.n < 0 || args.n > kMaxElems) return bad(fn, "numel outside [0, 2^40]");
  if (!known(args.dtype)) return unsupported(fn, "unknown dtype");
  if (args.n == 0) return FP8OPT_OK;
  if (null) return bad(fn, "NULL pointer");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  OpCall call;
  const int st = call.open(fn, stream, 0);
  if (st != FP8OPT_OK) return st;
  return call.done(fn, launch_act(act, fwd, args, call.sms, stream, call.mark));
}

// The activation kinds of the two GELU forms.
bool gelu_kind(int form, int* act) {
  *act = form == FP8OPT_GELU_TANH ? kActGeluTanh : kActGelu;
  return form == FP8OPT_GELU_ERF || form == FP8OPT_GELU_TANH;
}

int check_norm(const char* fn, int64_t rows, int64_t cols, int dtype, int wdtype) {
  if (rows < 0 || cols < 1 || cols > kMaxElems || rows > kMaxElems ||
      (rows > 0 && cols > kMaxElems / rows))
    return bad(fn, "rows < 0, cols < 1, or more than 2^40 elements");
  if (!known(dtype) || !known(wdtype)) return unsupported(fn, "unknown dtype");
  return FP8OPT_OK;
}

}  // namespace
}  // namespace fp8opt

extern "C" int fp8_act_save(const void* x, int64_t numel, int dtype, uint8_t* codes,
                            float* scales, void* stream) {
  return entry([&] {
    ActArgs a = {};
    a.x = x;
    a.n = numel;
    a.dtype = dtype;
    a.codes_out = codes;
    a.scales_out = scales;
    a.vec_ok = aligned_all(x, codes);
    return act_call("fp8_act_save", kActSave, true, a, !x || !codes || !scales, stream);
  });
}

extern "C" int fp8_act_load(const uint8_t* codes, const float* scales, int64_t numel,
                            int dtype, void* x, void* stream) {
  return entry([&] {
    ActArgs a = {};
    a.n = numel;
    a.dtype = dtype;
    a.codes = codes;
    a.scales = scales;
    a.out = x;
    a.vec_ok = aligned_all(x, codes);
    return act_call("fp8_act_load", kActSave, false, a, !x || !codes || !scales, stream);
  });
}

extern "C" int fp8_gelu(const void* x, int64_t numel, int dtype, int form, void* y,
                        uint8_t* codes, float* scales, void* stream) {
  return entry([&] {
    int act = 0;
    if (!gelu_kind(form, &act)) return unsupported("fp8_gelu", "unknown form");
    ActArgs a = {};
    a.x = x;
    a.n = numel;
    a.dtype = dtype;
    a.out = y;
    a.codes_out = codes;
    a.scales_out = scales;
    a.vec_ok = aligned_all(x, y, codes);
    return act_call("fp8_gelu", act, true, a, !x || !y || !codes || !scales, stream);
  });
}

extern "C" int fp8_gelu_backward(const void* dy, const uint8_t* codes, const float* scales,
                                 int64_t numel, int dtype, int form, void* dx, void* stream) {
  return entry([&] {
    int act = 0;
    if (!gelu_kind(form, &act)) return unsupported("fp8_gelu_backward", "unknown form");
    ActArgs a = {};
    a.x = dy;
    a.n = numel;
    a.dtype = dtype;
    a.codes = codes;
    a.scales = scales;
    a.out = dx;
    a.vec_ok = aligned_all(dy, dx, codes);
    return act_call("fp8_gelu_backward", act, false, a, !dy || !dx || !codes || !scales,
                    stream);
  });
}

extern "C" int fp8_layer_norm(const void* x, const void* weight, const void* bias,
                              int64_t rows, int64_t cols, int dtype, int wdtype, float eps,
                              void* y, float* mean, float* rstd, uint8_t* codes,
                              float* scales, void* stream_ptr) {
  return entry([&] {
    const char* fn = "fp8_layer_norm";
    int st = check_norm(fn, rows, cols, dtype, wdtype);
    if (st != FP8OPT_OK) return st;
    if (!(eps >= 0.0f) || std::isinf(eps)) return bad(fn, "eps is negative or not finite");
    if (rows == 0) return (int)FP8OPT_OK;
    if (!x || !weight || !y || !rstd) return bad(fn, "NULL pointer");
    const bool fp8 = codes != nullptr;
    if (fp8 != (scales != nullptr) || fp8 == (mean != nullptr))
      return bad(fn, "give mean, or codes and scales");
    LnForward a = {x, weight, bias, y, mean, rstd, codes, scales, rows, cols, dtype,
                   wdtype, kLnElements, eps};
    a.form = ln_form(aligned_all(x, y) && (reinterpret_cast<uintptr_t>(codes) & 7u) == 0,
                     aligned_all(weight, bias), cols, kLnFlatForward);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    OpCall call;
    if ((st = call.open(fn, stream, 0)) != FP8OPT_OK) return st;
    return call.done(fn, launch_ln_forward(a, call.sms, stream, call.mark));
  });
}

extern "C" int fp8_layer_norm_backward(const void* dy, const void* x, const float* mean,
                                       const uint8_t* codes, const float* scales,
                                       const float* rstd, const void* weight, int64_t rows,
                                       int64_t cols, int dtype, int wdtype, void* dx,
                                       void* dweight, void* dbias, void* stream_ptr) {
  return entry([&] {
    const char* fn = "fp8_layer_norm_backward";
    int st = check_norm(fn, rows, cols, dtype, wdtype);
    if (st != FP8OPT_OK) return st;
    if (!dweight || (rows > 0 && (!dy || !weight || !rstd || !dx)))
      return bad(fn, "NULL pointer");
    const bool fp8 = codes != nullptr;
    if (rows > 0 && (fp8 != (scales != nullptr) || fp8 == (mean != nullptr) ||
                     fp8 == (x != nullptr)))
      return bad(fn, "give x and mean, or codes and scales");
    LnBackward a = {dy, x, weight, mean, rstd, codes, scales, dx, dweight, dbias,
                    rows, cols, dtype, wdtype, kLnElements};
    a.form = ln_form(aligned_all(dy, x, dx) && (reinterpret_cast<uintptr_t>(codes) & 7u) == 0,
                     aligned_all(weight), cols, kLnFlatBackward);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    OpCall call;
    // the SM count sizes the grid, and the grid the scratch
    if ((st = call.open(fn, stream, 0)) != FP8OPT_OK) return st;
    const size_t bytes = ln_backward_scratch(a, call.sms);
    if ((st = call.open(fn, stream, bytes)) != FP8OPT_OK) return st;
    return call.done(fn, launch_ln_backward(a, call.scratch, call.sms, stream, call.mark));
  });
}

namespace fp8opt {
namespace {

// most_rows: the rows of x that the call takes.
int check_xent(const char* fn, const XentArgs& a, int64_t most_rows) {
  if (a.rows < 0 || a.rows > most_rows || a.dim < 1 || a.dim > kXentMostSummed || a.vocab < 1 ||
      a.vocab > kXentMost || a.rows > kMaxElems / a.dim || a.vocab > kMaxElems / a.dim)
    return bad(fn, "rows < 0, dim < 1, vocab < 1, or a size above its maximum");
  if (a.dtype != FP8OPT_BF16 && a.dtype != FP8OPT_F16)
    return unsupported(fn, "dtype is neither BF16 nor FP16");
  return FP8OPT_OK;
}

}  // namespace
}  // namespace fp8opt

extern "C" int fp8_linear_xent(const void* x, const void* w, const int64_t* target,
                               int64_t rows, int64_t dim, int64_t vocab, int dtype,
                               int64_t ignore_index, float* loss, float* lse,
                               void* stream_ptr) {
  return entry([&] {
    const char* fn = "fp8_linear_xent";
    XentArgs a = {};
    a.x = x;
    a.w = w;
    a.target = target;
    a.rows = rows;
    a.dim = dim;
    a.vocab = vocab;
    a.ignore = ignore_index;
    a.dtype = dtype;
    a.loss = loss;
    a.lse_out = lse;
    int st = check_xent(fn, a, kXentMost);
    if (st != FP8OPT_OK || rows == 0) return st;
    if (!x || !w || !target || !loss || !lse) return bad(fn, "NULL pointer");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    OpCall call;
    int* error = nullptr;
    if ((st = call.open(fn, stream, 0)) != FP8OPT_OK ||
        (st = call.open(fn, stream, xent_forward_scratch(a, call.sms))) != FP8OPT_OK ||
        (st = call.error_word(fn, stream, &error)) != FP8OPT_OK)
      return st;
    return call.done(fn, launch_xent_forward(a, call.scratch, error, call.sms, stream,
                                             call.mark));
  });
}

extern "C" int fp8_linear_xent_backward(const float* dloss, const void* x, const void* w,
                                        const int64_t* target, const float* lse, int64_t rows,
                                        int64_t dim, int64_t vocab, int dtype,
                                        int64_t ignore_index, void* dx, void* dw,
                                        void* stream_ptr) {
  return entry([&] {
    const char* fn = "fp8_linear_xent_backward";
    XentArgs a = {};
    a.x = x;
    a.w = w;
    a.target = target;
    a.rows = rows;
    a.dim = dim;
    a.vocab = vocab;
    a.ignore = ignore_index;
    a.dtype = dtype;
    a.dloss = dloss;
    a.lse = lse;
    a.dx = dx;
    a.dw = dw;
    int st = check_xent(fn, a, kXentMostSummed);
    if (st != FP8OPT_OK) return st;
    if (!dw || (rows > 0 && (!dloss || !x || !w || !target || !lse || !dx)))
      return bad(fn, "NULL pointer");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    OpCall call;
    int* error = nullptr;
    if ((st = call.open(fn, stream, 0)) != FP8OPT_OK) return st;
    const size_t bytes = rows > 0 ? xent_backward_scratch(a, call.sms) : 0;
    if ((st = call.open(fn, stream, bytes)) != FP8OPT_OK ||
        (st = call.error_word(fn, stream, &error)) != FP8OPT_OK)
      return st;
    return call.done(fn, launch_xent_backward(a, call.scratch, error, call.sms, stream,
                                              call.mark));
  });
}
