// Shared by the training operators (activation checkpoints, layer norm, the
// vocabulary's cross entropy): their call scope, launch records and element
// helpers.
#pragma once

#include <algorithm>
#include <mutex>

#include "fp8opt_internal.cuh"

namespace fp8opt {

// Elements that share one scale of an activation checkpoint.
constexpr int kActGroup = 128;

enum ActKind { kActSave = 0, kActGelu = 1, kActGeluTanh = 2 };

// One call of the activation kernels: forward reads x and writes codes_out,
// scales_out and (GELU) out; backward reads codes, scales and (GELU) x, the
// output's gradient, and writes out.
struct ActArgs {
  const void* x;
  int64_t n;
  int dtype;
  bool vec_ok;              // every buffer aligned for 16-byte accesses
  void* out;
  uint8_t* codes_out;
  float* scales_out;
  const uint8_t* codes;
  const float* scales;
};

cudaError_t launch_act(int act, bool fwd, const ActArgs& a, int sms,
                       cudaStream_t stream, LaunchMark mark);

// Longest row that a CTA keeps in registers.
constexpr int64_t kLnMaxRegCols = 8192;

// How layer norm reaches its rows: by elements; in vectors of eight, every row
// and the parameters starting at a 16-byte boundary; or in vectors of eight of
// the flat tensor, which does, though its rows may start anywhere (a row's
// threads then hold up to seven elements before it as well).
enum LnForm { kLnElements = 1, kLnFlat = 2, kLnVectors = 8 };

// kLnFlat from `least` columns: masking the ends costs a short row more than
// its element accesses.  65536 rows BF16, x kept, elements and flat: forward
// 321 columns 37.6 and 43.6 us, 385 49.4 and 43.8, 755 92.4 and 56.5; backward
// 129 27.3 and 29.2 us, 249 42.4 and 26.8, 755 176 and 92.5.
constexpr int64_t kLnFlatForward = 352, kLnFlatBackward = 192;

inline int ln_form(bool rows_aligned, bool params_aligned, int64_t cols, int64_t least) {
  if (rows_aligned && params_aligned && cols % 8 == 0) return kLnVectors;
  return rows_aligned && cols >= least && cols + 7 <= kLnMaxRegCols ? kLnFlat : kLnElements;
}

// Layer norm over rows of `cols` elements; x, y, dy and dx of type dtype, the
// parameters and their gradients of type wdtype.  codes and scales (one per
// row) hold xhat in 8 bits; without them mean and x are kept instead.
struct LnForward {
  const void* x;
  const void* weight;
  const void* bias;          // may be NULL
  void* y;
  float* mean;               // NULL with codes
  float* rstd;
  uint8_t* codes;
  float* scales;
  int64_t rows, cols;
  int dtype, wdtype;
  int form;                  // of the row accesses: an LnForm
  float eps;
};

struct LnBackward {
  const void* dy;
  const void* x;
  const void* weight;
  const float* mean;
  const float* rstd;
  const uint8_t* codes;
  const float* scales;
  void* dx;
  void* dw;
  void* db;                  // may be NULL
  int64_t rows, cols;
  int dtype, wdtype;
  int form;
};

cudaError_t launch_ln_forward(const LnForward& a, int sms, cudaStream_t stream,
                              LaunchMark mark);
size_t ln_backward_scratch(const LnBackward& a, int sms);
cudaError_t launch_ln_backward(const LnBackward& a, void* scratch, int sms,
                               cudaStream_t stream, LaunchMark mark);

// Most rows of a tensor of the cross entropy (coordinates are ints), and the
// longest sum of its products (dim, and backward the tokens): a tile's count of
// 64-deep blocks has 24 bits.
constexpr int64_t kXentMost = ((int64_t)1 << 31) - 1;
constexpr int64_t kXentMostSummed = 64 * (((int64_t)1 << 24) - 1);

// Cross entropy of the linear layer z = x w^T: x rows x dim, w vocab x dim, of
// type dtype (kBF16 or kF16).
struct XentArgs {
  const void* x;
  const void* w;
  const int64_t* target;
  int64_t rows, dim, vocab, ignore;
  int dtype;
  float* loss;               // forward
  float* lse_out;
  const float* dloss;        // backward
  const float* lse;
  void* dx;
  void* dw;
  // Distillation (ids not NULL): k words of a teacher's for each token, and their
  // logits, instead of target and ignore; lse is of z / temperature.
  const int64_t* ids;
  const void* logits;
  int k, logit_dtype;
  float temperature;
};

size_t xent_forward_scratch(const XentArgs& a, int sms);
size_t xent_backward_scratch(const XentArgs& a, int sms);
// error: a device word set to 1 when a wait in a kernel ran out.
cudaError_t launch_xent_forward(const XentArgs& a, char* scratch, int* error, int sms,
                                cudaStream_t stream, LaunchMark mark);
cudaError_t launch_xent_backward(const XentArgs& a, char* scratch, int* error, int sms,
                                 cudaStream_t stream, LaunchMark mark);

// The embedding: in is the table w (vocab x dim), out the rows y (rows x dim);
// backward in is dy and out dw.
struct EmbeddingArgs {
  const int64_t* ids;
  const void* in;
  void* out;
  int64_t rows, dim, vocab;
  int64_t padding;           // backward: a word that gets no gradient
  int dtype;
  float scale;
};

cudaError_t launch_embedding(const EmbeddingArgs& a, cudaStream_t stream, LaunchMark mark);
size_t embedding_backward_scratch(const EmbeddingArgs& a, int sms);
cudaError_t launch_embedding_backward(const EmbeddingArgs& a, char* scratch, int sms,
                                      cudaStream_t stream, LaunchMark mark);

// The clipped policy loss over `batch` sequences of `length` tokens.
struct PolicyArgs {
  const float* logp;
  const float* old_logp;
  const float* advantage;    // of every token (per_token), or of every sequence
  const uint8_t* mask;       // NULL: every token counts
  const float* ref_logp;     // NULL: no KL term
  int64_t batch, length;
  bool per_token, by_sequence;
  double clip_low, clip_high, kl_coef;
  float* stats;              // forward: loss, policy term, KL, clipped part
  float* weight_out;         // of each sequence's tokens
  const float* dloss;        // backward
  const float* weight;
  float* dlogp;
};

size_t policy_scratch(const PolicyArgs& a);
cudaError_t launch_policy(const PolicyArgs& a, char* scratch, cudaStream_t stream,
                          LaunchMark mark);
cudaError_t launch_policy_backward(const PolicyArgs& a, cudaStream_t stream, LaunchMark mark);

// Holds the library lock for one operator call, with the current device's SM
// count, the launch marks, and `scratch_bytes` of the stream's workspace
// (contents undefined; the call's own until its work on the stream ends).
// open() returns a status and records the error's text.
class OpCall {
 public:
  OpCall();
  int open(const char* fn, cudaStream_t stream, size_t scratch_bytes);
  int done(const char* fn, cudaError_t e);   // the call's status
  // The device's word in which kernels record that a wait of theirs ran out:
  // pinned host memory, so that a call made after such a kernel's end sees it
  // without waiting for the GPU, and fails.
  int error_word(const char* fn, cudaStream_t stream, int** device);
  char* scratch = nullptr;
  int sms = 0;
  LaunchMark mark = nullptr;

 private:
  std::unique_lock<std::mutex> lock_;
};

int record_error(int status, const char* what);

// Launches an operator's kernel; `early`: so that it may be set up, and its
// CTAs start, while the previous kernel of the stream ends (programmatic
// dependent launch).  Each kernel begins with begin_after_previous(), before
// which it reads and writes nothing in global memory.  Such a launch costs 1.5
// us more of the host's time, and saves about 2.5 us of the GPU's.
//
// A kernel launched early lives while its predecessor still writes what it will
// read, so none of its inputs is read-only in the sense of the non-coherent
// path: inputs are neither const __restrict__ parameters nor read with __ldg,
// but with plain, __ldca, __ldcg or __ldcs loads behind begin_after_previous().
template <class... Params, class... Args>
cudaError_t launch(bool early, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                   cudaStream_t stream, Args... args) {
  if (!early) {
    kernel<<<grid, block, smem, stream>>>(args...);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Whether a memory-bound kernel over this many elements is long enough (some 8
// us, at four bytes and more an element) for its launch to be an early one: a
// shorter one is over before the host has launched the next (128 x 768 norm:
// 6.8 us a call, 8.4 early; 16384 x 4096: 59.1 us, 56.6 early).
inline bool worth_early(int64_t elements) { return elements >= (int64_t)12 << 20; }

__device__ __forceinline__ void begin_after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// --------------------------------------------------------- element helpers

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Two fp32 values rounded to nearest even to a pair of DT (kBF16 or kF16),
// the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (DT == kF16) return f2_to_h2(make_float2(a, b));
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
  if (DT == kF32) static_cast<float*>(p)[i] = x;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)pack2<DT>(x, 0.0f);
}

}  // namespace fp8opt
