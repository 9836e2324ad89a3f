// 8-bit activation checkpoints and the GELU that saves and uses one.
//
// A checkpoint of a contiguous tensor is its E4M3 codes plus one fp32 scale
// per group of 128 consecutive elements (the last group may be shorter), in
// the cast's arithmetic taken per group: amax = max |x|, scale = 448 / amax
// (1 when amax is 0 or not finite, or the quotient is not finite), code =
// encode(x * scale); a value is read back as decode(code) * (1 / scale).  The
// group is short enough that one pass does it all: eight neighbouring threads
// hold a group, sixteen elements each, and take its amax with three shuffles.
//
// Bytes per element, e the element's size: save e + 1 + 4/128, load 1 + 4/128
// + e, GELU forward and backward 2 e + 1 + 4/128.  All four are bounded by
// HBM; a thread's loads are all issued before its first use.  16384 x 4096 read
// back to FP16: 30.2 us, 6.73 TB/s, 0.99 of the measured copy bandwidth; the
// GELU gradient (erf form) of 8192 x 16384 BF16: 104.9 us, 6.44 TB/s, 0.95.
//
// Buffers that are not aligned for 16-byte accesses take a path of one warp
// per group with element accesses, neighbouring lanes on neighbouring
// elements.
#include "ops_internal.cuh"

namespace fp8opt {

namespace {

constexpr int kPer = 16;                       // elements of one thread
constexpr int kLanes = kActGroup / kPer;       // threads of one group
static_assert(kLanes == 8, "three shuffles reduce a group");

// ----------------------------------------------------------------- GELU

__device__ __forceinline__ float ex2(float x) {   // 2^x, flushing below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {   // 1 / x to one ulp; 1/inf = 0
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
// The tanh form as a logistic: 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2 u)), with
// 2 u = x (kC0 + kC1 x^2), kC0 = 2 sqrt(2 / pi), kC1 = 0.044715 kC0.
constexpr float kC0 = 1.5957691216057308f;
constexpr float kC1 = 0.07135481282681852f;
// Beyond this magnitude both forms' derivative term x c'(x) is 0 in fp32;
// clamping x there keeps 0 from meeting an overflowed factor.
constexpr float kFar = 16.0f;

// Phi(x), and g = exp(-x^2 / 2).  For results in 16 bits: 1 - Phi(|x|) with
// Abramowitz and Stegun's formula 7.1.26 for erfc (its error, 1.5e-7 of erfc, is
// 0.75e-7 of Phi, and its roundings are up to 3e-7); the instructions bound the
// 16-bit gradient as much as HBM does.  FP32 has twice the bytes and room for a
// nearer form, off by at most 1.3e-7: below 1 an odd polynomial about 1/2, beyond
// it exp(-x^2 / 2) t P(t), t = 1 / (1 + 0.4 |x| / sqrt(2)), whose value, below
// 0.16, makes its roundings small.  Both are minimax fits of their own (reweighted
// least squares at Chebyshev points): 1.3e-10 absolute, 1.1e-7 relative.
template <int DT>
__device__ __forceinline__ float normal_cdf(float x, float& g) {
  const float z = fabsf(x) * 0.70710678118654752f;
  if (DT == kF32) {
    const float s = x * x;
    g = ex2(s * (-0.5f * kLog2e));
    float c = __fmaf_rn(-7.530306447733892e-06f, s, 0.00011314365110592917f);
    c = __fmaf_rn(c, s, -0.001185984699986875f);
    c = __fmaf_rn(c, s, 0.009973171167075634f);
    c = __fmaf_rn(c, s, -0.06649032980203629f);
    c = __fmaf_rn(c, s, 0.3989422917366028f);
    c = __fmaf_rn(x, c, 0.5f);
    const float t = rcp(__fmaf_rn(0.4f, z, 1.0f));
    float p = __fmaf_rn(-0.0566902682185173f, t, 0.11782621592283249f);
    p = __fmaf_rn(p, t, 0.00855597946792841f);
    p = __fmaf_rn(p, t, 0.10399360209703445f);
    p = __fmaf_rn(p, t, 0.10017447918653488f);
    p = __fmaf_rn(p, t, 0.11322233825922012f);
    p = __fmaf_rn(p, t, 0.11282133311033249f);
    const float q = p * t * g;
    return fabsf(x) < 1.0f ? c : x > 0.0f ? 1.0f - q : q;
  }
  const float t = rcp(__fmaf_rn(0.3275911f, z, 1.0f));
  float p = __fmaf_rn(1.061405429f, t, -1.453152027f);
  p = __fmaf_rn(p, t, 1.421413741f);
  p = __fmaf_rn(p, t, -0.284496736f);
  p = __fmaf_rn(p, t, 0.254829592f);
  g = ex2(x * x * (-0.5f * kLog2e));   // (here, not before p: 8192 x 16384 106.5 us)
  const float q = 0.5f * p * t * g;
  return x > 0.0f ? 1.0f - q : q;
}

template <int DT, bool TANH>
__device__ __forceinline__ float gelu(float x) {
  if (TANH) {
    const float u = x * __fmaf_rn(kC1, x * x, kC0);
    return x * rcp(1.0f + ex2(u * -kLog2e));
  }
  float g;
  return x * normal_cdf<DT>(x, g);
}

// d gelu / dx = c(x) + x c'(x)
template <int DT, bool TANH>
__device__ __forceinline__ float gelu_grad(float x) {
  const float xc = fminf(fmaxf(x, -kFar), kFar);   // NaN: the c term keeps it
  if (TANH) {
    // with e = exp(-|u|) and r = 1 / (1 + e): c is r or e r, and c (1 - c) =
    // e r^2 has no cancellation
    const float u = x * __fmaf_rn(kC1, x * x, kC0);
    const float e = ex2(fabsf(u) * -kLog2e);
    const float r = rcp(1.0f + e), er = e * r;
    const float du = __fmaf_rn(3.0f * kC1, xc * xc, kC0);
    return __fmaf_rn(xc * du, er * r, u < 0.0f ? er : r);
  }
  float g;
  const float c = normal_cdf<DT>(x, g);
  return __fmaf_rn(xc * 0.39894228040143268f, g, c);
}

// ------------------------------------------------------ sixteen elements

template <int DT>
struct Raw16 {
  uint4 v[DT == kF32 ? 4 : 2];
};

template <int DT>
__device__ __forceinline__ Raw16<DT> load_raw16(const void* p, int64_t i0) {
  Raw16<DT> r;
  const char* a = static_cast<const char*>(p) + i0 * (DT == kF32 ? 4 : 2);
#pragma unroll
  for (int k = 0; k < (DT == kF32 ? 4 : 2); ++k) r.v[k] = ld_once4(a + 16 * k);
  return r;
}

template <int DT>
__device__ __forceinline__ void widen16(const Raw16<DT>& r, float (&x)[kPer]) {
#pragma unroll
  for (int k = 0; k < (DT == kF32 ? 4 : 2); ++k) {
    const uint32_t w[4] = {r.v[k].x, r.v[k].y, r.v[k].z, r.v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (DT == kF32) {
        x[4 * k + j] = __uint_as_float(w[j]);
      } else {
        float2 f;
        if (DT == kF16) f = h2_to_f2(w[j]);
        else f = make_float2(__uint_as_float(w[j] << 16),
                             __uint_as_float(w[j] & 0xFFFF0000u));
        x[8 * k + 2 * j] = f.x;
        x[8 * k + 2 * j + 1] = f.y;
      }
    }
  }
}

// max |x| of the raw elements as fp32 bits (NaN above inf above finite).
template <int DT>
__device__ __forceinline__ uint32_t amax16(const Raw16<DT>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < (DT == kF32 ? 4 : 2); ++k) {
    const uint32_t w[4] = {r.v[k].x, r.v[k].y, r.v[k].z, r.v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = DT == kF32 ? max(m, w[j] & 0x7FFFFFFFu) : __vmaxu2(m, w[j] & 0x7FFF7FFFu);
  }
  if (DT == kF32) return m;
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  return DT == kBF16 ? h << 16 : __float_as_uint(h_to_f((uint16_t)h));
}

template <int DT>
__device__ __forceinline__ void store16(void* p, int64_t i0, const float (&x)[kPer]) {
  char* a = static_cast<char*>(p) + i0 * (DT == kF32 ? 4 : 2);
#pragma unroll
  for (int k = 0; k < (DT == kF32 ? 4 : 2); ++k) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (DT == kF32) w[j] = __float_as_uint(x[4 * k + j]);
      else w[j] = pack2<DT>(x[8 * k + 2 * j], x[8 * k + 2 * j + 1]);
    }
    __stcs(reinterpret_cast<uint4*>(a + 16 * k), make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// Sixteen codes of a group with a finite amax (non-finite values take the
// checked encoder).
__device__ __forceinline__ void encode16(const float (&x)[kPer], float scale,
                                         bool finite, uint8_t* codes, int64_t i0) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = mul2(make_float2(x[4 * j], x[4 * j + 1]), splat2(scale));
    const float2 b = mul2(make_float2(x[4 * j + 2], x[4 * j + 3]), splat2(scale));
    if (finite)
      w[j] = enc2<kE4M3>(a.x, a.y) | (enc2<kE4M3>(b.x, b.y) << 16);
    else
      w[j] = enc1_checked<kE4M3>(a.x) | (enc1_checked<kE4M3>(a.y) << 8) |
             (enc1_checked<kE4M3>(b.x) << 16) | (enc1_checked<kE4M3>(b.y) << 24);
  }
  __stcs(reinterpret_cast<uint4*>(codes + i0), make_uint4(w[0], w[1], w[2], w[3]));
}

__device__ __forceinline__ void decode16(uint4 c, float r, float (&x)[kPer]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = mul2(dec2<kE4M3>(w[j] & 0xFFFFu), splat2(r));
    const float2 b = mul2(dec2<kE4M3>(w[j] >> 16), splat2(r));
    x[4 * j] = a.x; x[4 * j + 1] = a.y; x[4 * j + 2] = b.x; x[4 * j + 3] = b.y;
  }
}

// ---------------------------------------------------------------- forward

// ACT: kActSave (y is not written), kActGelu or kActGeluTanh.
template <int DT, int ACT>
__device__ __forceinline__ float act_value(float x) {
  return gelu<DT, ACT == kActGeluTanh>(x);
}

// One group by a warp, element by element: any alignment, and a last group
// that is shorter.
template <int DT, int ACT>
__device__ __forceinline__ void forward_group(const void* x, int64_t n, int64_t g, void* y,
                                              uint8_t* codes, float* scales) {
  const int lane = threadIdx.x & 31;
  const int64_t base = g * kActGroup + lane;
  float v[4];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = base + 32 * j < n ? load1<DT>(x, base + 32 * j) : 0.0f;
    m = max(m, abs_bits(v[j]));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  const float scale = scale_from_amax_bits(m, 448.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t i = base + 32 * j;
    if (i >= n) continue;
    codes[i] = (uint8_t)enc1_checked<kE4M3>(__fmul_rn(v[j], scale));
    if (ACT != kActSave) store1<DT>(y, i, act_value<DT, ACT>(v[j]));
  }
  if (lane == 0) scales[g] = scale;
}

template <int DT, int ACT>
__device__ __forceinline__ void backward_group(const void* dy, const uint8_t* codes,
                                               const float* scales, int64_t n, int64_t g,
                                               void* out) {
  const float r = __fdiv_rn(1.0f, __ldcg(scales + g));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t i = g * kActGroup + 32 * j + (threadIdx.x & 31);
    if (i >= n) continue;
    float v = __fmul_rn(dec2<kE4M3>(codes[i]).x, r);
    if (ACT != kActSave) v = load1<DT>(dy, i) * gelu_grad<DT, ACT == kActGeluTanh>(v);
    store1<DT>(out, i, v);
  }
}

// All buffers aligned for 16-byte accesses: thread i takes elements [16 i, 16 i +
// 16) of the whole groups, and the last CTA what is left (tested per thread
// instead, the end of the tensor cost the GELU gradient 7%).
template <int DT, int ACT>
__global__ void __launch_bounds__(kThreads)
act_forward_kernel(const void* x, int64_t n, void* __restrict__ y,
                   uint8_t* __restrict__ codes, float* __restrict__ scales) {
  begin_after_previous();
  const int64_t whole = n / kActGroup * kActGroup;
  const int64_t i0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kPer;
  if (whole < n && blockIdx.x == gridDim.x - 1) {
    if (threadIdx.x < 32) forward_group<DT, ACT>(x, n, n / kActGroup, y, codes, scales);
    return;
  }
  const bool live = i0 < whole;     // the same for the eight threads of a group
  Raw16<DT> raw = {};
  if (live) raw = load_raw16<DT>(x, i0);
  uint32_t m = amax16<DT>(raw);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (!live) return;
  const float scale = scale_from_amax_bits(m, 448.0f);
  float v[kPer];
  widen16<DT>(raw, v);
  encode16(v, scale, m < 0x7F800000u, codes, i0);
  if ((threadIdx.x & (kLanes - 1)) == 0) scales[i0 / kActGroup] = scale;
  if (ACT != kActSave) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = act_value<DT, ACT>(v[j]);
    store16<DT>(y, i0, v);
  }
}

// ACT kActSave: x = decode(code) / scale; else dx = dy * gelu'(x).
template <int DT, int ACT>
__global__ void __launch_bounds__(kThreads)
act_backward_kernel(const void* dy, const uint8_t* codes, const float* scales, int64_t n,
                    void* __restrict__ out) {
  begin_after_previous();
  const int64_t whole = n / kActGroup * kActGroup;
  const int64_t i0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kPer;
  if (whole < n && blockIdx.x == gridDim.x - 1) {
    if (threadIdx.x < 32) backward_group<DT, ACT>(dy, codes, scales, n, n / kActGroup, out);
    return;
  }
  if (i0 >= whole) return;
  const uint4 c = ld_once4(codes + i0);
  const float s = __ldcg(scales + i0 / kActGroup);
  Raw16<DT> raw;
  if (ACT != kActSave) raw = load_raw16<DT>(dy, i0);
  float v[kPer];
  decode16(c, __fdiv_rn(1.0f, s), v);
  if (ACT != kActSave) {
    float d[kPer];
    widen16<DT>(raw, d);
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = d[j] * gelu_grad<DT, ACT == kActGeluTanh>(v[j]);
  }
  store16<DT>(out, i0, v);
}

// Any alignment: one warp per group.
template <int DT, int ACT, bool FWD>
__global__ void __launch_bounds__(kThreads) act_any_kernel(const ActArgs a) {
  begin_after_previous();
  const int64_t groups = (a.n + kActGroup - 1) / kActGroup;
  for (int64_t g = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); g < groups;
       g += (int64_t)gridDim.x * (kThreads / 32)) {
    if (FWD) forward_group<DT, ACT>(a.x, a.n, g, a.out, a.codes_out, a.scales_out);
    else backward_group<DT, ACT>(a.x, a.codes, a.scales, a.n, g, a.out);
  }
}

template <int DT, int ACT, bool FWD>
cudaError_t go(const ActArgs& a, int sms, cudaStream_t stream) {
  const bool early = worth_early(a.n);
  if (!a.vec_ok) {
    const int64_t blocks = (a.n + kActGroup * kThreads / 32 - 1) / (kActGroup * kThreads / 32);
    return launch(early, act_any_kernel<DT, ACT, FWD>,
                  (unsigned)(blocks < 16 * sms ? blocks : 16 * sms), kThreads, 0, stream, a);
  }
  const int64_t whole = a.n / kActGroup * kActGroup;
  const unsigned blocks = (unsigned)((whole + kPer * kThreads - 1) / (kPer * kThreads)) +
                          (whole < a.n ? 1u : 0u);
  if (FWD)
    return launch(early, act_forward_kernel<DT, ACT>, blocks, kThreads, 0, stream, a.x, a.n,
                  a.out, a.codes_out, a.scales_out);
  return launch(early, act_backward_kernel<DT, ACT>, blocks, kThreads, 0, stream, a.x, a.codes,
                a.scales, a.n, a.out);
}

template <int DT, bool FWD>
cudaError_t by_act(int act, const ActArgs& a, int sms, cudaStream_t s) {
  return act == kActSave   ? go<DT, kActSave, FWD>(a, sms, s)
         : act == kActGelu ? go<DT, kActGelu, FWD>(a, sms, s)
                           : go<DT, kActGeluTanh, FWD>(a, sms, s);
}

template <int DT>
cudaError_t launch_dt(int act, bool fwd, const ActArgs& a, int sms, cudaStream_t s) {
  return fwd ? by_act<DT, true>(act, a, sms, s) : by_act<DT, false>(act, a, sms, s);
}

}  // namespace

cudaError_t launch_act(int act, bool fwd, const ActArgs& a, int sms,
                       cudaStream_t stream, LaunchMark mark) {
  const int k = act == kActSave ? (fwd ? kActSaveK : kActLoadK)
                                : (fwd ? kGeluK : kGeluBackwardK);
  if (mark) mark(k, 0, stream);
  const cudaError_t e = a.dtype == kF32    ? launch_dt<kF32>(act, fwd, a, sms, stream)
                        : a.dtype == kBF16 ? launch_dt<kBF16>(act, fwd, a, sms, stream)
                                           : launch_dt<kF16>(act, fwd, a, sms, stream);
  if (mark) mark(k, 1, stream);
  return e;
}

}  // namespace fp8opt
