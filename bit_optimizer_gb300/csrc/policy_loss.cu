// The clipped policy loss with a KL term on the log probabilities of tokens,
//   r = exp(logp - old),  e = ref - logp,
//   l = -min(r A, clip(r, 1 - low, 1 + high) A) + kl_coef (exp(e) - 1 - e),
// its mean over the tokens that count, and dl / dlogp = -[not clipped] r A +
// kl_coef (1 - exp(e)).
//
// Bound by memory for large batches, by launches for small ones.  A warp takes
// up to kPiece tokens of one sequence and writes its sums; one CTA joins them in
// order, in fp64 (a batch's terms cancel down to their mean).
//
// Whether a token is clipped decides between its whole gradient and none, so it
// is decided exactly: logp - old, as the fp32 difference and its rounding error,
// against the border's logarithm in two floats.
#include <cmath>

#include "ops_internal.cuh"

namespace fp8opt {

namespace {

constexpr int kCtaThreads = 256, kCtaWarps = kCtaThreads / 32;
constexpr int kPiece = 1024;      // tokens of a warp
constexpr int kJoinThreads = 1024;

struct Border {
  float hi, lo;                   // log of the border
  float ratio;                    // the border
};

struct Policy {
  const float* logp;
  const float* old_logp;
  const float* advantage;
  const uint8_t* mask;
  const float* ref_logp;
  int64_t length, pieces, units;  // a unit: a piece of a sequence
  bool per_token;
  Border low, high;
  float kl_coef;
};

// exp(e) - 1 - e: the series e^2 (1 / 2! + e / 3! + ...) where the difference
// would cancel, to 2 / 12! of the result at |e| = 1.
__device__ __forceinline__ float kl_of(float e) {
  if (fabsf(e) > 1.0f) return expf(e) - 1.0f - e;
  float s = 1.0f / 39916800.0f;
  s = fmaf(s, e, 1.0f / 3628800.0f);
  s = fmaf(s, e, 1.0f / 362880.0f);
  s = fmaf(s, e, 1.0f / 40320.0f);
  s = fmaf(s, e, 1.0f / 5040.0f);
  s = fmaf(s, e, 1.0f / 720.0f);
  s = fmaf(s, e, 1.0f / 120.0f);
  s = fmaf(s, e, 1.0f / 24.0f);
  s = fmaf(s, e, 1.0f / 6.0f);
  s = fmaf(s, e, 0.5f);
  return e * e * s;
}

struct Token {
  float ratio;
  bool clipped;
};

__device__ __forceinline__ Token token_of(const Policy& p, float logp, float old, float a) {
  const float d = logp - old, back = d - logp;
  const float err = (logp - (d - back)) + (-old - back);   // logp - old = d + err
  const bool above = d > p.high.hi || (d == p.high.hi && err > p.high.lo);
  const bool below = d < p.low.hi || (d == p.low.hi && err < p.low.lo);
  return {expf(d), (a > 0.0f && above) || (a < 0.0f && below)};
}

// Calls f(token of the sequence, values) for the lane's tokens of a piece; VEC:
// four at a time, in 16-byte words.
template <bool VEC, class F>
__device__ __forceinline__ void each_token(const Policy& p, int64_t unit, F f) {
  const int lane = threadIdx.x & 31;
  const int64_t b = unit / p.pieces, t0 = (unit - b * p.pieces) * kPiece;
  const int64_t base = b * p.length;
  const int n = (int)min((int64_t)kPiece, p.length - t0);
  const float a_all = p.per_token ? 0.0f : p.advantage[b];
  if constexpr (VEC) {
#pragma unroll 2
    for (int i = 4 * lane; i < n; i += 128) {
      const int64_t at = base + t0 + i;
      const float4 lp = *reinterpret_cast<const float4*>(p.logp + at);
      const float4 old = *reinterpret_cast<const float4*>(p.old_logp + at);
      float4 ref = make_float4(0, 0, 0, 0), a = make_float4(a_all, a_all, a_all, a_all);
      uint32_t m = 0x01010101u;
      if (p.ref_logp != nullptr) ref = *reinterpret_cast<const float4*>(p.ref_logp + at);
      if (p.per_token) a = *reinterpret_cast<const float4*>(p.advantage + at);
      if (p.mask != nullptr) m = *reinterpret_cast<const uint32_t*>(p.mask + at);
      const float l4[4] = {lp.x, lp.y, lp.z, lp.w}, o4[4] = {old.x, old.y, old.z, old.w};
      const float r4[4] = {ref.x, ref.y, ref.z, ref.w}, a4[4] = {a.x, a.y, a.z, a.w};
      f(at, l4, o4, r4, a4, m);
    }
  } else {
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
      const int64_t at = base + t0 + i;
      const float l1[1] = {p.logp[at]}, o1[1] = {p.old_logp[at]};
      const float r1[1] = {p.ref_logp != nullptr ? p.ref_logp[at] : 0.0f};
      const float a1[1] = {p.per_token ? p.advantage[at] : a_all};
      f(at, l1, o1, r1, a1, p.mask != nullptr ? (uint32_t)p.mask[at] : 1u);
    }
  }
}

__device__ __forceinline__ bool counts(uint32_t m, int k) { return (m >> (8 * k) & 0xFFu) != 0; }

// A unit's sums.
struct Part {
  double policy, kl;
  int clipped, count;
};

__device__ __forceinline__ Part add(const Part& a, const Part& b) {
  return {a.policy + b.policy, a.kl + b.kl, a.clipped + b.clipped, a.count + b.count};
}

// Over groups of `width` lanes.
__device__ __forceinline__ Part reduce(Part p, int width) {
  for (int o = width / 2; o > 0; o >>= 1) {
    const Part q = {__shfl_xor_sync(0xFFFFFFFFu, p.policy, o),
                    __shfl_xor_sync(0xFFFFFFFFu, p.kl, o),
                    __shfl_xor_sync(0xFFFFFFFFu, p.clipped, o),
                    __shfl_xor_sync(0xFFFFFFFFu, p.count, o)};
    p = add(p, q);
  }
  return p;
}

template <bool VEC>
__device__ __forceinline__ Part part_of(const Policy& p, int64_t unit) {
  constexpr int N = VEC ? 4 : 1;
  float policy = 0.0f, kl = 0.0f;
  int clipped = 0, count = 0;
  each_token<VEC>(p, unit, [&](int64_t, const float (&lp)[N], const float (&old)[N],
                               const float (&ref)[N], const float (&a)[N], uint32_t m) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (!counts(m, k)) continue;
      const Token t = token_of(p, lp[k], old[k], a[k]);
      policy -= (t.clipped ? (a[k] > 0.0f ? p.high.ratio : p.low.ratio) : t.ratio) * a[k];
      if (p.ref_logp != nullptr) kl += kl_of(ref[k] - lp[k]);
      clipped += t.clipped;
      ++count;
    }
  });
  return reduce({(double)policy, (double)kl, clipped, count}, 32);
}

template <bool VEC>
__global__ void __launch_bounds__(kCtaThreads)
policy_kernel(const Policy p, Part* parts) {
  begin_after_previous();
  const int64_t unit = (int64_t)blockIdx.x * kCtaWarps + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  const Part r = part_of<VEC>(p, unit);
  if ((threadIdx.x & 31) == 0) parts[unit] = r;
}

// What the batch's sums come to: by_sequence, of the sequences' means, else of
// all tokens.
struct Total {
  double policy = 0.0, kl = 0.0, clipped = 0.0;
  long long count = 0;             // tokens, or sequences that have any
  __device__ __forceinline__ void take(const Part& p, bool by_sequence) {
    if (p.count == 0) return;
    const double w = by_sequence ? 1.0 / p.count : 1.0;
    policy += p.policy * w;
    kl += p.kl * w;
    clipped += p.clipped * w;
    count += by_sequence ? 1 : p.count;
  }
};

__global__ void __launch_bounds__(kJoinThreads)
policy_join_kernel(const Part* parts, int64_t batch, int64_t pieces, bool by_sequence,
                   double kl_coef, float* stats, float* weight) {
  __shared__ double sh[3][kJoinThreads / 32];
  __shared__ long long sh_count[kJoinThreads / 32];
  begin_after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // `width` neighbouring lanes to a sequence
  int width = 1;
  while (width < 32 && width < pieces) width *= 2;
  const int groups = kJoinThreads / width, mine = threadIdx.x / width;
  Total total;
  for (int64_t b0 = 0; b0 < batch; b0 += groups) {
    const int64_t b = b0 + mine;
    Part s = {0.0, 0.0, 0, 0};
    if (b < batch)
      for (int64_t i = threadIdx.x % width; i < pieces; i += width)
        s = add(s, parts[b * pieces + i]);
    s = reduce(s, width);
    if (b < batch && threadIdx.x % width == 0) {
      total.take(s, by_sequence);
      weight[b] = __int_as_float(s.count);      // for now
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    total.policy += __shfl_xor_sync(0xFFFFFFFFu, total.policy, o);
    total.kl += __shfl_xor_sync(0xFFFFFFFFu, total.kl, o);
    total.clipped += __shfl_xor_sync(0xFFFFFFFFu, total.clipped, o);
    total.count += __shfl_xor_sync(0xFFFFFFFFu, total.count, o);
  }
  if (lane == 0) {
    sh[0][warp] = total.policy;
    sh[1][warp] = total.kl;
    sh[2][warp] = total.clipped;
    sh_count[warp] = total.count;
  }
  __syncthreads();
  double sum[3] = {0.0, 0.0, 0.0};
  long long count = 0;
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    for (int k = 0; k < 3; ++k) sum[k] += sh[k][w];
    count += sh_count[w];
  }
  const double all = count > 0 ? 1.0 / (double)count : 0.0;
  if (threadIdx.x == 0) {
    stats[0] = (float)((sum[0] + kl_coef * sum[1]) * all);
    for (int k = 0; k < 3; ++k) stats[1 + k] = (float)(sum[k] * all);
  }
  // (each by the thread that wrote its count)
  if (threadIdx.x % width == 0) {
    for (int64_t b = mine; b < batch; b += groups) {
      const int c = __float_as_int(weight[b]);
      weight[b] = c == 0 ? 0.0f : (float)(by_sequence ? all / c : all);
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kCtaThreads)
policy_backward_kernel(const Policy p, const float* dloss, const float* weight, float* dlogp) {
  begin_after_previous();
  const int64_t unit = (int64_t)blockIdx.x * kCtaWarps + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  constexpr int N = VEC ? 4 : 1;
  const float g = *dloss * weight[unit / p.pieces];
  each_token<VEC>(p, unit, [&](int64_t at, const float (&lp)[N], const float (&old)[N],
                               const float (&ref)[N], const float (&a)[N], uint32_t m) {
    float d[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const Token t = token_of(p, lp[k], old[k], a[k]);
      float v = t.clipped ? 0.0f : -(t.ratio * a[k]);
      if (p.ref_logp != nullptr) {
        const float e = ref[k] - lp[k];
        v -= p.kl_coef * (fabsf(e) > 1.0f ? expf(e) - 1.0f : e + kl_of(e));
      }
      d[k] = counts(m, k) ? v * g : 0.0f;
    }
    if constexpr (VEC) *reinterpret_cast<float4*>(dlogp + at) = make_float4(d[0], d[1], d[2], d[3]);
    else dlogp[at] = d[0];
  });
}

// Of the ratio 1 + x.
Border border(double x) {
  const double l = std::log1p(x);
  Border b = {(float)l, 0.0f, (float)(1.0 + x)};
  if (std::isfinite(l)) b.lo = (float)(l - (double)b.hi);
  return b;
}

Policy policy_of(const PolicyArgs& a) {
  Policy p = {};
  p.logp = a.logp;
  p.old_logp = a.old_logp;
  p.advantage = a.advantage;
  p.mask = a.mask;
  p.ref_logp = a.ref_logp;
  p.length = a.length;
  p.pieces = (a.length + kPiece - 1) / kPiece;
  p.units = a.batch * p.pieces;
  p.per_token = a.per_token;
  p.low = border(-a.clip_low);
  p.high = border(a.clip_high);
  p.kl_coef = (float)a.kl_coef;
  return p;
}

bool vectors_ok(const PolicyArgs& a) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.logp) |
                        reinterpret_cast<uintptr_t>(a.old_logp) |
                        reinterpret_cast<uintptr_t>(a.ref_logp) |
                        reinterpret_cast<uintptr_t>(a.dlogp) |
                        (a.per_token ? reinterpret_cast<uintptr_t>(a.advantage) : 0);
  return a.length % 4 == 0 && (all & 15u) == 0 && (reinterpret_cast<uintptr_t>(a.mask) & 3u) == 0;
}

unsigned ctas(const Policy& p) { return (unsigned)((p.units + kCtaWarps - 1) / kCtaWarps); }

}  // namespace

size_t policy_scratch(const PolicyArgs& a) { return (size_t)policy_of(a).units * sizeof(Part); }

cudaError_t launch_policy(const PolicyArgs& a, char* scratch, cudaStream_t stream,
                          LaunchMark mark) {
  const Policy p = policy_of(a);
  Part* parts = reinterpret_cast<Part*>(scratch);
  cudaError_t e = cudaSuccess;
  if (p.units > 0) {
    if (mark) mark(kPolicyLossK, 0, stream);
    e = launch(true, vectors_ok(a) ? policy_kernel<true> : policy_kernel<false>, ctas(p),
               kCtaThreads, 0, stream, p, parts);
    if (mark) mark(kPolicyLossK, 1, stream);
  }
  if (e != cudaSuccess) return e;
  if (mark) mark(kPolicyJoinK, 0, stream);
  e = launch(true, policy_join_kernel, 1, kJoinThreads, 0, stream, (const Part*)parts, a.batch,
             p.pieces, a.by_sequence, a.kl_coef, a.stats, a.weight_out);
  if (mark) mark(kPolicyJoinK, 1, stream);
  return e;
}

cudaError_t launch_policy_backward(const PolicyArgs& a, cudaStream_t stream, LaunchMark mark) {
  const Policy p = policy_of(a);
  if (mark) mark(kPolicyBackwardK, 0, stream);
  const cudaError_t e =
      launch(worth_early(a.batch * a.length),
             vectors_ok(a) ? policy_backward_kernel<true> : policy_backward_kernel<false>,
             ctas(p), kCtaThreads, 0, stream, p, a.dloss, a.weight, a.dlogp);
  if (mark) mark(kPolicyBackwardK, 1, stream);
  return e;
}

}  // namespace fp8opt
