// The clipped policy loss with a KL term on the log probabilities of tokens,
//   r = exp(logp - old),  e = ref - logp,
//   l = -min(r A, clip(r, 1 - low, 1 + high) A) + kl_coef (exp(e) - 1 - e),
// its mean over the tokens that count, and dl / dlogp = -[not clipped] r A +
// kl_coef (1 - exp(e)).
//
// Bound by memory for large batches, by launches for small ones.  A warp takes a
// piece of one sequence; a CTA adds up what its warps have of a sequence, and one
// CTA joins the rest in order.  (A batch's terms cancel down to their mean: sums
// over warps are held in two floats, 48 bits.  In fp64, which the GB300 has little
// of, the join took 37 us for 8 sequences and 73 for 512.)  512 x 8192 tokens, half
// of them masked: 16 us, the gradient 10.4 to 11.6 us; the values of masked tokens
// are not read, and what is left is the latency of mask, values and join.  Both
// forward kernels are launched early, which makes them as fast as a single one for
// small batches (in one cluster 8 x 512 took 8.2 us, 64 x 1023 10.3; 7.4 and 7.7).
//
// Whether a token is clipped decides between its whole gradient and none, so it
// is decided exactly: logp - old, as the fp32 difference and its rounding error,
// against the border's logarithm in two floats.
#include <cmath>

#include "ops_internal.cuh"

namespace fp8opt {

namespace {

constexpr int kCtaThreads = 256, kCtaWarps = kCtaThreads / 32;
// Tokens of a warp: a multiple of 128, at most 32 of a lane.
constexpr int kLeastPiece = 128, kMostPiece = 1024;
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
  // A sequence is `pieces` units, each `warps` neighbouring warps of a CTA with
  // `piece` tokens each.
  int64_t length;
  unsigned pieces, units, warps;
  int piece;
  bool per_token;
  Border low, high;
  float kl_coef;
};

// exp(e) - 1 - e: the series e^2 (1 / 2! + e / 3! + ...) where the difference
// would cancel; what it leaves out is at most 2.6 / 12! of the result (at e = -1).
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
  const float d = logp - old;
  bool above = d > p.high.hi, below = d < p.low.hi;
  if (d == p.high.hi || d == p.low.hi) {      // then what d is off by decides
    const float back = d - logp, err = (logp - (d - back)) + (-old - back);
    above |= d == p.high.hi && err > p.high.lo;
    below |= d == p.low.hi && err < p.low.lo;
  }
  return {expf(d), (a > 0.0f && above) || (a < 0.0f && below)};
}

// The calling warp's unit, its sequence and the warp's first token of it.
struct Place {
  unsigned unit;
  int64_t b, t0;
};

__device__ __forceinline__ Place place_of(const Policy& p) {
  const unsigned warp = threadIdx.x >> 5;
  const unsigned unit = blockIdx.x * (kCtaWarps / p.warps) + warp / p.warps, b = unit / p.pieces;
  return {unit, (int64_t)b,
          ((int64_t)(unit - b * p.pieces) * p.warps + warp % p.warps) * p.piece};
}

__device__ __forceinline__ bool counts(uint32_t m, int k) { return (m >> (8 * k) & 0xFFu) != 0; }

// Calls f(first token, values, mask) for the lane's tokens of a piece of sequence b,
// from t0 on; VEC: four at a time, in 16-byte words.  Values of tokens that do not
// count are not read where all of a call's do not.
template <bool VEC, class F>
__device__ __forceinline__ void each_token(const Policy& p, int64_t b, int64_t t0, F f) {
  const int lane = threadIdx.x & 31;
  const int64_t base = b * p.length + t0;
  const int n = (int)min((int64_t)p.piece, p.length - t0);    // (may be below 0)
  const float a_all = p.per_token ? 0.0f : p.advantage[b];
  constexpr int N = VEC ? 4 : 1;
  // the masks of kAhead rounds, and while these are added the next ones'
  constexpr int kAhead = VEC ? 2 : 4;
  const auto masks = [&](int i0, uint32_t (&m)[kAhead]) {
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      const int i = i0 + r * 32 * N;
      m[r] = i < n ? (VEC ? 0x01010101u : 1u) : 0u;
      if (i < n && p.mask != nullptr) {
        if constexpr (VEC) m[r] = *reinterpret_cast<const uint32_t*>(p.mask + base + i);
        else m[r] = p.mask[base + i];
      }
    }
  };
  uint32_t m[kAhead];
  masks(N * lane, m);
  for (int i0 = N * lane; i0 < n; i0 += kAhead * 32 * N) {
    float lp[kAhead][N], old[kAhead][N], ref[kAhead][N], a[kAhead][N];
    const auto read = [&](float (&to)[N], const float* from, int64_t at) {
      if constexpr (VEC) {
        const float4 v = *reinterpret_cast<const float4*>(from + at);
        to[0] = v.x;
        to[1] = v.y;
        to[2] = v.z;
        to[3] = v.w;
      } else {
        to[0] = from[at];
      }
    };
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      const int64_t at = base + i0 + r * 32 * N;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        lp[r][k] = old[r][k] = ref[r][k] = 0.0f;
        a[r][k] = a_all;
      }
      if (m[r] != 0) {
        read(lp[r], p.logp, at);
        read(old[r], p.old_logp, at);
        if (p.ref_logp != nullptr) read(ref[r], p.ref_logp, at);
        if (p.per_token) read(a[r], p.advantage, at);
      }
    }
    uint32_t next[kAhead];
    masks(i0 + kAhead * 32 * N, next);
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      const int i = i0 + r * 32 * N;
      if (i < n) f(base + i, lp[r], old[r], ref[r], a[r], m[r]);
      m[r] = next[r];
    }
  }
}

// A sum in two floats: hi, and what it was off by so far.
struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two add(Two a, Two b) {
  const float s = a.hi + b.hi, back = s - a.hi;
  const float e = (a.hi - (s - back)) + (b.hi - back) + (a.lo + b.lo);
  if (nonfinite(s)) return {s, 0.0f};
  const float hi = s + e;
  return {hi, e - (hi - s)};
}

__device__ __forceinline__ Two scaled(Two a, Two k) {
  const float hi = a.hi * k.hi;
  if (nonfinite(hi)) return {hi, 0.0f};
  return {hi, fmaf(a.hi, k.hi, -hi) + (a.lo * k.hi + a.hi * k.lo)};
}

__device__ __forceinline__ Two shuffled(Two a, int o) {
  return {__shfl_xor_sync(0xFFFFFFFFu, a.hi, o), __shfl_xor_sync(0xFFFFFFFFu, a.lo, o)};
}

// 1 / x.  (In one float, means of sequences that cancel keep 2^-25 of theirs.)
__device__ __forceinline__ Two reciprocal(unsigned long long x) {
  const float hi = __ull2float_rn(x);
  const float lo = (float)(long long)(x - (unsigned long long)hi);
  const float q = 1.0f / hi, e = q * (fmaf(-q, hi, 1.0f) - q * lo);
  const float r = q + e;
  return {r, e - (r - q)};
}

// A unit's sums.
struct Part {
  Two policy, kl;
  int clipped, count;
};
constexpr int kPartWords = 6;
static_assert(sizeof(Part) == 4 * kPartWords, "");

__device__ __forceinline__ Part add(const Part& a, const Part& b) {
  return {add(a.policy, b.policy), add(a.kl, b.kl), a.clipped + b.clipped, a.count + b.count};
}

// Over groups of `width` lanes.
__device__ __forceinline__ Part reduce(Part p, int width) {
  for (int o = width / 2; o > 0; o >>= 1)
    p = add(p, {shuffled(p.policy, o), shuffled(p.kl, o),
                __shfl_xor_sync(0xFFFFFFFFu, p.clipped, o),
                __shfl_xor_sync(0xFFFFFFFFu, p.count, o)});
  return p;
}

template <bool VEC>
__device__ __forceinline__ Part part_of(const Policy& p, int64_t b, int64_t t0) {
  constexpr int N = VEC ? 4 : 1;
  float policy = 0.0f, kl = 0.0f;
  int clipped = 0, count = 0;
  each_token<VEC>(p, b, t0, [&](int64_t, const float (&lp)[N], const float (&old)[N],
                               const float (&ref)[N], const float (&a)[N], uint32_t m) {
    if (m == 0) return;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const Token t = token_of(p, lp[k], old[k], a[k]);
      const float r = t.clipped ? (a[k] > 0.0f ? p.high.ratio : p.low.ratio) : t.ratio;
      const float d = p.ref_logp != nullptr ? kl_of(ref[k] - lp[k]) : 0.0f;
      if (counts(m, k)) {
        policy -= r * a[k];
        kl += d;
        clipped += t.clipped;
        ++count;
      }
    }
  });
  // (a lane's at most 32 terms and the lanes' in fp32; from here on in two floats)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    policy += __shfl_xor_sync(0xFFFFFFFFu, policy, o);
    kl += __shfl_xor_sync(0xFFFFFFFFu, kl, o);
  }
  const unsigned n = __reduce_add_sync(0xFFFFFFFFu, (unsigned)clipped << 16 | (unsigned)count);
  return {{policy, 0.0f}, {kl, 0.0f}, (int)(n >> 16), (int)(n & 0xFFFFu)};
}
static_assert(kMostPiece < 1 << 16, "a piece's counts");

// What the batch's sums come to: by_sequence, of the sequences' means, else of
// all tokens.
struct Total {
  Two policy, kl, clipped;
  unsigned long long count;        // tokens, or sequences that have any
  __device__ __forceinline__ void take(const Part& p, bool by_sequence) {
    if (p.count == 0) return;
    const Two w = by_sequence ? reciprocal(p.count) : Two{1.0f, 0.0f};
    policy = add(policy, scaled(p.policy, w));
    kl = add(kl, scaled(p.kl, w));
    clipped = add(clipped, scaled({(float)(p.clipped & ~0xFFF), (float)(p.clipped & 0xFFF)}, w));
    count += by_sequence ? 1 : p.count;
  }
  __device__ __forceinline__ void reduce() {
    for (int o = 16; o > 0; o >>= 1) {
      policy = add(policy, shuffled(policy, o));
      kl = add(kl, shuffled(kl, o));
      clipped = add(clipped, shuffled(clipped, o));
      count += __shfl_xor_sync(0xFFFFFFFFu, count, o);
    }
  }
};

__global__ void __launch_bounds__(kJoinThreads)
policy_join_kernel(const Part* parts, int64_t batch, int64_t pieces, bool by_sequence,
                   float kl_coef, float* stats, float* weight) {
  __shared__ Total sh[kJoinThreads / 32];
  __shared__ unsigned long long sh_count;
  begin_after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // `width` neighbouring lanes to a sequence
  int width = 1;
  while (width < 32 && width < pieces) width *= 2;
  const int groups = kJoinThreads / width, mine = threadIdx.x / width;
  Total total = {};
  // (a warp without a sequence has nothing to add up: 32 warps' sums in two floats
  // take longer than the memory)
  const bool busy = warp * 32 / width < batch;
  for (int64_t b0 = 0; busy && b0 < batch; b0 += groups) {
    const int64_t b = b0 + mine;
    Part s = {};
    if (b < batch) {
#pragma unroll 4
      for (int64_t i = threadIdx.x % width; i < pieces; i += width)
        s = add(s, parts[b * pieces + i]);
    }
    s = reduce(s, width);
    if (b < batch && threadIdx.x % width == 0) {
      total.take(s, by_sequence);
      weight[b] = __int_as_float(s.count);      // for now
    }
  }
  if (busy) total.reduce();
  if (lane == 0) sh[warp] = total;
  __syncthreads();
  if (warp == 0) {
    total = sh[lane];
    if (batch * width > 32) total.reduce();
    if (lane == 0) sh_count = total.count;
  }
  __syncthreads();
  const unsigned long long count = sh_count;
  const Two all = count > 0 ? reciprocal(count) : Two{0.0f, 0.0f};
  if (threadIdx.x == 0) {
    const Two each[3] = {scaled(total.policy, all), scaled(total.kl, all),
                         scaled(total.clipped, all)};
    const Two loss = add(each[0], scaled(each[1], {kl_coef, 0.0f}));
    stats[0] = loss.hi;
    for (int k = 0; k < 3; ++k) stats[1 + k] = each[k].hi + each[k].lo;
  }
  // (each by the thread that wrote its count)
  if (threadIdx.x % width == 0) {
    for (int64_t b = mine; b < batch; b += groups) {
      const int c = __float_as_int(weight[b]);
      weight[b] = c == 0        ? 0.0f
                  : by_sequence ? reciprocal((unsigned long long)c * count).hi : all.hi;
    }
  }
}
static_assert(kJoinThreads / 32 == 32, "a lane to each warp's total");

template <bool VEC>
__global__ void __launch_bounds__(kCtaThreads)
policy_kernel(const Policy p, Part* parts) {
  __shared__ Part sh[kCtaWarps];
  begin_after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place at = place_of(p);
  if (at.unit < p.units) {
    const Part r = part_of<VEC>(p, at.b, at.t0);
    if (lane == 0) sh[warp] = r;
  }
  __syncthreads();
  // (a unit's first warp goes on)
  if (at.unit >= p.units || warp % p.warps != 0) return;
  const Part r = reduce(sh[warp + lane % p.warps], p.warps);
  if (lane == 0) parts[at.unit] = r;
}

template <bool VEC>
__global__ void __launch_bounds__(kCtaThreads)
policy_backward_kernel(const Policy p, const float* dloss, const float* weight, float* dlogp) {
  begin_after_previous();
  const Place place = place_of(p);
  if (place.unit >= p.units) return;
  constexpr int N = VEC ? 4 : 1;
  const float g = *dloss * weight[place.b];
  each_token<VEC>(p, place.b, place.t0, [&](int64_t at, const float (&lp)[N], const float (&old)[N],
                               const float (&ref)[N], const float (&a)[N], uint32_t m) {
    float d[N];
#pragma unroll
    for (int k = 0; k < N; ++k) d[k] = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (m == 0) break;
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

// The pieces are as large as they can be while there are kWarps of them (27 an SM):
// fewer sums to join.  Forward and backward in us with 2048, 4096 and 8192: 200 x 8192
// 11.3 and 6.3, 11.3 and 5.0, 14.7 and 7.0; 300 x 8192 13.4 and 8.5, 11.4 and 6.5, 14.1
// and 7.0; 512 x 8192 (4096 of the largest) 16.3 and 11.1 with the first two, 17.5 and
// 10.4; 1000 x 3000 15.1 and 8.4, 15.5 and 8.5, 18.9 and 8.3.
constexpr int64_t kWarps = 4096;

Policy policy_of(const PolicyArgs& a) {
  Policy p = {};
  p.logp = a.logp;
  p.old_logp = a.old_logp;
  p.advantage = a.advantage;
  p.mask = a.mask;
  p.ref_logp = a.ref_logp;
  p.length = a.length;
  const auto up = [](int64_t x, int64_t m) { return (x + m - 1) / m; };
  for (int most = kMostPiece;; most /= 2) {
    p.warps = 1;
    while (p.warps < kCtaWarps && (int64_t)p.warps * most < a.length) p.warps *= 2;
    p.pieces = (unsigned)up(a.length, (int64_t)p.warps * most);
    p.units = (unsigned)(a.batch * p.pieces);
    p.piece = p.pieces > 0 ? (int)(up(up(a.length, (int64_t)p.warps * p.pieces), 128) * 128) : most;
    if ((int64_t)p.units * p.warps >= kWarps || most == kLeastPiece) break;
  }
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

unsigned ctas(const Policy& p) {
  const unsigned units = kCtaWarps / p.warps;
  return (p.units + units - 1) / units;
}

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
             (int64_t)p.pieces, a.by_sequence, (float)a.kl_coef, a.stats, a.weight_out);
  if (mark) mark(kPolicyJoinK, 1, stream);
  return e;
}

// From here on the gradient's kernel takes longer than the host for its early launch
// (4096 x 100: 4.1 us, 6.1 launched late; 512 x 8192: 10.4 and 12.3).
constexpr int64_t kEarlyTokens = 1 << 18;

cudaError_t launch_policy_backward(const PolicyArgs& a, cudaStream_t stream, LaunchMark mark) {
  const Policy p = policy_of(a);
  if (mark) mark(kPolicyBackwardK, 0, stream);
  const cudaError_t e =
      launch(a.batch * a.length >= kEarlyTokens,
             vectors_ok(a) ? policy_backward_kernel<true> : policy_backward_kernel<false>,
             ctas(p), kCtaThreads, 0, stream, p, a.dloss, a.weight, a.dlogp);
  if (mark) mark(kPolicyBackwardK, 1, stream);
  return e;
}

}  // namespace fp8opt
