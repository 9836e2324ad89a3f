// Distillation from a teacher's top logits, on top of the vocabulary's cross
// entropy (linear_xent.cu): the teacher's entries of a token, made ready for the
// tiles' epilogues, which meet them in the order of the vocabulary.
//
// The entries of a token are its words with their share q of the softmax over
// the given ones, sorted by word; `start` says where in them each strip of
// kTeacherStrip words begins, so that a thread, whose row is a token, has its
// strip's entries without a search.  On average a strip meets very few (64 of 50257
// words: 0.16 of a row's 128), so a column that has one is picked out of the
// thread's registers by the six bits of its place among 64 (63 selections for a
// warp's 32 rows), instead of each column being compared with a list.  Read from
// TMEM a column at a time, with the entries' loads behind one another, they cost
// the gradients of 2048 x 768 x 50257 with 128 entries 90 us.
#pragma once

#include "ops_internal.cuh"

namespace fp8opt {
namespace {

constexpr int kTeacherStrip = 128;

// What a token's target stands for in the kernels that the cross entropy shares:
// one that counts, one without entries (ignored), one whose loss is NaN (vocab).
constexpr long long kTeacherLive = 0, kTeacherNone = -1;

struct Teacher {
  const uint32_t* words;     // [token][k], sorted
  const float* q;            // [token][k]
  const uint16_t* start;     // [token][strips + 1]
  float* z;                  // [token][k]: the words' logits (forward)
  int k, strips;
  float temperature;
  float factor;              // log2(e) / temperature
  const long long* ids;      // few tokens: the entries as they are given (z goes by
                             // them too); words, q and start are NULL then
};

// A row's entries in the columns of a strip, in order: the one that comes next and
// the one behind it, which is read while the first is waited for.
constexpr uint32_t kNoColumn = 0xFFFFFFFFu;
template <bool SHARES>
struct Entries {
  const uint32_t* words;     // the token's
  const float* q;
  int at, end;               // the entry that comes next, behind the strip's last
  int64_t c0;                // the strip's first word
  uint32_t column, column1;  // from c0 on; kNoColumn behind the last
  float share, share1;
  __device__ __forceinline__ void read(int i, uint32_t* column, float* share) const {
    *column = kNoColumn;
    if (i < end) {
      *column = (uint32_t)(words[i] - c0);
      if (SHARES) *share = q[i];
    }
  }
  __device__ __forceinline__ Entries(const Teacher& t, int64_t token, int first, int last,
                                     int64_t c)
      : words(t.words + token * t.k), q(t.q + token * t.k), at(first), end(last), c0(c),
        share(0.0f), share1(0.0f) {
    read(at, &column, &share);
    read(at + 1, &column1, &share1);
  }
  // Calls f(first entry, entry behind the last, their shares' sum, column - c, value)
  // for each of the row's words among the columns [c, c + 64), whose values are
  // get(0 .. 63).  The whole warp calls it, from left to right.
  template <class G, class F>
  __device__ __forceinline__ void take(uint32_t c, G get, F f) {
    while (__any_sync(0xFFFFFFFFu, column - c < 64u)) {
      const bool mine = column - c < 64u;
      const uint32_t i = mine ? column - c : 0;
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = i & 1 ? get(2 * j + 1) : get(2 * j);
#pragma unroll
      for (int bit = 1; bit < 6; ++bit) {
#pragma unroll
        for (int j = 0; j < 32 >> bit; ++j) v[j] = i >> bit & 1 ? v[2 * j + 1] : v[2 * j];
      }
      if (mine) {
        const int first = at;
        float sum = 0.0f;
        do {
          if (SHARES) sum += share;
          column = column1;
          share = share1;
          ++at;
          read(at + 1, &column1, &share1);
        } while (column - c == i);
        f(first, at, sum, (int)i, v[0]);
      }
    }
  }
};

// Most entries of a token, and a CTA's warps.
constexpr int kTeacherMost = 256, kTeacherWarps = 8;
static_assert(kTeacherMost == 32 * kTeacherWarps, "a thread to an entry");

template <int DT>
__device__ __forceinline__ float teacher_logit(const void* p, int64_t i) {
  if (DT == kF32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return DT == kBF16 ? __uint_as_float(h << 16) : h2_to_f2(h).x;
}

// The entries of `tokens` tokens from their ids and logits, a thread to an entry and
// `group` warps (1, 2, 4 or 8) to a token.  Entries whose id is negative are not
// given, and those whose share is 0 (of a logit of -inf) left out.  Backward, dloss
// is divided by the temperature.  `zeros`: words to set to zero besides.
//
// Bound by latency for few tokens (6 of 197 entries: 7 us; with a warp to a token
// 19), by the sort's instructions for many (8191 of 64 entries: 19 us with cold
// caches; 2279 of 217: 21, by counting each entry's smaller words 28).
__global__ void __launch_bounds__(32 * kTeacherWarps)
teacher_kernel(const long long* ids, const void* logits, int logit_dtype, int64_t tokens,
               int64_t vocab, int group, const Teacher t, uint32_t* __restrict__ words,
               float* __restrict__ q, uint16_t* __restrict__ start,
               long long* __restrict__ state, const float* dloss,
               float* __restrict__ dloss_out, int* __restrict__ zeros, int n_zeros) {
  __shared__ uint32_t sh_word[32 * kTeacherWarps];
  __shared__ float sh_share[32 * kTeacherWarps];
  __shared__ float sh_top[kTeacherWarps], sh_sum[kTeacherWarps];
  __shared__ int sh_wrong[kTeacherWarps], sh_count[kTeacherWarps];
  begin_after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % group, first = warp - sub;      // of the token's warps
  const int64_t token = (int64_t)blockIdx.x * (kTeacherWarps / group) + warp / group;
  const bool live = token < tokens;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < n_zeros; i += 32 * kTeacherWarps) zeros[i] = 0;
  const int j = 32 * sub + lane;
  constexpr uint32_t kOut = 0x7FFFFFFFu;    // behind every word
  const float none = __uint_as_float(0xFF800000u);
  uint32_t id = kOut;
  float share = none;
  bool wrong = false;
  if (live && j < t.k) {
    const int64_t at = token * t.k + j;
    const long long i = ids[at];
    const float l = logit_dtype == kF32    ? teacher_logit<kF32>(logits, at)
                    : logit_dtype == kBF16 ? teacher_logit<kBF16>(logits, at)
                                           : teacher_logit<kF16>(logits, at);
    wrong = i >= vocab || (i >= 0 && l != l);
    if (i >= 0 && !wrong) {
      id = (uint32_t)i;
      share = l;
    }
  }
  float top = share;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  wrong = __any_sync(0xFFFFFFFFu, wrong);
  if (lane == 0) {
    sh_top[warp] = top;
    sh_wrong[warp] = wrong;
  }
  __syncthreads();
  wrong = false;
  for (int w = first; w < first + group; ++w) {
    top = fmaxf(top, sh_top[w]);
    wrong |= sh_wrong[w] != 0;
  }
  wrong |= top == -none;
  const bool dead = !wrong && top == none;
  share = wrong || dead ? 0.0f : expf((share - top) / t.temperature);
  float sum = share;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) sh_sum[warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int w = first; w < first + group; ++w) sum += sh_sum[w];
  if (share > 0.0f) share = __fdiv_rn(share, sum);
  if (share == 0.0f) id = kOut;
  const int mine = __popc(__ballot_sync(0xFFFFFFFFu, id != kOut));
  if (lane == 0) sh_count[warp] = mine;
  // sorted by word, a bitonic network: entry j to thread j, shuffles within a warp
  const auto exchange = [&](int k, int d, uint32_t other, float other_share) {
    const bool least = ((j & k) == 0) == ((j & d) == 0);
    if (least ? other < id : other > id) {
      id = other;
      share = other_share;
    }
  };
  const auto shuffles = [&](int k, int most) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
      if (d <= most)
        exchange(k, d, __shfl_xor_sync(0xFFFFFFFFu, id, d),
                 __shfl_xor_sync(0xFFFFFFFFu, share, d));
  };
#pragma unroll
  for (int k = 2; k <= 32; k *= 2) shuffles(k, k / 2);
  for (int k = 64; k <= 32 * group; k *= 2) {
    for (int d = k / 2; d >= 32; d /= 2) {
      __syncthreads();
      sh_word[threadIdx.x] = id;
      sh_share[threadIdx.x] = share;
      __syncthreads();
      exchange(k, d, sh_word[threadIdx.x ^ d], sh_share[threadIdx.x ^ d]);
    }
    shuffles(k, 16);
  }
  __syncthreads();
  uint32_t* const strip_of = sh_word + 32 * first;
  int count = 0;
  for (int w = first; w < first + group; ++w) count += sh_count[w];
  strip_of[j] = id / kTeacherStrip;
  if (j < count) {
    words[token * t.k + j] = id;
    q[token * t.k + j] = share;
  }
  __syncthreads();
  if (!live) return;
  // the number of entries before each strip: a thread has neighbouring strips, looks
  // for the first one's and goes on from there (8191 tokens of 64 entries, 394
  // strips: 24 us with a search for each)
  const int per = (t.strips + 32 * group) / (32 * group), s0 = j * per;
  int n = 0;
  for (int step = count > 0 ? 1 << (31 - __clz(count)) : 0; step > 0; step >>= 1)
    if (n + step <= count && strip_of[n + step - 1] < (uint32_t)s0) n += step;
  uint16_t* const out = start + token * (t.strips + 1);
  for (int s = s0; s < min(s0 + per, t.strips + 1); ++s) {
    while (n < count && strip_of[n] < (uint32_t)s) ++n;
    out[s] = (uint16_t)n;
  }
  if (j == 0) {
    state[token] = wrong ? (long long)vocab : dead ? kTeacherNone : kTeacherLive;
    if (dloss != nullptr) dloss_out[token] = dloss[token] / t.temperature;
  }
}

// A token's loss from its entries' logits, the row's largest logit and the log of its
// sum of exponentials above that; a whole warp.  (lse, which adds the two up, is
// rounded to its own size, and z / t to its: with differences from the largest logit
// the loss of 64 entries at logits around 28 and t = 0.05 is off by 1.4e-7 on average
// instead of 7.6e-6, at t = 1 by 1.5e-7 instead of 9.4e-7.)  The first 32 entries are
// read when it is made.
struct TeacherLoss {
  int count = 0;
  float q = 0.0f, z = 0.0f;
  __device__ __forceinline__ TeacherLoss(const Teacher& t, int64_t token, bool any) {
    const int lane = threadIdx.x & 31;
    if (!any) return;
    count = t.start[token * (t.strips + 1) + t.strips];
    if (lane < t.k) {      // (what is behind `count` was never written, and is not used)
      q = t.q[token * t.k + lane];
      z = __ldcg(t.z + token * t.k + lane);
    }
  }
  __device__ __forceinline__ float operator()(const Teacher& t, int64_t token, float top,
                                              float log_sum) {
    float sum = 0.0f;
    for (int j = threadIdx.x & 31; j < count; j += 32) {
      if (j >= 32) {
        q = t.q[token * t.k + j];
        z = __ldcg(t.z + token * t.k + j);
      }
      sum += q * (logf(q) - (__fdiv_rn(z - top, t.temperature) - log_sum));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    return sum;
  }
};

}  // namespace
}  // namespace fp8opt
