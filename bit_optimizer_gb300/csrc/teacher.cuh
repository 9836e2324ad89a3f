// Distillation from a teacher's top logits, on top of the vocabulary's cross
// entropy (linear_xent.cu): the teacher's entries of a token, made ready for the
// tiles' epilogues, which meet them in the order of the vocabulary.
//
// The entries of a token are its words with their share q of the softmax over
// the given ones, sorted by word; `start` says where in them each tile of
// kTeacherTile words begins, so that a thread, whose row is a token, has its
// tile's entries without a search.  On average a tile meets very few (64 of 50257
// words: 0.33 of a row's 256), so a column that has one is picked out of the
// thread's registers by the six bits of its place among 64 (63 selections for a
// warp's 32 rows), instead of each column being compared with a list.  Read from
// TMEM a column at a time, with the entries' loads behind one another, they cost
// the gradients of 2048 x 768 x 50257 with 128 entries 90 us.
#pragma once

#include "ops_internal.cuh"

namespace fp8opt {
namespace {

constexpr int kTeacherTile = 256;

// What a token's target stands for in the kernels that the cross entropy shares:
// one that counts, one without entries (ignored), one whose loss is NaN (vocab).
constexpr long long kTeacherLive = 0, kTeacherNone = -1;

struct Teacher {
  const uint32_t* words;     // [token][k], sorted
  const float* q;            // [token][k]
  const uint16_t* start;     // [token][tiles + 1]
  float* z;                  // [token][k]: the words' logits (forward)
  int k, tiles;
  float temperature;
  float factor;              // log2(e) / temperature
};

// A row's entries in the columns of a strip, in order.
constexpr uint32_t kNoColumn = 0xFFFFFFFFu;
struct Entries {
  const uint32_t* words;     // the token's
  int at, end;
  int64_t c0;                // the strip's first word
  uint32_t column;           // of entry `at`, from c0 on; kNoColumn behind the last
  __device__ __forceinline__ void find() {
    column = at < end ? (uint32_t)(words[at] - c0) : kNoColumn;
  }
  __device__ __forceinline__ Entries(const uint32_t* w, int first, int last, int64_t c)
      : words(w), at(first), end(last), c0(c) {
    while (at < end && (int64_t)words[at] < c0) ++at;    // (of the tile's other half)
    find();
  }
  // Calls f(first entry, entry behind the last, column - c, value) for each of the
  // row's words among the columns [c, c + 64), whose values are get(0 .. 63).  The
  // whole warp calls it, from left to right.
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
        do {
          ++at;
          find();
        } while (column - c == i);
        f(first, at, (int)i, v[0]);
      }
    }
  }
};

// A CTA's warps, a token each.
constexpr int kTeacherWarps = 8;

template <int DT>
__device__ __forceinline__ float teacher_logit(const void* p, int64_t i) {
  if (DT == kF32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return DT == kBF16 ? __uint_as_float(h << 16) : h2_to_f2(h).x;
}

// The entries of `tokens` tokens from their ids and logits, a warp to a token and
// E of them to a lane.  Entries whose id is negative are not given, and those whose
// share is 0 (of a logit of -inf) left out.  Backward, dloss is divided by the
// temperature.
template <int DT, int E>
__global__ void __launch_bounds__(32 * kTeacherWarps)
teacher_kernel(const long long* ids, const void* logits, int64_t tokens, int64_t vocab,
               const Teacher t, uint32_t* __restrict__ words, float* __restrict__ q,
               uint16_t* __restrict__ start, long long* __restrict__ state, const float* dloss,
               float* __restrict__ dloss_out) {
  __shared__ uint4 sh_id[kTeacherWarps][8 * E];
  __shared__ uint32_t sh_word[kTeacherWarps][32 * E];
  begin_after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = (int64_t)blockIdx.x * kTeacherWarps + warp;
  if (token >= tokens) return;
  uint32_t* const word = sh_word[warp];
  constexpr uint32_t kOut = 0x7FFFFFFFu;    // behind every word
  const float none = __uint_as_float(0xFF800000u);
  uint32_t id[E];
  float share[E], top = none;
  bool wrong = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int j = lane + 32 * e;
    const long long i = j < t.k ? ids[token * t.k + j] : -1;
    const float l = j < t.k ? teacher_logit<DT>(logits, token * t.k + j) : none;
    wrong |= i >= vocab || (i >= 0 && l != l);
    id[e] = i >= 0 && i < vocab ? (uint32_t)i : kOut;
    share[e] = id[e] != kOut ? l : none;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) top = fmaxf(top, share[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  wrong = __any_sync(0xFFFFFFFFu, wrong || top == -none);
  const bool dead = !wrong && top == none;
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    share[e] = dead ? 0.0f : expf((share[e] - top) / t.temperature);
    sum += share[e];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  int count = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    share[e] = __fdiv_rn(share[e], sum);
    if (wrong || dead || share[e] == 0.0f) id[e] = kOut;
    count += id[e] != kOut;
    reinterpret_cast<uint32_t*>(sh_id[warp])[lane + 32 * e] = id[e];
  }
  count = __reduce_add_sync(0xFFFFFFFFu, count);
  __syncwarp();
  // an entry's place: the smaller words, and equal ones before it
  int at[E] = {};
#pragma unroll
  for (int b = 0; b < E; ++b) {
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const uint4 w = sh_id[warp][8 * b + i];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (b == e) {
          const int to = lane - 4 * i;      // equal ones count while they are before lane
          at[e] += (w.x < id[e] + (0 < to)) + (w.y < id[e] + (1 < to)) +
                   (w.z < id[e] + (2 < to)) + (w.w < id[e] + (3 < to));
        } else {
          const uint32_t limit = id[e] + (b < e ? 1 : 0);
          at[e] += (w.x < limit) + (w.y < limit) + (w.z < limit) + (w.w < limit);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (id[e] != kOut) {
      word[at[e]] = id[e];
      words[token * t.k + at[e]] = id[e];
      q[token * t.k + at[e]] = share[e];
    }
  }
  __syncwarp();
  // the number of words below each tile's first one, four tiles of a lane at a time
  const int highest = count > 0 ? 1 << (31 - __clz(count)) : 0;
  for (int64_t t0 = lane; t0 <= t.tiles; t0 += 4 * 32) {
    int n[4] = {};
    for (int step = highest; step > 0; step >>= 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n[k] + step <= count && (int64_t)word[n[k] + step - 1] < (t0 + 32 * k) * kTeacherTile)
          n[k] += step;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (t0 + 32 * k <= t.tiles)
        start[token * (t.tiles + 1) + t0 + 32 * k] = (uint16_t)n[k];
  }
  if (lane == 0) {
    state[token] = wrong ? (long long)vocab : dead ? kTeacherNone : kTeacherLive;
    if (dloss != nullptr) dloss_out[token] = dloss[token] / t.temperature;
  }
}

// A token's loss from its entries' logits and its lse; a whole warp.
__device__ __forceinline__ float teacher_loss(const Teacher& t, int64_t token, float lse) {
  const int count = t.start[token * (t.tiles + 1) + t.tiles];
  float sum = 0.0f;
  for (int j = threadIdx.x & 31; j < count; j += 32) {
    const float q = t.q[token * t.k + j];
    sum += q * (logf(q) - (__fdiv_rn(__ldcg(t.z + token * t.k + j), t.temperature) - lse));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return sum;
}

}  // namespace
}  // namespace fp8opt
