// Distillation from a teacher's top logits, on top of the vocabulary's cross
// entropy (linear_xent.cu): the teacher's entries of a token, made ready for the
// tiles' epilogues, which meet them in the order of the vocabulary.
//
// The entries of a token are its words with their share q of the softmax over
// the given ones, sorted by word; `start` says where in them each tile of
// kTeacherTile words begins, so that a thread, whose row is a token, has its
// tile's entries without a search.  On average a tile meets very few (64 of 50257
// words: 0.33 of a row's 256), so the epilogues fetch their logits one column of
// TMEM at a time instead of comparing every column with a list.
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

// Entry `at` of a token's up to `end` as a column from c0 on (its word is not
// below); kNoColumn behind the end.
constexpr uint32_t kNoColumn = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t column_of(const uint32_t* words, int at, int end, int64_t c0) {
  return at < end ? (uint32_t)(words[at] - c0) : kNoColumn;
}

// One column of the warp's lanes.
__device__ __forceinline__ float tmem_column(uint32_t addr) {
  uint32_t r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r)
      : "r"(addr)
      : "memory");
  return __uint_as_float(r);
}

// Calls f(first entry, entry behind the last, column, logit) for every word of the
// lane's token among the `cols` columns at `tmem`, which are the words from c0 on.
// The whole warp calls it; each column with an entry is read once.
template <class F>
__device__ __forceinline__ void each_entry(const uint32_t* words, int at, int end, int64_t c0,
                                           int cols, uint32_t tmem, F f) {
  while (at < end && (int64_t)words[at] < c0) ++at;      // (of the tile's other half)
  uint32_t column = column_of(words, at, end, c0);
  for (;;) {
    const uint32_t next = __reduce_min_sync(0xFFFFFFFFu, column);
    if (next >= (uint32_t)cols) break;
    const float z = tmem_column(tmem + next);
    if (column == next) {
      const int first = at;
      do column = column_of(words, ++at, end, c0);
      while (column == next);
      f(first, at, (int)next, z);
    }
    __syncwarp();
  }
}

// Most entries of a token, and a CTA's warps, a token each.
constexpr int kTeacherMost = 256, kTeacherWarps = 8;

template <int DT>
__device__ __forceinline__ float teacher_logit(const void* p, int64_t i) {
  if (DT == kF32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return DT == kBF16 ? __uint_as_float(h << 16) : h2_to_f2(h).x;
}

// The entries of `tokens` tokens from their ids and logits.  Entries whose id is
// negative are not given, and those whose share is 0 (of a logit of -inf) left
// out.  Backward, dloss is divided by the temperature.
template <int DT>
__global__ void __launch_bounds__(32 * kTeacherWarps)
teacher_kernel(const long long* ids, const void* logits, int64_t tokens, int64_t vocab,
               const Teacher t, uint32_t* __restrict__ words, float* __restrict__ q,
               uint16_t* __restrict__ start, long long* __restrict__ state, const float* dloss,
               float* __restrict__ dloss_out) {
  __shared__ uint32_t sh_id[kTeacherWarps][kTeacherMost], sh_word[kTeacherWarps][kTeacherMost];
  __shared__ float sh_q[kTeacherWarps][kTeacherMost];
  begin_after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = (int64_t)blockIdx.x * kTeacherWarps + warp;
  if (token >= tokens) return;
  uint32_t* const id = sh_id[warp];
  uint32_t* const word = sh_word[warp];
  float* const share = sh_q[warp];
  constexpr uint32_t kOut = 0x7FFFFFFFu;    // behind every word
  const float none = __uint_as_float(0xFF800000u);
  bool wrong = false;
  float top = none;
  for (int j = lane; j < t.k; j += 32) {
    const long long i = ids[token * t.k + j];
    const float l = teacher_logit<DT>(logits, token * t.k + j);
    wrong |= i >= vocab;
    id[j] = i >= 0 && i < vocab ? (uint32_t)i : kOut;
    share[j] = id[j] != kOut ? l : none;
    top = fmaxf(top, share[j]);
    wrong |= share[j] != share[j];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  wrong = __any_sync(0xFFFFFFFFu, wrong || top == -none);
  const bool dead = !wrong && top == none;
  __syncwarp();
  float sum = 0.0f;
  if (!wrong && !dead) {
    for (int j = lane; j < t.k; j += 32) {
      share[j] = expf((share[j] - top) / t.temperature);
      sum += share[j];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  int count = 0;
  if (!wrong && !dead) {
    for (int j = lane; j < t.k; j += 32) {
      share[j] = __fdiv_rn(share[j], sum);
      if (share[j] == 0.0f) id[j] = kOut;
      count += id[j] != kOut;
    }
  }
  count = __reduce_add_sync(0xFFFFFFFFu, count);
  __syncwarp();
  // an entry's place: the smaller words, and equal ones before it
  if (count > 0) {
    for (int j = lane; j < t.k; j += 32) {
      const uint32_t mine = id[j];
      if (mine == kOut) continue;
      int at = 0;
#pragma unroll 4
      for (int i = 0; i < t.k; ++i) at += id[i] < mine + (i < j);
      word[at] = mine;
      words[token * t.k + at] = mine;
      q[token * t.k + at] = share[j];
    }
  }
  __syncwarp();
  for (int64_t tile = lane; tile <= t.tiles; tile += 32) {
    const int64_t first = tile * kTeacherTile;
    int lo = 0, hi = count;                 // the first entry of a word >= first
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if ((int64_t)word[mid] < first) lo = mid + 1;
      else hi = mid;
    }
    start[token * (t.tiles + 1) + tile] = (uint16_t)lo;
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
