// The embedding lookup, y[i] = scale w[ids[i]], and the dense gradient of its
// table, dw[v] = scale * sum of dy[i] over the tokens i with ids[i] = v.
//
// forward   Bound by memory: every thread has four 16-byte vectors of the
//           result under way, each an id, its row's vector and a store.
//           16381 x 2048 BF16 over 50257 words: 16 us, 5.7 TB/s.
// backward  Each sum is in the tokens' order, without float atomics.  Up to
//           kFewTokens in one launch; else in three steps:
//           order   The tokens sorted by word, stably.  Up to kRankTokens each
//                   finds its place by comparing its key with all others; more, a
//                   radix sort of eight bits a pass, while other CTAs fill dw with
//                   zeros (which takes as long).
//           sums    A warp takes 8 to 32 consecutive tokens of the order and the
//                   columns that its lanes' 16-byte vectors cover, and adds rows
//                   of one word in fp32.  A word whose tokens lie within the
//                   chunk is written at once, a part of a word that goes on
//                   beyond it to scratch.  After the short sort, other warps fill
//                   the rows of words without tokens.
//           join    The parts of such words, in order.
// A frequent word's tokens are thereby spread over as many warps as any others.
// 65536 x 1024 BF16 over 50257 words: 57 to 58 us, of which the sort takes 12 alone
// and 22 with the zeros, the sums some 30 (170 MB), the join 8; bound by memory but
// for the sort's and the join's latencies.  Fewer tokens are bound by those and by
// the zeros: 2047 x 768, 21.5 us (77 MB of zeros alone 12).  Zeros for the highest
// words beside the sort and for the rest beside the sums gained nothing.
#include "ops_internal.cuh"

namespace fp8opt {

namespace {

constexpr int kCtaThreads = 256, kCtaWarps = kCtaThreads / 32;

// --------------------------------------------------------------- elements

// An element as it was loaded.
template <int DT>
__device__ __forceinline__ float value(uint32_t v) {
  if (DT == kF32) return __uint_as_float(v);
  return DT == kBF16 ? __uint_as_float(v << 16) : h2_to_f2(v).x;
}

// Elements of a lane's 16-byte vector.
template <int DT>
constexpr int kPer = DT == kF32 ? 4 : 8;

template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float (&e)[kPer<DT>]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == kF32) {
      e[k] = __uint_as_float(w[k]);
    } else {
      const float2 f = DT == kBF16 ? make_float2(__uint_as_float(w[k] << 16),
                                                 __uint_as_float(w[k] & 0xFFFF0000u))
                                   : h2_to_f2(w[k]);
      e[2 * k] = f.x;
      e[2 * k + 1] = f.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack(const float (&e)[kPer<DT>]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == kF32) w[k] = __float_as_uint(e[k]);
    else w[k] = pack2<DT>(e[2 * k], e[2 * k + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- forward

constexpr int kForwardVectors = 4;   // of a thread

// Rows of `vectors` 16-byte vectors.
template <int DT>
__global__ void __launch_bounds__(kCtaThreads)
embedding_kernel(const long long* ids, const uint4* w, int64_t rows, int64_t vectors,
                 int64_t vocab, float scale, uint4* __restrict__ y) {
  begin_after_previous();
  const int64_t total = rows * vectors;
  const int64_t i0 = (int64_t)blockIdx.x * (kForwardVectors * kCtaThreads) + threadIdx.x;
  uint4 v[kForwardVectors];
  bool known[kForwardVectors];
#pragma unroll
  for (int k = 0; k < kForwardVectors; ++k) {
    const int64_t i = i0 + k * kCtaThreads;
    known[k] = false;
    v[k] = make_uint4(0, 0, 0, 0);
    if (i < total) {
      const int64_t row = total <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / (uint32_t)vectors)
                                                 : i / vectors;
      const long long id = ids[row];
      known[k] = id >= 0 && id < vocab;
      if (known[k]) v[k] = w[id * vectors + (i - row * vectors)];
    }
  }
#pragma unroll
  for (int k = 0; k < kForwardVectors; ++k) {
    float e[kPer<DT>];
    unpack<DT>(v[k], e);
#pragma unroll
    for (int j = 0; j < kPer<DT>; ++j)
      e[j] = known[k] ? e[j] * scale : __uint_as_float(0x7FC00000u);
    const int64_t i = i0 + k * kCtaThreads;
    if (i < total) __stcs(y + i, pack<DT>(e));
  }
}

// Rows that start anywhere: a warp takes kRowPart elements of a row.  parts: of a
// row.  (The loads do not depend on whether the id or the column exists, so that
// all are under way.)
constexpr int kRowPart = 512;
template <int DT>
__global__ void __launch_bounds__(kCtaThreads)
embedding_any_kernel(const long long* ids, const void* w, int64_t rows, int64_t dim,
                     int64_t vocab, unsigned parts, float scale, void* y) {
  begin_after_previous();
  const unsigned unit = blockIdx.x * kCtaWarps + (threadIdx.x >> 5);
  const unsigned row = unit / parts;
  const int64_t c0 = (int64_t)(unit - row * parts) * kRowPart + (threadIdx.x & 31);
  if (row >= rows) return;
  const long long id = ids[row];
  const bool known = id >= 0 && id < vocab;
  const int n = (int)min((int64_t)kRowPart, dim - c0);       // of the lane's columns, 32 apart
  constexpr int kSize = DT == kF32 ? 4 : 2;
  const char* const from = static_cast<const char*>(w) + ((known ? id : 0) * dim + c0) * kSize;
  char* const to = static_cast<char*>(y) + ((int64_t)row * dim + c0) * kSize;
  if (n <= 0) return;
  uint32_t v[kRowPart / 32];
#pragma unroll
  for (int k = 0; k < kRowPart / 32; ++k) {
    const char* const p = from + (32 * k < n ? 32 * k * kSize : 0);
    if (kSize == 4) asm volatile("ld.global.b32 %0, [%1];" : "=r"(v[k]) : "l"(p));
    else {
      uint16_t h;
      asm volatile("ld.global.b16 %0, [%1];" : "=h"(h) : "l"(p));
      v[k] = h;
    }
  }
#pragma unroll
  for (int k = 0; k < kRowPart / 32; ++k) {
    if (32 * k < n)
      store1<DT>(to, 32 * k, known ? value<DT>(v[k]) * scale : __uint_as_float(0x7FC00000u));
  }
}

// ------------------------------------------------------------------ order

// A token's key: its word, or `vocab` where it takes no part (padding, or no
// word of the table), which sorts last.
__device__ __forceinline__ uint32_t key_of(long long id, uint32_t vocab, long long padding) {
  return id >= 0 && id < (long long)vocab && id != padding ? (uint32_t)id : vocab;
}

// Part `part` of `parts` of the zeros in `bytes` at p, which are elements of
// `size` bytes at any of their boundaries.
struct Fill {
  char* p;
  int64_t bytes;
  int size, part, parts;
};

// CTA `cta` of `ctas`.
__device__ __forceinline__ void fill_zeros(const Fill& f, int64_t cta, int64_t ctas) {
  const int64_t head = min((int64_t)(-reinterpret_cast<intptr_t>(f.p) & 15), f.bytes);
  const int64_t words = (f.bytes - head) / 16, tail = head + 16 * words;
  uint4* const q = reinterpret_cast<uint4*>(f.p + head);
  const int64_t lo = words / f.parts * f.part;
  const int64_t hi = f.part + 1 == f.parts ? words : words / f.parts * (f.part + 1);
  for (int64_t i = lo + cta * blockDim.x + threadIdx.x; i < hi; i += ctas * blockDim.x)
    q[i] = make_uint4(0, 0, 0, 0);
  // at most 15 bytes at either end
  if (f.part == 0 && cta == 0 && threadIdx.x < 16) {
    const int64_t a = (int64_t)threadIdx.x * f.size, b = tail + a;
    if (f.size == 2) {
      if (a < head) *reinterpret_cast<uint16_t*>(f.p + a) = 0;
      if (b < f.bytes) *reinterpret_cast<uint16_t*>(f.p + b) = 0;
    } else {
      if (a < head) *reinterpret_cast<uint32_t*>(f.p + a) = 0;
      if (b < f.bytes) *reinterpret_cast<uint32_t*>(f.p + b) = 0;
    }
  }
}

// Some tokens: the place of each is the number of smaller keys, and of equal ones
// before it.  A CTA places 32 tokens, its warps comparing them with a share of all
// keys each.  (4096 tokens over 50257 x 768, 5000 x 512: 25.2 and 16.4 us; by the
// radix sort 8192 take 25 and 20, by this one 38 and 27.)  CTAs that are launched
// early start where the previous kernel leaves room, many to an SM; kRankSmem bytes
// of shared memory, more than half of it, keep them to one each (4096 tokens over
// 5000 x 512: 14.8 us; launched late 16.4, early without it 29.9).
constexpr int64_t kRankTokens = 4096;
constexpr int kRankSmem = 200 << 10;
static_assert(kRankTokens * 4 <= kRankSmem - 4096, "the keys");

__global__ void __launch_bounds__(kCtaThreads)
embedding_rank_kernel(const long long* ids, int n, uint32_t vocab, long long padding,
                      uint32_t* __restrict__ keys, uint32_t* __restrict__ tokens) {
  extern __shared__ uint4 all4[];
  __shared__ int smaller[kCtaWarps][32];
  begin_after_previous();
  uint32_t* const all = reinterpret_cast<uint32_t*>(all4);
  const int share = ((n + kCtaWarps - 1) / kCtaWarps + 31) / 32 * 32;     // of a warp
#pragma unroll 8
  for (int i = threadIdx.x; i < share * kCtaWarps; i += kCtaThreads) {
    const long long id = ids[min(i, n - 1)];
    all[i] = i < n ? key_of(id, vocab, padding) : 0xFFFFFFFFu;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x * 32, i = first + lane;
  const uint32_t key = all[min(i, n - 1)];
  const int lo = warp * share, hi = lo + share;
  int count = 0;
  const auto below = [&](int a, int b, uint32_t limit) {
#pragma unroll 4
    for (int j = a / 4; j < b / 4; ++j) {
      const uint4 k = all4[j];
      count += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
    }
  };
  // equal keys count where they come before (limits: key + 1 and key)
  below(lo, min(hi, first), key + 1);
  for (int j = max(lo, first); j < min(hi, first + 32); ++j) count += all[j] < key + (j < i);
  below(max(lo, first + 32), hi, key);
  smaller[warp][lane] = count;
  __syncthreads();
  if (warp == 0 && i < n) {
    int at = 0;
#pragma unroll
    for (int w = 0; w < kCtaWarps; ++w) at += smaller[w][lane];
    keys[at] = key;
    tokens[at] = (uint32_t)i;
  }
}

// More tokens: a stable sort by eight bits of the key a pass, in tiles of a CTA
// each (a multiple of kSortStep tokens: 65536 tokens 59.6 us, with twice the step
// 62.4).  First the tiles' counts of each digit, for the first pass; every pass then
// counts the next one's, where its tokens go to (whole numbers: the order of the
// atomics does not matter).
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kDigits = 256;
constexpr int kRounds = 1, kSortStep = kRounds * kSortThreads;

struct SortPass {
  const long long* ids;      // the first pass's input; else NULL
  const uint32_t* keys;      // the later ones'
  const uint32_t* tokens;
  int64_t n, tile;
  int tiles, shift;
  uint32_t vocab;
  long long padding;
  uint32_t* counts;          // [tile][digit]
  uint32_t* next;            // the next pass's; NULL in the last one
  uint32_t* keys_out;
  uint32_t* tokens_out;
  __device__ __forceinline__ uint32_t key(int64_t i) const {
    return ids != nullptr ? key_of(ids[i], vocab, padding) : keys[i];
  }
};

// later: the counts of the `rest` later passes, set to zero.
__global__ void __launch_bounds__(kSortThreads)
embedding_count_kernel(SortPass s, uint32_t* later, int rest, Fill fill) {
  __shared__ uint32_t count[kDigits];
  begin_after_previous();
  if ((int)blockIdx.x >= s.tiles) {
    fill_zeros(fill, blockIdx.x - s.tiles, gridDim.x - s.tiles);
    return;
  }
  const int t = threadIdx.x;
  if (t < kDigits) count[t] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * s.tile, hi = min(lo + s.tile, s.n);
#pragma unroll 2
  for (int64_t i = lo + t; i < hi; i += kSortThreads)
    atomicAdd(&count[s.key(i) >> s.shift & (kDigits - 1)], 1u);
  for (int p = 0; p < rest; ++p)
    if (t < kDigits) later[((int64_t)p * s.tiles + blockIdx.x) * kDigits + t] = 0;
  __syncthreads();
  if (t < kDigits) s.counts[(int64_t)blockIdx.x * kDigits + t] = count[t];
}

// Every token to its place: those of smaller digits, of its digit in earlier
// tiles, in its tile's earlier warps and in its own warp come before it.
__global__ void __launch_bounds__(kSortThreads)
embedding_place_kernel(SortPass s, Fill fill) {
  constexpr int kGroups = kSortThreads / kDigits;
  __shared__ uint32_t base[kDigits], sums[kDigits / 32];
  __shared__ uint32_t of_group[kGroups][2][kDigits];
  __shared__ uint32_t before[kSortWarps][kDigits];   // a warp's tokens, then where they start
  begin_after_previous();
  if ((int)blockIdx.x >= s.tiles) {
    fill_zeros(fill, blockIdx.x - s.tiles, gridDim.x - s.tiles);
    return;
  }
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int64_t lo = blockIdx.x * s.tile, hi = min(lo + s.tile, s.n);
  // a warp's kRounds x 32 consecutive tokens
  uint32_t key[kRounds], token[kRounds];
  const auto read = [&](int64_t step) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int64_t i = step + warp * (kRounds * 32) + lane + 32 * r;
      key[r] = i < hi ? s.key(i) : 0;
      token[r] = i < hi && s.ids == nullptr ? s.tokens[i] : (uint32_t)i;
    }
  };
  read(lo);
  // of each digit, all tokens and those in earlier tiles; a quarter of the tiles to
  // a group of threads
  {
    const int group = t / kDigits, d = t % kDigits;
    uint32_t all = 0, mine = 0;
#pragma unroll 8
    for (int k = group; k < s.tiles; k += kGroups) {
      const uint32_t c = s.counts[(int64_t)k * kDigits + d];
      all += c;
      mine += k < (int)blockIdx.x ? c : 0;
    }
    of_group[group][0][d] = all;
    of_group[group][1][d] = mine;
  }
  __syncthreads();
  if (t < kDigits) {
    uint32_t all = 0, mine = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      all += of_group[g][0][t];
      mine += of_group[g][1][t];
    }
    uint32_t up = all;     // of the digits up to this one, first within the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, up, o);
      if (lane >= o) up += v;
    }
    if (lane == 31) sums[warp] = up;
    base[t] = up - all + mine;
  }
  __syncthreads();
  if (t < kDigits)
    for (int w = 0; w < warp; ++w) base[t] += sums[w];
  for (int64_t step = lo; step < hi; step += kSortStep) {
    for (int i = t; i < kSortWarps * kDigits; i += kSortThreads) (&before[0][0])[i] = 0;
    __syncthreads();
    uint32_t rank[kRounds];
    const int64_t i0 = step + warp * (kRounds * 32) + lane;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const bool in = i0 + 32 * r < hi;
      const int digit = in ? (int)(key[r] >> s.shift & (kDigits - 1)) : kDigits;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
      const unsigned earlier = same & ((1u << lane) - 1);
      rank[r] = __popc(earlier) + (in ? before[warp][digit] : 0);
      __syncwarp();
      if (in && earlier == 0) before[warp][digit] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (t < kDigits) {
      uint32_t at = base[t];
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = before[w][t];
        before[w][t] = at;
        at += c;
      }
      base[t] = at;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const bool in = i0 + 32 * r < hi;
      const uint32_t at =
          in ? before[warp][key[r] >> s.shift & (kDigits - 1)] + rank[r] : 0;
      if (in) {
        s.keys_out[at] = key[r];
        s.tokens_out[at] = token[r];
      }
      if (s.next != nullptr) {
        // one atomic for a word's tokens in the warp, where they go to one tile:
        // a frequent word's meet at one address
        const uint32_t to = at / (uint32_t)s.tile;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, in ? key[r] : ~0u);
        const int first = __ffs(same) - 1;
        const bool one = __shfl_sync(0xFFFFFFFFu, to, first) ==
                         __shfl_sync(0xFFFFFFFFu, to, 31 - __clz(same));
        if (in && (!one || lane == first))
          atomicAdd(&s.next[(int64_t)to * kDigits + (key[r] >> (s.shift + 8) & (kDigits - 1))],
                    one ? __popc(same) : 1u);
      }
    }
    if (step + kSortStep < hi) read(step + kSortStep);
    __syncthreads();
  }
}

// ------------------------------------------------------------------- sums

// Tokens of a warp, at most one to a lane: 32, or where that makes few warps, 16
// or 8 (whose rows are all under way at once).
constexpr int kMostChunk = 32, kLeastChunk = 8;
// Warps of a CTA, and where the chunks are the largest.  With eight and four at the
// largest: 65536 x 1024 58.1 and 62.2 us, 131072 x 768 74.3 and 77.8, 16381 x 2048 59.3
// and 64.2, but 16381 x 2047 76.9 and 73.4.  Below them it hardly matters (2047 x 768
// 21.8 both, 4096 x 768 26.0 and 26.6, 16384 x 768 31.4 and 31.1), but for the one launch
// of few tokens (256 x 768: 16.3 and 15.9; 100 x 769: 18.1 and 17.0).
constexpr int kSumWarps = 4, kMostSumWarps = 8;

struct Sums {
  const uint32_t* keys;
  const uint32_t* tokens;
  int64_t n, dim;
  uint32_t vocab;
  unsigned slices;             // of 32 lanes' columns
  int chunk;                   // tokens of a warp
  unsigned sums;               // warps that add; those behind them fill
  int group;                   // words of a filling warp; 0: dw is filled already
  const void* dy;
  float scale;
  float* parts;                // [chunk][2][dim]: the first word's, the last word's
  void* dw;
};

// A lane's columns of a slice: VEC, kPer in a row; else every 32nd from c on.
template <int DT, bool VEC>
struct Columns {
  static constexpr int E = kPer<DT>, kStep = VEC ? 1 : 32;
  int64_t c, dim;
  __device__ __forceinline__ Columns(int64_t slice, int64_t d)
      : c(slice * (32 * E) + (threadIdx.x & 31) * (VEC ? E : 1)), dim(d) {}
  // What a row of p has there; anything behind its end, which is not stored.  The
  // loads do not depend on whether the values count, so that many are under way
  // (volatile: else the compiler moves each behind the test of its count).
  struct Raw {
    uint32_t v[VEC ? 4 : E];
  };
  __device__ __forceinline__ Raw fetch(const void* p, int64_t row) const {
    constexpr int kSize = 16 / E;
    Raw r;
    const char* const from = static_cast<const char*>(p) + (row * dim + (c < dim ? c : 0)) * kSize;
    if constexpr (VEC) {
      asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3])
                   : "l"(from));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const char* const at = from + (c + j * kStep < dim ? j * kStep * kSize : 0);
        if constexpr (kSize == 4) {
          asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.v[j]) : "l"(at));
        } else {
          uint16_t h;
          asm volatile("ld.global.b16 %0, [%1];" : "=h"(h) : "l"(at));
          r.v[j] = h;
        }
      }
    }
    return r;
  }
  static __device__ __forceinline__ void add(const Raw& r, bool counts, float (&sum)[E]) {
    float e[E];
    if constexpr (VEC) {
      unpack<DT>(make_uint4(r.v[0], r.v[1], r.v[2], r.v[3]), e);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) e[j] = value<DT>(r.v[j]);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) sum[j] += counts ? e[j] : 0.0f;
  }
  __device__ __forceinline__ void store(void* p, int64_t row, const float (&e)[E]) const {
    if constexpr (VEC) {
      if (c < dim)
        *reinterpret_cast<uint4*>(static_cast<char*>(p) + (row * dim + c) * (16 / E)) =
            pack<DT>(e);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (c + j * kStep < dim) store1<DT>(p, row * dim + c + j * kStep, e[j]);
    }
  }
};

// Zeros in a row of dw, 16 bytes at a time wherever it starts; a whole warp.  (2047
// tokens over 50257 x 769: 24.5 us, by elements 30.5.)
template <int DT>
__device__ __forceinline__ void zero_row(void* dw, int64_t row, int64_t dim) {
  constexpr int kSize = DT == kF32 ? 4 : 2;
  char* const p = static_cast<char*>(dw) + row * dim * kSize;
  const int64_t bytes = dim * kSize;
  const int64_t head = min((int64_t)(-reinterpret_cast<intptr_t>(p) & 15), bytes);
  const int64_t words = (bytes - head) / 16;
  const int lane = threadIdx.x & 31;
  for (int64_t i = lane; i < words; i += 32)
    reinterpret_cast<uint4*>(p + head)[i] = make_uint4(0, 0, 0, 0);
  // at most 15 bytes at either end
  const int64_t a = lane * kSize, b = head + 16 * words + a;
  if (a < head) store1<DT>(p + a, 0, 0.0f);
  if (b < bytes) store1<DT>(p + b, 0, 0.0f);
}

// Zeros in the rows of the words [v0, v0 + group) that have no token: their place
// among the keys is searched for, a word to a lane.
template <int DT>
__device__ __forceinline__ void fill_absent(const Sums& s, int64_t v0) {
  const int64_t v = v0 + (threadIdx.x & 31);
  const bool mine = (threadIdx.x & 31) < s.group && v < (int64_t)s.vocab;
  int64_t lo = 0, hi = s.n;                  // the first key >= v
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if ((int64_t)s.keys[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  unsigned absent = __ballot_sync(0xFFFFFFFFu, mine && (lo == s.n || (int64_t)s.keys[lo] != v));
  for (; absent != 0; absent &= absent - 1)
    zero_row<DT>(s.dw, v0 + __ffs(absent) - 1, s.dim);
}

// Adds `count` <= 32 rows of dy, the lanes' tokens in order, to sum; where `ends`
// has a token's bit, put(its word) takes the sum, which starts again at 0.
constexpr int kAhead = 8;      // rows under way

template <int DT, bool VEC, class F>
__device__ __forceinline__ void add_rows(const Columns<DT, VEC>& columns, const void* dy,
                                         uint32_t word, uint32_t token, unsigned ends, int count,
                                         float (&sum)[kPer<DT>], F put) {
  for (int r = 0; r < count; r += kAhead) {
    typename Columns<DT, VEC>::Raw raw[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)     // (lanes without a token hold row 0's number)
      raw[k] = columns.fetch(dy, __shfl_sync(0xFFFFFFFFu, token, r + k));
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      columns.add(raw[k], r + k < count, sum);
      const uint32_t w = __shfl_sync(0xFFFFFFFFu, word, r + k);
      if (ends >> (r + k) & 1u) {
        put(w);
#pragma unroll
        for (int j = 0; j < kPer<DT>; ++j) sum[j] = 0.0f;
      }
    }
  }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(32 * kMostSumWarps)
embedding_sums_kernel(const Sums s) {
  begin_after_previous();
  constexpr int E = kPer<DT>;
  const int lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (unit >= s.sums) {
    if (s.group > 0) fill_absent<DT>(s, (int64_t)(unit - s.sums) * s.group);
    return;
  }
  const int64_t chunk = unit / s.slices, slice = unit - (unsigned)chunk * s.slices;
  const int64_t first = chunk * s.chunk, at = first + lane;
  if (first >= s.n) return;
  const uint32_t none = s.vocab;
  const bool mine = lane < s.chunk && at < s.n;
  const uint32_t key = mine ? s.keys[at] : none;
  const uint32_t token = mine ? s.tokens[at] : 0;
  uint32_t before = none, after = none;
  if (first > 0) before = s.keys[first - 1];
  if (first + s.chunk < s.n) after = s.keys[first + s.chunk];
  uint32_t next = __shfl_down_sync(0xFFFFFFFFu, key, 1);
  if (lane == s.chunk - 1) next = after;
  const unsigned live = __ballot_sync(0xFFFFFFFFu, key != none);
  const unsigned ends = __ballot_sync(0xFFFFFFFFu, key != none && (next != key));
  if (live == 0) return;
  bool goes_on = before == __shfl_sync(0xFFFFFFFFu, key, 0);   // from the chunk before
  const int count = __popc(live);                              // (those without a part come last)

  const Columns<DT, VEC> columns(slice, s.dim);
  const int64_t c0 = columns.c;
  constexpr int kStep = columns.kStep;
  float sum[E];
#pragma unroll
  for (int j = 0; j < E; ++j) sum[j] = 0.0f;
  const auto put = [&](uint32_t word, float* part) {
    if (part != nullptr) {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (c0 + j * kStep < s.dim) part[c0 + j * kStep] = sum[j];
    } else {
      float e[E];
#pragma unroll
      for (int j = 0; j < E; ++j) e[j] = sum[j] * s.scale;
      columns.store(s.dw, word, e);
    }
  };
  float* const parts = s.parts + chunk * 2 * s.dim;
  add_rows<DT, VEC>(columns, s.dy, key, token, ends, count, sum, [&](uint32_t word) {
    put(word, goes_on ? parts : nullptr);
    goes_on = false;
  });
  if (!(ends >> (count - 1) & 1u)) put(0, goes_on ? parts : parts + s.dim);
}

// Few tokens: one launch.  A warp takes `group` words and a slice of the columns,
// looks for their tokens among all ids, puts them in order and adds their rows, and
// writes zeros for the words without any.
constexpr int kFewTokens = 256;

template <int DT, bool VEC>
__global__ void __launch_bounds__(32 * kSumWarps)
embedding_few_kernel(const Sums s, const long long* ids, long long padding) {
  __shared__ uint32_t keys[kFewTokens];
  // a token's word, from the group's first on, and its number: found, then in order
  __shared__ uint16_t found[kSumWarps][kFewTokens], ordered[kSumWarps][kFewTokens];
  begin_after_previous();
  constexpr int E = kPer<DT>, kBlocks = kFewTokens / 32;
  const int n = (int)s.n, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kFewTokens; i += 32 * kSumWarps)
    keys[i] = i < n ? key_of(ids[i], s.vocab, padding) : s.vocab;
  __syncthreads();
  const unsigned unit = blockIdx.x * kSumWarps + warp, g = unit / s.slices;
  const int64_t v0 = (int64_t)g * s.group;
  if (v0 >= (int64_t)s.vocab) return;
  const Columns<DT, VEC> columns(unit - g * s.slices, s.dim);
  const uint32_t words = (uint32_t)min((int64_t)s.group, (int64_t)s.vocab - v0);
  int count = 0;
  unsigned present = 0;
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const uint32_t word = keys[32 * j + lane] - (uint32_t)v0;
    const bool mine = word < words;
    const unsigned here = __ballot_sync(0xFFFFFFFFu, mine);
    if (mine) {
      const int at = count + __popc(here & ((1u << lane) - 1));
      found[warp][at] = (uint16_t)(word << 8 | (32 * j + lane));
      present |= 1u << word;
    }
    count += __popc(here);
  }
  present = __reduce_or_sync(0xFFFFFFFFu, present);
  const float zero[E] = {};
  for (uint32_t w = 0; w < words; ++w)
    if (!(present >> w & 1u)) columns.store(s.dw, v0 + w, zero);
  if (count == 0) return;
  __syncwarp();
  for (int i = lane; i < count; i += 32) {       // (all different)
    const uint16_t mine = found[warp][i];
    int at = 0;
    for (int j = 0; j < count; ++j) at += found[warp][j] < mine;
    ordered[warp][at] = mine;
  }
  __syncwarp();
  float sum[E] = {};
  for (int i = 0; i < count; i += 32) {
    const uint32_t mine = i + lane < count ? ordered[warp][i + lane] : 0;
    const uint32_t next = i + lane + 1 < count ? ordered[warp][i + lane + 1] >> 8 : 0xFFFFu;
    const unsigned ends = __ballot_sync(0xFFFFFFFFu, i + lane < count && next != mine >> 8);
    add_rows<DT, VEC>(columns, s.dy, mine >> 8, mine & 0xFFu, ends, min(count - i, 32), sum,
                      [&](uint32_t word) {
                        float e[E];
#pragma unroll
                        for (int j = 0; j < E; ++j) e[j] = sum[j] * s.scale;
                        columns.store(s.dw, v0 + word, e);
                      });
  }
}
static_assert(kFewTokens == 256, "a token's number has eight bits");

// The words that go on from one chunk to the next: a word's last part in the
// chunk where it starts, then the first parts of the chunks that it reaches, in
// order.  A CTA for every chunk, with the word that goes on behind it.  Up to
// kFewParts parts: the CTA where the word starts adds them, a thread to four
// columns.  More: all CTAs that the word goes on behind take 32 columns each in
// turn, ranges of parts side by side.  CTAs of 128 threads, of 64 for narrow tables:
// most end at once, and more are resident (131072 tokens over 50257 x 512: 60.4 us,
// with 256 threads 65.5).
constexpr int kFewParts = 16, kJoinColumns = 32, kJoinLanes = kJoinColumns / 4;
constexpr int kNarrow = 256;      // columns

// The last number in [lo, hi) for which f holds, which holds for lo and, if for
// any number, for all smaller ones.  A whole warp; 32 probes a round, neighbours
// first.
template <class F>
__device__ __forceinline__ int64_t last_of(int64_t lo, int64_t hi, F f) {
  int64_t step = 1;
  while (hi - lo > 1) {
    const int64_t at = lo + (threadIdx.x % 32 + 1) * step;
    const int holds = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && f(at)));
    if (holds < 32) hi = min(hi, lo + (holds + 1) * step);
    lo += holds * step;
    step = (hi - lo + 32) / 33;
  }
  return lo;
}

template <int DT, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads)
embedding_join_kernel(const Sums s, bool vec) {
  constexpr int kJoinRanges = kJoinThreads / kJoinLanes;
  __shared__ float4 sh[kJoinRanges][kJoinLanes];
  begin_after_previous();
  const int64_t chunk = blockIdx.x, last = (chunk + 1) * s.chunk - 1;
  if (last + 1 >= s.n) return;
  const int64_t chunks = (s.n + s.chunk - 1) / s.chunk;
  // lanes 0 to 15: the last keys of the chunks before this one; 16 to 31: the
  // first ones of those behind the next
  static_assert(kFewParts == 16, "half a warp");
  const int probe = threadIdx.x & 31;
  const int64_t at = probe < 16 ? chunk - 1 - probe : chunk + 2 + probe - 16;
  uint32_t there = s.vocab;
  if (at >= 0 && at < chunks) there = s.keys[probe < 16 ? (at + 1) * s.chunk - 1 : at * s.chunk];
  const uint32_t key = s.keys[last], next = s.keys[last + 1];
  if (key == s.vocab || next != key) return;
  const unsigned others = __ballot_sync(0xFFFFFFFFu, there != key);
  // the first and the last chunk of the word
  int64_t from = chunk - (__ffs(others & 0xFFFFu | 0x10000u) - 1);
  int64_t to = chunk + 1 + __ffs(others >> 16 | 0x10000u) - 1;
  if (from == chunk - 16)
    from = -last_of(-from, 1, [&](int64_t c) { return s.keys[(1 - c) * s.chunk - 1] == key; });
  if (to == chunk + 17)
    to = last_of(to, chunks, [&](int64_t c) { return s.keys[c * s.chunk] == key; });
  const int64_t count = to - from + 1;
  const auto part = [&](int64_t i, int64_t c) {
    const float* p = s.parts + ((from + i) * 2 + (i == 0 ? 1 : 0)) * s.dim + c;
    if (vec) return *reinterpret_cast<const float4*>(p);
    return make_float4(p[0], c + 1 < s.dim ? p[1] : 0.0f, c + 2 < s.dim ? p[2] : 0.0f,
                       c + 3 < s.dim ? p[3] : 0.0f);
  };
  // parts [a, b) of four columns
  const auto sum_of = [&](int64_t a, int64_t b, int64_t c) {
    float4 sum = make_float4(0, 0, 0, 0);
    for (int64_t i = a; i < b; i += 8) {
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = i + k < b ? part(i + k, c) : make_float4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        sum = make_float4(sum.x + v[k].x, sum.y + v[k].y, sum.z + v[k].z, sum.w + v[k].w);
    }
    return sum;
  };
  const auto put = [&](const float4& sum, int64_t c) {
    const float e[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < s.dim) store1<DT>(s.dw, (int64_t)key * s.dim + c + j, e[j] * s.scale);
  };
  if (count <= kFewParts) {
    if (chunk != from) return;
    for (int64_t c = 4 * threadIdx.x; c < s.dim; c += 4 * kJoinThreads)
      put(sum_of(0, count, c), c);
    return;
  }
  const int lane = threadIdx.x % kJoinLanes, range = threadIdx.x / kJoinLanes;
  const int64_t a = count * range / kJoinRanges, b = count * (range + 1) / kJoinRanges;
  for (int64_t c0 = (chunk - from) * kJoinColumns; c0 < s.dim; c0 += (count - 1) * kJoinColumns) {
    const int64_t c = c0 + 4 * lane;
    sh[range][lane] = c < s.dim ? sum_of(a, b, c) : make_float4(0, 0, 0, 0);
    __syncthreads();
    if (range == 0 && c < s.dim) {
      float4 sum = sh[0][lane];
#pragma unroll 8
      for (int r = 1; r < kJoinRanges; ++r) {
        const float4 v = sh[r][lane];
        sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
      }
      put(sum, c);
    }
    __syncthreads();
  }
}

int64_t element_size(int dtype) { return dtype == kF32 ? 4 : 2; }

bool vectors_ok(const void* a, const void* b, int64_t dim, int dtype) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
           (uintptr_t)(dim * element_size(dtype))) & 15u) == 0;
}

int64_t blocks(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Words of a warp that fills, so that every SM has some 32 of them.
int group_of(int64_t words, int sms) {
  int group = 32;
  while (group > 1 && blocks(words, group) < 32 * sms) group /= 2;
  return group;
}

struct Scratch {
  size_t keys[2] = {0, 0}, tokens[2] = {0, 0}, counts = 0, parts = 0, bytes = 0;
  int64_t tile = 0;
  int tiles = 0, passes = 0;
};

// The largest chunk with which every SM still has kSumUnits warps.
constexpr int64_t kSumUnits = 16;
static_assert(kFewTokens > kMostChunk, "the chunked path always has several chunks");
int chunk_of(const EmbeddingArgs& a, int sms) {
  const int64_t slices = blocks(a.dim, 32 * (a.dtype == kF32 ? kPer<kF32> : kPer<kF16>));
  int chunk = kMostChunk;
  while (chunk > kLeastChunk && blocks(a.rows, chunk) * slices < kSumUnits * sms) chunk /= 2;
  return chunk;
}

Scratch backward_scratch(const EmbeddingArgs& a, int sms) {
  Scratch s;
  const auto take = [&](int64_t bytes) {
    const size_t at = s.bytes;
    s.bytes += (size_t)((bytes + 255) / 256 * 256);
    return at;
  };
  if (a.rows <= kFewTokens) return s;
  for (int i = 0; i < (a.rows <= kRankTokens ? 1 : 2); ++i) {
    s.keys[i] = take(a.rows * 4);
    s.tokens[i] = take(a.rows * 4);
  }
  if (a.rows > kRankTokens) {
    s.tile = blocks(blocks(a.rows, 2 * sms), kSortStep) * kSortStep;
    s.tiles = (int)blocks(a.rows, s.tile);
    for (int64_t v = a.vocab; v > 0; v >>= 8) ++s.passes;    // (keys go up to vocab)
    s.counts = take((int64_t)s.passes * s.tiles * kDigits * 4);
  }
  s.parts = take(blocks(a.rows, chunk_of(a, sms)) * 2 * a.dim * 4);
  return s;
}

template <int DT>
cudaError_t forward(const EmbeddingArgs& a, cudaStream_t stream) {
  const long long* ids = reinterpret_cast<const long long*>(a.ids);
  const bool early = worth_early(a.rows * a.dim);
  if (vectors_ok(a.in, a.out, a.dim, DT)) {
    const int64_t vectors = a.dim / kPer<DT>;
    return launch(early, embedding_kernel<DT>,
                  (unsigned)blocks(a.rows * vectors, kForwardVectors * kCtaThreads), kCtaThreads, 0,
                  stream, ids, static_cast<const uint4*>(a.in), a.rows, vectors, a.vocab, a.scale,
                  static_cast<uint4*>(a.out));
  }
  return launch(early, embedding_any_kernel<DT>,
                (unsigned)blocks(a.rows * blocks(a.dim, kRowPart), kCtaWarps), kCtaThreads, 0,
                stream, ids, a.in, a.rows, a.dim, a.vocab, (unsigned)blocks(a.dim, kRowPart),
                a.scale, a.out);
}

template <int DT>
cudaError_t backward(const EmbeddingArgs& a, char* scratch, int sms, cudaStream_t stream,
                     LaunchMark mark) {
  const Scratch l = backward_scratch(a, sms);
  const auto at = [&](size_t offset) { return reinterpret_cast<uint32_t*>(scratch + offset); };
  const int64_t size = element_size(DT);
  Fill fill = {static_cast<char*>(a.out), a.vocab * a.dim * size, (int)size, 0, 1};
  const long long* ids = reinterpret_cast<const long long*>(a.ids);
  const bool vec = vectors_ok(a.in, a.out, a.dim, DT);
  cudaError_t e = cudaSuccess;
  Sums s = {};
  s.n = a.rows;
  s.dim = a.dim;
  s.vocab = (uint32_t)a.vocab;
  s.slices = (unsigned)blocks(a.dim, 32 * kPer<DT>);
  s.dy = a.in;
  s.scale = a.scale;
  s.dw = a.out;
  if (a.rows <= kFewTokens) {
    s.group = group_of(a.vocab * (int64_t)s.slices, sms);
    if (mark) mark(kEmbeddingSumsK, 0, stream);
    e = launch(worth_early(a.vocab * a.dim),
               vec ? embedding_few_kernel<DT, true> : embedding_few_kernel<DT, false>,
               (unsigned)blocks(blocks(a.vocab, s.group) * s.slices, kSumWarps), 32 * kSumWarps,
               0, stream, s, ids, (long long)a.padding);
    if (mark) mark(kEmbeddingSumsK, 1, stream);
    return e;
  }
  int last = 0;
  if (mark) mark(kEmbeddingOrderK, 0, stream);
  if (a.rows <= kRankTokens) {
    const int n = (int)a.rows;
    e = cudaFuncSetAttribute(embedding_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRankSmem);
    if (e == cudaSuccess)
      e = launch(true, embedding_rank_kernel, (unsigned)blocks(n, 32), kCtaThreads, kRankSmem,
                 stream, ids, n, (uint32_t)a.vocab, (long long)a.padding, at(l.keys[0]),
                 at(l.tokens[0]));
    s.group = group_of(a.vocab, sms);
  } else {
    SortPass p = {};
    p.n = a.rows;
    p.tile = l.tile;
    p.tiles = l.tiles;
    p.vocab = (uint32_t)a.vocab;
    p.padding = a.padding;
    p.ids = ids;
    p.counts = at(l.counts);
    // two CTAs an SM, those that sort first
    const int ctas = std::max(2 * sms, l.tiles + sms);
    const int64_t pass = (int64_t)l.tiles * kDigits;
    fill.parts = l.passes + 1;
    e = launch(true, embedding_count_kernel, ctas, kSortThreads, 0, stream, p, p.counts + pass,
               l.passes - 1, fill);
    for (int i = 0; e == cudaSuccess && i < l.passes; ++i) {
      p.keys = at(l.keys[last]);
      p.tokens = at(l.tokens[last]);
      if (i > 0) {
        p.ids = nullptr;
        p.counts += pass;
        p.shift += 8;
        last ^= 1;
      }
      p.next = i + 1 < l.passes ? p.counts + pass : nullptr;
      p.keys_out = at(l.keys[last]);
      p.tokens_out = at(l.tokens[last]);
      fill.part = i + 1;
      e = launch(true, embedding_place_kernel, ctas, kSortThreads, 0, stream, p, fill);
    }
  }
  if (mark) mark(kEmbeddingOrderK, 1, stream);
  if (e != cudaSuccess) return e;
  s.keys = at(l.keys[last]);
  s.tokens = at(l.tokens[last]);
  s.chunk = chunk_of(a, sms);
  s.parts = reinterpret_cast<float*>(scratch + l.parts);
  const int64_t chunks = blocks(a.rows, s.chunk);
  s.sums = (unsigned)(chunks * s.slices);
  const int64_t fillers = s.group > 0 ? blocks(a.vocab, s.group) : 0;
  const int warps = s.chunk == kMostChunk ? kMostSumWarps : kSumWarps;
  if (mark) mark(kEmbeddingSumsK, 0, stream);
  e = launch(true, vec ? embedding_sums_kernel<DT, true> : embedding_sums_kernel<DT, false>,
             (unsigned)blocks((int64_t)s.sums + fillers, warps), 32 * warps, 0, stream, s);
  if (mark) mark(kEmbeddingSumsK, 1, stream);
  if (e != cudaSuccess) return e;
  if (mark) mark(kEmbeddingJoinK, 0, stream);
  const bool narrow = a.dim <= kNarrow;
  e = launch(true, narrow ? embedding_join_kernel<DT, 64> : embedding_join_kernel<DT, 128>,
             (unsigned)chunks, narrow ? 64 : 128, 0, stream, s, a.dim % 4 == 0);
  if (mark) mark(kEmbeddingJoinK, 1, stream);
  return e;
}

}  // namespace

size_t embedding_backward_scratch(const EmbeddingArgs& a, int sms) {
  return backward_scratch(a, sms).bytes;
}

cudaError_t launch_embedding(const EmbeddingArgs& a, cudaStream_t stream, LaunchMark mark) {
  if (mark) mark(kEmbeddingK, 0, stream);
  const cudaError_t e = a.dtype == kF32    ? forward<kF32>(a, stream)
                        : a.dtype == kBF16 ? forward<kBF16>(a, stream)
                                           : forward<kF16>(a, stream);
  if (mark) mark(kEmbeddingK, 1, stream);
  return e;
}

cudaError_t launch_embedding_backward(const EmbeddingArgs& a, char* scratch, int sms,
                                      cudaStream_t stream, LaunchMark mark) {
  if (a.rows == 0)
    return cudaMemsetAsync(a.out, 0, (size_t)(a.vocab * a.dim * element_size(a.dtype)), stream);
  if (a.dtype == kF32) return backward<kF32>(a, scratch, sms, stream, mark);
  return a.dtype == kBF16 ? backward<kBF16>(a, scratch, sms, stream, mark)
                          : backward<kF16>(a, scratch, sms, stream, mark);
}

}  // namespace fp8opt
