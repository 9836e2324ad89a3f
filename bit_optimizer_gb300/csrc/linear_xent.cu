// Softmax cross entropy of a linear layer over a large vocabulary: logits
// z = x w^T (tokens x vocabulary), loss = lse(z) - z[target], without the
// logits ever being in memory as a whole.
//
// forward   One product on the tensor cores.  A tile's epilogue reduces its
//           logits, still in TMEM, to each token's maximum and sum of
//           exponentials (base 2, fp32, the difference taken before it is
//           scaled) and takes the target's logit where it meets it; a small
//           kernel joins the parts of a token in order.
// backward  The vocabulary goes in pieces.  For each piece the logits are
//           computed again and turned into p = (exp(z - lse) - [target]) *
//           dloss in the operands' 16-bit type, tokens x piece, in scratch;
//           then dx += p w_piece (fp32 in scratch) and dw_piece = p^T x.  p is
//           scaled by a power of two and max |dloss| against underflow in
//           FP16: the one rounding to 16 bits besides the results', random per
//           element and of the size of the operands' own (a token whose dloss
//           is far below the largest has a scale of its own: see dloss_shift()).
//           A launch holds one
//           piece's dx and dw and the next piece's p, so that its end, where
//           pairs run out of tiles, comes once a piece and is filled with the
//           short tiles of p.
//
// Every product is the same persistent kernel on pairs of CTAs (cta_group::2),
// one tile of 256 x 256 at a time: a producer warp in each CTA copies its half
// of A and B by TMA into six stages of 64-deep blocks, the leader's MMA warp
// issues tcgen05.mma into one of two TMEM accumulators, eight epilogue warps
// in each CTA empty the other, and a scheduler warp looks tiles up ahead of
// everybody.  x and w are K-major in the logits product; w in dx, and both
// operands of dw, are read MN-major, so nothing is transposed in memory.
//
// Bound by the tensor cores: 8192 x 2048 x 50257 forward 0.92 ms, 1.83 PFLOP/s in
// calls in a row (cuBLAS' measured burst: 1.91); in loops of seconds the power
// limit lowers the clock for both (8192 x 1024: 1.73 PFLOP/s; cuBLAS 1.70).  The
// gradients of 8191 x 2048: 3.2 ms, 1.58 PFLOP/s, the tensor pipe active 87% of the
// cycles.  Few tokens are bound by reading w: 24 x 768 x 200000, 55 us, 5.6
// TB/s.  What a step brought: single CTAs with tiles of 128 x 256 and four
// stages, a launch for each product: 353 us forward and 1540 us backward at 8192
// x 2048 x 20224; pairs, which need two thirds of the L2 traffic, six stages and
// joint launches: 343 and 1400, once the tile look-up had a warp of its own (in
// the producer warp it left the pipe idle 4000 clocks a tile: 444 and 1900); p,
// dx and dw stored in whole lines: 254 us instead of 612 backward at width 128.
//
// Tokens whose target is `ignore` have no loss and give no gradient whatever
// is in their row of x: their p is 0 and dw reads a copy of x in which such
// rows are zero.  Rows that TMA cannot read (a row length that is not a
// multiple of 8, unaligned tensors) are copied to a 16-byte pitch.
#include "ops_internal.cuh"
#include "tensor_core.cuh"

namespace fp8opt {

namespace {

// A pair of CTAs takes a tile of 256 x tile_n: 128 rows of A and half of B each.
constexpr int kTileM = 256, kTileN = 256, kBlockK = 64, kGemmStages = 6;
constexpr int kHalfM = kTileM / 2, kStageA = kHalfM * kBlockK * 2;
constexpr int kStageB = kTileN / 2 * kBlockK * 2;
// Eight epilogue warps (two for each quarter of the lanes, each with half of the
// columns), a producer, an MMA and a scheduler warp.
constexpr int kEpilogueWarps = 8, kGemmThreads = 32 * (kEpilogueWarps + 3);
constexpr int kTurnBytes = 4096;   // of an epilogue warp
constexpr int kGemmSmem =
    1024 + kGemmStages * (kStageA + kStageB) + kEpilogueWarps * kTurnBytes;

constexpr float kLog2eF = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

enum GemmMode { kStats = 0, kStatsSwapped, kProbs, kDx, kDw };

// One product C[m, n] = sum_k A[m, k] B[n, k] in tiles of 256 x tile_n, k in
// `splits` ranges of `kper` blocks, and what its tiles are for.
struct GemmShape {
  int mode;
  int tiles_m, tiles_n, tile_n, kblocks, kper, splits;
  int b_mn0, b_k0;         // B's coordinates of n = 0 and k = 0 (A's are 0)
  int a_mn, b_mn;          // MN-major operands
  int first;               // kDx: the first piece
  int64_t v0;              // first vocabulary row of the piece
  uint16_t* probs;         // kProbs: [token][piece]
  // A's rows where they all lie in the leader's half of one row of tiles (a
  // multiple of 8, K-major): only these are copied, the leader alone, and the
  // rest of its stage, like the other CTA's, keeps what was there, which makes
  // rows of C that nobody reads.  (Copies that end past a tensor are slow to
  // fill up with zeros.)  0: any other A.
  int a_rows;
  __host__ __device__ int tiles() const { return tiles_m * tiles_n * splits; }
};
struct GemmJob {
  CUtensorMap a, b;
  GemmShape shape;
};

// What the tiles' epilogues read and write.
struct GemmOut {
  int64_t tokens;          // rows of x in this call
  int64_t vocab, dim;
  const long long* target;
  long long ignore;
  // kStats
  float2* partial;         // [part of the vocabulary][token]: maximum, sum of exponentials
  float* target_logit;     // [token]
  // kProbs
  const float* lse;
  const float* dloss;
  const float* top;        // largest finite |dloss|
  int64_t piece;           // columns of probs
  // kDx, kDw
  float* dx_sum;           // [split][token][dim_pitch]
  int64_t dim_pitch;
  void* dw;
};

// One launch: up to three products that do not depend on one another, those
// with the longest tiles first.  (Two of them tile by tile in turn, which would
// put p's long epilogues between longer products, was slower, 1.92 against 1.51
// ms at 8192 x 1024: pairs that work on one product at a time read the same
// operands at about the same time.)
constexpr int kMaxJobs = 3;
struct GemmArgs {
  GemmJob job[kMaxJobs];
  int jobs;
  GemmOut out;
  // Tiles handed out beyond the first two of each pair, to whichever pair gets
  // free; NULL: a pair takes every so many-th tile (they are equally long).
  int* next;
  int* error;              // set to 1 when a wait ran out
};

// p is held as (exp(z - lse) - [target]) * (2^b dloss / max |dloss|) *
// kProbScale: below 2^15, and in FP16 without underflow down to 2^-39.  (A common
// dloss then leaves p as it is: multiplied in before the rounding, it would give
// every token the same rounding error.)
constexpr float kProbScale = 32768.0f;

// b of a token: 0 for a dloss within 2^12 of the largest.  A smaller one would
// push the token's small probabilities below FP16's range, and its dx with them
// (1 / 50257 of 2^-20 keeps three bits).  So 2^-b is left out of p and put where
// it is exact: on the token's row of dx, in fp32, and on its row of dw's copy of
// x (in FP16 exact until x 2^-b is below 2^-14; beyond that its part of dw is
// off by at most 2^-37 of a like token's of the largest dloss).
constexpr int kFullRange = 12;
__device__ __forceinline__ int dloss_shift(float dloss, float top) {
  if (dloss == 0.0f || top == 0.0f || nonfinite(dloss)) return 0;
  return max(ilogbf(top) - ilogbf(dloss) - kFullRange, 0);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return pack2<BF16 ? kBF16 : kF16>(a, b);
}

// An epilogue warp's 4 KB of shared memory: 32 rows of 128 bytes, in which its
// lanes, a row each, turn over to eight lanes a row, so that global memory is
// read and written in whole lines (straight from the lanes, 16 bytes of 32
// rows at a time, the stores of p took twice the time of the product).  The
// 16-byte words of a row are permuted so that both ways are free of conflicts.
struct Turn {
  uint4 w[32][8];
  __device__ __forceinline__ uint4& at(int row, int word) { return w[row][word ^ (row & 7)]; }
};
static_assert(sizeof(Turn) == kTurnBytes, "");

// 64 results of each lane's row as 16-bit values, at out + row * pitch; rows
// below `rows`, columns below `cols`.
template <bool BF16>
__device__ __forceinline__ void store_rows16(Turn& turn, uint16_t* out, int64_t pitch, int rows,
                                             int cols, const float (&v)[64]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    turn.at(lane, j) =
        make_uint4(pack16<BF16>(v[8 * j], v[8 * j + 1]), pack16<BF16>(v[8 * j + 2], v[8 * j + 3]),
                   pack16<BF16>(v[8 * j + 4], v[8 * j + 5]),
                   pack16<BF16>(v[8 * j + 6], v[8 * j + 7]));
  __syncwarp();
  const int word = lane & 7, c = 8 * word, row0 = lane >> 3;
  uint16_t* p = out + row0 * pitch + c;
  const int64_t step = 4 * pitch;
  // (with rows of whole 16-byte words, cols is a multiple of 8 as well)
  if ((((uint64_t)reinterpret_cast<uintptr_t>(out) | (uint64_t)pitch * 2) & 15u) == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i, p += step)
      if (c < cols && 4 * i + row0 < rows)
        *reinterpret_cast<uint4*>(p) = turn.at(4 * i + row0, word);
  } else {
    // rows that start anywhere: a row at a time, a pair of columns to a lane, in
    // aligned pairs of the row's memory
    const int n = min(64, cols);
    for (int i = 0; i < rows && i < 32; ++i) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(&turn.at(i, lane >> 2))[lane & 3];
      const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w, 1);
      uint16_t* q = out + i * pitch;
      const bool odd = (reinterpret_cast<uintptr_t>(q) & 2u) != 0;
      const uint32_t both = odd ? w >> 16 | next << 16 : w;
      const int first = 2 * lane + (odd ? 1 : 0);
      if (odd && lane == 0 && n > 0) q[0] = (uint16_t)w;
      if (first + 1 < n) *reinterpret_cast<uint32_t*>(q + first) = both;
      else if (first < n) q[first] = (uint16_t)both;
    }
  }
  __syncwarp();
}

// Adds (or, `first`, stores) 32 columns of each lane's row to out + row *
// pitch, fp32 at a 16-byte pitch; rows below `rows`.
__device__ __forceinline__ void add_rows32(Turn& turn, float* out, int64_t pitch, int rows,
                                           bool first, const uint32_t (&r)[32]) {
  const int lane = threadIdx.x & 31, word = lane & 7, row0 = lane >> 3;
  float* const p = out + row0 * pitch + 4 * word;
  const int64_t step = 4 * pitch;
  float4 s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!first && 4 * i + row0 < rows) s[i] = *reinterpret_cast<const float4*>(p + i * step);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    turn.at(lane, j) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 w = turn.at(4 * i + row0, word);
    if (4 * i + row0 < rows)
      *reinterpret_cast<float4*>(p + i * step) =
          make_float4(s[i].x + __uint_as_float(w.x), s[i].y + __uint_as_float(w.y),
                      s[i].z + __uint_as_float(w.z), s[i].w + __uint_as_float(w.w));
  }
  __syncwarp();
}

// exp(a + shift) and exp(b + shift) of two accumulators.  The difference is
// taken before it is scaled to base 2: its rounding error does not grow with
// the logits.
__device__ __forceinline__ float2 exp_pair(uint32_t a, uint32_t b, float shift) {
  const float2 d = mul2(add2(make_float2(__uint_as_float(a), __uint_as_float(b)), splat2(shift)),
                        splat2(kLog2eF));
  return make_float2(exp2_approx(d.x), exp2_approx(d.y));
}

// An epilogue thread's part of a tile: one row and `cols` columns from `c0` on
// (rows and columns of C; the columns lie in TMEM at `tmem`).
struct Strip {
  uint32_t tmem;
  int64_t row, c0;
  int cols, index;         // index: column strip of the whole product
};

// What an epilogue needs of its row, read while the tile is being computed.
struct RowIn {
  long long target;
  float lse, dloss, top;
};

__device__ __forceinline__ RowIn row_in(const GemmShape& g, const GemmOut& o, int64_t row) {
  RowIn in = {-1, 0.0f, 0.0f, 0.0f};
  if (g.mode == kStats || g.mode == kProbs) {
    if (row < o.tokens) {
      in.target = o.target[row];
      if (g.mode == kProbs) {
        in.lse = o.lse[row];
        in.dloss = o.dloss[row];
      }
    }
  }
  if (g.mode == kProbs || g.mode == kDw) in.top = *o.top;
  return in;
}

// Two parts of a token's logits: maximum, and sum of exponentials above it.
__device__ __forceinline__ float2 join_stats(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x);
  return make_float2(top, a.y * exp2_approx((a.x - top) * kLog2eF) +
                              b.y * exp2_approx((b.x - top) * kLog2eF));
}

// A token's running maximum and sum of exponentials, and its target's logit.  The
// maximum starts at fp32's lowest number, which is above no logit but -inf and
// makes its exponential 0 (from -inf the difference of two would be NaN).
constexpr float kLowest = -3.402823466e38f;
struct Stats {
  float top = kLowest, sum = 0.0f, at_target = 0.0f;
  // 32 more logits, of which the first `valid` count; the target's is number
  // rel, if it is among them.
  __device__ __forceinline__ void add(uint32_t (&r)[32], int valid, int rel) {
    if (valid < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j >= valid) r[j] = 0xFF800000u;
    }
    if (__any_sync(0xFFFFFFFFu, rel >= 0 && rel < 32)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (rel == j) at_target = __uint_as_float(r[j]);
    }
    float m[4] = {top, top, top, top};
#pragma unroll
    for (int j = 0; j < 32; ++j) m[j & 3] = fmaxf(m[j & 3], __uint_as_float(r[j]));
    m[0] = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    float2 s[2] = {make_float2(sum * exp2_approx((top - m[0]) * kLog2eF), 0.0f),
                   make_float2(0.0f, 0.0f)};
    top = m[0];
#pragma unroll
    for (int j = 0; j < 32; j += 2)
      s[j / 2 & 1] = add2(s[j / 2 & 1], exp_pair(r[j], r[j + 1], -top));
    s[0] = add2(s[0], s[1]);
    sum = s[0].x + s[0].y;
  }
};

// The strip's logits: maximum and sum of exponentials.
__device__ __forceinline__ void stats_strip(const GemmOut& o, const Strip& t, const RowIn& in) {
  const long long target = in.target;
  const int rel = target >= t.c0 && target < t.c0 + t.cols && target < o.vocab
                      ? (int)(target - t.c0) : -1;
  const int valid = (int)min((int64_t)t.cols, o.vocab - t.c0);   // may be <= 0
  Stats s;
  tmem_columns(t.tmem, t.cols, [&](int c, uint32_t (&r)[32], uint32_t (&q)[32]) {
    s.add(r, valid - c, rel - c);
    s.add(q, valid - c - 32, rel - c - 32);
  });
  if (t.row < o.tokens) {
    o.partial[(int64_t)t.index * o.tokens + t.row] = make_float2(s.top, s.sum);
    if (rel >= 0) o.target_logit[t.row] = s.at_target;
  }
}

// The same with the operands swapped: the tile's rows are the vocabulary's, its
// columns the tokens (tile_n covers them, at most kSwapTokens).  Through the
// warp's shared memory the logits of 32 rows and 32 columns are turned over, a
// token to each lane; a warp's statistics of its two ranges of tokens run on
// from tile to tile, and a CTA writes its own once, at the end.
struct SwappedStats {
  Stats s[2];
  __device__ __forceinline__ void add(const GemmShape& g, const GemmOut& o, uint32_t tmem,
                                      int64_t v0, int half, Turn& turn) {
    const int lane = threadIdx.x & 31;
    const int valid = (int)min((int64_t)32, max(o.vocab - v0, (int64_t)0));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = 32 * half + 64 * k;
      if (c >= g.tile_n) break;
      uint32_t r[32];
      tmem_load32(tmem + c, r);
      tmem_wait(r);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        turn.at(lane, j) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        r[j] = reinterpret_cast<const uint32_t*>(&turn.at(j, lane >> 2))[lane & 3];
      __syncwarp();
      const int64_t token = c + lane;
      const long long target = token < o.tokens ? o.target[token] : -1;
      const int rel = target >= v0 && target < v0 + 32 && target < o.vocab ? (int)(target - v0)
                                                                            : -1;
      s[k].add(r, valid, rel);
      if (rel >= 0) o.target_logit[token] = s[k].at_target;
    }
  }
  // Every epilogue warp; turns: all warps' shared memory.
  __device__ __forceinline__ void finish(const GemmOut& o, int warp, Turn* turns) {
    const int lane = threadIdx.x & 31;
    float2* const mine = reinterpret_cast<float2*>(&turns[warp]);
    for (int k = 0; k < 2; ++k) mine[32 * k + lane] = make_float2(s[k].top, s[k].sum);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (warp % 4 != 0) return;
    for (int k = 0; k < 2; ++k) {
      const int64_t token = 32 * (warp / 4) + 64 * k + lane;
      if (token >= o.tokens) continue;
      float2 a = make_float2(kLowest, 0.0f);
      for (int w = 0; w < 4; ++w)
        a = join_stats(a, reinterpret_cast<const float2*>(&turns[warp + w])[32 * k + lane]);
      o.partial[(int64_t)blockIdx.x * o.tokens + token] = a;
    }
  }
};

// The strip's logits turned into p.
template <bool BF16>
__device__ __forceinline__ void probs_strip(const GemmShape& g, const GemmOut& o,
                                            const Strip& t, const RowIn& in, Turn& turn) {
  const bool live = t.row < o.tokens;
  float shift = 0.0f, k = 0.0f;
  int rel = -1;
  if (live && in.target != o.ignore) {
    const float own = ldexpf(in.dloss, dloss_shift(in.dloss, in.top));
    k = (in.top == 0.0f ? own : __fdiv_rn(own, in.top)) * kProbScale;
    shift = -in.lse;
    const long long at = in.target - g.v0 - t.c0;
    if (at >= 0 && at < t.cols) rel = (int)at;
    if (in.target < 0 || in.target >= o.vocab) k = __uint_as_float(0x7FC00000u);
  }
  const bool zero = k == 0.0f;      // an ignored token, whatever its logits are
  const int valid = (int)min((int64_t)t.cols, o.vocab - g.v0 - t.c0);
  const int64_t row0 = t.row - (threadIdx.x & 31);
  uint16_t* const out = g.probs + row0 * o.piece + t.c0;
  const int rows = (int)min((int64_t)32, o.tokens - row0);
  tmem_columns(t.tmem, t.cols, [&](int c, uint32_t (&r)[32], uint32_t (&q)[32]) {
    float v[64];
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 e = exp_pair(r[j], r[j + 1], shift), f = exp_pair(q[j], q[j + 1], shift);
      v[j] = e.x;
      v[j + 1] = e.y;
      v[32 + j] = f.x;
      v[33 + j] = f.y;
    }
    if (__any_sync(0xFFFFFFFFu, rel >= c && rel < c + 64)) {
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (rel == c + j) v[j] -= 1.0f;
    }
#pragma unroll
    for (int j = 0; j < 64; ++j) v[j] = zero ? 0.0f : v[j] * k;
    if (c + 64 > valid) {           // columns past the vocabulary's end are 0
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (c + j >= valid) v[j] = 0.0f;
    }
    store_rows16<BF16>(turn, out + c, o.piece, rows, 64, v);
  });
}

// This piece's part of dx, added to the earlier ones'.  `none`: the split has
// no k in this piece, and nothing was accumulated.
__device__ __forceinline__ void dx_strip(const GemmShape& g, const GemmOut& o, const Strip& t,
                                         int split, bool none, Turn& turn) {
  const int64_t row0 = t.row - (threadIdx.x & 31);
  float* const sum = o.dx_sum + (split * o.tokens + row0) * o.dim_pitch + t.c0;
  const int rows = (int)min((int64_t)32, o.tokens - row0);
  tmem_columns(t.tmem, t.cols, [&](int c, uint32_t (&r)[32], uint32_t (&q)[32]) {
    if (none) {
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = q[j] = 0;
    }
    add_rows32(turn, sum + c, o.dim_pitch, rows, g.first, r);
    add_rows32(turn, sum + c + 32, o.dim_pitch, rows, g.first, q);
  });
}

template <bool BF16>
__device__ __forceinline__ void dw_strip(const GemmShape& g, const GemmOut& o, const Strip& t,
                                         const RowIn& in, Turn& turn) {
  const int64_t v0 = g.v0 + t.row - (threadIdx.x & 31);
  const int cols = (int)min((int64_t)t.cols, o.dim - t.c0);
  const int rows = (int)min((int64_t)32, o.vocab - v0);
  uint16_t* const out = static_cast<uint16_t*>(o.dw) + v0 * o.dim + t.c0;
  tmem_columns(t.tmem, t.cols, [&](int c, uint32_t (&r)[32], uint32_t (&q)[32]) {
    float v[64];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = __uint_as_float(r[j]) * (1.0f / kProbScale) * in.top;
      v[32 + j] = __uint_as_float(q[j]) * (1.0f / kProbScale) * in.top;
    }
    store_rows16<BF16>(turn, out + c, o.dim, rows, cols - c, v);
  });
}

// A tile as the warps of one CTA need it.  `work` is what its MMA warp reads:
// blocks of k, tile_n / 16 and the operands' order (see its accessors).
struct Tile {
  uint32_t work;
  int job, m, n, split;
  int a_mn, b_mn;          // this CTA's coordinates in A and B ...
  int a_k, b_k;            // ... and those of the first block of k
  int a_rows;              // GemmShape's
  int pad[2];
};
constexpr uint32_t kNoWork = 0xFFFFFFFFu;
__device__ __forceinline__ int work_blocks(uint32_t w) { return (int)(w & 0xFFFFFFu); }
__device__ __forceinline__ int work_tile_n(uint32_t w) { return (int)(w >> 24 & 31u) * 16; }
__device__ __forceinline__ bool work_a_mn(uint32_t w) { return w >> 29 & 1u; }
__device__ __forceinline__ bool work_b_mn(uint32_t w) { return w >> 30 & 1u; }
static_assert(sizeof(Tile) == 48, "three 16-byte words");
static_assert(kXentMostSummed <= kBlockK * 0xFFFFFFll, "a tile's blocks fit work_blocks");

__device__ __forceinline__ Tile locate(const GemmArgs& args, int tile, int rank) {
  Tile t = {};
  GemmShape g = args.job[0].shape;
#pragma unroll
  for (int j = 1; j < kMaxJobs; ++j) {
    if (t.job == j - 1 && j < args.jobs && tile >= g.tiles()) {
      tile -= g.tiles();
      g = args.job[j].shape;
      t.job = j;
    }
  }
  t.m = tile % g.tiles_m;
  t.n = tile / g.tiles_m % g.tiles_n;
  t.split = tile / g.tiles_m / g.tiles_n;
  const int kb0 = t.split * g.kper, blocks = max(min(g.kper, g.kblocks - kb0), 0);
  t.work = (uint32_t)blocks | (uint32_t)(g.tile_n / 16) << 24 | (uint32_t)g.a_mn << 29 |
           (uint32_t)g.b_mn << 30;
  t.a_mn = t.m * kTileM + rank * kHalfM;
  t.a_rows = g.a_rows;
  t.b_mn = g.b_mn0 + t.n * g.tile_n + rank * (g.tile_n / 2);
  t.a_k = kb0 * kBlockK;
  t.b_k = g.b_k0 + kb0 * kBlockK;
  return t;
}

// Tiles are handed out as pairs get free.  One warp of each CTA does nothing
// else: the leader's takes the next tile from a counter and passes it to the
// other CTA's, and each writes it, looked up, to a ring of four that its CTA's
// other warps follow.  The counter's, the pair's and the look-up's latencies
// are thereby hidden behind the tiles in the ring (in the producer warp they
// cost 4000 clocks a tile, which the stages' depth could not cover).
constexpr int kRing = 4;
struct GemmBarriers {
  uint64_t full[kGemmStages], empty[kGemmStages], acc_full[2], acc_empty[2], drained;
  uint64_t tile_full[kRing], tile_empty[kRing];
  uint64_t pair_full, pair_empty;   // the other CTA's, the leader's
  int pair_tile;
  uint32_t tmem;
  Tile tile[kRing];
};

// A position in the ring; next() waits for the following tile and returns it,
// null when the wait ran out; done() gives its slot back.  A whole warp calls
// them, or one thread (WARP false).
template <bool WARP>
struct TileReader {
  int slot = 0, phase = 0;
  __device__ __forceinline__ const Tile* next(GemmBarriers& bar) {
    bool ok = mbar_wait(&bar.tile_full[slot], phase);
    if (WARP) ok = __all_sync(0xFFFFFFFFu, ok);
    return ok ? &bar.tile[slot] : nullptr;
  }
  __device__ __forceinline__ void done(GemmBarriers& bar) {
    if (WARP) __syncwarp();
    if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(&bar.tile_empty[slot]);
    if (++slot == kRing) slot = 0, phase ^= 1;
  }
};

template <bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
gemm_kernel(const __grid_constant__ GemmArgs args) {
  extern __shared__ uint8_t dyn[];
  __shared__ GemmBarriers bar;
  uint8_t* const stages = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kGemmStages; ++i) {
      mbar_init(&bar.full[i], 1);     // the leader's: its own, with both CTAs' bytes
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.acc_full[i], 1);
      mbar_init(&bar.acc_empty[i], 2 * kEpilogueWarps);    // the leader's: of both CTAs
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar.tile_full[i], 1);
      // the epilogue warps, the producer and, in the leader, the MMA warp
      mbar_init(&bar.tile_empty[i], kEpilogueWarps + 1 + (leader ? 1 : 0));
    }
    mbar_init(&bar.pair_full, 1);
    mbar_init(&bar.pair_empty, 1);
    mbar_init(&bar.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(&bar.tmem);
  tcgen_fence_before();
  __syncthreads();
  cluster_sync();
  tcgen_fence_after();
  const uint32_t tmem = bar.tmem;
  bool ok = true;
  // the set-up above runs while the previous launch of the stream ends
  begin_after_previous();

  if (warp == kEpilogueWarps + 2) {
    if ((threadIdx.x & 31) == 0) {
      int total = 0;
      for (int j = 0; j < args.jobs; ++j) total += args.job[j].shape.tiles();
      const int pairs = (int)gridDim.x / 2;
      int slot = 0, phase = 0, pair_phase = 0;
      int tile = (int)blockIdx.x / 2, second = tile + pairs, asked = -1;
      for (;;) {
        if (leader) {
          if (tile >= total) tile = -1;
          if (!(ok = mbar_wait(&bar.pair_empty, pair_phase ^ 1))) break;
          cluster_store(cluster_addr(&bar.pair_tile, 1), tile);
          cluster_arrive(cluster_addr(&bar.pair_full, 1));
        } else {
          if (!(ok = mbar_wait<true>(&bar.pair_full, pair_phase))) break;
          tile = *const_cast<volatile int*>(&bar.pair_tile);
          if (tile >= -1) cluster_arrive_relaxed(cluster_addr(&bar.pair_empty, 0));
        }
        pair_phase ^= 1;
        Tile t = {kNoWork};
        if (tile >= 0) t = locate(args, tile, (int)rank);
        if (!(ok = mbar_wait(&bar.tile_empty[slot], phase ^ 1))) break;
        const uint4* from = reinterpret_cast<const uint4*>(&t);
        uint4* to = reinterpret_cast<uint4*>(&bar.tile[slot]);
        to[0] = from[0];
        to[1] = from[1];
        to[2] = from[2];
        mbar_arrive(&bar.tile_full[slot]);
        if (++slot == kRing) slot = 0, phase ^= 1;
        if (tile < 0) break;
        if (leader) {   // (with a counter, the first two tiles of a pair are fixed)
          if (args.next == nullptr) {
            tile += pairs;
          } else {
            tile = second >= 0 ? second : 2 * pairs + asked;
            second = -1;
            if (tile < total) asked = atomicAdd(args.next, 1);
          }
        }
      }
    }
  } else if (warp == kEpilogueWarps) {
    if ((threadIdx.x & 31) == 0) {
      for (int j = 0; j < args.jobs; ++j) {
        tma_prefetch_map(&args.job[j].a);
        tma_prefetch_map(&args.job[j].b);
      }
      int s = 0, phase = 0;
      uint32_t loads = 0;
      TileReader<false> reader;
      for (;;) {
        const Tile* next = reader.next(bar);
        if (!(ok = next != nullptr)) break;
        const Tile t = *next;
        if (t.work == kNoWork) break;
        reader.done(bar);
        const CUtensorMap* const map_a = &args.job[t.job].a;
        const CUtensorMap* const map_b = &args.job[t.job].b;
        const int blocks = work_blocks(t.work), half_n = work_tile_n(t.work) / 2;
        const bool a_mn = work_a_mn(t.work), b_mn = work_b_mn(t.work);
        const uint32_t bytes_a = t.a_rows > 0 ? t.a_rows * (kBlockK * 2) : 2 * kStageA;
        const uint32_t bytes = bytes_a + 2 * half_n * (kBlockK * 2);
        const bool copies_a = leader || t.a_rows == 0;
        for (int kb = 0; kb < blocks; ++kb) {
          if (!(ok = mbar_wait(&bar.empty[s], phase ^ 1))) break;
          uint8_t* a = stages + s * (kStageA + kStageB);
          uint8_t* b = a + kStageA;
          const uint32_t full = cluster_addr(&bar.full[s], 0);
          if (leader) mbar_expect(&bar.full[s], bytes);
          ++loads;
          const int ka = t.a_k + kb * kBlockK, kk = t.b_k + kb * kBlockK;
          if (a_mn) {
            for (int i = 0; i < kHalfM / 64; ++i)
              tma_load(a + i * (kBlockK * 128), map_a, t.a_mn + 64 * i, ka, full);
          } else if (copies_a) {
            tma_load(a, map_a, ka, t.a_mn, full);
          }
          if (b_mn) {
            for (int i = 0; i < half_n / 64; ++i)
              tma_load(b + i * (kBlockK * 128), map_b, t.b_mn + 64 * i, kk, full);
          } else {
            tma_load(b, map_b, kk, t.b_mn, full);
          }
          if (++s == kGemmStages) s = 0, phase ^= 1;
        }
        if (!ok) break;
      }
      // every copy lands before the pair's shared memory is given up (the
      // leader's barriers count the other CTA's copies too)
      for (int i = 0; leader && i < kGemmStages; ++i)
        if (loads > (uint32_t)i)
          ok = mbar_wait(&bar.full[i], (loads - 1 - i) / kGemmStages & 1) && ok;
      // and so does every arrival from the MMA warp, which commits to both CTAs:
      // the last ones of the stages, and the very last one, which in the leader
      // its own MMA warp waits for
      for (int i = 0; ok && i < kGemmStages; ++i)
        if (loads > (uint32_t)i)
          ok = mbar_wait<true>(&bar.empty[i], (loads - 1 - i) / kGemmStages & 1);
      if (!leader) ok = mbar_wait<true>(&bar.drained, 0) && ok;
    }
  } else if (warp == kEpilogueWarps + 1) {
    if (leader && (threadIdx.x & 31) == 0) {
      int s = 0, phase = 0, buf = 0, acc_phase = 0;
      TileReader<false> reader;
      for (;;) {
        const Tile* next = reader.next(bar);
        if (!(ok = next != nullptr)) break;
        const uint32_t work = next->work;
        if (work == kNoWork) break;
        reader.done(bar);
        const int blocks = work_blocks(work);
        const bool a_mn = work_a_mn(work), b_mn = work_b_mn(work);
        const uint32_t idesc = mma_desc(BF16, a_mn, b_mn, kTileM, work_tile_n(work));
        const uint32_t step_a = a_mn ? 16 * 128 : 32, step_b = b_mn ? 16 * 128 : 32;
        if (!(ok = mbar_wait(&bar.acc_empty[buf], acc_phase ^ 1))) break;
        tcgen_fence_after();
        const uint32_t d = tmem + buf * kTileN;
        for (int kb = 0; kb < blocks; ++kb) {
          if (!(ok = mbar_wait(&bar.full[s], phase))) break;
          tcgen_fence_after();
          const uint32_t a = smem_addr(stages + s * (kStageA + kStageB));
          const uint64_t da = operand_desc(a, a_mn, kBlockK * 128);
          const uint64_t db = operand_desc(a + kStageA, b_mn, kBlockK * 128);
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            mma_f16(d, da + (k * step_a >> 4), db + (k * step_b >> 4), idesc, kb + k > 0);
          mma_commit(&bar.empty[s]);
          if (++s == kGemmStages) s = 0, phase ^= 1;
        }
        if (!ok) break;
        mma_commit(&bar.acc_full[buf]);
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1;
      }
      // and every product ends before TMEM is
      mma_commit(&bar.drained);
      ok = mbar_wait(&bar.drained, 0) && ok;
    }
  } else {
    TileReader<true> reader;
    Turn* const turns = reinterpret_cast<Turn*>(stages + kGemmStages * (kStageA + kStageB));
    Turn& turn = turns[warp];
    SwappedStats swapped;
    int buf = 0, phase = 0;
    // A tile's row inputs are asked for one tile ahead, so that their latency
    // lies under the tile before.
    const auto read = [&](Tile* t, RowIn* in) {
      const Tile* next = reader.next(bar);
      if (next == nullptr) return false;
      *t = *next;
      if (t->work == kNoWork) return true;
      reader.done(bar);
      *in = row_in(args.job[t->job].shape, args.out,
                   (int64_t)t->m * kTileM + rank * kHalfM + (threadIdx.x & 127));
      return true;
    };
    Tile t;
    RowIn in;
    ok = read(&t, &in);
    while (ok && t.work != kNoWork) {
      const GemmShape& g = args.job[t.job].shape;
      const int half = warp / 4, cols = work_tile_n(t.work) / 2;
      const Strip strip = {tmem + buf * kTileN + half * cols + ((uint32_t)(warp % 4) << 21),
                           (int64_t)t.m * kTileM + rank * kHalfM + (threadIdx.x & 127),
                           ((int64_t)t.n * 2 + half) * cols, cols, 2 * t.n + half};
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar.acc_full[buf], phase));
      if (!ok) break;
      tcgen_fence_after();
      Tile after;
      RowIn in_after;
      if (!(ok = read(&after, &in_after))) break;
      if (g.mode == kStats) stats_strip(args.out, strip, in);
      else if (g.mode == kStatsSwapped)
        swapped.add(g, args.out, tmem + buf * kTileN + ((uint32_t)(warp % 4) << 21),
                    strip.row - (threadIdx.x & 31), half, turn);
      else if (g.mode == kProbs) probs_strip<BF16>(g, args.out, strip, in, turn);
      else if (g.mode == kDx) dx_strip(g, args.out, strip, t.split, work_blocks(t.work) == 0, turn);
      else dw_strip<BF16>(g, args.out, strip, in, turn);
      tcgen_fence_before();
      __syncwarp();
      // (the accumulators have been read: nothing else needs an order here)
      if ((threadIdx.x & 31) == 0)
        cluster_arrive_relaxed(cluster_addr(&bar.acc_empty[buf], 0));
      buf ^= 1;
      if (buf == 0) phase ^= 1;
      t = after;
      in = in_after;
    }
    if (args.job[0].shape.mode == kStatsSwapped) swapped.finish(args.out, warp, turns);
  }
  if (!ok) *args.error = 1;
  __syncwarp();
  tcgen_fence_before();
  cluster_sync();
  tcgen_fence_after();
  if (warp == 0) tmem_free(tmem);
}

// Joins the column strips of 32 tokens, a token to each lane (neighbouring
// tokens' statistics lie side by side): warp k takes strips k, k + 32, ... in
// order, then the 32 warps' results are joined in order.
__global__ void __launch_bounds__(1024, 2)
xent_join_kernel(const float2* partial, int strips, int64_t tokens, int64_t vocab,
                 const long long* target, long long ignore, const float* target_logit,
                 float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  const float2 none = make_float2(kLowest, 0.0f);
  begin_after_previous();
  float2 s = none;
  for (int i = warp; i < strips; i += 8 * 32) {
    float2 p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      p[k] = i + 32 * k < strips && row < tokens
                 ? __ldcg(partial + (int64_t)(i + 32 * k) * tokens + row) : none;
#pragma unroll
    for (int k = 0; k < 8; ++k) s = join_stats(s, p[k]);
  }
  sh[warp][lane] = s;
  __syncthreads();
  // warp w joins token w of the block
  s = sh[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = join_stats(s, make_float2(__shfl_xor_sync(0xFFFFFFFFu, s.x, o),
                                  __shfl_xor_sync(0xFFFFFFFFu, s.y, o)));
  const int64_t mine = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && mine < tokens) {
    const float l = s.x + logf(s.y);
    lse[mine] = l;
    const long long t = target[mine];
    loss[mine] = t == ignore ? 0.0f
               : t >= 0 && t < vocab ? l - target_logit[mine] : __uint_as_float(0x7FC00000u);
  }
}

// Threads and CTAs an SM of the copying kernel: every CTA looks through all tokens'
// dloss, so few large ones (65000 x 1024: 265 us with eight of 256 threads, 103;
// 2048 x 768: 10.1 and 8.5).
constexpr int kCopyThreads = 512, kCopyCtas = 3;

// The largest finite |dloss| of the tokens that count (one that is not finite
// spoils its own token's dx, not the others'), for every thread of the CTA.
__device__ float top_dloss(const float* dloss, const long long* target, long long ignore,
                           int64_t rows) {
  __shared__ uint32_t sh[kCopyThreads / 32];
  uint32_t most = 0;
#pragma unroll 4
  for (int64_t r = threadIdx.x; r < rows; r += kCopyThreads) {
    const float d = dloss[r];
    if (target[r] != ignore && !nonfinite(d)) most = max(most, abs_bits(d));
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCopyThreads / 32; ++i) most = max(most, sh[i]);
  return __uint_as_float(most);
}

// x 2^-b of two elements, in their type.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, int b, bool bf16) {
  const float2 f = bf16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u))
                        : h2_to_f2(w);
  const float lo = ldexpf(f.x, -b), hi = ldexpf(f.y, -b);
  return bf16 ? pack2<kBF16>(lo, hi) : pack2<kF16>(lo, hi);
}

// Rows of a matrix at a 16-byte pitch.  With dloss, those of x for dw: zero for
// an ignored token, with the token's 2^-b; then top gets the largest |dloss|
// (every CTA finds it for itself: 12 bytes a token, from L2), and `plain`, unless
// NULL, the rows as they are.
__global__ void __launch_bounds__(kCopyThreads)
xent_copy_kernel(const uint16_t* src, int64_t rows, int64_t dim, int64_t pitch, bool vec,
                 bool bf16, const long long* target, long long ignore, const float* dloss,
                 float* top, uint16_t* __restrict__ dst, uint16_t* __restrict__ plain) {
  begin_after_previous();
  const int lane = threadIdx.x & 31;   // a warp to a row
  float most = 0.0f;
  if (dloss != nullptr) {
    most = top_dloss(dloss, target, ignore, rows);
    if (blockIdx.x == 0 && threadIdx.x == 0) *top = most;
  }
  constexpr int kRows = kCopyThreads / 32;
  for (int64_t r = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * kRows) {
    const bool zero = dloss != nullptr && target[r] == ignore;
    const int b = dloss != nullptr && !zero ? dloss_shift(dloss[r], most) : 0;
    // one 16-byte word of the row
    const auto put = [&](int64_t c, uint4 v) {
      if (plain != nullptr) *reinterpret_cast<uint4*>(plain + r * pitch + c) = v;
      if (zero) v = make_uint4(0, 0, 0, 0);
      if (b > 0)
        v = make_uint4(scaled_pair(v.x, b, bf16), scaled_pair(v.y, b, bf16),
                       scaled_pair(v.z, b, bf16), scaled_pair(v.w, b, bf16));
      *reinterpret_cast<uint4*>(dst + r * pitch + c) = v;
    };
    if (vec) {
      const uint4* s = reinterpret_cast<const uint4*>(src + r * dim);
      for (int64_t c = lane; c < dim / 8; c += 4 * 32) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = c + 32 * k < dim / 8 ? __ldcg(s + c + 32 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + 32 * k < dim / 8) put(8 * (c + 32 * k), v[k]);
      }
    } else {
      // (the pitch is a multiple of 8 and dst aligned; src may be neither)
      const uint16_t* from = src + r * dim;
      const bool even = (reinterpret_cast<uintptr_t>(from) & 2u) == 0;
#pragma unroll 2
      for (int64_t c = 8 * lane; c < pitch; c += 8 * 32) {
        uint32_t w[4] = {0, 0, 0, 0};
        const uint16_t* p = from + c;
        if (c + 8 > dim) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < dim) w[k / 2] |= (uint32_t)p[k] << (16 * (k & 1));
        } else if (even) {
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = reinterpret_cast<const uint32_t*>(p)[k];
        } else {   // the first element, three words that start at the second, the last
          const uint32_t* q = reinterpret_cast<const uint32_t*>(p + 1);
          const uint32_t first = p[0], a = q[0], b2 = q[1], d = q[2], last = p[7];
          w[0] = first | a << 16;
          w[1] = a >> 16 | b2 << 16;
          w[2] = b2 >> 16 | d << 16;
          w[3] = d >> 16 | last << 16;
        }
        put(c, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}

// dx from its fp32 parts: the splits added in order, scaled back (with the
// token's own 2^-b), rounded; 0 for an ignored token.  Eight columns a thread (the
// parts' pitch is a multiple of 128).  The bound on CTAs gives a thread the 64
// registers that five splits' loads take; left to itself the compiler chose 32 to
// 40 and spilled (24 x 768: 8.6 to 8.2 us).
template <bool BF16>
__global__ void __launch_bounds__(256, 4)
xent_dx_kernel(const float* sum, int splits, int64_t tokens, int64_t dim, int64_t pitch,
               const long long* target, long long ignore, const float* dloss, const float* top,
               uint16_t* __restrict__ dx) {
  begin_after_previous();
  const float most = *top;
  const int64_t groups = (dim + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < tokens * groups;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / groups, c = (i - r * groups) * 8;
    const float4* a = reinterpret_cast<const float4*>(sum + r * pitch + c);
    const int64_t next = tokens * pitch / 4;
    float4 v[2] = {a[0], a[1]};
    for (int s = 1; s < splits; s += 5) {     // five splits' loads at a time
      float4 b[5][2];
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        const bool in = s + k < splits;
        b[k][0] = in ? a[(s + k) * next] : make_float4(0, 0, 0, 0);
        b[k][1] = in ? a[(s + k) * next + 1] : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < 5; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[h] = make_float4(v[h].x + b[k][h].x, v[h].y + b[k][h].y, v[h].z + b[k][h].z,
                             v[h].w + b[k][h].w);
    }
    float e[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    const bool zero = target[r] == ignore;
    const float back = ldexpf(most, -dloss_shift(dloss[r], most));
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = zero ? 0.0f : e[j] * (1.0f / kProbScale) * back;
    uint16_t* out = dx + r * dim + c;
    if (c + 8 <= dim && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
      *reinterpret_cast<uint4*>(out) =
          make_uint4(pack16<BF16>(e[0], e[1]), pack16<BF16>(e[2], e[3]),
                     pack16<BF16>(e[4], e[5]), pack16<BF16>(e[6], e[7]));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < dim) out[j] = (uint16_t)pack16<BF16>(e[j], 0.0f);
    }
  }
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

// rows x cols of 16-bit elements at a pitch, read in boxes of 64 columns.
cudaError_t make_map(CUtensorMap* map, bool bf16, const void* base, int64_t rows, int64_t cols,
                     int64_t pitch, int box_rows) {
  EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, ones[2] = {1, 1};
  const CUresult r = encode(
      map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
      const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

unsigned gemm_ctas(int64_t tiles, int sms) {
  return 2 * (unsigned)std::min(tiles, (int64_t)sms / 2);
}

cudaError_t launch_gemm(GemmArgs& g, bool bf16, int sms, cudaStream_t stream) {
  auto kernel = bf16 ? gemm_kernel<true> : gemm_kernel<false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
  if (e != cudaSuccess) return e;
  // the longest tiles first: the short ones even out the end
  std::sort(g.job, g.job + g.jobs,
            [](const GemmJob& a, const GemmJob& b) { return a.shape.kper > b.shape.kper; });
  int64_t tiles = 0;
  for (int i = 0; i < g.jobs; ++i) tiles += g.job[i].shape.tiles();
  return launch(true, kernel, gemm_ctas(tiles, sms), kGemmThreads, kGemmSmem, stream, g);
}

// Rows that TMA can read as they are.
bool direct(const void* p, int64_t dim) {
  return dim % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// For dw's copy of x: what its rows depend on, and where else they go.
struct CopyFor {
  const int64_t* target = nullptr;
  int64_t ignore = 0;
  const float* dloss = nullptr;
  float* top = nullptr;
  char* plain = nullptr;
};

cudaError_t copy_rows(const void* src, int64_t rows, int64_t dim, int64_t pitch, bool bf16,
                      char* dst, int sms, cudaStream_t stream, const CopyFor& f = CopyFor()) {
  constexpr int kRows = kCopyThreads / 32;
  const int64_t grid = std::min((rows + kRows - 1) / kRows, (int64_t)kCopyCtas * sms);
  return launch(true, xent_copy_kernel, (unsigned)grid, kCopyThreads, 0, stream,
                static_cast<const uint16_t*>(src), rows, dim, pitch,
                direct(src, dim) && pitch == dim, bf16,
                reinterpret_cast<const long long*>(f.target), (long long)f.ignore, f.dloss, f.top,
                reinterpret_cast<uint16_t*>(dst), reinterpret_cast<uint16_t*>(f.plain));
}

// Tokens of one forward launch: bounds the scratch of the tiles' statistics.
constexpr int64_t kForwardTokens = 65536;
// Columns of a piece.  A launch is one piece's gradients and the next piece's
// p, and dw's tiles, as long as the tokens are many, have to be a small part of
// a pair's share of it: the share over the tile's length is 3 piece dim /
// (pairs 65536), asked to be 6 (kShare columns of a 1-wide x per pair).  8192 x
// 1024 x 50257: 2.30 ms with 32 MiB of p a piece, 1.60 with 6 times the tile.
// Beyond that 128 MiB, up to 256: longer launches have fewer ends (2048 x 768:
// 0.49 ms with 32 MiB, 0.36 with 128; 8192 x 2048: 3.14 either way).
constexpr int64_t kPieceBytes = 128ll << 20, kMostPieceBytes = 256ll << 20, kShare = 131072;

int64_t piece_columns(const XentArgs& a, int sms) {
  const int64_t row = 2 * up(a.rows, kTileM);
  const int64_t want = std::max(kPieceBytes / row, kShare * (sms / 2) / a.dim);
  const int64_t fit = std::max(std::min(want, kMostPieceBytes / row) / kTileN, (int64_t)1);
  const int64_t pieces = (a.vocab + fit * kTileN - 1) / (fit * kTileN);
  return up((a.vocab + pieces - 1) / pieces, kTileN);   // of even size
}

// Width of the tiles that cover dim columns: 128 or 256 (a CTA's half is read in
// boxes of 64).
int width_of(int64_t dim) {
  const int64_t tiles = (dim + kTileN - 1) / kTileN;
  return (int)up((dim + tiles - 1) / tiles, 128);
}

int blocks_of(int64_t k) { return (int)((k + kBlockK - 1) / kBlockK); }

// Ranges of k for dx: its tiles are few and long when the tokens are few, so
// they are cut until one is at most half of a pair's share of a launch, into 8
// or, while the parts fit 64 MiB, up to 16 (more cost more to add up).  2048 x
// 768 x 50257: 312 us; at most the share, 323; a third, 330; a sixth, 345.
int dx_splits(const XentArgs& a, int64_t piece, int sms) {
  const int64_t tiles_t = up(a.rows, kTileM) / kTileM;
  const int64_t tiles_d = (a.dim + width_of(a.dim) - 1) / width_of(a.dim);
  const int64_t dx = tiles_t * tiles_d * blocks_of(piece);
  const int64_t dw = up(piece, kTileM) / kTileM * tiles_d * blocks_of(a.rows);
  const int64_t probs = tiles_t * (piece / kTileN) * blocks_of(a.dim);
  const int64_t share = std::max((dx + dw + probs) / (sms / 2) / 2, (int64_t)4);
  const int64_t fit = (64ll << 20) / (a.rows * tiles_d * width_of(a.dim) * 4);
  return (int)std::min((blocks_of(piece) + share - 1) / share,
                       std::min(std::max(fit, (int64_t)8), (int64_t)16));
}

class Layout {
 public:
  size_t take(int64_t bytes) {
    const size_t at = bytes_;
    bytes_ += (size_t)up(bytes, 256);
    return at;
  }
  size_t bytes() const { return bytes_; }

 private:
  size_t bytes_ = 0;
};

// Few tokens: the vocabulary's rows take the tiles' 256 rows and the tokens
// their columns, as many as there are; a stage then holds little besides w,
// which is all that has to be read.  24 x 768 x 50257: 19.9 us, 27.3 with the
// tokens as rows (mostly past x's end); 128 x 768 x 200000: 56 us against 75.
constexpr int64_t kSwapTokens = 128;

struct ForwardScratch {
  size_t x = 0, w = 0, partial = 0, logit = 0, bytes = 0;
  bool swapped = false;
  int64_t strips = 0;
};
ForwardScratch forward_scratch(const XentArgs& a, int sms) {
  ForwardScratch s;
  Layout l;
  const int64_t pitch = up(a.dim, 8), tokens = std::min(a.rows, kForwardTokens);
  if (!direct(a.x, a.dim)) s.x = l.take(a.rows * pitch * 2);
  if (!direct(a.w, a.dim)) s.w = l.take(a.vocab * pitch * 2);
  s.swapped = a.rows <= kSwapTokens;
  // a CTA's share of the vocabulary, or half a tile's columns
  s.strips = s.swapped ? gemm_ctas(up(a.vocab, kTileM) / kTileM, sms)
                       : 2 * (up(a.vocab, kTileN) / kTileN);
  s.partial = l.take(s.strips * tokens * 8);
  s.logit = l.take(tokens * 4);
  s.bytes = l.bytes();
  return s;
}

struct BackwardScratch {
  size_t next = 0, x = 0, x_plain = 0, w = 0, top = 0, probs[2] = {0, 0}, dx = 0, bytes = 0;
  int64_t piece = 0, pieces = 0;
  int splits = 1;
};
BackwardScratch backward_scratch(const XentArgs& a, int sms) {
  BackwardScratch s;
  Layout l;
  const int64_t pitch = up(a.dim, 8);
  s.piece = piece_columns(a, sms);
  s.pieces = (a.vocab + s.piece - 1) / s.piece;
  s.splits = dx_splits(a, s.piece, sms);
  s.next = l.take((s.pieces + 1) * 4);     // the launches' counters
  s.top = l.take(4);                       // max |dloss|
  s.x = l.take(a.rows * pitch * 2);
  if (!direct(a.x, a.dim)) s.x_plain = l.take(a.rows * pitch * 2);
  if (!direct(a.w, a.dim)) s.w = l.take(a.vocab * pitch * 2);
  for (int i = 0; i < 2 && i < s.pieces; ++i) s.probs[i] = l.take(a.rows * s.piece * 2);
  s.dx = l.take(s.splits * a.rows * up(a.dim, width_of(a.dim)) * 4);
  s.bytes = l.bytes();
  return s;
}

}  // namespace

size_t xent_forward_scratch(const XentArgs& a, int sms) { return forward_scratch(a, sms).bytes; }
size_t xent_backward_scratch(const XentArgs& a, int sms) { return backward_scratch(a, sms).bytes; }

cudaError_t launch_xent_forward(const XentArgs& a, char* scratch, int* error, int sms,
                                cudaStream_t stream, LaunchMark mark) {
  const ForwardScratch s = forward_scratch(a, sms);
  const bool bf16 = a.dtype == kBF16;
  const int64_t pitch = up(a.dim, 8);
  const char* x = static_cast<const char*>(a.x);
  const char* w = static_cast<const char*>(a.w);
  cudaError_t e = cudaSuccess;
  if (!direct(a.x, a.dim)) {
    e = copy_rows(a.x, a.rows, a.dim, pitch, bf16, scratch + s.x, sms, stream);
    x = scratch + s.x;
  }
  if (e == cudaSuccess && !direct(a.w, a.dim)) {
    e = copy_rows(a.w, a.vocab, a.dim, pitch, bf16, scratch + s.w, sms, stream);
    w = scratch + s.w;
  }
  for (int64_t t0 = 0; e == cudaSuccess && t0 < a.rows; t0 += kForwardTokens) {
    const int64_t tokens = std::min(a.rows - t0, kForwardTokens);
    GemmArgs g = {};
    g.error = error;
    g.jobs = 1;
    const int tiles_t = (int)(up(tokens, kTileM) / kTileM), kb = blocks_of(a.dim);
    const int tiles_v = (int)(up(a.vocab, kTileN) / kTileN);
    if (s.swapped)
      g.job[0].shape = {kStatsSwapped, tiles_v, 1, (int)up(tokens, 32), kb, kb, 1};
    else
      g.job[0].shape = {kStats, tiles_t, tiles_v, kTileN, kb, kb, 1};
    g.out.tokens = tokens;
    g.out.vocab = a.vocab;
    g.out.dim = a.dim;
    g.out.target = reinterpret_cast<const long long*>(a.target) + t0;
    g.out.ignore = a.ignore;
    g.out.partial = reinterpret_cast<float2*>(scratch + s.partial);
    g.out.target_logit = reinterpret_cast<float*>(scratch + s.logit);
    CUtensorMap& of_x = s.swapped ? g.job[0].b : g.job[0].a;
    CUtensorMap& of_w = s.swapped ? g.job[0].a : g.job[0].b;
    e = make_map(&of_x, bf16, x + t0 * pitch * 2, tokens, a.dim, pitch,
                 s.swapped ? g.job[0].shape.tile_n / 2 : kHalfM);
    if (e == cudaSuccess)
      e = make_map(&of_w, bf16, w, a.vocab, a.dim, pitch, s.swapped ? kHalfM : kTileN / 2);
    if (e != cudaSuccess) break;
    if (mark) mark(kXentLogitsK, 0, stream);
    e = launch_gemm(g, bf16, sms, stream);
    if (mark) mark(kXentLogitsK, 1, stream);
    if (e != cudaSuccess) break;
    if (mark) mark(kXentJoinK, 0, stream);
    e = launch(true, xent_join_kernel, (unsigned)((tokens + 31) / 32), 1024, 0, stream,
                     (const float2*)g.out.partial, (int)s.strips, tokens, a.vocab, g.out.target,
                     g.out.ignore, (const float*)g.out.target_logit, a.loss + t0,
                     a.lse_out + t0);
    if (mark) mark(kXentJoinK, 1, stream);
  }
  return e;
}

cudaError_t launch_xent_backward(const XentArgs& a, char* scratch, int* error, int sms,
                                 cudaStream_t stream, LaunchMark mark) {
  const bool bf16 = a.dtype == kBF16;
  if (a.rows == 0) return cudaMemsetAsync(a.dw, 0, (size_t)(a.vocab * a.dim) * 2, stream);
  const BackwardScratch s = backward_scratch(a, sms);
  const int64_t pitch = up(a.dim, 8);
  const int width = width_of(a.dim);
  const long long* target = reinterpret_cast<const long long*>(a.target);
  // the logits' x, and dw's: zero for ignored tokens, scaled for a small dloss
  const bool x_direct = direct(a.x, a.dim);
  const char* x = x_direct ? static_cast<const char*>(a.x) : scratch + s.x_plain;
  const char* x_dw = scratch + s.x;
  const char* w = static_cast<const char*>(a.w);
  int* next = reinterpret_cast<int*>(scratch + s.next);
  float* top = reinterpret_cast<float*>(scratch + s.top);
  cudaError_t e = cudaMemsetAsync(next, 0, (size_t)(s.pieces + 1) * 4, stream);
  if (mark) mark(kXentPrepareK, 0, stream);
  if (e == cudaSuccess)
    e = copy_rows(a.x, a.rows, a.dim, pitch, bf16, scratch + s.x, sms, stream,
                  {a.target, a.ignore, a.dloss, top, x_direct ? nullptr : scratch + s.x_plain});
  if (e == cudaSuccess && !direct(a.w, a.dim)) {
    e = copy_rows(a.w, a.vocab, a.dim, pitch, bf16, scratch + s.w, sms, stream);
    w = scratch + s.w;
  }
  if (mark) mark(kXentPrepareK, 1, stream);
  if (e != cudaSuccess) return e;

  // x and w as K-major operands of the logits, and MN-major ones of dw and dx;
  // p as dx's K-major and dw's MN-major operand
  CUtensorMap x_k, w_k, x_mn, w_mn, p_k[2], p_mn[2];
  const int a_rows = a.rows <= kHalfM ? (int)up(a.rows, 8) : 0, box = a_rows > 0 ? a_rows : kHalfM;
  if ((e = make_map(&x_k, bf16, x, a.rows, a.dim, pitch, box)) != cudaSuccess ||
      (e = make_map(&w_k, bf16, w, a.vocab, a.dim, pitch, kTileN / 2)) != cudaSuccess ||
      (e = make_map(&x_mn, bf16, x_dw, a.rows, a.dim, pitch, kBlockK)) != cudaSuccess ||
      (e = make_map(&w_mn, bf16, w, a.vocab, a.dim, pitch, kBlockK)) != cudaSuccess)
    return e;
  for (int i = 0; i < 2 && i < s.pieces; ++i) {
    const char* p = scratch + s.probs[i];
    if ((e = make_map(&p_k[i], bf16, p, a.rows, s.piece, s.piece, box)) != cudaSuccess ||
        (e = make_map(&p_mn[i], bf16, p, a.rows, s.piece, s.piece, kBlockK)) != cudaSuccess)
      return e;
  }

  GemmArgs g = {};
  g.error = error;
  GemmOut& o = g.out;
  o.tokens = a.rows;
  o.vocab = a.vocab;
  o.dim = a.dim;
  o.target = target;
  o.ignore = a.ignore;
  o.lse = a.lse;
  o.dloss = a.dloss;
  o.top = top;
  o.piece = s.piece;
  o.dx_sum = reinterpret_cast<float*>(scratch + s.dx);
  o.dim_pitch = up(a.dim, width);
  o.dw = a.dw;
  const int tiles_t = (int)(up(a.rows, kTileM) / kTileM);
  const int tiles_d = (int)(o.dim_pitch / width);
  // Launch i: the gradients of piece i - 1 and the probabilities of piece i.
  for (int64_t i = 0; i <= s.pieces; ++i) {
    g.jobs = 0;
    g.next = next + i;
    if (i > 0) {
      const int64_t v0 = (i - 1) * s.piece, cols = std::min(s.piece, a.vocab - v0);
      const int at = (int)((i - 1) & 1), kb = blocks_of(cols);
      g.job[g.jobs++] = {p_k[at], w_mn,
                         {kDx, tiles_t, tiles_d, width, kb, (kb + s.splits - 1) / s.splits,
                          s.splits, 0, (int)v0, 0, 1, i == 1, v0, nullptr, a_rows}};
      g.job[g.jobs++] = {p_mn[at], x_mn,
                         {kDw, (int)(up(cols, kTileM) / kTileM), tiles_d, width,
                          blocks_of(a.rows), blocks_of(a.rows), 1, 0, 0, 1, 1, 0, v0, nullptr, 0}};
    }
    if (i < s.pieces) {
      const int64_t v0 = i * s.piece, cols = std::min(s.piece, a.vocab - v0);
      g.job[g.jobs++] = {x_k, w_k,
                         {kProbs, tiles_t, (int)(up(cols, kTileN) / kTileN), kTileN,
                          blocks_of(a.dim), blocks_of(a.dim), 1, (int)v0, 0, 0, 0, 0, v0,
                          reinterpret_cast<uint16_t*>(scratch + s.probs[i & 1]), a_rows}};
    }
    if (mark) mark(kXentGradsK, 0, stream);
    e = launch_gemm(g, bf16, sms, stream);
    if (mark) mark(kXentGradsK, 1, stream);
    if (e != cudaSuccess) return e;
  }
  if (mark) mark(kXentDxK, 0, stream);
  e = launch(true, bf16 ? xent_dx_kernel<true> : xent_dx_kernel<false>,
                   (unsigned)std::min((a.rows * ((a.dim + 7) / 8) + 255) / 256, (int64_t)8 * sms), 256,
                   0, stream, (const float*)o.dx_sum, s.splits, a.rows, a.dim, o.dim_pitch, target,
                   (long long)a.ignore, a.dloss, (const float*)top,
                   static_cast<uint16_t*>(a.dx));
  if (mark) mark(kXentDxK, 1, stream);
  return e;
}

}  // namespace fp8opt
