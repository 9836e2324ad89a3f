// Softmax cross entropy of a linear layer over a large vocabulary: logits
// z = x w^T (tokens x vocabulary), loss = lse(z) - z[target], without the
// logits ever being in memory as a whole.
//
// forward   One product on the tensor cores.  A tile's epilogue reduces its
//           logits, still in TMEM, to each token's maximum and sum of
//           exponentials over the tile's columns (base-2, fp32) and takes the
//           target's logit where it lies in the tile; a small kernel joins the
//           tiles of a token in column order.
// backward  The vocabulary goes in pieces.  For each piece the logits are
//           computed again and turned into p = (exp(z - lse) - [target]) *
//           dloss in the operands' 16-bit type, tokens x piece, in scratch;
//           then dx += p w_piece (fp32 in scratch between pieces) and dw_piece
//           = p^T x.  p is scaled by a power of two taken from max |dloss|, so
//           that FP16 holds it without underflow, and the results are scaled
//           back in fp32: the one rounding to 16 bits besides the results'.
//           Where p rounds, the error is random per element and of the size
//           of the operands' own rounding.
//
// Every product is the same kernel: persistent CTAs of six warps, one tile of
// 128 x 256 at a time.  Warp 4 feeds four stages of 64-deep operand blocks by
// TMA, warp 5 issues tcgen05.mma into one of two TMEM accumulators, warps 0 to
// 3 empty the other one, a row of the tile to each thread.  x and w are K-major
// in the logits product; w in dx, and both operands of dw, are read MN-major,
// so nothing is ever transposed in memory.
//
// Tokens whose target is `ignore` have no loss and give no gradient whatever
// is in their row of x: their p is 0 and dw reads a copy of x in which such
// rows are zero.  The copy also brings rows that TMA cannot read (a row
// length that is not a multiple of 8, unaligned tensors) to a 16-byte pitch.
#include "ops_internal.cuh"
#include "tensor_core.cuh"

namespace fp8opt {

namespace {

constexpr int kTileM = 128, kTileN = 256, kBlockK = 64, kGemmStages = 4;
constexpr int kStageA = kTileM * kBlockK * 2, kStageB = kTileN * kBlockK * 2;
constexpr int kGemmThreads = 192;
constexpr int kGemmSmem = 1024 + kGemmStages * (kStageA + kStageB);
constexpr float kLog2eF = 1.4426950408889634f, kLn2F = 0.69314718055994531f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

enum GemmMode { kStats = 0, kProbs, kDx, kDw };

// One product C[m, n] = sum_k A[m, k] B[n, k] and what becomes of its tiles.
struct GemmJob {
  CUtensorMap a, b;
  int mode;
  int tiles_m, tiles_n, kblocks;
  int a_mn0, a_k0, b_mn0, b_k0;   // coordinates of element (0, 0)
  int a_mn, b_mn;                 // MN-major operands
};

struct GemmOut {
  int64_t tokens;          // rows of x in this call
  int64_t vocab, dim;
  const long long* target;
  long long ignore;
  // kStats
  float2* partial;         // [column tile][token]: maximum, sum of exponentials
  float* target_logit;     // [token]
  // kProbs
  const float* lse;
  const float* dloss;
  const float* scale;      // 2^k and 2^-k
  uint16_t* probs;         // [token][piece]
  int64_t piece;           // columns of probs
  int64_t v0;              // first column of the piece
  // kDx, kDw
  float* dx_sum;           // [token][dim], NULL when there is one piece
  int first, last;         // first and last piece
  void* dx;
  void* dw;
};

struct GemmArgs {
  GemmJob job;
  GemmOut out;
  int* error;              // set to 1 when a wait ran out
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return pack2<BF16 ? kBF16 : kF16>(a, b);
}

// Stores n <= 32 results of one row as 16-bit values.
template <bool BF16>
__device__ __forceinline__ void store_row16(uint16_t* p, const float (&v)[32], int n) {
  if (n >= 32 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      reinterpret_cast<uint4*>(p)[j] =
          make_uint4(pack16<BF16>(v[8 * j], v[8 * j + 1]), pack16<BF16>(v[8 * j + 2], v[8 * j + 3]),
                     pack16<BF16>(v[8 * j + 4], v[8 * j + 5]),
                     pack16<BF16>(v[8 * j + 6], v[8 * j + 7]));
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) p[j] = (uint16_t)pack16<BF16>(v[j], 0.0f);
  }
}

// The tile's logits of one token: running maximum and sum of exponentials.
__device__ __forceinline__ void stats_row(const GemmOut& o, uint32_t tmem, int64_t row, int n_tile) {
  const int64_t n0 = (int64_t)n_tile * kTileN;
  const bool live = row < o.tokens;
  const long long target = live ? o.target[row] : -1;
  const int64_t rel = target >= 0 && target < o.vocab ? target - n0 : -1;
  float top = -1e30f, sum = 0.0f, at_target = 0.0f;
#pragma unroll 1
  for (int c = 0; c < kTileN; c += 32) {
    if (n0 + c >= o.vocab) break;
    uint32_t r[32];
    tmem_load32(tmem + c, r);
    tmem_wait();
    const int64_t left = o.vocab - n0 - c;
    if (left < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j >= left) r[j] = 0xFF800000u;
    }
    if (__any_sync(0xFFFFFFFFu, rel >= c && rel < c + 32)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (rel == c + j) at_target = __uint_as_float(r[j]);
    }
    float m = top;
#pragma unroll
    for (int j = 0; j < 32; ++j) m = fmaxf(m, __uint_as_float(r[j]));
    sum *= exp2_approx((top - m) * kLog2eF);
    top = m;
    const float shift = -m * kLog2eF;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 32; ++j)
      s[j & 3] += exp2_approx(__fmaf_rn(__uint_as_float(r[j]), kLog2eF, shift));
    sum += (s[0] + s[1]) + (s[2] + s[3]);
    __syncwarp();
  }
  if (live) {
    o.partial[(int64_t)n_tile * o.tokens + row] = make_float2(top, sum);
    if (rel >= 0 && rel < kTileN) o.target_logit[row] = at_target;
  }
}

// The tile's logits of one token turned into p.
template <bool BF16>
__device__ __forceinline__ void probs_row(const GemmOut& o, uint32_t tmem, int64_t row, int n_tile) {
  const int64_t n0 = (int64_t)n_tile * kTileN;   // within the piece
  const bool live = row < o.tokens;
  float shift = 0.0f, k = 0.0f;
  int64_t rel = -1;
  if (live) {
    const long long target = o.target[row];
    if (target != o.ignore) {
      k = o.dloss[row] * o.scale[0];
      shift = -o.lse[row] * kLog2eF;
      rel = target - o.v0 - n0;
      if (target < 0 || target >= o.vocab) k = __uint_as_float(0x7FC00000u);
    }
  }
  const bool zero = k == 0.0f;      // an ignored token, whatever its logits are
#pragma unroll 1
  for (int c = 0; c < kTileN; c += 32) {
    uint32_t r[32];
    tmem_load32(tmem + c, r);
    tmem_wait();
    const int64_t left = o.vocab - o.v0 - n0 - c;   // columns past the end are 0
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = exp2_approx(__fmaf_rn(__uint_as_float(r[j]), kLog2eF, shift));
    if (__any_sync(0xFFFFFFFFu, rel >= c && rel < c + 32)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (rel == c + j) v[j] -= 1.0f;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = zero ? 0.0f : v[j] * k;
    if (left < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j >= left) v[j] = 0.0f;
    }
    if (live) store_row16<BF16>(o.probs + row * o.piece + n0 + c, v, 32);
    __syncwarp();
  }
}

// dx of one token: this piece's part added to the earlier ones', and on the
// last piece scaled back and rounded.
template <bool BF16>
__device__ __forceinline__ void dx_row(const GemmOut& o, uint32_t tmem, int64_t row, int n_tile) {
  const int64_t n0 = (int64_t)n_tile * kTileN;
  const bool live = row < o.tokens;
  const bool zero = live && o.target[row] == o.ignore;
  const float back = o.scale[1];
#pragma unroll 1
  for (int c = 0; c < kTileN; c += 32) {
    if (n0 + c >= o.dim) break;
    uint32_t r[32];
    tmem_load32(tmem + c, r);
    tmem_wait();
    const int left = (int)min((int64_t)32, o.dim - n0 - c);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
    // dx_sum has a pitch of whole tiles, so its accesses need no bound
    float* sum = o.dx_sum + row * ((o.dim + kTileN - 1) / kTileN * kTileN) + n0 + c;
    if (live && !o.first) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 s = reinterpret_cast<const float4*>(sum)[j];
        v[4 * j] += s.x;
        v[4 * j + 1] += s.y;
        v[4 * j + 2] += s.z;
        v[4 * j + 3] += s.w;
      }
    }
    if (live && !o.last) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        reinterpret_cast<float4*>(sum)[j] =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    if (live && o.last) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = zero ? 0.0f : v[j] * back;
      store_row16<BF16>(static_cast<uint16_t*>(o.dx) + row * o.dim + n0 + c, v, left);
    }
    __syncwarp();
  }
}

template <bool BF16>
__device__ __forceinline__ void dw_row(const GemmOut& o, uint32_t tmem, int64_t row, int n_tile) {
  const int64_t n0 = (int64_t)n_tile * kTileN;
  const int64_t v0 = o.v0 + row;
  const float back = o.scale[1];
#pragma unroll 1
  for (int c = 0; c < kTileN; c += 32) {
    if (n0 + c >= o.dim) break;
    uint32_t r[32];
    tmem_load32(tmem + c, r);
    tmem_wait();
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * back;
    if (v0 < o.vocab)
      store_row16<BF16>(static_cast<uint16_t*>(o.dw) + v0 * o.dim + n0 + c, v,
                        (int)min((int64_t)32, o.dim - n0 - c));
    __syncwarp();
  }
}

struct GemmBarriers {
  uint64_t full[kGemmStages], empty[kGemmStages], acc_full[2], acc_empty[2], drained;
  uint32_t tmem;
};

template <bool BF16>
__global__ void __launch_bounds__(kGemmThreads, 1)
gemm_kernel(const __grid_constant__ GemmArgs args) {
  extern __shared__ uint8_t dyn[];
  __shared__ GemmBarriers bar;
  uint8_t* const stages = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
  const GemmJob& job = args.job;
  const int warp = threadIdx.x >> 5;
  const int tiles = job.tiles_m * job.tiles_n;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kGemmStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.acc_full[i], 1);
      mbar_init(&bar.acc_empty[i], 4);
    }
    mbar_init(&bar.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(&bar.tmem);
  tcgen_fence_before();
  __syncthreads();
  tcgen_fence_after();
  const uint32_t tmem = bar.tmem;
  bool ok = true;

  if (warp == 4) {
    if ((threadIdx.x & 31) == 0) {
      tma_prefetch_map(&job.a);
      tma_prefetch_map(&job.b);
      int s = 0, phase = 0;
      uint32_t loads = 0;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const int m = job.a_mn0 + tile % job.tiles_m * kTileM;
        const int n = job.b_mn0 + tile / job.tiles_m * kTileN;
        for (int kb = 0; kb < job.kblocks; ++kb) {
          if (!(ok = mbar_wait(&bar.empty[s], phase ^ 1))) break;
          uint8_t* a = stages + s * (kStageA + kStageB);
          uint8_t* b = a + kStageA;
          mbar_expect(&bar.full[s], kStageA + kStageB);
          ++loads;
          const int ka = job.a_k0 + kb * kBlockK, kk = job.b_k0 + kb * kBlockK;
          if (job.a_mn) {
            for (int i = 0; i < kTileM / 64; ++i)
              tma_load(a + i * (kBlockK * 128), &job.a, m + 64 * i, ka, &bar.full[s]);
          } else {
            tma_load(a, &job.a, ka, m, &bar.full[s]);
          }
          if (job.b_mn) {
            for (int i = 0; i < kTileN / 64; ++i)
              tma_load(b + i * (kBlockK * 128), &job.b, n + 64 * i, kk, &bar.full[s]);
          } else {
            tma_load(b, &job.b, kk, n, &bar.full[s]);
          }
          if (++s == kGemmStages) s = 0, phase ^= 1;
        }
      }
      // every copy lands before the CTA's shared memory is given up
      for (int i = 0; i < kGemmStages; ++i)
        if (loads > i)
          ok = mbar_wait(&bar.full[i], (loads - 1 - i) / kGemmStages & 1) && ok;
    }
  } else if (warp == 5) {
    if ((threadIdx.x & 31) == 0) {
      const uint32_t idesc = mma_desc(BF16, job.a_mn, job.b_mn, kTileM, kTileN);
      const uint32_t step_a = job.a_mn ? 16 * 128 : 32, step_b = job.b_mn ? 16 * 128 : 32;
      int s = 0, phase = 0, buf = 0, acc_phase = 0;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        if (!(ok = mbar_wait(&bar.acc_empty[buf], acc_phase ^ 1))) break;
        tcgen_fence_after();
        const uint32_t d = tmem + buf * kTileN;
        for (int kb = 0; kb < job.kblocks; ++kb) {
          if (!(ok = mbar_wait(&bar.full[s], phase))) break;
          tcgen_fence_after();
          const uint32_t a = smem_addr(stages + s * (kStageA + kStageB));
          const uint64_t da = operand_desc(a, job.a_mn, kBlockK * 128);
          const uint64_t db = operand_desc(a + kStageA, job.b_mn, kBlockK * 128);
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            mma_f16(d, da + (k * step_a >> 4), db + (k * step_b >> 4), idesc, kb + k > 0);
          mma_commit(&bar.empty[s]);
          if (++s == kGemmStages) s = 0, phase ^= 1;
        }
        mma_commit(&bar.acc_full[buf]);
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1;
      }
      // and every product ends before TMEM is
      mma_commit(&bar.drained);
      ok = mbar_wait(&bar.drained, 0) && ok;
    }
  } else {
    int buf = 0, phase = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      ok = mbar_wait(&bar.acc_full[buf], phase);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        ok = false;
        break;
      }
      tcgen_fence_after();
      const int64_t row = (int64_t)(tile % job.tiles_m) * kTileM + threadIdx.x;
      const int n = tile / job.tiles_m;
      const uint32_t t = tmem + buf * kTileN + ((uint32_t)warp << 21);
      if (job.mode == kStats) stats_row(args.out, t, row, n);
      else if (job.mode == kProbs) probs_row<BF16>(args.out, t, row, n);
      else if (job.mode == kDx) dx_row<BF16>(args.out, t, row, n);
      else dw_row<BF16>(args.out, t, row, n);
      tcgen_fence_before();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.acc_empty[buf]);
      buf ^= 1;
      if (buf == 0) phase ^= 1;
    }
  }
  if (!ok) *args.error = 1;
  __syncwarp();
  tcgen_fence_before();
  __syncthreads();
  tcgen_fence_after();
  if (warp == 0) tmem_free(tmem);
}

// Joins a token's column tiles: lane l takes tiles l, l + 32, ..., in order.
__global__ void __launch_bounds__(256)
xent_join_kernel(const float2* __restrict__ partial, int tiles, int64_t tokens, int64_t vocab,
                 const long long* __restrict__ target, long long ignore,
                 const float* __restrict__ target_logit, float* __restrict__ loss,
                 float* __restrict__ lse) {
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= tokens) return;
  float m = -1e30f, s = 0.0f;
  for (int i = threadIdx.x & 31; i < tiles; i += 32) {
    const float2 p = __ldg(partial + (int64_t)i * tokens + row);
    const float top = fmaxf(m, p.x);
    s = s * exp2_approx((m - top) * kLog2eF) + p.y * exp2_approx((p.x - top) * kLog2eF);
    m = top;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, o), s2 = __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const float top = fmaxf(m, m2);
    s = s * exp2_approx((m - top) * kLog2eF) + s2 * exp2_approx((m2 - top) * kLog2eF);
    m = top;
  }
  if ((threadIdx.x & 31) == 0) {
    const float l = m + logf(s);
    lse[row] = l;
    const long long t = target[row];
    loss[row] = t == ignore ? 0.0f
              : t >= 0 && t < vocab ? l - target_logit[row] : __uint_as_float(0x7FC00000u);
  }
}

// Rows of a matrix at a 16-byte pitch, those of ignored tokens zero (target
// NULL: none is).
__global__ void __launch_bounds__(256)
xent_copy_kernel(const uint16_t* __restrict__ src, int64_t rows, int64_t dim, int64_t pitch,
                 const long long* __restrict__ target, long long ignore,
                 uint16_t* __restrict__ dst, bool vec) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const bool zero = target != nullptr && target[r] == ignore;
    if (vec) {
      const uint4* s = reinterpret_cast<const uint4*>(src + r * dim);
      uint4* d = reinterpret_cast<uint4*>(dst + r * pitch);
      for (int64_t c = threadIdx.x; c < dim / 8; c += 256)
        d[c] = zero ? make_uint4(0, 0, 0, 0) : s[c];
    } else {
      for (int64_t c = threadIdx.x; c < pitch; c += 256)
        dst[r * pitch + c] = zero || c >= dim ? (uint16_t)0 : src[r * dim + c];
    }
  }
}

// scale[0] = the power of two that brings max |dloss| of the tokens that count
// to [2^14, 2^15), scale[1] = its inverse; 1 when the maximum is 0 or not
// finite.  (|exp(z - lse) - [target]| is at most 1, so |p| < 2^15.)
__global__ void __launch_bounds__(1024)
xent_scale_kernel(const float* __restrict__ dloss, const long long* __restrict__ target,
                  long long ignore, int64_t tokens, float* __restrict__ scale) {
  __shared__ uint32_t sh[32];
  uint32_t m = 0;
  for (int64_t i = threadIdx.x; i < tokens; i += 1024)
    if (target[i] != ignore) m = max(m, abs_bits(dloss[i]));
  m = block_max_u32<1024>(m, sh);
  if (threadIdx.x == 0) {
    int e = (int)(m >> 23) - 127;                 // 2^e <= max < 2^(e + 1)
    if (m == 0 || m >= 0x7F800000u) e = 14;
    const int k = min(max(14 - e, -126), 126);
    scale[0] = __int_as_float((127 + k) << 23);
    scale[1] = __int_as_float((127 - k) << 23);
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

cudaError_t launch_gemm(const GemmArgs& g, bool bf16, int sms, cudaStream_t stream) {
  auto kernel = bf16 ? gemm_kernel<true> : gemm_kernel<false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)g.job.tiles_m * g.job.tiles_n;
  kernel<<<(unsigned)(tiles < sms ? tiles : sms), kGemmThreads, kGemmSmem, stream>>>(g);
  return cudaGetLastError();
}

// Rows that TMA can read as they are.
bool direct(const void* p, int64_t dim) {
  return dim % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

cudaError_t copy_rows(const void* src, int64_t rows, int64_t dim, int64_t pitch,
                      const int64_t* target, int64_t ignore, char* dst, int sms,
                      cudaStream_t stream) {
  const int64_t grid = rows < 8 * sms ? rows : 8 * sms;
  xent_copy_kernel<<<(unsigned)grid, 256, 0, stream>>>(
      static_cast<const uint16_t*>(src), rows, dim, pitch,
      reinterpret_cast<const long long*>(target), ignore, reinterpret_cast<uint16_t*>(dst),
      direct(src, dim) && pitch == dim);
  return cudaGetLastError();
}

// Tokens of one forward launch: bounds the scratch of the tiles' statistics.
constexpr int64_t kForwardTokens = 65536;
// Bytes of p aimed at for one piece of the vocabulary.
constexpr int64_t kPieceBytes = 64ll << 20;

int64_t piece_columns(int64_t tokens, int64_t vocab) {
  const int64_t fit = kPieceBytes / 2 / up(tokens, kTileM) / kTileN * kTileN;
  return std::min(std::max(fit, (int64_t)kTileN), up(vocab, kTileN));
}

// Layouts of the scratch.
struct ForwardScratch {
  size_t x = 0, w = 0, partial = 0, logit = 0, bytes = 0;
};
ForwardScratch forward_scratch(const XentArgs& a) {
  ForwardScratch s;
  size_t at = 0;
  const auto take = [&](int64_t n) {
    const size_t p = at;
    at += (size_t)up(n, 256);
    return p;
  };
  const int64_t pitch = up(a.dim, 8);
  const int64_t tokens = std::min(a.rows, kForwardTokens);
  if (!direct(a.x, a.dim)) s.x = take(a.rows * pitch * 2);
  if (!direct(a.w, a.dim)) s.w = take(a.vocab * pitch * 2);
  s.partial = take(up(a.vocab, kTileN) / kTileN * tokens * 8);
  s.logit = take(tokens * 4);
  s.bytes = at;
  return s;
}

struct BackwardScratch {
  size_t x = 0, w = 0, scale = 0, probs = 0, dx = 0, bytes = 0;
  int64_t piece = 0;
};
BackwardScratch backward_scratch(const XentArgs& a) {
  BackwardScratch s;
  size_t at = 0;
  const auto take = [&](int64_t n) {
    const size_t p = at;
    at += (size_t)up(n, 256);
    return p;
  };
  const int64_t pitch = up(a.dim, 8);
  s.piece = piece_columns(a.rows, a.vocab);
  s.x = take(a.rows * pitch * 2);
  if (!direct(a.w, a.dim)) s.w = take(a.vocab * pitch * 2);
  s.scale = take(8);
  s.probs = take(a.rows * s.piece * 2);
  if (s.piece < a.vocab) s.dx = take(a.rows * up(a.dim, kTileN) * 4);
  s.bytes = at;
  return s;
}

}  // namespace

size_t xent_forward_scratch(const XentArgs& a) { return forward_scratch(a).bytes; }
size_t xent_backward_scratch(const XentArgs& a) { return backward_scratch(a).bytes; }

cudaError_t launch_xent_forward(const XentArgs& a, char* scratch, int* error, int sms,
                                cudaStream_t stream, LaunchMark mark) {
  const ForwardScratch s = forward_scratch(a);
  const bool bf16 = a.dtype == kBF16;
  const int64_t pitch = up(a.dim, 8);
  const char* x = static_cast<const char*>(a.x);
  const char* w = static_cast<const char*>(a.w);
  cudaError_t e = cudaSuccess;
  if (!direct(a.x, a.dim)) {
    e = copy_rows(a.x, a.rows, a.dim, pitch, nullptr, 0, scratch + s.x, sms, stream);
    x = scratch + s.x;
  }
  if (e == cudaSuccess && !direct(a.w, a.dim)) {
    e = copy_rows(a.w, a.vocab, a.dim, pitch, nullptr, 0, scratch + s.w, sms, stream);
    w = scratch + s.w;
  }
  for (int64_t t0 = 0; e == cudaSuccess && t0 < a.rows; t0 += kForwardTokens) {
    const int64_t tokens = std::min(a.rows - t0, kForwardTokens);
    GemmArgs g = {};
    g.error = error;
    g.job.mode = kStats;
    g.job.tiles_m = (int)(up(tokens, kTileM) / kTileM);
    g.job.tiles_n = (int)(up(a.vocab, kTileN) / kTileN);
    g.job.kblocks = (int)(up(a.dim, kBlockK) / kBlockK);
    g.out.tokens = tokens;
    g.out.vocab = a.vocab;
    g.out.dim = a.dim;
    g.out.target = reinterpret_cast<const long long*>(a.target) + t0;
    g.out.ignore = a.ignore;
    g.out.partial = reinterpret_cast<float2*>(scratch + s.partial);
    g.out.target_logit = reinterpret_cast<float*>(scratch + s.logit);
    e = make_map(&g.job.a, bf16, x + t0 * pitch * 2, tokens, a.dim, pitch, kTileM);
    if (e == cudaSuccess) e = make_map(&g.job.b, bf16, w, a.vocab, a.dim, pitch, kTileN);
    if (e != cudaSuccess) break;
    if (mark) mark(kXentLogitsK, 0, stream);
    e = launch_gemm(g, bf16, sms, stream);
    if (mark) mark(kXentLogitsK, 1, stream);
    if (e != cudaSuccess) break;
    if (mark) mark(kXentJoinK, 0, stream);
    xent_join_kernel<<<(unsigned)((tokens + 7) / 8), 256, 0, stream>>>(
        g.out.partial, g.job.tiles_n, tokens, a.vocab, g.out.target, a.ignore,
        g.out.target_logit, a.loss + t0, a.lse_out + t0);
    if (mark) mark(kXentJoinK, 1, stream);
    e = cudaGetLastError();
  }
  return e;
}

cudaError_t launch_xent_backward(const XentArgs& a, char* scratch, int* error, int sms,
                                 cudaStream_t stream, LaunchMark mark) {
  const bool bf16 = a.dtype == kBF16;
  if (a.rows == 0) return cudaMemsetAsync(a.dw, 0, (size_t)(a.vocab * a.dim) * 2, stream);
  const BackwardScratch s = backward_scratch(a);
  const int64_t pitch = up(a.dim, 8);
  const char* x = scratch + s.x;   // rows of ignored tokens zero
  const char* w = static_cast<const char*>(a.w);
  if (mark) mark(kXentPrepareK, 0, stream);
  cudaError_t e = copy_rows(a.x, a.rows, a.dim, pitch, a.target, a.ignore, scratch + s.x, sms,
                            stream);
  if (e == cudaSuccess && !direct(a.w, a.dim)) {
    e = copy_rows(a.w, a.vocab, a.dim, pitch, nullptr, 0, scratch + s.w, sms, stream);
    w = scratch + s.w;
  }
  float* scale = reinterpret_cast<float*>(scratch + s.scale);
  xent_scale_kernel<<<1, 1024, 0, stream>>>(a.dloss, reinterpret_cast<const long long*>(a.target),
                                            a.ignore, a.rows, scale);
  if (mark) mark(kXentPrepareK, 1, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  // x and w as K-major operands of the logits, and MN-major ones of dw and dx;
  // p as dx's K-major and dw's MN-major operand
  CUtensorMap x_k, w_k, x_mn, w_mn, p_k, p_mn;
  const char* p = scratch + s.probs;
  if ((e = make_map(&x_k, bf16, x, a.rows, a.dim, pitch, kTileM)) != cudaSuccess ||
      (e = make_map(&w_k, bf16, w, a.vocab, a.dim, pitch, kTileN)) != cudaSuccess ||
      (e = make_map(&x_mn, bf16, x, a.rows, a.dim, pitch, kBlockK)) != cudaSuccess ||
      (e = make_map(&w_mn, bf16, w, a.vocab, a.dim, pitch, kBlockK)) != cudaSuccess ||
      (e = make_map(&p_k, bf16, p, a.rows, s.piece, s.piece, kTileM)) != cudaSuccess ||
      (e = make_map(&p_mn, bf16, p, a.rows, s.piece, s.piece, kBlockK)) != cudaSuccess)
    return e;

  GemmArgs g = {};
  g.error = error;
  GemmOut& o = g.out;
  o.tokens = a.rows;
  o.vocab = a.vocab;
  o.dim = a.dim;
  o.target = reinterpret_cast<const long long*>(a.target);
  o.ignore = a.ignore;
  o.lse = a.lse;
  o.dloss = a.dloss;
  o.scale = scale;
  o.probs = reinterpret_cast<uint16_t*>(scratch + s.probs);
  o.piece = s.piece;
  o.dx_sum = reinterpret_cast<float*>(scratch + s.dx);
  o.dx = a.dx;
  o.dw = a.dw;
  const int tiles_t = (int)(up(a.rows, kTileM) / kTileM);
  const int tiles_d = (int)(up(a.dim, kTileN) / kTileN);
  for (int64_t v0 = 0; v0 < a.vocab; v0 += s.piece) {
    const int64_t cols = std::min(s.piece, a.vocab - v0);
    o.v0 = v0;
    o.first = v0 == 0;
    o.last = v0 + cols == a.vocab;
    GemmJob& j = g.job;
    j = GemmJob{x_k, w_k, kProbs, tiles_t, (int)(up(cols, kTileN) / kTileN),
                (int)(up(a.dim, kBlockK) / kBlockK), 0, 0, (int)v0, 0, 0, 0};
    if (mark) mark(kXentProbsK, 0, stream);
    e = launch_gemm(g, bf16, sms, stream);
    if (mark) mark(kXentProbsK, 1, stream);
    if (e != cudaSuccess) return e;
    if (mark) mark(kXentGradsK, 0, stream);
    j = GemmJob{p_k, w_mn, kDx, tiles_t, tiles_d, (int)(up(cols, kBlockK) / kBlockK),
                0, 0, 0, (int)v0, 0, 1};
    e = launch_gemm(g, bf16, sms, stream);
    if (e == cudaSuccess) {
      j = GemmJob{p_mn, x_mn, kDw, (int)(up(cols, kTileM) / kTileM), tiles_d,
                  (int)(up(a.rows, kBlockK) / kBlockK), 0, 0, 0, 0, 1, 1};
      e = launch_gemm(g, bf16, sms, stream);
    }
    if (mark) mark(kXentGradsK, 1, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fp8opt
