// Layer norm, forward: y = xhat w + b with xhat = (x - mean) rstd over each
// row, mean = sum x / C, rstd = 1 / sqrt(sum (x - mean)^2 / C + eps).  For the
// backward pass it keeps mean and rstd, or (FP8) the E4M3 codes of xhat with
// one scale per row, 448 / max |xhat|, and rstd.
//
// Bound by HBM: e bytes in, e out, 1 more for the codes.  A row stays in
// registers between its three uses (sum, centred squares, result), so the
// variance is the two-pass one, without cancellation, at the price of one read;
// the next rows are on their way through the ring meanwhile, and weight and
// bias wait in shared memory (read from L1 they were evicted by the rows: 77.8
// us).  16384 x 4096 BF16 with codes: 56.6 us, 5.93 TB/s, 0.87 of the measured
// copy bandwidth; 65536 x 1024 without: 47 us, 0.83.  Rows that start anywhere
// take scalar reads of weight and bias and masked ends: 65536 x 767 59 us, 0.50
// (768: 34 us), 32768 x 1501 53 us (by elements 99), 32768 x 2041 58 (111); just
// above a power of two half of a row's threads idle: 32768 x 2049 107 (159).
#include "layer_norm.cuh"

namespace fp8opt {

namespace {

// Threads of a CTA, one CTA to an SM (128 registers a thread).
constexpr int kFwdThreads = 512, kFwdCtas = 1;

// Rows in flight of a thread's ring, and the ring's bytes.
template <int DT>
constexpr int kStages = DT == kF32 ? 2 : 4;
template <int DT, int VPT>
constexpr int kRingBytes = kStages<DT> * VPT * (DT == kF32 ? 32 : 16) * kFwdThreads;

// Sum of the elements as a tree of pairs, so that its rounding error grows
// with the logarithm of their number.
template <int N>
__device__ __forceinline__ float tree_sum(const float2* x) {
  float2 s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = x[i];
#pragma unroll
  for (int h = N / 2; h > 0; h /= 2)
#pragma unroll
    for (int i = 0; i < h; ++i) s[i] = add2(s[i], s[i + h]);
  return s[0].x + s[0].y;
}

template <int DT, int VEC, int TPR, int VPT, bool FP8, bool FULL>
__global__ void __launch_bounds__(kFwdThreads, kFwdCtas)
ln_forward_kernel(const LnForward a) {
  constexpr int NT = kFwdThreads, RPC = NT / TPR, Q = DT == kF32 ? 2 : 1, ST = kStages<DT>;
  __shared__ RowSums<TPR> sums[RPC];
  // Weight and bias as fp32, then the ring [ST][VPT][Q][NT].  VEC 8: [2]
  // [VPT][2][TPR] quads, so that a warp's quads lie side by side; VEC 1:
  // [2][TPR * 8 * VPT] elements; kLnFlat: pairs of both, element c at [c mod 8]
  // [c / 8], where the elements e of a warp's vectors lie side by side for
  // every shift.
  extern __shared__ uint4 shared[];
  const int slot = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const int cols = (int)a.cols;
  const size_t es = DT == kF32 ? 4 : 2;
  const int64_t step = (int64_t)gridDim.x * RPC;
  int turn = 0;
  int64_t r = (int64_t)blockIdx.x * RPC + slot;
  float* const sw = reinterpret_cast<float*>(shared);
  float* const sb = sw + TPR * 8 * VPT;
  float2* const pairs = reinterpret_cast<float2*>(shared);
  uint4* const ring = shared + TPR * 4 * VPT;
  const auto at = [&](int stage, int v, int q) -> uint4* {
    return ring + ((stage * VPT + v) * Q + q) * NT + threadIdx.x;
  };
  const int shift = VEC == kLnFlat ? (int)(r * a.cols & 7) : 0, end = cols + shift;
  const auto fetch = [&](int stage, int64_t row) {
    if (row < a.rows) {
      const char* p = static_cast<const char*>(a.x) + ((size_t)row * a.cols - shift) * es;
      const int left = VEC == kLnFlat ? ln_left(a.rows - row, a.cols, shift) : 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = ln_col<TPR, 8>(v, 0, t);
        if (FULL || c < end)
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            if constexpr (VEC == kLnFlat) {
              const int n = ln_bytes(left - c, (int)es, 16 * q, 16);
              if (n > 0) copy_async<16>(at(stage, v, q), p + c * es + 16 * q, n);
            } else {
              copy_async<16>(at(stage, v, q), p + c * es + 16 * q);
            }
          }
      }
    }
    copy_commit();
  };
  begin_after_previous();
  if constexpr (VEC != 1) {
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(i, r + i * step);
  }
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < ST; ++i)   // what lies past the row's end stays zero
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (!ln_in<TPR, 8, FULL>(v, 0, t, cols))
#pragma unroll
          for (int q = 0; q < Q; ++q) *at(i, v, q) = make_uint4(0, 0, 0, 0);
  }
  for (int i = threadIdx.x; i < TPR * VPT; i += NT) {
    float w[8], b[8];
    constexpr int PV = VEC == 8 ? 8 : 1;
    ln_param<PV, TPR>(a.weight, a.wdtype, 0.0f, i / TPR, i % TPR, cols, w);
    ln_param<PV, TPR>(a.bias, a.wdtype, 0.0f, i / TPR, i % TPR, cols, b);
    if constexpr (VEC == 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at4 = (i / TPR * 2 + h) * TPR + i % TPR;
        reinterpret_cast<float4*>(sw)[at4] =
            make_float4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
        reinterpret_cast<float4*>(sb)[at4] =
            make_float4(b[4 * h], b[4 * h + 1], b[4 * h + 2], b[4 * h + 3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = ln_col<TPR, 1>(i / TPR, e, i % TPR);
        if constexpr (VEC == kLnFlat) {
          pairs[(c & 7) * (TPR * VPT) + (c >> 3)] = make_float2(w[e], b[e]);
        } else {
          sw[c] = w[e];
          sb[c] = b[e];
        }
      }
    }
  }
  // where the elements e of vector 0 of thread 0 lie (masked ones before the
  // row: at the end of the line before, never before the first)
  int at_e[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned u = (unsigned)(8 + e - shift);   // its column + 8
    at_e[e] = (int)((u & 7u) * (TPR * VPT) + (u >> 3)) + t - 1;
  }
  __syncthreads();
  for (int stage = 0; r < a.rows; r += step, stage = stage + 1 == ST ? 0 : stage + 1) {
    float2 x[4 * VPT];
    if constexpr (VEC != 1) {
      copy_wait<ST - 2>();
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        LnRaw<DT, 8> raw;
        float f[8];
        if (VEC == kLnFlat && ln_col<TPR, 8>(v, 0, t) >= end) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[4 * v + j] = splat2(0.0f);
          continue;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) raw.v[q] = *at(stage, v, q);
        ln_widen<DT, 8>(raw, f);
        if (VEC == kLnFlat) ln_mask(f, ln_col<TPR, 8>(v, 0, t), shift, end);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * v + j] = make_float2(f[2 * j], f[2 * j + 1]);
      }
      fetch(stage == 0 ? ST - 1 : stage - 1, r + (ST - 1) * step);
    } else {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const LnRaw<DT, 1> raw = ln_load<DT, 1, TPR>(
            static_cast<const char*>(a.x) + (size_t)r * a.cols * es, v, t, cols);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * v + j] = make_float2(raw.f[2 * j], raw.f[2 * j + 1]);
      }
    }
    // (what lies past the row's end is zero in both)
    const float s = tree_sum<4 * VPT>(x);
    const float mean = row_reduce<kOne, TPR>(s, 0.0f, sums[slot], turn, slot).x / (float)cols;
    float2 sq[4] = {splat2(0.0f), splat2(0.0f), splat2(0.0f), splat2(0.0f)};
    float m = 0.0f;   // (a NaN passes it by, and is found in the sum of squares)
#pragma unroll
    for (int i = 0; i < 4 * VPT; ++i) {
      if constexpr (VEC == kLnFlat) {
        if (ln_col<TPR, 8>(i / 4, 0, t) >= end) continue;
        if (i % 4 == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i + j] = add2(x[i + j], splat2(-mean));
          ln_mask(x + i, ln_col<TPR, 8>(i / 4, 0, t), shift, end);
        }
      } else {
        x[i] = add2(x[i], splat2(-mean));
        if (!ln_in<TPR, VEC, FULL>(i / 4, 2 * (i % 4), t, cols)) x[i].x = 0.0f;
        if (!ln_in<TPR, VEC, FULL>(i / 4, 2 * (i % 4) + 1, t, cols)) x[i].y = 0.0f;
      }
      sq[i % 4] = fma2(x[i], x[i], sq[i % 4]);
      if (FP8) m = fmaxf(fmaxf(m, fabsf(x[i].x)), fabsf(x[i].y));
    }
    const float2 qm = row_reduce<FP8 ? kMax : kOne, TPR>(tree_sum<4>(sq), m, sums[slot], turn,
                                                         slot);
    const float q = qm.x;
    const float rstd = __frsqrt_rn(q / (float)cols + a.eps);
    if (t == 0) {
      a.rstd[r] = rstd;
      if (!FP8) a.mean[r] = mean;
    }
    float scale = 1.0f, to_code = 1.0f;
    bool finite = true;
    if constexpr (FP8) {
      // |x - mean| * rstd rounds monotonically, so this is max |xhat|
      const uint32_t amax = abs_bits(qm.y * rstd);
      scale = scale_from_amax_bits(amax, 448.0f);
      finite = amax < 0x7F800000u;
      if (t == 0) a.scales[r] = scale;
      // xhat * scale = (x - mean) * 448 / max |x - mean|: taken so, the codes
      // carry the rounding of one quotient instead of rstd's and the scale's
      to_code = __fdiv_rn(448.0f, qm.y);
      if (scale == 1.0f || nonfinite(to_code)) to_code = rstd * scale;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (VEC == kLnFlat && ln_col<TPR, 8>(v, 0, t) >= end) continue;
      float y[8], z[8];
      float4 w4[2], b4[2];
      if constexpr (VEC == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w4[h] = reinterpret_cast<const float4*>(sw)[(2 * v + h) * TPR + t];
          b4[h] = reinterpret_cast<const float4*>(sb)[(2 * v + h) * TPR + t];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 h = mul2(x[4 * v + j], splat2(rstd));
        float2 w, b;
        if constexpr (VEC == 8) {
          w = (j & 1) ? make_float2(w4[j / 2].z, w4[j / 2].w)
                      : make_float2(w4[j / 2].x, w4[j / 2].y);
          b = (j & 1) ? make_float2(b4[j / 2].z, b4[j / 2].w)
                      : make_float2(b4[j / 2].x, b4[j / 2].y);
        } else if constexpr (VEC == kLnFlat) {
          const float2 p0 = pairs[at_e[2 * j] + v * TPR], p1 = pairs[at_e[2 * j + 1] + v * TPR];
          w = make_float2(p0.x, p1.x);
          b = make_float2(p0.y, p1.y);
        } else {
          const int c0 = ln_col<TPR, 1>(v, 2 * j, t), c1 = ln_col<TPR, 1>(v, 2 * j + 1, t);
          w = make_float2(sw[c0], sw[c1]);
          b = make_float2(sb[c0], sb[c1]);
        }
        const float2 p = fma2(h, w, b);
        y[2 * j] = p.x;
        y[2 * j + 1] = p.y;
        if constexpr (FP8) {
          const float2 c = mul2(x[4 * v + j], splat2(to_code));
          z[2 * j] = c.x;
          z[2 * j + 1] = c.y;
        }
      }
      char* const out = static_cast<char*>(a.y) + (size_t)r * a.cols * es;
      if constexpr (VEC == kLnFlat) ln_store_flat<DT, TPR>(out, v, t, shift, end, y);
      else ln_store<DT, VEC, TPR>(out, v, t, cols, y);
      if constexpr (FP8) {
        uint8_t* codes = a.codes + (size_t)r * a.cols;
        if constexpr (VEC == 8) {
          const int c = ln_col<TPR, 8>(v, 0, t);
          if (FULL || c < cols)
            __stcs(reinterpret_cast<uint2*>(codes + c),
                   finite ? enc8<kE4M3, false>(z) : enc8<kE4M3, true>(z));
        } else if constexpr (VEC == kLnFlat) {
          const int c = ln_col<TPR, 8>(v, 0, t);
          const uint2 p = finite ? enc8<kE4M3, false>(z) : enc8<kE4M3, true>(z);
          if (c >= shift && c + 8 <= end) {
            __stcs(reinterpret_cast<uint2*>(codes - shift + c), p);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (c + e >= shift && c + e < end)
                codes[c + e - shift] = (uint8_t)((e < 4 ? p.x : p.y) >> (8 * (e & 3)));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = ln_col<TPR, 1>(v, e, t);
            if (c < cols) codes[c] = (uint8_t)enc1_checked<kE4M3>(z[e]);
          }
        }
      }
    }
  }
}

// Sum and max over a CTA, for every thread.
template <int NT>
__device__ float2 cta_sum_max(float s, uint32_t m, float2* sh) {
  s = warp_sum(s);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(s, __uint_as_float(m));
  __syncthreads();
  s = 0.0f;
  m = 0;
  for (int i = 0; i < NT / 32; ++i) {
    s += sh[i].x;
    m = max(m, __float_as_uint(sh[i].y));
  }
  return make_float2(s, __uint_as_float(m));
}

// Rows too long for the registers of a CTA: three passes over the row, the
// later two from L2.
template <int DT, bool FP8>
__global__ void __launch_bounds__(1024)
ln_forward_long_kernel(const LnForward a) {
  __shared__ float2 sh[32];
  begin_after_previous();
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const int64_t at = r * a.cols;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) s += load1<DT>(a.x, at + c);
    const float mean = cta_sum_max<1024>(s, 0u, sh).x / (float)a.cols;
    float q = 0.0f;
    uint32_t m = 0;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float d = load1<DT>(a.x, at + c) - mean;
      q = __fmaf_rn(d, d, q);
      m = max(m, abs_bits(d));
    }
    const float2 qm = cta_sum_max<1024>(q, m, sh);
    const float rstd = __frsqrt_rn(qm.x / (float)a.cols + a.eps);
    const float scale = scale_from_amax_bits(abs_bits(qm.y * rstd), 448.0f);
    if (threadIdx.x == 0) {
      a.rstd[r] = rstd;
      if (FP8) a.scales[r] = scale;
      else a.mean[r] = mean;
    }
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float xhat = (load1<DT>(a.x, at + c) - mean) * rstd;
      const float w = a.weight ? ln_param1(a.weight, a.wdtype, c) : 1.0f;
      const float b = a.bias ? ln_param1(a.bias, a.wdtype, c) : 0.0f;
      store1<DT>(a.y, at + c, __fmaf_rn(xhat, w, b));
      if (FP8) a.codes[at + c] = (uint8_t)enc1_checked<kE4M3>(xhat * scale);
    }
  }
}

template <int DT, int VEC, int TPR, int VPT, bool FP8, bool FULL>
cudaError_t go_form(const LnForward& a, int sms, cudaStream_t stream) {
  constexpr int RPC = kFwdThreads / TPR;
  auto kernel = ln_forward_kernel<DT, VEC, TPR, VPT, FP8, FULL>;
  const int smem = (VEC != 1 ? kRingBytes<DT, VPT> : 0) + 2 * (int)sizeof(float) * TPR * 8 * VPT;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t grid = ln_grid((a.rows + RPC - 1) / RPC, (int64_t)sms * kFwdCtas, a.form);
  return launch(worth_early(a.rows * a.cols), kernel, (unsigned)grid, kFwdThreads, smem, stream, a);
}

template <int DT, int VEC, int TPR, int VPT>
cudaError_t go(const LnForward& a, int sms, cudaStream_t stream) {
  if constexpr (VEC == 8) {
    if (a.cols == TPR * VPT * 8)
      return a.codes != nullptr ? go_form<DT, VEC, TPR, VPT, true, true>(a, sms, stream)
                                : go_form<DT, VEC, TPR, VPT, false, true>(a, sms, stream);
  }
  return a.codes != nullptr ? go_form<DT, VEC, TPR, VPT, true, false>(a, sms, stream)
                            : go_form<DT, VEC, TPR, VPT, false, false>(a, sms, stream);
}

// As many elements a thread as its registers take: the reductions, which cost
// the same whatever a thread holds, then weigh least (16384 x 4096 with codes:
// 61.7 us with 16 elements a thread, 59.1 with 32).
template <int DT, int VEC>
cudaError_t by_cols(const LnForward& a, int sms, cudaStream_t stream) {
  const int64_t span = ln_span(a.cols, VEC);
  if constexpr (VEC != kLnFlat)
    if (span <= 256) return go<DT, VEC, 32, 1>(a, sms, stream);
  if (span <= 512) return go<DT, VEC, 32, 2>(a, sms, stream);
  if (span <= 1024) return go<DT, VEC, 32, 4>(a, sms, stream);
  if (span <= 2048) return go<DT, VEC, 64, 4>(a, sms, stream);
  if (span <= 4096) return go<DT, VEC, 128, 4>(a, sms, stream);
  return go<DT, VEC, 256, 4>(a, sms, stream);
}

template <int DT>
cudaError_t by_type(const LnForward& a, int sms, cudaStream_t stream) {
  if (a.cols > kLnMaxRegCols) {
    const int64_t most = (int64_t)sms * 2;
    const unsigned grid = (unsigned)(a.rows < most ? a.rows : most);
    return launch(worth_early(a.rows * a.cols), a.codes != nullptr ? ln_forward_long_kernel<DT, true>
                                           : ln_forward_long_kernel<DT, false>,
                        grid, 1024, 0, stream, a);
  }
  if (a.form == kLnVectors) return by_cols<DT, 8>(a, sms, stream);
  if (a.form == kLnFlat) return by_cols<DT, kLnFlat>(a, sms, stream);
  return by_cols<DT, 1>(a, sms, stream);
}

}  // namespace

cudaError_t launch_ln_forward(const LnForward& a, int sms, cudaStream_t stream,
                              LaunchMark mark) {
  if (mark) mark(kLayerNormK, 0, stream);
  const cudaError_t e = a.dtype == kF32    ? by_type<kF32>(a, sms, stream)
                        : a.dtype == kBF16 ? by_type<kBF16>(a, sms, stream)
                                           : by_type<kF16>(a, sms, stream);
  if (mark) mark(kLayerNormK, 1, stream);
  return e;
}

}  // namespace fp8opt
