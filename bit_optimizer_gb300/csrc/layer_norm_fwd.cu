// Layer norm, forward: y = xhat w + b with xhat = (x - mean) rstd over each
// row, mean = sum x / C, rstd = 1 / sqrt(sum (x - mean)^2 / C + eps).  For the
// backward pass it keeps mean and rstd, or (FP8) the E4M3 codes of xhat with
// one scale per row, 448 / max |xhat|, and rstd.
//
// Bound by HBM: e bytes in, e out, 1 more for the codes.  A row stays in
// registers between its three uses (sum, centred squares, result), so the
// variance is the two-pass one, without cancellation, at the price of one read.
#include "layer_norm.cuh"

namespace fp8opt {

namespace {

template <int DT, int VEC, int TPR, int VPT, int NT, bool FP8>
__global__ void __launch_bounds__(NT)
ln_forward_kernel(const LnForward a) {
  constexpr int RPC = NT / TPR;
  __shared__ RowSums<TPR> sums[RPC];
  const int slot = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const int cols = (int)a.cols;
  const size_t es = DT == kF32 ? 4 : 2;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * RPC + slot; r < a.rows;
       r += (int64_t)gridDim.x * RPC) {
    const char* row = static_cast<const char*>(a.x) + (size_t)r * a.cols * es;
    LnRaw<DT, VEC> raw[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) raw[v] = ln_load<DT, VEC, TPR>(row, v, t, cols);
    float x[8 * VPT];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      ln_widen<DT, VEC>(raw[v], x + 8 * v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[8 * v + e];   // zero past the row's end
    }
    const float mean = row_sum2<TPR>(s, 0.0f, sums[slot], turn, slot).x / (float)cols;
    float q = 0.0f;
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float& c = x[8 * v + e];
        c = ln_in<TPR, VEC>(v, e, t, cols) ? c - mean : 0.0f;
        q = __fmaf_rn(c, c, q);
        if (FP8) m = max(m, abs_bits(c));
      }
    float2 sq = make_float2(0.0f, 0.0f);
    if constexpr (FP8) {
      // the row's max |x - mean| beside its sum of squares
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      q = warp_sum(q);
      if constexpr (TPR > 32) {
        if ((t & 31) == 0) sums[slot].w[turn][t >> 5] = make_float2(q, __uint_as_float(m));
        row_barrier<TPR>(slot);
        q = 0.0f;
        m = 0;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) {
          const float2 w = sums[slot].w[turn][i];
          q += w.x;
          m = max(m, __float_as_uint(w.y));
        }
        turn ^= 1;
      }
      sq.x = q;
    } else {
      sq = row_sum2<TPR>(q, 0.0f, sums[slot], turn, slot);
    }
    const float rstd = __frsqrt_rn(sq.x / (float)cols + a.eps);
    if (t == 0) {
      a.rstd[r] = rstd;
      if (!FP8) a.mean[r] = mean;
    }
    float scale = 1.0f;
    bool finite = true;
    if constexpr (FP8) {
      // |x - mean| * rstd rounds monotonically, so this is max |xhat|
      const uint32_t amax = abs_bits(__uint_as_float(m) * rstd);
      scale = scale_from_amax_bits(amax, 448.0f);
      finite = amax < 0x7F800000u;
      if (t == 0) a.scales[r] = scale;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float w[8], b[8], y[8];
      ln_param<VEC, TPR>(a.weight, a.wdtype, 1.0f, v, t, cols, w);
      ln_param<VEC, TPR>(a.bias, a.wdtype, 0.0f, v, t, cols, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[8 * v + e] *= rstd;
        y[e] = __fmaf_rn(x[8 * v + e], w[e], b[e]);
      }
      ln_store<DT, VEC, TPR>(static_cast<char*>(a.y) + (size_t)r * a.cols * es, v, t, cols, y);
      if constexpr (FP8) {
        uint8_t* codes = a.codes + (size_t)r * a.cols;
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = x[8 * v + e] * scale;
        if constexpr (VEC == 8) {
          const int c = ln_col<TPR, 8>(v, 0, t);
          if (c < cols)
            __stcs(reinterpret_cast<uint2*>(codes + c),
                   finite ? enc8<kE4M3, false>(z) : enc8<kE4M3, true>(z));
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

template <int DT, int VEC, int TPR, int VPT, int NT>
void go(const LnForward& a, int sms, cudaStream_t stream) {
  const int64_t ctas = (a.rows + NT / TPR - 1) / (NT / TPR);
  const int64_t most = (int64_t)sms * (2048 / NT);
  const unsigned grid = (unsigned)(ctas < most ? ctas : most);
  if (a.codes != nullptr)
    ln_forward_kernel<DT, VEC, TPR, VPT, NT, true><<<grid, NT, 0, stream>>>(a);
  else
    ln_forward_kernel<DT, VEC, TPR, VPT, NT, false><<<grid, NT, 0, stream>>>(a);
}

template <int DT, int VEC>
void by_cols(const LnForward& a, int sms, cudaStream_t stream) {
  if (a.cols <= 256) go<DT, VEC, 32, 1, 128>(a, sms, stream);
  else if (a.cols <= 512) go<DT, VEC, 32, 2, 128>(a, sms, stream);
  else if (a.cols <= 1024) go<DT, VEC, 32, 4, 128>(a, sms, stream);
  else if (a.cols <= 2048) go<DT, VEC, 128, 2, 128>(a, sms, stream);
  else if (a.cols <= 4096) go<DT, VEC, 128, 4, 128>(a, sms, stream);
  else go<DT, VEC, 512, 4, 512>(a, sms, stream);
}

template <int DT>
void by_type(const LnForward& a, int sms, cudaStream_t stream) {
  if (a.cols > kLnMaxRegCols) {
    const int64_t most = (int64_t)sms * 2;
    const unsigned grid = (unsigned)(a.rows < most ? a.rows : most);
    if (a.codes != nullptr) ln_forward_long_kernel<DT, true><<<grid, 1024, 0, stream>>>(a);
    else ln_forward_long_kernel<DT, false><<<grid, 1024, 0, stream>>>(a);
  } else if (a.vec_ok) {
    by_cols<DT, 8>(a, sms, stream);
  } else {
    by_cols<DT, 1>(a, sms, stream);
  }
}

}  // namespace

cudaError_t launch_ln_forward(const LnForward& a, int sms, cudaStream_t stream,
                              LaunchMark mark) {
  if (mark) mark(kLayerNormK, 0, stream);
  if (a.dtype == kF32) by_type<kF32>(a, sms, stream);
  else if (a.dtype == kBF16) by_type<kBF16>(a, sms, stream);
  else by_type<kF16>(a, sms, stream);
  if (mark) mark(kLayerNormK, 1, stream);
  return cudaGetLastError();
}

}  // namespace fp8opt
