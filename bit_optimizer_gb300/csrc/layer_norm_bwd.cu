// Layer norm, backward.  With h = dy w and xhat = (x - mean) rstd (or read
// from its E4M3 codes):
//   dx = rstd (h - mean_c(h) - xhat mean_c(h xhat)),
//   dw = sum_rows dy xhat,   db = sum_rows dy.
//
// One pass over dy and x (or the codes): a thread owns fixed columns and keeps
// their dw and db sums in registers over all the rows its CTA visits; a CTA's
// row slots are then added in shared memory in slot order, its sums go to
// global memory, and a second small kernel adds the CTAs' sums in CTA order.
// No atomics, so the result does not depend on the schedule.
//
// Bound by HBM: 3 e bytes per element, or 2 e + 1 from the codes.  The next
// row's loads are issued before the current row's reductions.
#include "layer_norm.cuh"

namespace fp8opt {

namespace {

// The saved side of a row: x, or the codes of xhat.
template <int DT, int VEC, bool FP8>
struct LnSaved {
  LnRaw<DT, VEC> x;
};
template <int DT>
struct LnSaved<DT, 8, true> {
  uint2 c;
};
template <int DT>
struct LnSaved<DT, 1, true> {
  uint8_t c[8];
};

template <int DT, int VEC, bool FP8, int TPR>
__device__ __forceinline__ LnSaved<DT, VEC, FP8> ln_load_saved(const LnBackward& a, int64_t r,
                                                              int v, int t, int cols) {
  LnSaved<DT, VEC, FP8> s;
  if constexpr (!FP8) {
    s.x = ln_load<DT, VEC, TPR>(
        static_cast<const char*>(a.x) + (size_t)r * a.cols * (DT == kF32 ? 4 : 2), v, t, cols);
  } else if constexpr (VEC == 8) {
    const int c = ln_col<TPR, 8>(v, 0, t);
    s.c = make_uint2(0, 0);
    if (c < cols) s.c = ld_once2(a.codes + r * a.cols + c);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<TPR, 1>(v, e, t);
      s.c[e] = c < cols ? a.codes[r * a.cols + c] : 0;
    }
  }
  return s;
}

// xhat of eight elements: (x - sub) * mul, with sub = mean and mul = rstd, or
// sub = 0 and mul = 1 / scale.
template <int DT, int VEC, bool FP8>
__device__ __forceinline__ void ln_xhat(const LnSaved<DT, VEC, FP8>& s, float sub, float mul,
                                        float* x) {
  if constexpr (!FP8) {
    ln_widen<DT, VEC>(s.x, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (x[e] - sub) * mul;
  } else {
    if constexpr (VEC == 8) {
      float d[8];
      dec8<kE4M3>(s.c, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = d[e] * mul;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = dec2<kE4M3>(s.c[e]).x * mul;
    }
  }
}

template <int DT, int VEC, int TPR, int VPT, int NT, int CTAS, bool FP8>
__global__ void __launch_bounds__(NT, CTAS)
ln_backward_kernel(const LnBackward a, float* __restrict__ partial) {
  constexpr int RPC = NT / TPR;
  __shared__ RowSums<TPR> sums[RPC];
  extern __shared__ float merge[];   // [2][cols], used when RPC > 1
  const int slot = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const int cols = (int)a.cols;
  const size_t es = DT == kF32 ? 4 : 2;
  const float inv_c = 1.0f / (float)cols;
  const int64_t step = (int64_t)gridDim.x * RPC;
  int turn = 0;

  float aw[8 * VPT], ab[8 * VPT];
#pragma unroll
  for (int i = 0; i < 8 * VPT; ++i) aw[i] = ab[i] = 0.0f;

  int64_t r = (int64_t)blockIdx.x * RPC + slot;
  LnRaw<DT, VEC> dy[VPT];
  LnSaved<DT, VEC, FP8> sv[VPT];
  float mul = 0.0f, sub = 0.0f, rstd = 0.0f;
  if (r < a.rows) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      dy[v] = ln_load<DT, VEC, TPR>(static_cast<const char*>(a.dy) + (size_t)r * a.cols * es, v,
                                    t, cols);
      sv[v] = ln_load_saved<DT, VEC, FP8, TPR>(a, r, v, t, cols);
    }
    rstd = __ldg(a.rstd + r);
    if (FP8) mul = __ldg(a.scales + r);
    else sub = __ldg(a.mean + r);
  }
  while (r < a.rows) {
    const int64_t rn = r + step;
    LnRaw<DT, VEC> dyn[VPT];
    LnSaved<DT, VEC, FP8> svn[VPT];
    float muln = 0.0f, subn = 0.0f, rstdn = 0.0f;
    if (rn < a.rows) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        dyn[v] = ln_load<DT, VEC, TPR>(static_cast<const char*>(a.dy) + (size_t)rn * a.cols * es,
                                       v, t, cols);
        svn[v] = ln_load_saved<DT, VEC, FP8, TPR>(a, rn, v, t, cols);
      }
      rstdn = __ldg(a.rstd + rn);
      if (FP8) muln = __ldg(a.scales + rn);
      else subn = __ldg(a.mean + rn);
    }
    // The values are made twice, before and after the reduction, from the raw
    // words: keeping them would take twice the registers.
    const float k = FP8 ? __fdiv_rn(1.0f, mul) : rstd;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float g[8], x[8], w[8];
      ln_widen<DT, VEC>(dy[v], g);
      ln_xhat<DT, VEC, FP8>(sv[v], sub, k, x);
      ln_param<VEC, TPR>(a.weight, a.wdtype, 0.0f, v, t, cols, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!ln_in<TPR, VEC>(v, e, t, cols)) x[e] = 0.0f;   // g is 0 there
        const float h = g[e] * w[e];
        s1 += h;
        s2 = __fmaf_rn(h, x[e], s2);
        aw[8 * v + e] = __fmaf_rn(g[e], x[e], aw[8 * v + e]);
        ab[8 * v + e] += g[e];
      }
    }
    const float2 s = row_sum2<TPR>(s1, s2, sums[slot], turn, slot);
    const float m1 = s.x * inv_c, m2 = s.y * inv_c;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float g[8], x[8], w[8];
      ln_widen<DT, VEC>(dy[v], g);
      ln_xhat<DT, VEC, FP8>(sv[v], sub, k, x);
      ln_param<VEC, TPR>(a.weight, a.wdtype, 0.0f, v, t, cols, w);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        g[e] = rstd * __fmaf_rn(-x[e], m2, __fmaf_rn(g[e], w[e], -m1));
      ln_store<DT, VEC, TPR>(static_cast<char*>(a.dx) + (size_t)r * a.cols * es, v, t, cols, g);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      dy[v] = dyn[v];
      sv[v] = svn[v];
    }
    mul = muln;
    sub = subn;
    rstd = rstdn;
    r = rn;
  }

  float* out = partial + (size_t)blockIdx.x * 2 * cols;
  for (int s = 0; s < RPC; ++s) {
    if (slot == s) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = ln_col<TPR, VEC>(v, e, t);
          if (c >= cols) continue;
          if (RPC == 1) {
            out[c] = aw[8 * v + e];
            out[cols + c] = ab[8 * v + e];
          } else if (s == 0) {
            merge[c] = aw[8 * v + e];
            merge[cols + c] = ab[8 * v + e];
          } else {
            merge[c] += aw[8 * v + e];
            merge[cols + c] += ab[8 * v + e];
          }
        }
    }
    if (RPC > 1) __syncthreads();
  }
  if (RPC > 1)
    for (int c = threadIdx.x; c < 2 * cols; c += NT) out[c] = merge[c];
}

// dw and db of 32 columns: the `parts` partial sums, 32 at a time, then the 32
// sums of this block, each in order.
__global__ void __launch_bounds__(1024)
ln_param_grad_kernel(const float* __restrict__ partial, int64_t parts, int64_t cols,
                     int wdtype, void* dw, void* db) {
  __shared__ float sh[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  void* out = blockIdx.y == 0 ? dw : db;
  float s = 0.0f;
  if (c < cols)
    for (int64_t p = threadIdx.y; p < parts; p += 32)
      s += __ldcg(partial + (p * 2 + blockIdx.y) * cols + c);
  sh[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // warp y adds column y of the block
  s = warp_sum(sh[threadIdx.x][threadIdx.y]);
  const int64_t at = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && at < cols && out != nullptr) {
    if (wdtype == kF32) store1<kF32>(out, at, s);
    else if (wdtype == kBF16) store1<kBF16>(out, at, s);
    else store1<kF16>(out, at, s);
  }
}

// ------------------------------------- rows too long for a CTA's registers

template <int DT, bool FP8>
__device__ __forceinline__ float long_xhat(const LnBackward& a, int64_t i, float sub, float k) {
  if (FP8) return dec2<kE4M3>(a.codes[i]).x * k;
  return (load1<DT>(a.x, i) - sub) * k;
}

template <int DT, bool FP8>
__global__ void __launch_bounds__(1024)
ln_backward_long_dx_kernel(const LnBackward a) {
  __shared__ float2 sh[32];
  const float inv_c = 1.0f / (float)a.cols;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const int64_t at = r * a.cols;
    const float rstd = a.rstd[r];
    const float sub = FP8 ? 0.0f : a.mean[r];
    const float k = FP8 ? __fdiv_rn(1.0f, a.scales[r]) : rstd;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float h = load1<DT>(a.dy, at + c) * ln_param1(a.weight, a.wdtype, c);
      s1 += h;
      s2 = __fmaf_rn(h, long_xhat<DT, FP8>(a, at + c, sub, k), s2);
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(s1, s2);
    __syncthreads();
    s1 = s2 = 0.0f;
    for (int i = 0; i < 32; ++i) {
      s1 += sh[i].x;
      s2 += sh[i].y;
    }
    const float m1 = s1 * inv_c, m2 = s2 * inv_c;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float h = load1<DT>(a.dy, at + c) * ln_param1(a.weight, a.wdtype, c);
      store1<DT>(a.dx, at + c,
                 rstd * __fmaf_rn(-long_xhat<DT, FP8>(a, at + c, sub, k), m2, h - m1));
    }
  }
}

// Partial dw and db of rows [y rows_per, (y + 1) rows_per), one thread a column.
template <int DT, bool FP8>
__global__ void __launch_bounds__(256)
ln_backward_long_cols_kernel(const LnBackward a, int64_t rows_per, float* __restrict__ partial) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  const int64_t r1 = min(a.rows, (int64_t)(blockIdx.y + 1) * rows_per);
  float sw = 0.0f, sb = 0.0f;
  for (int64_t r = (int64_t)blockIdx.y * rows_per; r < r1; ++r) {
    const float k = FP8 ? __fdiv_rn(1.0f, __ldg(a.scales + r)) : __ldg(a.rstd + r);
    const float sub = FP8 ? 0.0f : __ldg(a.mean + r);
    const float g = load1<DT>(a.dy, r * a.cols + c);
    sw = __fmaf_rn(g, long_xhat<DT, FP8>(a, r * a.cols + c, sub, k), sw);
    sb += g;
  }
  float* out = partial + (size_t)blockIdx.y * 2 * a.cols;
  out[c] = sw;
  out[a.cols + c] = sb;
}

constexpr int kLongParts = 16;   // row ranges of the long rows' dw and db

// Rows a CTA visits at a time, and how many CTAs run, for the kernel that
// by_cols() picks.
struct Shape {
  int rpc, nt, ctas;
};
Shape shape_of(int64_t cols) {
  if (cols <= 1024) return {8, 256, 2};
  if (cols <= 2048) return {2, 256, 2};
  if (cols <= 4096) return {1, 256, 2};
  return {1, 512, 1};
}

unsigned grid_of(const LnBackward& a, int sms) {
  const Shape s = shape_of(a.cols);
  const int64_t need = (a.rows + s.rpc - 1) / s.rpc, most = (int64_t)sms * s.ctas;
  return (unsigned)(need < most ? need : most);
}

template <int DT, int VEC, int TPR, int VPT, int NT, int CTAS>
void go(const LnBackward& a, float* partial, unsigned grid, cudaStream_t stream) {
  const size_t smem = NT / TPR > 1 ? 2 * sizeof(float) * (size_t)a.cols : 0;
  if (a.codes != nullptr)
    ln_backward_kernel<DT, VEC, TPR, VPT, NT, CTAS, true><<<grid, NT, smem, stream>>>(a, partial);
  else
    ln_backward_kernel<DT, VEC, TPR, VPT, NT, CTAS, false><<<grid, NT, smem, stream>>>(a, partial);
}

template <int DT, int VEC>
void by_cols(const LnBackward& a, float* p, unsigned grid, cudaStream_t s) {
  if (a.cols <= 256) go<DT, VEC, 32, 1, 256, 2>(a, p, grid, s);
  else if (a.cols <= 512) go<DT, VEC, 32, 2, 256, 2>(a, p, grid, s);
  else if (a.cols <= 1024) go<DT, VEC, 32, 4, 256, 2>(a, p, grid, s);
  else if (a.cols <= 2048) go<DT, VEC, 128, 2, 256, 2>(a, p, grid, s);
  else if (a.cols <= 4096) go<DT, VEC, 256, 2, 256, 2>(a, p, grid, s);
  else go<DT, VEC, 512, 2, 512, 1>(a, p, grid, s);
}

template <int DT>
int64_t by_type(const LnBackward& a, float* p, int sms, cudaStream_t s) {
  if (a.rows == 0) return 0;
  if (a.cols > kLnMaxRegColsBackward) {
    const unsigned grid = (unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms);
    const int64_t parts = a.rows < kLongParts ? a.rows : kLongParts;
    const int64_t rows_per = (a.rows + parts - 1) / parts;
    const dim3 cg((unsigned)((a.cols + 255) / 256), (unsigned)parts);
    if (a.codes != nullptr) {
      ln_backward_long_dx_kernel<DT, true><<<grid, 1024, 0, s>>>(a);
      ln_backward_long_cols_kernel<DT, true><<<cg, 256, 0, s>>>(a, rows_per, p);
    } else {
      ln_backward_long_dx_kernel<DT, false><<<grid, 1024, 0, s>>>(a);
      ln_backward_long_cols_kernel<DT, false><<<cg, 256, 0, s>>>(a, rows_per, p);
    }
    return parts;
  }
  const unsigned grid = grid_of(a, sms);
  if (a.vec_ok) by_cols<DT, 8>(a, p, grid, s);
  else by_cols<DT, 1>(a, p, grid, s);
  return grid;
}

}  // namespace

size_t ln_backward_scratch(const LnBackward& a, int sms) {
  if (a.rows == 0) return 0;
  const size_t parts = a.cols > kLnMaxRegColsBackward ? kLongParts : grid_of(a, sms);
  return parts * 2 * (size_t)a.cols * sizeof(float);
}

cudaError_t launch_ln_backward(const LnBackward& a, void* scratch, int sms, cudaStream_t stream,
                               LaunchMark mark) {
  float* p = static_cast<float*>(scratch);
  if (mark) mark(kLayerNormBackwardK, 0, stream);
  int64_t parts = 0;
  if (a.dtype == kF32) parts = by_type<kF32>(a, p, sms, stream);
  else if (a.dtype == kBF16) parts = by_type<kBF16>(a, p, sms, stream);
  else parts = by_type<kF16>(a, p, sms, stream);
  if (mark) mark(kLayerNormBackwardK, 1, stream);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (mark) mark(kLayerNormParamsK, 0, stream);
  ln_param_grad_kernel<<<dim3((unsigned)((a.cols + 31) / 32), a.db != nullptr ? 2 : 1),
                         dim3(32, 32), 0, stream>>>(p, parts, a.cols, a.wdtype, a.dw, a.db);
  if (mark) mark(kLayerNormParamsK, 1, stream);
  return cudaGetLastError();
}

}  // namespace fp8opt
