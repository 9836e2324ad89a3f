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
// Bound by HBM, 3 e bytes per element, or 2 e + 1 from the codes, and close
// behind by instructions (63% of the issue slots).  The coming rows' copies run
// through a ring in shared memory: held in registers, two rows ahead was all
// there was room for, and a 16381 x 2048 gradient from codes took 57 us; now
// 35.0 us, 4.79 TB/s, 0.71 of the measured copy bandwidth; 65536 x 1024 from x:
// 0.82.  With the row slots' sums added one slot after the other the end of a
// CTA alone took 30 us; side by side it is one pass.
// Rows that start anywhere, from x (by elements): 32768 x 1501 83 us, 0.52 (183),
// 32768 x 2041 84 us (237), 32768 x 2049 161 us (301).
#include "layer_norm.cuh"

namespace fp8opt {

namespace {

// Threads of an SM (128 registers each), in one or two CTAs: each CTA writes
// one pair of partial sums.
constexpr int kBwdThreads = 512;

// Bytes of a vector of eight elements: of dy (and x), and of the saved side.
template <int DT>
constexpr int kVecBytes = DT == kF32 ? 32 : 16;
template <int DT, bool FP8>
constexpr int kSavedBytes = FP8 ? 8 : kVecBytes<DT>;
template <int DT>
constexpr int kStages = DT == kF32 ? 3 : 4;

template <int DT, int VPT, int NT, bool FP8>
constexpr int kRingBytes = kStages<DT> * VPT * NT * (kVecBytes<DT> + kSavedBytes<DT, FP8>);

// xhat of eight elements: (x - sub) * mul, with sub = mean and mul = rstd, or
// the code's value * mul with mul = 1 / scale.
template <bool FP8>
__device__ __forceinline__ void ln_xhat(const float* x, float sub, float mul, float2* out) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    out[j] = make_float2(x[2 * j], x[2 * j + 1]);
    if (!FP8) out[j] = add2(out[j], splat2(-sub));
    out[j] = mul2(out[j], splat2(mul));
  }
}

template <int DT, int VEC, int TPR, int VPT, int NT, bool FP8, bool FULL>
__global__ void __launch_bounds__(NT, kBwdThreads / NT)
ln_backward_kernel(const LnBackward a, float* __restrict__ partial) {
  constexpr int RPC = NT / TPR, ST = kStages<DT>, Q = DT == kF32 ? 2 : 1;
  __shared__ RowSums<TPR> sums[RPC];
  // the ring: dy [ST][VPT][Q][NT] of 16 bytes, then x alike or the codes
  // [ST][VPT][NT] of 8; afterwards the row slots' sums [RPC][2][cols]
  extern __shared__ uint4 ring[];
  const int slot = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const int cols = (int)a.cols;
  const size_t es = DT == kF32 ? 4 : 2;
  const float inv_c = 1.0f / (float)cols;
  const int64_t step = (int64_t)gridDim.x * RPC;
  int turn = 0;
  begin_after_previous();

  const auto at_dy = [&](int stage, int v, int q) -> uint4* {
    return ring + ((stage * VPT + v) * Q + q) * NT + threadIdx.x;
  };
  uint4* const ring2 = ring + ST * VPT * Q * NT;
  const auto at_x = [&](int stage, int v, int q) -> uint4* {
    return ring2 + ((stage * VPT + v) * Q + q) * NT + threadIdx.x;
  };
  const auto at_code = [&](int stage, int v) -> uint2* {
    return reinterpret_cast<uint2*>(ring2) + (stage * VPT + v) * NT + threadIdx.x;
  };
  int64_t r = (int64_t)blockIdx.x * RPC + slot;
  const int shift = VEC == kLnFlat ? (int)(r * a.cols & 7) : 0, end = cols + shift;
  const auto fetch = [&](int stage, int64_t row) {
    if (row < a.rows) {
      const size_t at = (size_t)row * a.cols - shift;
      const int left = VEC == kLnFlat ? ln_left(a.rows - row, a.cols, shift) : 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = ln_col<TPR, 8>(v, 0, t);
        if (!FULL && c >= end) continue;
        if constexpr (VEC == kLnFlat) {
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const int n = ln_bytes(left - c, (int)es, 16 * q, 16);
            const size_t off = (at + c) * es + 16 * q;
            if (n <= 0) continue;
            copy_async<16>(at_dy(stage, v, q), static_cast<const char*>(a.dy) + off, n);
            if (!FP8) copy_async<16>(at_x(stage, v, q), static_cast<const char*>(a.x) + off, n);
          }
          if (FP8) copy_async<8>(at_code(stage, v), a.codes + at + c, ln_bytes(left - c, 1, 0, 8));
        } else {
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const size_t off = (at + c) * es + 16 * q;
            copy_async<16>(at_dy(stage, v, q), static_cast<const char*>(a.dy) + off);
            if (!FP8) copy_async<16>(at_x(stage, v, q), static_cast<const char*>(a.x) + off);
          }
          if (FP8) copy_async<8>(at_code(stage, v), a.codes + at + c);
        }
      }
    }
    copy_commit();
  };

  float2 w[4 * VPT], aw[4 * VPT], ab[4 * VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    float p[8];
    if constexpr (VEC == kLnFlat)
      ln_param_flat<TPR>(a.weight, a.wdtype, v, t, shift, end, p);
    else
      ln_param<VEC, TPR>(a.weight, a.wdtype, 0.0f, v, t, cols, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[4 * v + j] = make_float2(p[2 * j], p[2 * j + 1]);
      aw[4 * v + j] = ab[4 * v + j] = make_float2(0.0f, 0.0f);
    }
  }

  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < ST; ++i)   // what lies past the row's end stays zero
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (!ln_in<TPR, 8, FULL>(v, 0, t, cols)) {
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            *at_dy(i, v, q) = make_uint4(0, 0, 0, 0);
            if (!FP8) *at_x(i, v, q) = make_uint4(0, 0, 0, 0);
          }
          if (FP8) *at_code(i, v) = make_uint2(0, 0);
        }
  }
  if constexpr (VEC != 1) {
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(i, r + i * step);
  }
  // a row's rstd, and its mean or scale, are read one row ahead
  const float* const other = FP8 ? a.scales : a.mean;
  float rstd_next = 0.0f, other_next = 1.0f;
  if (r < a.rows) {
    rstd_next = __ldca(a.rstd + r);
    other_next = __ldca(other + r);
  }
  for (int stage = 0; r < a.rows; r += step, stage = stage + 1 == ST ? 0 : stage + 1) {
    const float rstd = rstd_next;
    const float sub = FP8 ? 0.0f : other_next;
    const float mul = FP8 ? __fdiv_rn(1.0f, other_next) : rstd;
    if (r + step < a.rows) {
      rstd_next = __ldca(a.rstd + r + step);
      other_next = __ldca(other + r + step);
    }
    if constexpr (VEC != 1) copy_wait<ST - 2>();
    float2 g[4 * VPT], x[4 * VPT];
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float d[8], e[8];
      if (VEC == kLnFlat && ln_col<TPR, 8>(v, 0, t) >= end) {
#pragma unroll
        for (int j = 0; j < 4; ++j) g[4 * v + j] = x[4 * v + j] = splat2(0.0f);
        continue;
      }
      if constexpr (VEC != 1) {
        LnRaw<DT, 8> raw;
#pragma unroll
        for (int q = 0; q < Q; ++q) raw.v[q] = *at_dy(stage, v, q);
        ln_widen<DT, 8>(raw, d);
        if constexpr (FP8) {
          dec8<kE4M3>(*at_code(stage, v), e);
        } else {
#pragma unroll
          for (int q = 0; q < Q; ++q) raw.v[q] = *at_x(stage, v, q);
          ln_widen<DT, 8>(raw, e);
        }
      } else {
        const size_t at = (size_t)r * a.cols;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = ln_col<TPR, 1>(v, k, t);
          d[k] = e[k] = 0.0f;
          if (c < cols) {
            d[k] = load1<DT>(a.dy, at + c);
            e[k] = FP8 ? dec2<kE4M3>(a.codes[at + c]).x : load1<DT>(a.x, at + c);
          }
        }
      }
      ln_xhat<FP8>(e, sub, mul, x + 4 * v);
      if constexpr (VEC == kLnFlat) {
        const int c = ln_col<TPR, 8>(v, 0, t);
        ln_mask(d, c, shift, end);
        ln_mask(x + 4 * v, c, shift, end);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * v + j;
        g[i] = make_float2(d[2 * j], d[2 * j + 1]);
        // past the row's end dy is 0, and xhat must not be a NaN there
        if constexpr (VEC != kLnFlat) {
          if (!ln_in<TPR, VEC, FULL>(v, 2 * j, t, cols)) x[i].x = 0.0f;
          if (!ln_in<TPR, VEC, FULL>(v, 2 * j + 1, t, cols)) x[i].y = 0.0f;
        }
        aw[i] = fma2(g[i], x[i], aw[i]);
        ab[i] = add2(ab[i], g[i]);
        g[i] = mul2(g[i], w[i]);
        s1 = add2(s1, g[i]);
        s2 = fma2(g[i], x[i], s2);
      }
    }
    if constexpr (VEC != 1) fetch(stage == 0 ? ST - 1 : stage - 1, r + (ST - 1) * step);
    const float2 s = row_reduce<kTwo, TPR>(s1.x + s1.y, s2.x + s2.y, sums[slot], turn, slot);
    const float2 m1 = splat2(-s.x * inv_c), m2 = splat2(-s.y * inv_c), k = splat2(rstd);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float d[8];
      if (VEC == kLnFlat && ln_col<TPR, 8>(v, 0, t) >= end) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = mul2(k, fma2(x[4 * v + j], m2, add2(g[4 * v + j], m1)));
        d[2 * j] = y.x;
        d[2 * j + 1] = y.y;
      }
      char* const out = static_cast<char*>(a.dx) + (size_t)r * a.cols * es;
      if constexpr (VEC == kLnFlat) ln_store_flat<DT, TPR>(out, v, t, shift, end, d);
      else ln_store<DT, VEC, TPR>(out, v, t, cols, d);
    }
  }

  // The CTA's sums: the row slots side by side in shared memory (the ring is
  // drained first), then added in slot order.
  float* const out = partial + (size_t)blockIdx.x * 2 * cols;
  float* const merge = reinterpret_cast<float*>(ring);
  if (RPC > 1) {
    copy_wait<0>();
    __syncthreads();
  }
  float* const mine = RPC > 1 ? merge + slot * 2 * cols : out;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const float2* s[2] = {aw + 4 * v, ab + 4 * v};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* p = mine + h * cols;
      if constexpr (VEC == 8) {
        const int c = ln_col<TPR, 8>(v, 0, t);
        if (c < cols) {
          float4* q = reinterpret_cast<float4*>(p + c);
          q[0] = make_float4(s[h][0].x, s[h][0].y, s[h][1].x, s[h][1].y);
          q[1] = make_float4(s[h][2].x, s[h][2].y, s[h][3].x, s[h][3].y);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = ln_col<TPR, VEC>(v, j, t) - shift;
          if (c >= 0 && c < cols) p[c] = (j & 1) ? s[h][j / 2].y : s[h][j / 2].x;
        }
      }
    }
  }
  if (RPC > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * cols; c += NT) {
      float v = merge[c];
#pragma unroll
      for (int i = 1; i < RPC; ++i) v += merge[i * 2 * cols + c];
      out[c] = v;
    }
  }
}

// dw and db of 32 columns: the `parts` partial sums, 32 at a time, then the 32
// sums of this block, each in order.
__global__ void __launch_bounds__(1024)
ln_param_grad_kernel(const float* partial, int64_t parts, int64_t cols,
                     int wdtype, void* dw, void* db) {
  __shared__ float sh[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  void* out = blockIdx.y == 0 ? dw : db;
  float s = 0.0f;
  begin_after_previous();
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
  begin_after_previous();
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
  begin_after_previous();
  if (c >= a.cols) return;
  const int64_t r1 = min(a.rows, (int64_t)(blockIdx.y + 1) * rows_per);
  float sw = 0.0f, sb = 0.0f;
  for (int64_t r = (int64_t)blockIdx.y * rows_per; r < r1; ++r) {
    const float k = FP8 ? __fdiv_rn(1.0f, __ldca(a.scales + r)) : __ldca(a.rstd + r);
    const float sub = FP8 ? 0.0f : __ldca(a.mean + r);
    const float g = load1<DT>(a.dy, r * a.cols + c);
    sw = __fmaf_rn(g, long_xhat<DT, FP8>(a, r * a.cols + c, sub, k), sw);
    sb += g;
  }
  float* out = partial + (size_t)blockIdx.y * 2 * a.cols;
  out[c] = sw;
  out[a.cols + c] = sb;
}

constexpr int kLongParts = 16;   // row ranges of the long rows' dw and db

// Rows that a CTA of the kernel that by_cols() picks visits at a time.
int rows_per_cta(int64_t cols) {   // (cols: with the shift)
  return cols <= 512 ? 16 : cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
}

unsigned grid_of(const LnBackward& a, int sms) {
  const int64_t rpc = rows_per_cta(ln_span(a.cols, a.form));
  return (unsigned)ln_grid((a.rows + rpc - 1) / rpc, sms, a.form);
}

template <int DT, int VEC, int TPR, int VPT, bool FP8, bool FULL>
cudaError_t go_form(const LnBackward& a, float* partial, unsigned grid, cudaStream_t stream) {
  constexpr int NT = kBwdThreads, RPC = NT / TPR;
  auto kernel = ln_backward_kernel<DT, VEC, TPR, VPT, NT, FP8, FULL>;
  const int ring = VEC != 1 ? kRingBytes<DT, VPT, NT, FP8> : 0;
  const int merge = RPC > 1 ? RPC * 2 * (int)sizeof(float) * (int)a.cols : 0;
  const int smem = ring > merge ? ring : merge;
  if (smem > 47 * 1024) {   // with the static arrays beside it, above 48 KB
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch(worth_early(a.rows * a.cols), kernel, grid, NT, smem, stream, a, partial);
}

template <int DT, int VEC, int TPR, int VPT>
cudaError_t go(const LnBackward& a, float* p, unsigned grid, cudaStream_t s) {
  if constexpr (VEC == 8) {
    if (a.cols == TPR * VPT * 8)
      return a.codes != nullptr ? go_form<DT, VEC, TPR, VPT, true, true>(a, p, grid, s)
                                : go_form<DT, VEC, TPR, VPT, false, true>(a, p, grid, s);
  }
  return a.codes != nullptr ? go_form<DT, VEC, TPR, VPT, true, false>(a, p, grid, s)
                            : go_form<DT, VEC, TPR, VPT, false, false>(a, p, grid, s);
}

template <int DT, int VEC>
cudaError_t by_cols(const LnBackward& a, float* p, unsigned grid, cudaStream_t s) {
  const int64_t span = ln_span(a.cols, VEC);
  if (span <= 256) return go<DT, VEC, 32, 1>(a, p, grid, s);
  if (span <= 512) return go<DT, VEC, 32, 2>(a, p, grid, s);
  if (span <= 1024) return go<DT, VEC, 64, 2>(a, p, grid, s);
  if (span <= 2048) return go<DT, VEC, 128, 2>(a, p, grid, s);
  if (span <= 4096) return go<DT, VEC, 256, 2>(a, p, grid, s);
  return go<DT, VEC, 512, 2>(a, p, grid, s);
}

template <int DT>
cudaError_t by_type(const LnBackward& a, float* p, int sms, cudaStream_t s, int64_t* parts) {
  *parts = 0;
  if (a.rows == 0) return cudaSuccess;
  if (a.cols > kLnMaxRegCols) {
    const unsigned grid = (unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms);
    *parts = a.rows < kLongParts ? a.rows : kLongParts;
    const int64_t rows_per = (a.rows + *parts - 1) / *parts;
    const dim3 cg((unsigned)((a.cols + 255) / 256), (unsigned)*parts);
    const bool fp8 = a.codes != nullptr;
    const cudaError_t e = launch(true, fp8 ? ln_backward_long_dx_kernel<DT, true>
                                           : ln_backward_long_dx_kernel<DT, false>,
                                       grid, 1024, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch(true, fp8 ? ln_backward_long_cols_kernel<DT, true>
                            : ln_backward_long_cols_kernel<DT, false>,
                        cg, 256, 0, s, a, rows_per, p);
  }
  const unsigned grid = grid_of(a, sms);
  *parts = grid;
  if (a.form == kLnVectors) return by_cols<DT, 8>(a, p, grid, s);
  if (a.form == kLnFlat) return by_cols<DT, kLnFlat>(a, p, grid, s);
  return by_cols<DT, 1>(a, p, grid, s);
}

}  // namespace

size_t ln_backward_scratch(const LnBackward& a, int sms) {
  if (a.rows == 0) return 0;
  const size_t parts = a.cols > kLnMaxRegCols ? kLongParts : grid_of(a, sms);
  return parts * 2 * (size_t)a.cols * sizeof(float);
}

cudaError_t launch_ln_backward(const LnBackward& a, void* scratch, int sms, cudaStream_t stream,
                               LaunchMark mark) {
  float* p = static_cast<float*>(scratch);
  if (mark) mark(kLayerNormBackwardK, 0, stream);
  int64_t parts = 0;
  cudaError_t e = a.dtype == kF32    ? by_type<kF32>(a, p, sms, stream, &parts)
                  : a.dtype == kBF16 ? by_type<kBF16>(a, p, sms, stream, &parts)
                                     : by_type<kF16>(a, p, sms, stream, &parts);
  if (mark) mark(kLayerNormBackwardK, 1, stream);
  if (e != cudaSuccess) return e;
  if (mark) mark(kLayerNormParamsK, 0, stream);
  e = launch(true, ln_param_grad_kernel,
                   dim3((unsigned)((a.cols + 31) / 32), a.db != nullptr ? 2 : 1), dim3(32, 32), 0,
                   stream, (const float*)p, parts, a.cols, a.wdtype, a.dw, a.db);
  if (mark) mark(kLayerNormParamsK, 1, stream);
  return e;
}

}  // namespace fp8opt
