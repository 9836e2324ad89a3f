// Row ownership shared by the layer norm kernels.
//
// A row of C elements is held in the registers of TPR threads, 8 * VPT
// elements each, so that a row is read from HBM once however often its values
// are used.  VEC = 8: vector v of thread t holds elements [8 (v TPR + t), + 8)
// (C and the buffers allow 16-byte accesses); VEC = 1: its element e is number
// (8 v + e) TPR + t, so that neighbouring threads read neighbouring elements
// of rows that start anywhere.  VEC = kLnFlat: the vectors are those of the flat
// tensor; the first one of a row begins `shift` = (row C) mod 8 elements before
// the row, and the vectors at its ends are masked.  A CTA's row slots step by a
// multiple of 8 rows, so that shift, and with it what a thread holds of the
// parameters and their gradients, is the same for all rows of a slot.
#pragma once

#include "ops_internal.cuh"

namespace fp8opt {

template <int TPR, int VEC>
__device__ __forceinline__ int ln_col(int v, int e, int t) {
  return VEC != 1 ? (v * TPR + t) * 8 + e : (v * 8 + e) * TPR + t;
}

// Whether that element lies in the row (for VEC = 8 the whole vector does or
// does not).  FULL: the row fills its threads' registers, and every element
// does: the tests and selections were a tenth of the kernels' instructions,
// which is what bounds them beside HBM.
template <int TPR, int VEC, bool FULL>
__device__ __forceinline__ bool ln_in(int v, int e, int t, int cols) {
  return FULL || ln_col<TPR, VEC>(v, VEC == 8 ? 0 : e, t) < cols;
}

// kLnFlat: of the vector at c, counted from the first vector's start, the
// elements from shift to end = shift + C belong to the row.
__device__ __forceinline__ void ln_mask(float* x, int c, int shift, int end) {
  if (c < shift || c + 8 > end) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < shift || c + e >= end) x[e] = 0.0f;
  }
}

__device__ __forceinline__ void ln_mask(float2* x, int c, int shift, int end) {
  if (c < shift || c + 8 > end) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + 2 * e < shift || c + 2 * e >= end) x[e].x = 0.0f;
      if (c + 2 * e + 1 < shift || c + 2 * e + 1 >= end) x[e].y = 0.0f;
    }
  }
}

// Rows of one slot that are to have the same shift: CTAs of a launch of at most
// `most`, when some visit more than one row a slot.
inline int64_t ln_grid(int64_t ctas, int64_t most, int form) {
  if (form == kLnFlat && most >= 8) most &= ~(int64_t)7;
  return ctas < most ? ctas : most;
}

// Columns that the threads of a row have to hold.
inline int64_t ln_span(int64_t cols, int form) { return form == kLnFlat ? cols + 7 : cols; }

// Eight elements of vector v as raw words (VEC 8) or widened values (VEC 1);
// the elements past the row's end are zero.
template <int DT, int VEC>
struct LnRaw {
  uint4 v[DT == kF32 ? 2 : 1];
};
template <int DT>
struct LnRaw<DT, 1> {
  float f[8];
};

template <int DT, int VEC, int TPR>
__device__ __forceinline__ LnRaw<DT, VEC> ln_load(const void* row, int v, int t, int cols) {
  LnRaw<DT, VEC> r;
  if constexpr (VEC == 8) {
    const int c = ln_col<TPR, 8>(v, 0, t);
    const bool in = c < cols;
#pragma unroll
    for (int k = 0; k < (DT == kF32 ? 2 : 1); ++k) {
      r.v[k] = make_uint4(0, 0, 0, 0);
      if (in) r.v[k] = ld_once4(static_cast<const char*>(row) +
                                (int64_t)c * (DT == kF32 ? 4 : 2) + 16 * k);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<TPR, 1>(v, e, t);
      r.f[e] = c < cols ? load1<DT>(row, c) : 0.0f;
    }
  }
  return r;
}

template <int DT, int VEC>
__device__ __forceinline__ void ln_widen(const LnRaw<DT, VEC>& r, float* x) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int k = 0; k < (DT == kF32 ? 2 : 1); ++k) {
      const uint32_t w[4] = {r.v[k].x, r.v[k].y, r.v[k].z, r.v[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (DT == kF32) {
          x[4 * k + j] = __uint_as_float(w[j]);
        } else if (DT == kF16) {
          const float2 f = h2_to_f2(w[j]);
          x[2 * j] = f.x;
          x[2 * j + 1] = f.y;
        } else {
          x[2 * j] = __uint_as_float(w[j] << 16);
          x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = r.f[e];
  }
}

// Eight results of vector v to a row of DT.
template <int DT, int VEC, int TPR>
__device__ __forceinline__ void ln_store(void* row, int v, int t, int cols, const float* x) {
  if constexpr (VEC == 8) {
    const int c = ln_col<TPR, 8>(v, 0, t);
    if (c >= cols) return;
    char* p = static_cast<char*>(row) + (int64_t)c * (DT == kF32 ? 4 : 2);
    if constexpr (DT == kF32) {
      __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
      __stcs(reinterpret_cast<uint4*>(p),
             make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]),
                        pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7])));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<TPR, 1>(v, e, t);
      if (c < cols) store1<DT>(row, c, x[e]);
    }
  }
}

// kLnFlat: the same to the row at `row` (elements of a row of another CTA lie
// in its end vectors).
template <int DT, int TPR>
__device__ __forceinline__ void ln_store_flat(char* row, int v, int t, int shift, int end,
                                              const float* x) {
  const int c = ln_col<TPR, 8>(v, 0, t);
  if (c >= shift && c + 8 <= end) {
    ln_store<DT, 8, TPR>(row - shift * (DT == kF32 ? 4 : 2), v, t, end, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= shift && c + e < end) store1<DT>(row, c + e - shift, x[e]);
  }
}

// One element of a parameter vector of any element type.
__device__ __forceinline__ float ln_param1(const void* p, int dtype, int64_t c) {
  return dtype == kF32 ? load1<kF32>(p, c)
       : dtype == kBF16 ? load1<kBF16>(p, c) : load1<kF16>(p, c);
}

// Eight elements of a parameter vector (the type is the same for the whole
// grid, so the branch is uniform); `missing` where there is none.
template <int VEC, int TPR>
__device__ __forceinline__ void ln_param(const void* p, int dtype, float missing, int v,
                                         int t, int cols, float* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = missing;
  if (p == nullptr) return;
  if constexpr (VEC == 8) {
    const int c = ln_col<TPR, 8>(v, 0, t);
    if (c >= cols) return;
    if (dtype == kF32) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + 1);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
      const uint4 a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + c));
      LnRaw<kF16, 8> r;
      r.v[0] = a;
      if (dtype == kF16) {
        ln_widen<kF16, 8>(r, x);
      } else {
        LnRaw<kBF16, 8> q;
        q.v[0] = a;
        ln_widen<kBF16, 8>(q, x);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<TPR, 1>(v, e, t);
      if (c < cols) x[e] = ln_param1(p, dtype, c);
    }
  }
}

// kLnFlat: the same of a thread's share of a row that begins at shift.
template <int TPR>
__device__ __forceinline__ void ln_param_flat(const void* p, int dtype, int v, int t, int shift,
                                              int end, float* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = ln_col<TPR, 8>(v, e, t);
    x[e] = c >= shift && c < end ? ln_param1(p, dtype, c - shift) : 0.0f;
  }
}

// ------------------------------------------------------------ the row ring
//
// With vectors a thread copies its own share of the coming rows into shared
// memory with cp.async, STAGES - 1 rows ahead, and reads back only what it
// copied itself, so the ring needs no barrier: HBM latency is covered by
// copies in flight instead of by registers or more threads.

template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* global) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(smem);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(global) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(global) : "memory");
}

// The first `bytes` of them, and zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* global, int bytes) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(smem);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(d), "l"(global), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                 ::"r"(d), "l"(global), "r"(bytes) : "memory");
}

// Elements from the start of the row's first vector to the tensor's end, where
// that matters (kLnFlat: the last vector ends where the tensor does).
__device__ __forceinline__ int ln_left(int64_t rows, int64_t cols, int shift) {
  return (int)min(rows * cols, (int64_t)1 << 20) + shift;
}

__device__ __forceinline__ int ln_bytes(int elements, int size, int skip, int most) {
  return min(max(elements * size - skip, 0), most);
}

__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Two sums over the TPR threads of a row, in a fixed order, for every one of
// them.  Rows of more than one warp meet at the row's own barrier, so the rows
// of a CTA run independently; the buffers alternate (turn), so one barrier per
// reduction is enough: a warp writes buffer b again only after the barrier of
// the reduction in between, which every warp passes after reading b.
template <int TPR>
struct RowSums {
  float2 w[2][TPR / 32];
};

template <int TPR>
__device__ __forceinline__ void row_barrier(int row_slot) {
  asm volatile("bar.sync %0, %1;" ::"r"(row_slot + 1), "n"(TPR) : "memory");
}

// A second sum (TWO), or a maximum beside the sum (MAX: of non-negative
// values, by their bits).
enum RowPair { kOne, kTwo, kMax };

template <RowPair KIND, int TPR>
__device__ __forceinline__ float2 row_reduce(float a, float b, RowSums<TPR>& s, int& turn,
                                             int row_slot) {
  a = warp_sum(a);
  if (KIND == kTwo) b = warp_sum(b);
  if (KIND == kMax) b = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(b)));
  if constexpr (TPR > 32) {
    const int t = threadIdx.x % TPR;
    if ((t & 31) == 0) s.w[turn][t >> 5] = make_float2(a, b);
    row_barrier<TPR>(row_slot);
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      const float2 w = s.w[turn][i];
      a += w.x;
      if (KIND == kTwo) b += w.y;
      if (KIND == kMax) b = fmaxf(b, w.y);
    }
    turn ^= 1;
  }
  return make_float2(a, b);
}

}  // namespace fp8opt
