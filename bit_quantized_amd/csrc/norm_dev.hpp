// Shared by the kernels of the gated residual and modulated norm (norm.hip,
// norm_bwd.hip) and of the rotation (rope.hip): cross-lane sums, vectors of
// eight values in bf16 or fp32, and the sample a row belongs to.
#pragma once

#include "ft_device.hpp"
#include "ft_kernels.h"

namespace ft {
namespace norm_dev {

// One DPP step: the value of another lane of the same 16.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
      0, static_cast<int>(__float_as_uint(x)), CTRL, 0xF, 0xF, true)));
}
// Sum over each aligned group of N lanes (a power of two up to 64), in every
// lane of it: quad permutes, mirrors of 8 and 16 lanes, then lane exchanges.
// The order is fixed.
template <int N>
__device__ __forceinline__ float lanes_sum(float x) {
  if constexpr (N >= 2) x += dpp<0xB1>(x);    // lane ^ 1
  if constexpr (N >= 4) x += dpp<0x4E>(x);    // lane ^ 2
  if constexpr (N >= 8) x += dpp<0x141>(x);   // mirrored in 8: the other quad
  if constexpr (N >= 16) x += dpp<0x140>(x);  // mirrored in 16: the other half
  if constexpr (N >= 32) x += __shfl_xor(x, 16);
  if constexpr (N >= 64) x += __shfl_xor(x, 32);
  return x;
}
// Eight values as they lie in memory: bf16 (F32 = 0) or fp32 (1).
template <int F32>
struct Raw8;
template <>
struct Raw8<0> {
  u32x4 w;
  __device__ __forceinline__ void load(const void* p, int64_t i8) {
    w = reinterpret_cast<const u32x4*>(p)[i8];
  }
  __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int e) const {
    return (e & 1) ? bf16hi_to_f32(w[e >> 1]) : bf16lo_to_f32(w[e >> 1]);
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = cvt_pk_bf16(f[2 * e], f[2 * e + 1]);
  }
  __device__ __forceinline__ void store(void* p, int64_t i8) const {
    reinterpret_cast<u32x4*>(p)[i8] = w;
  }
};
template <>
struct Raw8<1> {
  u32x4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i8) {
    a = reinterpret_cast<const u32x4*>(p)[2 * i8];
    b = reinterpret_cast<const u32x4*>(p)[2 * i8 + 1];
  }
  __device__ __forceinline__ void zero() { a = b = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e < 4 ? a[e & 3] : b[e & 3]);
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = __float_as_uint(f[e]);
      b[e] = __float_as_uint(f[4 + e]);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i8) const {
    reinterpret_cast<u32x4*>(p)[2 * i8] = a;
    reinterpret_cast<u32x4*>(p)[2 * i8 + 1] = b;
  }
};
// An optional bf16 row factor; a missing one reads as `none`.
__device__ __forceinline__ Raw8<0> factor(const uint16_t* p, int64_t i8, uint32_t none) {
  Raw8<0> v;
  if (p) v.load(p, i8);
  else v.w = u32x4{none, none, none, none};
  return v;
}
constexpr uint32_t kOnes = 0x3F803F80u;   // two bf16 1.0

// The sample of a row: the last one that starts at or before it, the first
// for rows before all.
__device__ __forceinline__ int sample_of(const NormArgs& a, int row) {
  if (a.n_seg == 1) return 0;
  if (!a.seg) return row / a.rows_per_seg;
  int lo = 0, hi = a.n_seg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.seg[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// Rows [first, last) of sample b, inside [0, M): with sample_of, every row is
// in exactly one of them if the offsets ascend.
__device__ __forceinline__ int sample_first(const NormArgs& a, int b) {
  if (b <= 0) return 0;
  if (b >= a.n_seg) return static_cast<int>(a.M);
  if (!a.seg) return b * a.rows_per_seg;
  const int s = a.seg[b];
  return s < 0 ? 0 : s > a.M ? static_cast<int>(a.M) : s;
}

}  // namespace norm_dev
}  // namespace ft
