// The gated residual after one sub-block of a DiT block and the modulated
// norm before the next (forward):
//   r = x + alpha gate_b (post_weight N_post(y)),  h = (1 + scale_b) (weight N(r)) + shift_b
//
// Memory bound: x and y are read once, r and h written once; between them
// are about 15 operations per value.  A row lives in registers from its
// loads to its stores, so both norms take their mean first and then the mean
// of the squared distances from it (no difference of large sums).  One wave
// takes a row where there are rows enough to fill the chip, so that its sums
// need no LDS and no barrier; a workgroup of four waves takes one where
// there are few, or more than 4096 channels.
#include "norm_dev.hpp"

namespace ft {

using namespace norm_dev;

namespace {

// Sum over the WPR waves of a row; `slot` is this sum's own LDS place.
template <int WPR>
__device__ __forceinline__ float row_sum(float x, float* slot, int wave) {
  x = lanes_sum<64>(x);
  if constexpr (WPR == 1) {
    return x;
  } else {
    if ((threadIdx.x & 63) == 0) slot[wave] = x;
    __syncthreads();
    float s = slot[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) s += slot[i];
    return s;
  }
}

// Mean (LAYER) and 1 / deviation of the C values v, zero past the row's end.
template <int WPR, int NV>
__device__ __forceinline__ void row_stats(const float (&v)[NV][8], const bool (&ok)[NV], int kind,
                                          float inv_c, float eps, float* slots, int wave,
                                          float& mean, float& rstd) {
  mean = 0.0f;
  if (kind == 2) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[i][e];
    mean = row_sum<WPR>(s, slots, wave) * inv_c;
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float qi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = v[i][e] - mean;
      qi = __builtin_fmaf(t, t, qi);
    }
    q += ok[i] ? qi : 0.0f;
  }
  rstd = 1.0f / __builtin_sqrtf(row_sum<WPR>(q, slots + 4, wave) * inv_c + eps);
}

// Y: 0 no y, 1 y as it is, 2 y normalized.  F32: the stream's type.
template <int WPR, int NV, int F32, int Y>
__global__ __launch_bounds__(256) void k_norm_fwd(const NormArgs a) {
  __shared__ float slots[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = WPR == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  if (row >= a.M) return;          // whole waves; with WPR > 1 the grid is exact
  const int nv = static_cast<int>(a.C >> 3);
  const int at = WPR == 1 ? lane : static_cast<int>(threadIdx.x);
  const int64_t row8 = row * nv;
  const int b = sample_of(a, static_cast<int>(row));
  const int64_t mod8 = b * (a.ld_mod >> 3);
  const float inv_c = 1.0f / static_cast<float>(a.C);

  bool ok[NV];
  Raw8<F32> xr[NV];
  Raw8<0> yr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c8 = at + i * 64 * WPR;
    ok[i] = c8 < nv;
    xr[i].zero();
    yr[i].zero();
    if (ok[i]) {
      xr[i].load(a.x, row8 + c8);
      if constexpr (Y > 0) yr[i].load(a.y, row8 + c8);
    }
  }
  float v[NV][8];
  float mean_y = 0.0f, rstd_y = 1.0f;
  if constexpr (Y > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = yr[i].get(e);
    if constexpr (Y == 2)
      row_stats<WPR>(v, ok, a.post_norm, inv_c, a.eps, slots, wave, mean_y, rstd_y);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c8 = at + i * 64 * WPR;
      if (!ok[i]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        continue;
      }
      const Raw8<0> w = factor(a.post_weight, c8, kOnes);
      const Raw8<0> g = factor(a.gate, mod8 + c8, kOnes);
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = Y == 2 ? (v[i][e] - mean_y) * rstd_y : v[i][e];
        o[e] = xr[i].get(e) + (a.alpha * g.get(e)) * (n * w.get(e));
      }
      // the norm reads r as it is held, rounded to the stream's type
      xr[i].set(o);
      xr[i].store(a.r, row8 + c8);
    }
  } else if (a.r) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (ok[i]) xr[i].store(a.r, row8 + at + i * 64 * WPR);
  }
  float mean = 0.0f, rstd = 1.0f;
  if (a.h) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = xr[i].get(e);
    row_stats<WPR>(v, ok, a.norm, inv_c, a.eps, slots + 8, wave, mean, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c8 = at + i * 64 * WPR;
      if (!ok[i]) continue;
      const Raw8<0> w = factor(a.weight, c8, kOnes);
      const Raw8<0> sc = factor(a.scale, mod8 + c8, 0u);
      const Raw8<0> sh = factor(a.shift, mod8 + c8, 0u);
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = __builtin_fmaf((v[i][e] - mean) * rstd * w.get(e), 1.0f + sc.get(e), sh.get(e));
      Raw8<0> out;
      out.set(o);
      out.store(a.h, row8 + c8);
    }
  }
  if (a.stats && at == 0)
    reinterpret_cast<f32x4*>(a.stats)[row] = f32x4{mean, rstd, mean_y, rstd_y};
}

template <int WPR, int NV>
hipError_t go(const NormArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(WPR == 1 ? (a.M + 3) / 4 : a.M));
  const int y = !a.y ? 0 : a.post_norm == 0 ? 1 : 2;
#define FT_NF(F, Y) hipLaunchKernelGGL((k_norm_fwd<WPR, NV, F, Y>), grid, dim3(256), 0, st, a)
  if (a.f32) { if (y == 0) FT_NF(1, 0); else if (y == 1) FT_NF(1, 1); else FT_NF(1, 2); }
  else { if (y == 0) FT_NF(0, 0); else if (y == 1) FT_NF(0, 1); else FT_NF(0, 2); }
#undef FT_NF
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  const int nv = static_cast<int>(a.C >> 3);
  if (a.M >= 1024 && nv <= 512) {
    if (nv <= 64) return go<1, 1>(a, st);
    if (nv <= 128) return go<1, 2>(a, st);
    if (nv <= 256) return go<1, 4>(a, st);
    if (nv <= 384) return go<1, 6>(a, st);
    return go<1, 8>(a, st);
  }
  if (nv <= 256) return go<4, 1>(a, st);
  if (nv <= 512) return go<4, 2>(a, st);
  if (nv <= 1024) return go<4, 4>(a, st);
  return go<4, 8>(a, st);
}

}  // namespace ft
