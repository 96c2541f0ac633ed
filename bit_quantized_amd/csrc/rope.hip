// Rotary positions with several axes on query and key heads, with an
// optional RMS norm of each head before the rotation, forward and backward:
//   t = w x rstd,  rstd = 1 / sqrt(mean(x^2) + eps);   out = R t
//   backward: u = R^T d;  dw = sum u x rstd;
//             dx = rstd (w u - n mean(w u n)),  n = x rstd
//
// Memory bound: every head is read and written once.  A head is D / 8 lanes
// with eight values each, rounded up to a power of two, so a wave holds
// 64 / LPH heads of one row, and a lane's pairs are the same for every head
// of the row: their sines and cosines are computed once per row, from the
// position and the table of frequencies in the launch's arguments (no table
// in memory to read), while the first heads are on their way.  A lane's
// eight values are four whole pairs in either layout: one 16-byte piece, or
// two of 8 bytes a half apart, so no lane needs another's values but for the
// norm's sum.  The angle is taken in turns, p * (hi + lo) with the fraction of
// p * hi exact, because the hardware's sine and cosine take turns; at
// position 2^24 the angle is still good to 2^-20 of a turn.
//
// Measured with norms, 24 query and 24 key heads of 128 at 4608 rows: forward
// 24 us (4.7 TB/s), backward 33 us (5.1 TB/s) and 4 us for the norm weights'
// sums; 16380 rows of 16 and 4 heads in halves layout 37 us (4.5 TB/s).
#include <algorithm>

#include "norm_dev.hpp"

namespace ft {

using namespace norm_dev;

namespace {

constexpr int kWaves = 4;

// sin and cos of position p times the frequency hi + lo (turns).  No
// contraction: r - rint(r) taken as one fused operation on p * hi would hold
// the rounding error e of r already.
__device__ __forceinline__ void turn(float p, float hi, float lo, float& s, float& c) {
#pragma clang fp contract(off)
  const float r = p * hi;
  const float e = __builtin_fmaf(p, hi, -r);
  const float f = (r - __builtin_rintf(r)) + __builtin_fmaf(p, lo, e);
  s = __builtin_amdgcn_sinf(f);
  c = __builtin_amdgcn_cosf(f);
}

// Eight values of a head: at a0 .. +7 (PAIRS), or at a0 .. +3 and a1 .. +3.
template <bool HALVES>
__device__ __forceinline__ Raw8<0> load8(const uint16_t* p, int a0, int a1) {
  Raw8<0> v;
  if constexpr (HALVES) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p + a0), y = *reinterpret_cast<const u32x2*>(p + a1);
    v.w = u32x4{x[0], x[1], y[0], y[1]};
  } else {
    v.w = *reinterpret_cast<const u32x4*>(p + a0);
  }
  return v;
}
template <bool HALVES>
__device__ __forceinline__ void store8(uint16_t* p, int a0, int a1, const Raw8<0>& v) {
  if constexpr (HALVES) {
    *reinterpret_cast<u32x2*>(p + a0) = u32x2{v.w[0], v.w[1]};
    *reinterpret_cast<u32x2*>(p + a1) = u32x2{v.w[2], v.w[3]};
  } else {
    *reinterpret_cast<u32x4*>(p + a0) = v.w;
  }
}

// LPH lanes per head.  BWD: the transposed rotation, and the norm's gradient.
template <int LPH, bool HALVES, bool BWD>
__global__ __launch_bounds__(kWaves * 64) void k_rope(const RopeArgs a, int rows_per_wave,
                                                       int head_splits) {
  constexpr int HPW = 64 / LPH;          // heads of a wave
  constexpr int UN = 2;                  // heads in flight per lane (3 and 4: fewer waves, slower)
  __shared__ float dwl[BWD ? kWaves * 2 * LPH * 8 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int vec = lane % LPH, hsub = lane / LPH;
  const int D = a.t.D, np = a.t.n_pairs;
  const bool in_head = vec * 8 < D;
  const bool turned = vec * 4 < np;      // the lane's four pairs (the last lane's may be fewer)
  // where the lane's values lie; those past the pairs are eight in a row
  const int a0 = !HALVES ? 8 * vec : turned ? 4 * vec : 8 * vec;
  const int a1 = turned ? np + 4 * vec : 8 * vec + 4;
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.0f;
  const float inv_d = 1.0f / static_cast<float>(D);
  float hi[4], lo[4];
  int ax[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = vec * 4 + i;
    const bool has = j < np;
    hi[i] = has ? a.t.turn_hi[has ? j : 0] : 0.0f;
    lo[i] = has ? a.t.turn_lo[has ? j : 0] : 0.0f;
    ax[i] = has ? a.t.axis[has ? j : 0] : 0;
  }
  Raw8<0> wt[2];
#pragma unroll
  for (int si = 0; si < 2; ++si) {
    wt[si].w = u32x4{kOnes, kOnes, kOnes, kOnes};
    if (a.side[si].weight && in_head) wt[si] = load8<HALVES>(a.side[si].weight, a0, a1);
  }
  const int step = HPW * head_splits;

  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * rows_per_wave;
  const int64_t row1 = min(row0 + rows_per_wave, a.M);
  for (int64_t row = row0; row < row1; ++row) {
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pos[i] = a.pos[row * a.t.n_axes + ax[i]];
    float sn[4], cs[4];
    bool have = false;
#pragma unroll
    for (int si = 0; si < 2; ++si) {
      const RopeSide& s = a.side[si];
      const bool norm = s.weight != nullptr;
      const uint16_t* in = s.in + row * s.ld_in;
      const uint16_t* xin = s.x + row * s.ld_x;
      uint16_t* outp = s.out + row * s.ld_out;
      for (int h0 = static_cast<int>(blockIdx.y) * HPW; h0 < s.heads; h0 += step * UN) {
        Raw8<0> v[UN], xv[UN];
        bool ok[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          const int h = h0 + u * step + hsub;
          ok[u] = in_head && h < s.heads;
          v[u].zero();
          xv[u].zero();
          if (ok[u]) {
            v[u] = load8<HALVES>(in + static_cast<int64_t>(h) * D, a0, a1);
            if (BWD && norm) xv[u] = load8<HALVES>(xin + static_cast<int64_t>(h) * D, a0, a1);
          }
        }
        if (!have) {
          have = true;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            turn(static_cast<float>(pos[i]), hi[i], lo[i], sn[i], cs[i]);
            if (BWD) sn[i] = -sn[i];
          }
        }
        // the rotation of a lane's four pairs
        auto rotate = [&](float(&t)[8]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int p = HALVES ? i : 2 * i, q = HALVES ? i + 4 : 2 * i + 1;
            const float x = t[p], y = t[q];
            t[p] = x * cs[i] - y * sn[i];
            t[q] = __builtin_fmaf(x, sn[i], y * cs[i]);
          }
        };
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          if (h0 + u * step >= s.heads) break;       // uniform
          float t[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] = v[u].get(e);
          if constexpr (!BWD) {
            if (norm) {
              float q = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) q = __builtin_fmaf(t[e], t[e], q);
              const float rstd = 1.0f / __builtin_sqrtf(lanes_sum<LPH>(q) * inv_d + a.eps);
#pragma unroll
              for (int e = 0; e < 8; ++e) t[e] = t[e] * rstd * wt[si].get(e);
            }
            rotate(t);
          } else {
            rotate(t);
            if (norm) {
              float q = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) q = __builtin_fmaf(xv[u].get(e), xv[u].get(e), q);
              const float rstd = 1.0f / __builtin_sqrtf(lanes_sum<LPH>(q) * inv_d + a.eps);
              float m = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float n = xv[u].get(e) * rstd;
                dw[si][e] = __builtin_fmaf(t[e], n, dw[si][e]);
                t[e] *= wt[si].get(e);
                m = __builtin_fmaf(t[e], n, m);
              }
              m = lanes_sum<LPH>(m) * inv_d;
#pragma unroll
              for (int e = 0; e < 8; ++e) t[e] = rstd * (t[e] - xv[u].get(e) * rstd * m);
            }
          }
          if (ok[u]) {
            Raw8<0> o;
            o.set(t);
            store8<HALVES>(outp + static_cast<int64_t>(h0 + u * step + hsub) * D, a0, a1, o);
          }
        }
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    // the heads of a wave, then the waves, added in a fixed order
#pragma unroll
    for (int si = 0; si < 2; ++si)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = dw[si][e];
#pragma unroll
        for (int k = LPH; k < 64; k *= 2) v += __shfl_xor(v, k);
        const int at = HALVES ? (e < 4 ? a0 + e : a1 + e - 4) : a0 + e;
        if (hsub == 0 && in_head) dwl[(wave * 2 + si) * LPH * 8 + at] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kWaves * 64) {
      const int si = i / D, d = i % D;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += dwl[(w * 2 + si) * LPH * 8 + d];
      a.part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = v;
    }
  }
}

// The weights' gradients: the workgroups' sums added in a fixed order, 64
// threads for four values.
constexpr int kQuads = 4, kWays = 64;
__global__ __launch_bounds__(kQuads* kWays) void k_rope_reduce(const RopeArgs a, int n) {
  __shared__ f32x4 acc[kWays][kQuads];
  const int D = a.t.D;
  const int quad = threadIdx.x % kQuads, way = threadIdx.x / kQuads;
  const int i = (static_cast<int>(blockIdx.x) * kQuads + quad) * 4;      // 2 D is a multiple of 16
  f32x4 v = {0, 0, 0, 0};
#pragma unroll 8
  for (int g = way; g < n; g += kWays)
    v += *reinterpret_cast<const f32x4*>(a.part + static_cast<int64_t>(g) * 2 * D + i);
  acc[way][quad] = v;
  __syncthreads();
  if (threadIdx.x >= kQuads * 4) return;
  const int q = threadIdx.x / 4, e = threadIdx.x % 4;                    // one value each
  float s = 0.0f;
  for (int w = 0; w < kWays; ++w) s += acc[w][q][e];
  const int at = (static_cast<int>(blockIdx.x) * kQuads + q) * 4 + e;
  void* out = a.side[at / D].dweight;
  if (!out) return;
  if (a.grad_f32) static_cast<float*>(out)[at % D] = s;
  else static_cast<uint16_t*>(out)[at % D] = static_cast<uint16_t>(cvt_pk_bf16(s, 0.0f));
}

// With weight gradients a wave walks several rows, so that at most 1024
// workgroups leave partial sums; without, where a grid of one row a wave would
// pass the 32 bits that its threads are counted in.
constexpr int64_t kMaxPart = 1024, kMaxWgs = 1 << 22;
int rows_per_wave(int64_t M, bool part) {
  const int64_t per = (part ? kMaxPart : kMaxWgs) * kWaves;
  return static_cast<int>((M + per - 1) / per);
}

template <int LPH>
hipError_t go(const RopeArgs& a, bool bwd, hipStream_t st) {
  const int rpw = std::max(1, rows_per_wave(a.M, a.part != nullptr));
  const uint32_t wgs = static_cast<uint32_t>((a.M + kWaves * rpw - 1) / (kWaves * rpw));
  if (wgs > 0) {
    // few rows: the heads of a row are divided over workgroups
    const int hpw = 64 / LPH;
    const int groups = (std::max(a.side[0].heads, a.side[1].heads) + hpw - 1) / hpw;
    const int splits = a.part || wgs >= 512 ? 1 : std::max(1, std::min<int>(groups, static_cast<int>(1024 / wgs)));
    const dim3 grid(wgs, static_cast<uint32_t>(splits));
#define FT_RO(H, B) hipLaunchKernelGGL((k_rope<LPH, H, B>), grid, dim3(kWaves * 64), 0, st, a, rpw, splits)
    if (a.t.layout) { if (bwd) FT_RO(true, true); else FT_RO(true, false); }
    else { if (bwd) FT_RO(false, true); else FT_RO(false, false); }
#undef FT_RO
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!a.part) return hipSuccess;
  hipLaunchKernelGGL(k_rope_reduce, dim3(2 * a.t.D / (4 * kQuads)), dim3(kQuads * kWays), 0, st, a,
                     static_cast<int>(wgs));
  return hipGetLastError();
}

}  // namespace

size_t rope_part_bytes(int64_t M, int D) {
  const int64_t rpw = std::max(1, rows_per_wave(M, true));
  return static_cast<size_t>((M + kWaves * rpw - 1) / (kWaves * rpw)) * 2 * D * sizeof(float);
}

hipError_t launch_rope(const RopeArgs& a, bool bwd, hipStream_t st) {
  const int v = a.t.D / 8;
  if (v <= 8) return go<8>(a, bwd, st);
  if (v <= 16) return go<16>(a, bwd, st);
  return go<32>(a, bwd, st);
}

}  // namespace ft
