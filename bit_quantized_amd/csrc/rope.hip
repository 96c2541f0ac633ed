// Rotary positions with several axes on query and key heads, with an
// optional RMS norm of each head before the rotation, forward and backward:
//   t = w x rstd,  rstd = 1 / sqrt(mean(x^2) + eps);   out = R t
//   backward: u = R^T d;  dw = sum u x rstd;
//             dx = rstd (w u - n mean(w u n)),  n = x rstd
//
// Memory bound: every head is read and written once.  A head is D / 8 lanes
// with eight values each (16-byte loads), rounded up to a power of two, so a
// wave holds 64 / LPH heads of one row, and a lane's pairs are the same for
// every head of the row: their sines and cosines are computed once per row,
// from the position and the table of frequencies in the launch's arguments
// (no table in memory to read).  The angle is taken in turns, p * (hi + lo)
// with the fraction of p * hi exact, because the hardware's sine and cosine
// take turns; at position 2^24 the angle is still good to 2^-20 of a turn.
#include <algorithm>

#include "norm_dev.hpp"

namespace ft {

using namespace norm_dev;

namespace {

constexpr int kWaves = 4;

// sin and cos of position p times the frequency of pair j.
__device__ __forceinline__ void turn(float p, float hi, float lo, float& s, float& c) {
  const float r = p * hi;
  const float e = __builtin_fmaf(p, hi, -r);
  const float f = (r - __builtin_rintf(r)) + __builtin_fmaf(p, lo, e);
  s = __builtin_amdgcn_sinf(f);
  c = __builtin_amdgcn_cosf(f);
}

// LPH lanes per head; HALVES: pair j is (j, j + n_pairs), whose partner
// vector sits n_pairs / 8 lanes away; BWD: the transposed rotation, and
// the norm's gradient.  DW: the weights' gradients too.
template <int LPH, bool HALVES, bool BWD>
__global__ __launch_bounds__(kWaves * 64) void k_rope(const RopeArgs a, int rows_per_wave,
                                                       int head_splits) {
  constexpr int HPW = 64 / LPH;          // heads of a wave
  constexpr int NP = HALVES ? 8 : 4;     // pairs a lane's vector meets
  constexpr int UN = 4;                  // heads in flight per lane
  __shared__ float dwl[BWD ? kWaves * 2 * LPH * 8 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int vec = lane % LPH, hsub = lane / LPH;
  const int D = a.t.D, np = a.t.n_pairs;
  const bool in_head = vec * 8 < D;
  // the lane's pairs, their axes and frequencies
  const int hv = np >> 3;                // HALVES: vectors of a half
  const bool second = HALVES && vec >= hv;
  const bool turned = vec * 8 < 2 * np;
  const int partner = second ? lane - hv : lane + hv;
  float hi[NP], lo[NP];
  int ax[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int j = HALVES ? (second ? vec - hv : vec) * 8 + i : vec * 4 + i;
    const bool has = turned && j < np;
    hi[i] = has ? a.t.turn_hi[has ? j : 0] : 0.0f;
    lo[i] = has ? a.t.turn_lo[has ? j : 0] : 0.0f;
    ax[i] = has ? a.t.axis[has ? j : 0] : 0;
  }
  const float inv_d = 1.0f / static_cast<float>(D);
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.0f;

  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * rows_per_wave;
  const int64_t row1 = min(row0 + rows_per_wave, a.M);
  for (int64_t row = row0; row < row1; ++row) {
    float sn[NP], cs[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float p = static_cast<float>(a.pos[row * a.t.n_axes + ax[i]]);
      turn(p, hi[i], lo[i], sn[i], cs[i]);
      if (BWD) sn[i] = -sn[i];
      if (HALVES && !second) sn[i] = -sn[i];   // out_a = t_a cos - t_b sin, out_b = t_b cos + t_a sin
    }
    // the rotation of a lane's eight values
    auto rotate = [&](float(&t)[8]) {
      if constexpr (HALVES) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = __shfl(t[e], partner);
          t[e] = turned ? __builtin_fmaf(o, sn[e], t[e] * cs[e]) : t[e];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = t[2 * i], y = t[2 * i + 1];
          t[2 * i] = x * cs[i] - y * sn[i];
          t[2 * i + 1] = __builtin_fmaf(x, sn[i], y * cs[i]);
        }
      }
    };
#pragma unroll
    for (int si = 0; si < 2; ++si) {
      const RopeSide& s = a.side[si];
      const bool norm = s.weight != nullptr;
      Raw8<0> wr;
      wr.w = u32x4{kOnes, kOnes, kOnes, kOnes};
      if (norm && in_head) wr.load(s.weight, vec);
      const int step = HPW * head_splits;
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
            v[u].load(s.in + row * s.ld_in + static_cast<int64_t>(h) * D, vec);
            if (BWD && norm) xv[u].load(s.x + row * s.ld_x + static_cast<int64_t>(h) * D, vec);
          }
        }
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
              for (int e = 0; e < 8; ++e) t[e] = t[e] * rstd * wr.get(e);
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
                t[e] *= wr.get(e);
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
            o.store(s.out + row * s.ld_out + static_cast<int64_t>(h0 + u * step + hsub) * D, vec);
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
        if (hsub == 0) dwl[(wave * 2 + si) * LPH * 8 + vec * 8 + e] = v;
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

// The weights' gradients: the workgroups' sums added in order, 16 threads a value.
constexpr int kCols = 16, kWays = 16;
__global__ __launch_bounds__(kCols* kWays) void k_rope_reduce(const RopeArgs a, int n) {
  __shared__ float acc[kWays][kCols];
  const int D = a.t.D;
  const int col = threadIdx.x % kCols, way = threadIdx.x / kCols;
  const int i = static_cast<int>(blockIdx.x) * kCols + col;      // 2 D is a multiple of 16
  float v = 0.0f;
  for (int g = way; g < n; g += kWays) v += a.part[static_cast<int64_t>(g) * 2 * D + i];
  acc[way][col] = v;
  __syncthreads();
  if (way != 0) return;
  v = acc[0][col];
#pragma unroll
  for (int w = 1; w < kWays; ++w) v += acc[w][col];
  void* out = a.side[i / D].dweight;
  if (!out) return;
  if (a.grad_f32) static_cast<float*>(out)[i % D] = v;
  else static_cast<uint16_t*>(out)[i % D] = static_cast<uint16_t>(cvt_pk_bf16(v, 0.0f));
}

// With weight gradients a wave walks several rows, so that at most 512
// workgroups leave partial sums.
constexpr int64_t kMaxPart = 512;
int rows_per_wave(int64_t M, bool part) {
  return part ? static_cast<int>((M + kMaxPart * kWaves - 1) / (kMaxPart * kWaves)) : 1;
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
  hipLaunchKernelGGL(k_rope_reduce, dim3(2 * a.t.D / kCols), dim3(kCols * kWays), 0, st, a,
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
