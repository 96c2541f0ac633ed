// Attention inside packed documents, backward.  With P from the forward's
// lse (p_ij = exp(s_ij - lse_i)) and delta_i = do_i . o_i:
//   dP = dO V^T,  dS = P (dP - delta) scale [(1 - tanh^2)],
//   dQ = dS K,  dK = dS^T Q,  dV = P^T dO
//
// Two kernels, so that every sum has one owner and a fixed order (no
// atomics): k_attn_dq walks the keys of 128 queries and also leaves delta;
// k_attn_dkv walks the queries of 128 keys, over all query heads of the key
// head.  S and dP are formed in both: 7 products of M^2 D instead of 5, for
// no traffic of partial dQ.  As in the forward each wave owns 32 rows, the
// scores are computed with the owned rows as columns, so that a lane's
// accumulator is the operand of the product that follows, and P and dS are
// rounded to bf16 there (relative 2^-9).
#include "attn_dev.hpp"

namespace ft {

using namespace attn_dev;

namespace {

constexpr int BM = 128;

// ds = p (dp - delta) [slope]; p from the score s and lse2 = lse / ln 2.
template <bool CAP>
__device__ __forceinline__ void p_and_ds(float s, float dp, float lse2, float delta, float c1,
                                         float c2, bool hidden, float& p, float& ds) {
  float slope = 1.0f;
  float t;
  if constexpr (CAP) {
    const float th = tanh_f32(s * c1);
    t = __builtin_fmaf(c2, th, -lse2);
    slope = 1.0f - th * th;
  } else {
    t = __builtin_fmaf(s, c1, -lse2);
  }
  p = hidden ? 0.0f : __builtin_amdgcn_exp2f(t);
  ds = p * (dp - delta);
  if constexpr (CAP) ds *= slope;
}

template <int D, bool CAP>
__global__ __launch_bounds__(256, 2) void k_attn_dq(const AttnArgs a, uint32_t tiles) {
  constexpr int KS = D / 16, DB = D / 32, BN = 64;
  constexpr int TB = BN * D * 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * TB];   // [buffer][K, V]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int head = static_cast<int>(id / tiles);
  DocTile dt;
  if (!find_tile<BM>(a, static_cast<int>(id % tiles), dt)) return;
  const int kvh = head / (a.Hq / a.Hkv);
  const int qi = dt.row0 + wave * 32 + l32;
  const bool live = qi < dt.hi;
  uint16_t* dqrow = a.dq + static_cast<int64_t>(qi) * a.ld_dq + head * D;
  if (!dt.keys) {
    if (live) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) reinterpret_cast<u32x4*>(dqrow)[2 * i + half] = u32x4{0, 0, 0, 0};
    }
    return;
  }
  const int len = dt.hi - dt.lo;
  const int q0 = dt.row0 - dt.lo;
  const int seen = a.mask == 0 ? len : max(q0 + dt.rows, dt.prefix);
  const int nt = (seen + BN - 1) / BN;
  const uint16_t* kp = a.k + static_cast<int64_t>(dt.lo) * a.ld_k + kvh * D;
  const uint16_t* vp = a.v + static_cast<int64_t>(dt.lo) * a.ld_v + kvh * D;
  auto fetch = [&](int t) {
    uint8_t* buf = lds + (t & 1) * 2 * TB;
    stage<D, BN, 4>(kp + static_cast<int64_t>(t) * BN * a.ld_k, a.ld_k, len - t * BN, buf, wave, lane);
    stage<D, BN, 4>(vp + static_cast<int64_t>(t) * BN * a.ld_v, a.ld_v, len - t * BN, buf + TB, wave, lane);
  };
  fetch(0);
  u32x4 q[KS], g[KS];
  float delta = 0.0f, lse2 = 0.0f;
  {
    const u32x4* qrow = reinterpret_cast<const u32x4*>(a.q + static_cast<int64_t>(qi) * a.ld_q + head * D);
    const u32x4* grow = reinterpret_cast<const u32x4*>(a.d_o + static_cast<int64_t>(qi) * a.ld_do + head * D);
    const u32x4* orow = reinterpret_cast<const u32x4*>(a.o_in + static_cast<int64_t>(qi) * a.ld_o + head * D);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks] = g[ks] = u32x4{0, 0, 0, 0};
      if (live) {
        q[ks] = qrow[2 * ks + half];
        g[ks] = grow[2 * ks + half];
        const u32x4 ov = orow[2 * ks + half];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          delta = __builtin_fmaf(bf16lo_to_f32(ov[e]), bf16lo_to_f32(g[ks][e]), delta);
          delta = __builtin_fmaf(bf16hi_to_f32(ov[e]), bf16hi_to_f32(g[ks][e]), delta);
        }
      }
    }
    delta = halves_sum(delta);
    if (live) {
      lse2 = a.lse[head * a.M + qi] * kLog2e;
      if (half == 0) a.delta[head * a.M + qi] = delta;
    }
  }
  uint32_t koff[KS], coff[DB][2];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) koff[ks] = row_off<D>(l32, half, ks);
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 2; ++i) coff[db][i] = col_off<D>(lane, db, i);
  f32x16 acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) acc[db] = zero16();
  const float c1 = CAP ? a.scale / a.softcap : a.scale * kLog2e;
  const float c2 = a.softcap * kLog2e;
  const int wq0 = q0 + wave * 32;
  const int end = a.mask == 0 ? len : min(len, max(wq0 + l32 + 1, dt.prefix));
  staged_barrier();
  for (int t = 0; t < nt; ++t) {
    if (t + 1 < nt) fetch(t + 1);
    const uint8_t* kt = lds + (t & 1) * 2 * TB;
    const uint8_t* vt = kt + TB;
    const int last = t * BN + BN - 1;
    const bool edge = last >= len || (a.mask != 0 && last > wq0 && last >= dt.prefix);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        s = mfma_bf16_32x32x16(lds_read_b128(kt + kb * 32 * 2 * D + koff[ks]), q[ks], s);
        dp = mfma_bf16_32x32x16(lds_read_b128(vt + kb * 32 * 2 * D + koff[ks]), g[ks], dp);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const bool hidden = edge && t * BN + kb * 32 + acc_row(r, half) >= end;
        float p, ds;
        p_and_ds<CAP>(s[r], dp[r], lse2, delta, c1, c2, hidden, p, ds);
        s[r] = ds;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 d = pack8(s, 8 * h);
        const uint8_t* kk = kt + (kb * 32 + h * 16) * 2 * D;
#pragma unroll
        for (int db = 0; db < DB; ++db)
          acc[db] = mfma_bf16_32x32x16(col_read(kk, coff[db][0], coff[db][1]), d, acc[db]);
      }
    }
    staged_barrier();
  }
  if (live) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = a.scale;
        const u32x2 w = {cvt_pk_bf16(acc[db][4 * i] * f, acc[db][4 * i + 1] * f),
                         cvt_pk_bf16(acc[db][4 * i + 2] * f, acc[db][4 * i + 3] * f)};
        *reinterpret_cast<u32x2*>(dqrow + db * 32 + 8 * i + 4 * half) = w;
      }
  }
}

// 128 keys of one key head; a wave owns 32.
template <int D, bool CAP>
__global__ __launch_bounds__(256, 1) void k_attn_dkv(const AttnArgs a, uint32_t tiles) {
  constexpr int KS = D / 16, DB = D / 32, BQ = 64;
  constexpr int TB = BQ * D * 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * TB];       // [buffer][Q, dO]
  __shared__ __attribute__((aligned(16))) float stat[2][2][BQ];     // [buffer][lse2, delta]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int kvh = static_cast<int>(id / tiles);
  DocTile dt;
  if (!find_tile<BM>(a, static_cast<int>(id % tiles), dt)) return;
  const int kj = dt.row0 + wave * 32 + l32;              // this lane's key
  const bool live = kj < dt.hi;
  uint16_t* dkrow = a.dk + static_cast<int64_t>(kj) * a.ld_dk + kvh * D;
  uint16_t* dvrow = a.dv + static_cast<int64_t>(kj) * a.ld_dv + kvh * D;
  if (!dt.keys) {
    if (live) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        reinterpret_cast<u32x4*>(dkrow)[2 * i + half] = u32x4{0, 0, 0, 0};
        reinterpret_cast<u32x4*>(dvrow)[2 * i + half] = u32x4{0, 0, 0, 0};
      }
    }
    return;
  }
  const int len = dt.hi - dt.lo;
  const int k0 = dt.row0 - dt.lo;                        // in the document
  // the first query that sees a key of the workgroup; whole tiles of 64
  const int first = a.mask == 0 || k0 < dt.prefix ? 0 : k0 / BQ;
  const int nt = (len + BQ - 1) / BQ - first;
  const int group = a.Hq / a.Hkv;
  const int total = nt * group;                          // (query head, tile) pairs
  auto fetch = [&](int it) {
    const int h = kvh * group + it / nt;
    const int t = first + it % nt;
    uint8_t* buf = lds + (it & 1) * 2 * TB;
    const int64_t row = dt.lo + static_cast<int64_t>(t) * BQ;
    stage<D, BQ, 4>(a.q + row * a.ld_q + h * D, a.ld_q, len - t * BQ, buf, wave, lane);
    stage<D, BQ, 4>(a.d_o + row * a.ld_do + h * D, a.ld_do, len - t * BQ, buf + TB, wave, lane);
  };
  // lse and delta of a tile, through registers (rows past the end: p = 0)
  float nstat = 0.0f;
  auto fetch_stat = [&](int it) {
    if (threadIdx.x < 2 * BQ) {
      const int h = kvh * group + it / nt;
      const int i = threadIdx.x & (BQ - 1), t = first + it % nt;
      const bool in = t * BQ + i < len;
      const int64_t at = h * a.M + dt.lo + t * BQ + i;
      if (threadIdx.x < BQ) nstat = in ? a.lse[at] * kLog2e : __builtin_inff();
      else nstat = in ? a.delta[at] : 0.0f;
    }
  };
  auto put_stat = [&](int it) {
    if (threadIdx.x < 2 * BQ) stat[it & 1][threadIdx.x / BQ][threadIdx.x & (BQ - 1)] = nstat;
  };
  fetch(0);
  fetch_stat(0);
  u32x4 k[KS], v[KS];
  {
    const u32x4* krow = reinterpret_cast<const u32x4*>(a.k + static_cast<int64_t>(kj) * a.ld_k + kvh * D);
    const u32x4* vrow = reinterpret_cast<const u32x4*>(a.v + static_cast<int64_t>(kj) * a.ld_v + kvh * D);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      k[ks] = v[ks] = u32x4{0, 0, 0, 0};
      if (live) {
        k[ks] = krow[2 * ks + half];
        v[ks] = vrow[2 * ks + half];
      }
    }
  }
  uint32_t roff[KS], coff[DB][2];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) roff[ks] = row_off<D>(l32, half, ks);
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 2; ++i) coff[db][i] = col_off<D>(lane, db, i);
  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) dk[db] = dv[db] = zero16();
  const float c1 = CAP ? a.scale / a.softcap : a.scale * kLog2e;
  const float c2 = a.softcap * kLog2e;
  const int wk0 = k0 + wave * 32;                        // the wave's first key
  const int key = wk0 + l32;
  put_stat(0);
  staged_barrier();
  for (int it = 0; it < total; ++it) {
    if (it + 1 < total) {
      fetch(it + 1);
      fetch_stat(it + 1);
    }
    const uint8_t* qt = lds + (it & 1) * 2 * TB;
    const uint8_t* gt = qt + TB;
    const float* ls = stat[it & 1][0];
    const float* de = stat[it & 1][1];
    const int t = first + it % nt;
    // some query of the tile does not see some key of the wave
    const bool edge = a.mask != 0 && t * BQ < wk0 + 31 && wk0 + 31 >= dt.prefix;
#pragma unroll
    for (int qb = 0; qb < 2; ++qb) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        s = mfma_bf16_32x32x16(lds_read_b128(qt + qb * 32 * 2 * D + roff[ks]), k[ks], s);
        dp = mfma_bf16_32x32x16(lds_read_b128(gt + qb * 32 * 2 * D + roff[ks]), v[ks], dp);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 lse2 = *reinterpret_cast<const f32x4*>(ls + qb * 32 + 8 * j + 4 * half);
        const f32x4 delta = *reinterpret_cast<const f32x4*>(de + qb * 32 + 8 * j + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * j + e;
          const int query = t * BQ + qb * 32 + 8 * j + 4 * half + e;
          const bool hidden = edge && key > query && key >= dt.prefix;
          float p, ds;
          p_and_ds<CAP>(s[r], dp[r], lse2[e], delta[e], c1, c2, hidden, p, ds);
          s[r] = p;
          dp[r] = ds;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 pp = pack8(s, 8 * h), dd = pack8(dp, 8 * h);
        const uint32_t at = (qb * 32 + h * 16) * 2 * D;
#pragma unroll
        for (int db = 0; db < DB; ++db) {
          dv[db] = mfma_bf16_32x32x16(col_read(gt + at, coff[db][0], coff[db][1]), pp, dv[db]);
          dk[db] = mfma_bf16_32x32x16(col_read(qt + at, coff[db][0], coff[db][1]), dd, dk[db]);
        }
      }
    }
    if (it + 1 < total) put_stat(it + 1);
    staged_barrier();
  }
  if (live) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = a.scale;
        const u32x2 wk = {cvt_pk_bf16(dk[db][4 * i] * f, dk[db][4 * i + 1] * f),
                          cvt_pk_bf16(dk[db][4 * i + 2] * f, dk[db][4 * i + 3] * f)};
        const u32x2 wv = {cvt_pk_bf16(dv[db][4 * i], dv[db][4 * i + 1]),
                          cvt_pk_bf16(dv[db][4 * i + 2], dv[db][4 * i + 3])};
        *reinterpret_cast<u32x2*>(dkrow + db * 32 + 8 * i + 4 * half) = wk;
        *reinterpret_cast<u32x2*>(dvrow + db * 32 + 8 * i + 4 * half) = wv;
      }
  }
}

}  // namespace

hipError_t launch_attn_bwd(const AttnArgs& a, int D, hipStream_t st) {
  const uint32_t tiles = static_cast<uint32_t>(tiles_of<BM>(a));
#define FT_AB(DD, C)                                                                              \
  do {                                                                                            \
    hipLaunchKernelGGL((k_attn_dq<DD, C>), dim3(tiles * static_cast<uint32_t>(a.Hq)), dim3(256),  \
                       0, st, a, tiles);                                                          \
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;                              \
    hipLaunchKernelGGL((k_attn_dkv<DD, C>), dim3(tiles * static_cast<uint32_t>(a.Hkv)),           \
                       dim3(256), 0, st, a, tiles);                                               \
  } while (0)
  if (D == 128) { if (a.softcap > 0) FT_AB(128, true); else FT_AB(128, false); }
  else { if (a.softcap > 0) FT_AB(64, true); else FT_AB(64, false); }
#undef FT_AB
  return hipGetLastError();
}

}  // namespace ft
