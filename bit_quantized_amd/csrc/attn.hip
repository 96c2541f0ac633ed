// Attention inside packed documents, forward:
//   o_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  s_ij = scale q_i . k_j (capped by a tanh)
// in one pass over the keys with the running maximum and sum of each query.
//
// A workgroup takes 32 to 256 queries of one document and head, a wave 32
// of them; where there are few workgroups, groups of waves take the same
// queries and divide the key tiles, and are joined at the end (their
// maxima, sums and outputs through LDS).  Key and value tiles of 64 rows
// go through LDS, loaded one or two tiles ahead.  The products run as
// 32x32x16 bf16 matrix instructions on the transposed problem: S^T = K Q^T
// leaves a query's scores in two lanes (32 apart), so the softmax needs one
// exchange per tile and its statistics are one value per lane; and the
// accumulator's rows are, in order, the reduction slots of O^T = V^T P^T, if
// V's columns are read with the same order of rows.  So P never leaves its
// registers.  P is rounded to bf16 for that product (at most 2^-8
// of it, as the output is); scores, statistics and the output accumulate in fp32.
//
// A tile costs a wave about as long in the vector units (exponentials, sums,
// maxima: 750 cycles) as in the matrix unit (1024), and both are there for
// all waves of a SIMD at once.  Four waves that run freely overlap them by
// chance: 53% of the cycles have a matrix product at work (24 heads of 128,
// 4608 keys).  With 256 queries, the two waves of a SIMD take turns: a barrier
// splits a tile's time in half, in which four waves have their products and
// four their softmax, and the products' LDS reads are ordered to run eight
// products ahead: 64%, and 15% fewer cycles.  The clock pays most of that
// back (2.2 -> 2.0 GHz: the card is at its power), so the time falls by 6%:
// 268 -> 252 us, 1.04 PFLOP/s; a large bf16 matrix product runs at 1.57.
#include "attn_dev.hpp"

namespace ft {

using namespace attn_dev;

namespace {

// Registers for two waves a SIMD, also where LDS leaves one: more than 256
// would be of two kinds, with moves between them (5 to 20% slower).
#pragma clang diagnostic ignored "-Wpass-failed"

// NW waves of 32 queries each, in G groups that divide the tiles of BN keys.
template <int D, bool CAP, int NW, int G, int BN>
__global__ __launch_bounds__(64 * NW, D == 64 && NW == 8 ? 4 : 2) void k_attn_fwd(const AttnArgs a, uint32_t tiles) {
  constexpr int W = NW / G;              // waves of a group
  constexpr int KS = D / 16, DB = D / 32, KB = BN / 32, BM = 32 * W;
  constexpr int TB = BN * D * 2;         // bytes of a tile
  // (two objects: with one, the compiler waits for all loads in flight before
  // the transposing reads)
  constexpr bool TURNS = W == 8;        // half of the waves in turn with the others
  constexpr int NB = TURNS ? 3 : 2;
  __shared__ __attribute__((aligned(16))) uint8_t klds[NB * G * TB];
  __shared__ __attribute__((aligned(16))) uint8_t vlds[NB * G * TB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / W, l32 = lane & 31, half = lane >> 5;
  const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int head = static_cast<int>(id / tiles);
  DocTile dt;
  if (!find_tile<BM>(a, static_cast<int>(id % tiles), dt)) return;
  const int kvh = head / (a.Hq / a.Hkv);
  const int w0 = wave % W * 32;                          // the wave's first query
  const int qi = dt.row0 + w0 + l32;              // this lane's query
  const bool live = qi < dt.hi;
  uint16_t* orow = a.o + static_cast<int64_t>(qi) * a.ld_o + head * D;
  if (!dt.keys) {
    if (live && group == 0) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) reinterpret_cast<u32x4*>(orow)[2 * i + half] = u32x4{0, 0, 0, 0};
      if (a.lse && half == 0) a.lse[head * a.M + qi] = kNegInf;
    }
    return;
  }
  // the tiles that some query of the workgroup sees
  const int len = dt.hi - dt.lo;
  const int q0 = dt.row0 - dt.lo;                        // in the document
  const int seen = a.mask == 0 ? len : max(q0 + dt.rows, dt.prefix);
  const int nt = (seen + BN - 1) / BN;
  const uint16_t* kp = a.k + static_cast<int64_t>(dt.lo) * a.ld_k + kvh * D;
  const uint16_t* vp = a.v + static_cast<int64_t>(dt.lo) * a.ld_v + kvh * D;
  const Stager<D, BN * G, NW> ks(a.ld_k, wave, lane), vs(a.ld_v, wave, lane);       // G tiles at a time
  auto fetch_k = [&](int t, int buf) { ks(kp, t, len, klds + buf * G * TB); };
  auto fetch_v = [&](int t, int buf) { vs(vp, t, len, vlds + buf * G * TB); };
  fetch_k(0, 0);
  fetch_v(0, 0);
  if constexpr (TURNS) fetch_k(1, 1);
  u32x4 q[KS];
  {
    const uint16_t* qrow = a.q + static_cast<int64_t>(qi) * a.ld_q + head * D;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks] = u32x4{0, 0, 0, 0};
      if (live) q[ks] = reinterpret_cast<const u32x4*>(qrow)[2 * ks + half];
    }
  }
  const uint32_t kbase = row_base<D>(l32, half), vbase = col_base<D>(lane);
  f32x16 o[DB], s[KB];
  u32x4 p[2 * KB];
#pragma unroll
  for (int db = 0; db < DB; ++db) o[db] = zero16();
  float m = -3e38f, l = 0.0f;           // (finite: a group may see only hidden keys of a query)
  // scores in units of log 2: score * c1, or c2 tanh(score * c1)
  const float c1 = CAP ? a.scale / a.softcap : a.scale * kLog2e;
  const float c2 = a.softcap * kLog2e;
  const int wq0 = q0 + w0;                               // in the document
  auto scores = [&](int buf) {
    const uint8_t* kt = klds + (buf * G + group) * TB;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      s[kb] = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        s[kb] = mfma_bf16_32x32x16(lds_read_b128(kt + kb * 32 * 2 * D + (kbase ^ row_step(ks))), q[ks], s[kb]);
    }
  };
  auto outputs = [&](int buf) {
    const uint8_t* vt = vlds + (buf * G + group) * TB;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* vk = vt + (kb * 32 + h * 16) * 2 * D;
#pragma unroll
        for (int db = 0; db < DB; ++db)
          o[db] = mfma_bf16_32x32x16(col_read(vk, vbase ^ col_step<D>(db, 0), vbase ^ col_step<D>(db, 1)), p[2 * kb + h], o[db]);
      }
  };
  // In the turns' products the reads run AHEAD products before their use.
  auto order = [] {
    constexpr int PV = 2 * KB * DB, QK = KB * KS, AHEAD = 8;   // two reads a product, one read
#define FT_ORDER(what, n) __builtin_amdgcn_sched_group_barrier(what, n, 0)
    constexpr int PRODUCT = 0x8, READ = 0x100;
    FT_ORDER(READ, 2 * AHEAD);
#pragma unroll
    for (int j = 0; j < PV + QK; ++j) {
      FT_ORDER(PRODUCT, 1);
      if (j + AHEAD < PV) FT_ORDER(READ, 2);
      else if (j + AHEAD < PV + QK) FT_ORDER(READ, 1);
    }
#undef FT_ORDER
  };
  auto softmax = [&](int t) {
    if constexpr (CAP) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        tanh16(s[kb], c1);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[kb][r] *= c2;
      }
    }
    const int last = t * BN + BN - 1;
    if (last >= len || (a.mask != 0 && last > wq0 && last >= dt.prefix)) {
      // the tile's keys from `end` on are hidden from this lane's query
      const int end = (a.mask == 0 ? len : min(len, max(wq0 + l32 + 1, dt.prefix))) - t * BN - 4 * half;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (kb * 32 + acc_row(r) >= end) s[kb][r] = kNegInf;
    }
    float mt = s[0][0];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) mt = fmaxf(mt, s[kb][r]);
    mt = halves_max(mt);
    if constexpr (!CAP) mt *= c1;
    // The statistics follow the maximum only when some query's rose by more
    // than 2^8: until then p stays below 256, and the output needs no
    // rescaling (its relative precision is the same).
    if (__any(mt > m + 8.0f)) {
      const float mn = fmaxf(m, mt);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[db][r] *= f;
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float sum = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[kb][r] = __builtin_amdgcn_exp2f(CAP ? s[kb][r] - m : __builtin_fmaf(s[kb][r], c1, -m));
        sum += s[kb][r];
      }
      l += sum;
#pragma unroll
      for (int h = 0; h < 2; ++h) p[2 * kb + h] = pack8(s[kb], 8 * h);
    }
  };
  if constexpr (!TURNS) {
    staged_barrier();
    const int steps = (nt + G - 1) / G;
    for (int i = 0; i < steps; ++i) {
      if (i + 1 < steps) {
        fetch_k(i + 1, (i + 1) & 1);
        fetch_v(i + 1, (i + 1) & 1);
      }
      const int t = i * G + group;
      if (t < nt) {
        scores(i & 1);
        softmax(t);
        outputs(i & 1);
      }
      staged_barrier();
    }
    // join the groups, half of them to the other half at a time
#pragma unroll
    for (int h = G / 2; h >= 1; h /= 2) {
      f32x4* const part = reinterpret_cast<f32x4*>(klds) + (group % h * W + wave % W) * (DB * 4 * 64) + lane;
      float* const stat = reinterpret_cast<float*>(vlds) + (group % h * W + wave % W) * 128 + lane;
      if (group >= h && group < 2 * h) {
        stat[0] = m;
        stat[64] = l;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            part[(db * 4 + i) * 64] = f32x4{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]};
      }
      __syncthreads();
      if (group < h) {
        const float m2 = stat[0], mn = fmaxf(m, m2);
        const float f = __builtin_amdgcn_exp2f(m - mn), f2 = __builtin_amdgcn_exp2f(m2 - mn);
        m = mn;
        l = l * f + stat[64] * f2;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 v = part[(db * 4 + i) * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[db][4 * i + e] = o[db][4 * i + e] * f + v[e] * f2;
          }
      }
      if (h > 1) __syncthreads();
    }
    if (group > 0) return;
  } else {
    // Step t of the first half of the waves: products (outputs of tile t - 1,
    // scores of tile t), barrier, softmax of t, barrier; of the second half:
    // softmax of t - 1, barrier, products, barrier.  So K of t and V of t - 1
    // are read during step t; K of t + 2 and V of t + 1 are loaded in it,
    // into the third buffers, and waited for at the end of step t + 1.
    constexpr int IN = 2 * Stager<D, BN * G, NW>::N;          // loads of a wave in a step
    int b0 = 2, b1 = 0, b2 = 1;                           // the buffers of tiles t - 1, t and t + 1
    auto turn = [&] {
      const int b = b0;
      b0 = b1;
      b1 = b2;
      b2 = b;
    };
    staged_barrier<IN / 2>();                             // (all but the last loads: K of tile 1)
    if (wave < NW / 2) {
      scores(0);
      staged_barrier<63>();
      fetch_k(2, b0);
      fetch_v(1, b2);
      softmax(0);
      staged_barrier<IN>();
      turn();
      for (int t = 1; t < nt; ++t) {
        outputs(b0);
        scores(b1);
        order();
        staged_barrier<63>();
        fetch_k(t + 2, b0);
        fetch_v(t + 1, b2);
        softmax(t);
        staged_barrier<IN>();
        turn();
      }
      outputs(b0);
    } else {
      fetch_k(2, b0);
      fetch_v(1, b2);
      staged_barrier<63>();
      scores(0);
      staged_barrier<IN>();
      turn();
      for (int t = 1; t < nt; ++t) {
        fetch_k(t + 2, b0);
        fetch_v(t + 1, b2);
        softmax(t - 1);
        staged_barrier<63>();
        outputs(b0);
        scores(b1);
        order();
        staged_barrier<IN>();
        turn();
      }
      softmax(nt - 1);
      outputs(b0);
    }
    // no load may land in LDS after the workgroup has left it
    __builtin_amdgcn_s_waitcnt(0x0F70);
  }
  l = halves_sum(l);
  const float inv = 1.0f / l;
  if (live) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 w = {cvt_pk_bf16(o[db][4 * i] * inv, o[db][4 * i + 1] * inv),
                         cvt_pk_bf16(o[db][4 * i + 2] * inv, o[db][4 * i + 3] * inv)};
        *reinterpret_cast<u32x2*>(orow + db * 32 + 8 * i + 4 * half) = w;
      }
    if (a.lse && half == 0)
      a.lse[head * a.M + qi] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

template <int D, int NW, int G, int BN = 64>
hipError_t go(const AttnArgs& a, hipStream_t st) {
  const uint32_t tiles = static_cast<uint32_t>(tiles_of<32 * NW / G>(a));
  const dim3 grid(tiles * static_cast<uint32_t>(a.Hq));
  if (a.softcap > 0) hipLaunchKernelGGL((k_attn_fwd<D, true, NW, G, BN>), grid, dim3(64 * NW), 0, st, a, tiles);
  else hipLaunchKernelGGL((k_attn_fwd<D, false, NW, G, BN>), grid, dim3(64 * NW), 0, st, a, tiles);
  return hipGetLastError();
}

}  // namespace

// Workgroups of W waves by G groups.  What counts is how many of the 256 CUs
// have work, and how long a workgroup's walk over the keys is.
// Up to one workgroup a CU, a single wave owns 32 queries and four groups
// share the keys (64 queries by two groups / 32 by four: 2 heads of 64, 4096
// keys 31.9 / 25.2 us, 8 heads, 1024 keys 11.6 / 10.5, 256 keys 5.9 / 6.2;
// heads of 128, whose tiles for four groups are 32 keys: 8 heads, 1024 keys
// 18.6 / 16.2, 512 keys 12.1 / 11.3, and by two groups of one wave 11.0).
// Then 64 queries by two groups (12 heads of 64, 1024 keys: 128 queries 17.4
// us, by two groups 14.3, 64 by two 12.2; 24 heads of 128, 512 keys: 15.2,
// 14.8, 13.5), up to one workgroup a CU, or where documents and masks
// make their lengths differ up to two (of heads of 64; 2711 tokens in eight
// documents, 12 heads: 37, 32, 22 us).  Heads of 64 take two groups
// always (24 heads, 4608 keys: 176 -> 170 us; causal 115 -> 102), heads of 128
// up to one workgroup a CU (1024 keys: 26.9 -> 24.3 us; 1365 keys, more than
// one: 48 -> 56).
hipError_t launch_attn_fwd(const AttnArgs& a, int D, hipStream_t st) {
  const int64_t n32 = (a.M + 31) / 32 * a.Hq, n64 = (a.M + 63) / 64 * a.Hq, n128 = (a.M + 127) / 128 * a.Hq;
  const int64_t each = a.M / a.n_doc;
  if (D == 64) {
    if (n32 <= 256 && each > 256) return go<64, 4, 4>(a, st);
    return n64 <= 256 || (uneven(a) && a.M * a.Hq <= 512 * 64) ? go<64, 4, 2>(a, st) : go<64, 8, 2>(a, st);
  }
  if (n32 <= 256) return each > 640 ? go<128, 4, 4, 32>(a, st) : go<128, 2, 2>(a, st);
  if (n64 <= 256) return go<128, 4, 2>(a, st);
  if (n128 <= 256) return go<128, 8, 2>(a, st);
  return wide_tiles(a) ? go<128, 8, 1>(a, st) : go<128, 4, 1>(a, st);
}

}  // namespace ft
