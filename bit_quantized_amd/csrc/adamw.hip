// One AdamW step over many tensors (adapters: hundreds of them, each small)
// in one launch.  Per element, every operation rounded once to fp32:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = decay p - rate m / (sqrt(v) lift + eps)
//
// Memory bound: 22 to 28 bytes an element with 32-bit states, 8 to 10 with
// 8-bit ones.  A workgroup takes 2048 elements of one tensor, found through
// a table of chunks made once for the set of tensors, so that the grid is
// full however the elements are spread over tensors; a thread takes eight
// consecutive elements (16-byte accesses), and 16 threads the 128 elements
// of a block of 8-bit states, whose new scale is a maximum over 16 lanes.
//
// The 8-bit states are the exact same function of the inputs on every
// machine that rounds fp32 operations correctly, so no operation on their
// way is contracted or approximated.
#include "norm_dev.hpp"

#pragma clang fp contract(off)

namespace ft {

using namespace norm_dev;

namespace {

// The largest code's value in units of the smallest: (16 + 15) 2^(e - 1).
constexpr float kMostM = 31.0f * 64.0f;       // 3 exponent bits and a sign
constexpr float kMostV = 31.0f * 16384.0f;    // 4 exponent bits
constexpr float kTiny = 1e-35f;               // a block below this is zero

// What a code (sign taken off) stands for, in units of the smallest code.
// As an fp32 bit pattern the code's exponent and fraction are in place at
// bit 19; 2^(126 - ...) is added to the exponent field, and the lowest
// exponent has no leading one.
__device__ __forceinline__ float code_value(uint32_t c) {
  const uint32_t e = c >> 4;
  const float f = __uint_as_float((c << 19) + (130u << 23));    // (1 + f/16) 2^(e + 3)
  return e ? f : static_cast<float>(c);
}
// y >= 0 in those units to a code: `bits` (19) are added below the last
// kept bit, then the rest is cut.  Below 16 (no leading one) y + 16 has its
// last bit where the codes of [16, 32) have theirs.
__device__ __forceinline__ uint32_t code_of(float y, uint32_t bits, uint32_t top) {
  const bool low = y < 16.0f;
  const float z = low ? y + 16.0f : y;
  // (16 + f) 2^(e - 1) has the exponent field 131 + (e - 1): the field minus
  // 130 is the code's exponent, one less where 16 was added
  const uint32_t u = (__float_as_uint(z) + bits) >> 19;
  const uint32_t c = u - (130u << 4) - (low ? 16u : 0u);
  return c < top ? c : top;
}
__device__ __forceinline__ uint32_t mix(uint32_t i, uint32_t key) {
  uint32_t h = i * 0x9E3779B1u + key;
  h = (h ^ (h >> 16)) * 0x6A09E667u;
  h = (h ^ (h >> 15)) * 0xBB67AE85u;
  return h ^ (h >> 16);
}

// P: 0 fp32, 1 bf16 rounded at random, 2 bf16 copy of an fp32 master.
template <int P, int GF32, int Q8>
__global__ __launch_bounds__(256) void k_adamw(const AdamwArgs a) {
  const AdamwChunk ch = a.chunks[blockIdx.x];
  const AdamwEntry en = a.entries[ch.tensor];
  const int64_t i0 = static_cast<int64_t>(ch.chunk) * kAdamwChunk + threadIdx.x * 8;
  const int64_t left = en.n - i0;                // elements of this thread, at most 8
  // a block of 8-bit states is worked on to its end (its scale is a maximum
  // over 16 lanes), with zeros past the tensor's
  if ((Q8 ? en.n - (i0 & ~static_cast<int64_t>(127)) : left) <= 0) return;
  const int64_t at = en.at + i0;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  float p[8], g[8], m[8], v[8];
  if (left >= 8) {
    Raw8<P == 1 ? 0 : 1> pr;
    Raw8<GF32> gr;
    pr.load(P == 2 ? static_cast<const void*>(en.master) : en.p, i0 >> 3);
    gr.load(en.g, i0 >> 3);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = pr.get(e);
      g[e] = gr.get(e);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = g[e] = 0.0f;
      if (e < left) {
        p[e] = P == 2   ? en.master[i0 + e]
               : P == 0 ? static_cast<const float*>(en.p)[i0 + e]
                        : bf16_to_f32(static_cast<const uint16_t*>(en.p)[i0 + e]);
        g[e] = GF32 ? static_cast<const float*>(en.g)[i0 + e]
                    : bf16_to_f32(static_cast<const uint16_t*>(en.g)[i0 + e]);
      }
    }
  }
  if constexpr (Q8) {
    const u32x2 mc = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.m) + at);
    const u32x2 vc = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.v) + at);
    const float ms = a.m_scale[at >> 7] * (1.0f / kMostM);
    const float vs = a.v_scale[at >> 7] * (1.0f / kMostV);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t cm = (mc[e >> 2] >> (8 * (e & 3))) & 0xFFu;
      const uint32_t cv = (vc[e >> 2] >> (8 * (e & 3))) & 0xFFu;
      const float mv = code_value(cm & 127u) * ms;
      const float rv = code_value(cv) * vs;
      m[e] = e < left ? (cm & 128u ? -mv : mv) : 0.0f;
      v[e] = e < left ? rv * rv : 0.0f;
    }
  } else {
    // (the arena runs on to a multiple of 128 past the tensor)
    Raw8<1> mr, vr;
    mr.load(static_cast<const float*>(a.m) + at, 0);
    vr.load(static_cast<const float*>(a.v) + at, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      m[e] = mr.get(e);
      v[e] = vr.get(e);
    }
  }
  float root[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float gg = g[e] * gs;
    m[e] = m[e] * a.b1 + gg * a.b1c;
    v[e] = v[e] * a.b2 + (gg * gg) * a.b2c;
    root[e] = Q8 ? __builtin_sqrtf(v[e]) : __builtin_amdgcn_sqrtf(v[e]);
    p[e] = p[e] * a.decay - (m[e] * __builtin_amdgcn_rcpf(root[e] * a.lift + a.eps)) * a.rate;
  }
  uint32_t rnd[8];
  if constexpr (Q8 || P == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) rnd[e] = mix(static_cast<uint32_t>(at) + e, a.key);
  }
  if constexpr (Q8) {
    float mm = 0.0f, vm = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mm = fmaxf(mm, __builtin_fabsf(m[e]));
      vm = fmaxf(vm, root[e]);
    }
    mm = lanes_max<16>(mm);
    vm = lanes_max<16>(vm);
    const float mu = mm > kTiny ? (1.0f / mm) * kMostM : 0.0f;
    const float vu = vm > kTiny ? (1.0f / vm) * kMostV : 0.0f;
    u32x2 mc = {0, 0}, vc = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t cm = code_of(__builtin_fabsf(m[e]) * mu, rnd[e] >> 13, 127u);
      cm |= m[e] < 0.0f ? 128u : 0u;
      uint32_t cv = code_of(root[e] * vu, (rnd[e] * 0x9E3779B1u) >> 13, 255u);
      cv = cv == 0u && root[e] > 0.0f ? 1u : cv;
      mc[e >> 2] |= cm << (8 * (e & 3));
      vc[e >> 2] |= cv << (8 * (e & 3));
    }
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.m) + at) = mc;
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.v) + at) = vc;
    if ((threadIdx.x & 15) == 0) {
      a.m_scale[at >> 7] = mm;
      a.v_scale[at >> 7] = vm;
    }
  } else {
    if (left >= 8) {
      Raw8<1> o;
      o.set(m);
      o.store(static_cast<float*>(a.m) + at, 0);
      o.set(v);
      o.store(static_cast<float*>(a.v) + at, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) {
          static_cast<float*>(a.m)[at + e] = m[e];
          static_cast<float*>(a.v)[at + e] = v[e];
        }
    }
  }
  uint32_t lowp[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (P == 1) lowp[e] = (__float_as_uint(p[e]) + ((rnd[e] * 0x510E527Fu) >> 16)) >> 16;
    else lowp[e] = 0;
  }
  if (left >= 8) {
    if constexpr (P == 1) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = lowp[2 * e] | (lowp[2 * e + 1] << 16);
      static_cast<u32x4*>(en.p)[i0 >> 3] = w;
    } else {
      Raw8<1> o;
      o.set(p);
      o.store(P == 2 ? static_cast<void*>(en.master) : en.p, i0 >> 3);
      if constexpr (P == 2) {
        Raw8<0> lo;
        lo.set(p);
        lo.store(en.p, i0 >> 3);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) {
        if constexpr (P == 0) static_cast<float*>(en.p)[i0 + e] = p[e];
        if constexpr (P == 1) static_cast<uint16_t*>(en.p)[i0 + e] = static_cast<uint16_t>(lowp[e]);
        if constexpr (P == 2) {
          en.master[i0 + e] = p[e];
          static_cast<uint16_t*>(en.p)[i0 + e] = static_cast<uint16_t>(cvt_pk_bf16(p[e], 0.0f));
        }
      }
  }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(a.n_chunks));
#define FT_AW(P, G, Q) hipLaunchKernelGGL((k_adamw<P, G, Q>), grid, dim3(256), 0, st, a)
#define FT_AWG(P) \
  do { if (a.g_f32) { if (a.q8) FT_AW(P, 1, 1); else FT_AW(P, 1, 0); } \
       else { if (a.q8) FT_AW(P, 0, 1); else FT_AW(P, 0, 0); } } while (0)
  if (a.p_kind == 0) FT_AWG(0);
  else if (a.p_kind == 1) FT_AWG(1);
  else FT_AWG(2);
#undef FT_AWG
#undef FT_AW
  return hipGetLastError();
}

}  // namespace ft
