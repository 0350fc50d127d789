// An AdamW step over a list of tensors, in one pass:
//
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every operation is FP32, rounded on its own in the order written (no fused
// multiply-adds), so a step gives the same bits whatever kernel, list or device
// computes it: what 8-bit codes need, whose neighbours lie percents apart.
//
// States in 8 bits: blocks of 256 consecutive elements of a tensor with one FP32
// scale s each.
//   m       = s c |c|,  c in -127 .. 127    s = max |m| / 127^2
//   sqrt(v) = s c^2,    c in 0 .. 255       s = max sqrt(v) / 255^2
// The codes are nearest in c.  Squares give small values of a block finer steps
// than a linear code: the smallest nonzero one is 6e-5 (m) and 1.5e-5 (sqrt v) of
// the block's largest.  A nonzero sqrt(v) keeps a code of at least 1: as 0 it would leave
// eps alone to divide m.
//
// A warp takes 256 elements at a time, eight a lane, so that a block's maxima are
// two warp reductions.  Bound by HBM: bfloat16 parameters and gradients move 22
// bytes an element with states in FP32, 10 with states in 8 bits.
#pragma once

#include <cmath>

#include "clip.cuh"

namespace poot {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamBlock = 256;     // elements of a scale, and of a warp's turn
// Shared memory of a block with states in 8 bits: two chunks a warp, of up to 4
// + 4 bytes of p and g and two codes an element
constexpr int kAdamStage = kAdamBlock * (4 + 4 + 2);
constexpr int kAdamSmem = 2 * kAdamWarps * kAdamStage;
constexpr int kAdamTable = 384;     // tensors of one launch
constexpr int kAdamTableFew = 48;   // short lists: less to pass to the launch

template <int T>
struct AdamTable {
  void* p[T];
  const void* g[T];
  void* m[T];
  void* v[T];
  float* ms[T];
  float* vs[T];
  void* copy[T];
  long long n[T];
  long long first[T + 1];  // first chunk of 256 elements of each tensor
  float decay[T];          // 1 - lr wd; with lr on the device wd
  unsigned char types[T];  // GradDtype of p, g << 2, copy << 4; kAdamVec
  int count;
};
constexpr int kAdamVec = 64;  // every pointer is on a 16-byte boundary

struct AdamArgs {
  // read on the device where not nullptr
  const float* lr_dev;
  const long long* step_dev;
  const float* grad_scale_dev;
  double lr, log_b1, log_b2;
  long long step;
  float b1, omb1, b2, omb2, eps, grad_scale;
  float minus_zero;             // -0, unknown to the compiler: see adam_product
  float step_size, root_scale;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};

// Which eight elements of a chunk a lane has: every 32nd, of which `n` of the
// 256 exist (the others are zero); two fours, 128 apart; or consecutive ones, in shared
// memory and where they are stored.
enum AdamLane : int { kAdamEach = 0, kAdamFours = 1, kAdamEight = 2 };

template <int DT, int VEC>
struct AdamLoad {
  uint32_t w[DT == kGradF32 ? 8 : 4];
  __device__ __forceinline__ void load(const void* base, long long e0, int n, int lane) {
    if constexpr (VEC == kAdamEight) {
      const uint4* p = static_cast<const uint4*>(base) + lane * (DT == kGradF32 ? 2 : 1);
#pragma unroll
      for (int i = 0; i < (DT == kGradF32 ? 2 : 1); ++i) {
        const uint4 a = p[i];
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
      }
    } else if constexpr (VEC && DT == kGradF32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + e0) + lane;
      const uint4 a = p[0], b = p[32];
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else if constexpr (VEC) {
      const uint2* p = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + e0) + lane;
      const uint2 a = p[0], b = p[32];
      w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
    } else if constexpr (DT == kGradF32) {
      const uint32_t* p = static_cast<const uint32_t*>(base) + e0;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j * 32 + lane < n ? p[j * 32 + lane] : 0u;
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(base) + e0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int a = j * 64 + lane, b = a + 32;
        w[j] = (a < n ? (uint32_t)p[a] : 0u) | (b < n ? (uint32_t)p[b] << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (DT == kGradF32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = ep_unpack_t<DT>(w[j]);
        f[2 * j] = a.x;
        f[2 * j + 1] = a.y;
      }
    }
  }
};

template <int DT, int VEC>
__device__ __forceinline__ void adam_store(void* base, long long e0, int n, int lane, const float (&f)[8]) {
  if constexpr (VEC == kAdamEight && DT == kGradF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e0) + lane * 2;
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else if constexpr (VEC == kAdamEight) {
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e0)[lane] =
        make_uint4(ep_pack_t<DT>(f[0], f[1]), ep_pack_t<DT>(f[2], f[3]), ep_pack_t<DT>(f[4], f[5]), ep_pack_t<DT>(f[6], f[7]));
  } else if constexpr (VEC && DT == kGradF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e0) + lane;
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[32] = make_float4(f[4], f[5], f[6], f[7]);
  } else if constexpr (VEC) {
    uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + e0) + lane;
    p[0] = make_uint2(ep_pack_t<DT>(f[0], f[1]), ep_pack_t<DT>(f[2], f[3]));
    p[32] = make_uint2(ep_pack_t<DT>(f[4], f[5]), ep_pack_t<DT>(f[6], f[7]));
  } else {
    using E = GradElem<DT>;
    typename E::type* p = static_cast<typename E::type*>(base) + e0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * 32 + lane < n) p[j * 32 + lane] = E::round(f[j]);
  }
}

// ---- codes -------------------------------------------------------------------
template <int VEC>
struct AdamCodes {
  uint32_t w[2];  // byte j & 3 of word j >> 2
  __device__ __forceinline__ void load(const void* base, long long e0, int n, int lane) {
    const unsigned char* p = static_cast<const unsigned char*>(base) + e0;
    if constexpr (VEC == kAdamEight) {
      const uint2 a = reinterpret_cast<const uint2*>(p)[lane];
      w[0] = a.x;
      w[1] = a.y;
    } else if constexpr (VEC) {
      w[0] = reinterpret_cast<const uint32_t*>(p)[lane];
      w[1] = reinterpret_cast<const uint32_t*>(p)[32 + lane];
    } else {
      w[0] = w[1] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 32 + lane < n) w[j >> 2] |= (uint32_t)p[j * 32 + lane] << (8 * (j & 3));
    }
  }
  __device__ __forceinline__ void store(void* base, long long e0, int n, int lane) const {
    unsigned char* p = static_cast<unsigned char*>(base) + e0;
    if constexpr (VEC == kAdamEight) {
      reinterpret_cast<uint2*>(p)[lane] = make_uint2(w[0], w[1]);
    } else if constexpr (VEC) {
      reinterpret_cast<uint32_t*>(p)[lane] = w[0];
      reinterpret_cast<uint32_t*>(p)[32 + lane] = w[1];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 32 + lane < n) p[j * 32 + lane] = (unsigned char)(w[j >> 2] >> (8 * (j & 3)));
    }
  }
};

// Two FP32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 adam_add(float2 a, float2 b) {
  add_f32x2(a.x, a.y, b.x, b.y);
  return a;
}
__device__ __forceinline__ float2 adam_mul(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 s, t;\n\t"
      "mov.b64 s, {%2, %3};\n\t"
      "mov.b64 t, {%4, %5};\n\t"
      "mul.rn.f32x2 s, s, t;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 adam_fma(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 s, t, u;\n\t"
      "mov.b64 s, {%2, %3};\n\t"
      "mov.b64 t, {%4, %5};\n\t"
      "mov.b64 u, {%6, %7};\n\t"
      "fma.rn.f32x2 s, s, t, u;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 adam_both(float v) { return make_float2(v, v); }
// (packed operands take no sign)
__device__ __forceinline__ float2 adam_neg(float2 v) { return adam_mul(v, adam_both(-1.0f)); }

// Bytes j and j + 1 of a word as floats: in the low bits of 2^23's, which is then
// taken off (conversions run at an eighth of the rate).
__device__ __forceinline__ float2 adam_bytes(uint32_t w, int j, float off) {
  const float2 t = make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | (j & 3))),
                               __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | ((j & 3) + 1))));
  return adam_add(t, adam_both(off));
}
// w ^ 0x80808080: c + 128 in 0 .. 255
__device__ __forceinline__ float2 adam_m(uint32_t w, int j, float scale) {
  const float2 c = adam_bytes(w ^ 0x80808080u, j, -8388736.0f);
  // (c |c| is exact)
  return adam_mul(adam_both(scale), make_float2(__fmul_rn(c.x, fabsf(c.x)), __fmul_rn(c.y, fabsf(c.y))));
}
__device__ __forceinline__ float2 adam_root(uint32_t w, int j, float scale) {
  const float2 c = adam_bytes(w, j, -8388608.0f);
  return adam_mul(adam_both(scale), adam_mul(c, c));
}

// The scale of a block whose largest value has the bits `most` (as integers, those of
// absolute values order like the values, infinities and NaN above), and what
// turns a value into the square of its code.  A block that is not finite gets
// the scale NaN, and so reads as NaN throughout.
struct AdamScale {
  float scale, inverse;
};
template <int TOP>
__device__ __forceinline__ AdamScale adam_scale(uint32_t most) {
  constexpr float kSquare = TOP * TOP, kPart = 1.0 / (TOP * TOP);
  const float f = __uint_as_float(most);
  if (most >= 0x7f800000u) return {NAN, 0.0f};
  // (below 2^-110, where the inverse would overflow, a block counts as zero; sqrt(v) is above 2^-75 or zero)
  if (f < 7.703719777548943e-34f) return {0.0f, 0.0f};
  return {__fmul_rn(f, kPart), __fmul_rn(__frcp_rn(f), kSquare)};
}

// 2^23 + c for two integers c nearest to sqrt(y), y in 0 .. 255^2 (1 + 2^-22): c + 1 from y >
// (c + 1/2)^2 on.  The square root is approximate; taken 2^-10 low, its rounding is the result or
// one less, and the comparison, exact in FP32, decides.
__device__ __forceinline__ float2 adam_code(float2 y) {
  float2 s, up;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(y.x));
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(y.y));
  // (beside 2^23 only integers are left)
  const float2 t = adam_add(adam_add(s, adam_both(-0.0009765625f)), adam_both(8388608.0f));
  const float2 half = adam_add(t, adam_both(-8388607.5f)), edge = adam_mul(half, half);
  asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(up.x) : "f"(y.x), "f"(edge.x));
  asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(up.y) : "f"(y.y), "f"(edge.y));
  return adam_add(t, up);
}
// The low bytes of four.
__device__ __forceinline__ uint32_t adam_pack(float2 a, float2 b) {
  const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

struct AdamHyper {
  float b1, omb1, b2, omb2, eps, grad_scale, step_size, root_scale, lr, minus_zero;
};

// a b rounded, for a sum: the assembler fuses a packed product with the addition behind it, .rn or
// not, but not a product that is one already (adding -0 changes nothing).
__device__ __forceinline__ float2 adam_product(const AdamHyper& h, float2 a, float b) {
  return adam_fma(a, adam_both(b), adam_both(h.minus_zero));
}

// sqrt(v) correctly rounded, for v of 2^-100 .. 2^100: from an approximate 1 /
// sqrt(v) one coupled Newton step for sqrt and half its reciprocal, then the
// remainder v - g^2, exact in an FMA, added back (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).
__device__ __forceinline__ float2 adam_sqrt(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v.y));
  float2 g = adam_mul(v, y), h = adam_mul(y, adam_both(-0.5f));  // h: minus half the reciprocal
  const float2 e = adam_fma(h, g, adam_both(0.5f));
  g = adam_fma(g, e, g);
  h = adam_fma(h, e, h);
  return adam_fma(adam_fma(g, g, adam_neg(v)), h, g);
}

// 1 / d for d of 2^-100 .. 2^100: an approximate one and a Newton step, rounded to nearest.
__device__ __forceinline__ float2 adam_reciprocal(float2 d) {
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return adam_fma(adam_fma(adam_neg(d), r, adam_both(1.0f)), r, r);
}

// m / d rounded to nearest likewise, for d of 2^-60 .. 2^60 and m of 2^-75 or more (below, the
// remainder may be subnormal and the last place off by one).
__device__ __forceinline__ float2 adam_div(float2 m, float2 d) {
  const float2 n = adam_neg(d), r = adam_reciprocal(d);
  const float2 q = adam_mul(m, r);
  return adam_fma(adam_fma(n, q, m), r, q);
}

// The largest and the smallest of three, NaN where one is.
__device__ __forceinline__ float adam_max(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float adam_min(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A lane's eight elements: m and v updated, sqrt(v) and the new p; `most`: the largest v.
// Whether all the warp's v are of 2^-100 .. 2^100.  All 32 lanes call it.
__device__ __forceinline__ bool adam_update(const AdamHyper& h, float decay, const float (&gs)[8], float (&p)[8],
                                            float (&m)[8], float (&v)[8], float (&root)[8], float& most) {
  float lo = INFINITY, hi = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 g = adam_mul(make_float2(gs[j], gs[j + 1]), adam_both(h.grad_scale));
    const float2 a = adam_add(adam_product(h, make_float2(m[j], m[j + 1]), h.b1), adam_product(h, g, h.omb1));
    const float2 b = adam_add(adam_product(h, make_float2(v[j], v[j + 1]), h.b2),
                              adam_product(h, adam_mul(g, g), h.omb2));
    m[j] = a.x;
    m[j + 1] = a.y;
    v[j] = b.x;
    v[j + 1] = b.y;
    lo = adam_min(lo, b.x, b.y);
    hi = adam_max(hi, b.x, b.y);
  }
  most = hi;
  // (zeros, of elements that have had no gradient yet, and NaN take the second way)
  const bool plain =
      __all_sync(0xffffffffu, lo >= 7.888609052210118e-31f && hi <= 1.2676506002282294e30f && h.eps <= 1e15f);
  if (plain) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 r = adam_sqrt(make_float2(v[j], v[j + 1]));
      const float2 d = adam_add(adam_product(h, r, h.root_scale), adam_both(h.eps));
      const float2 q = adam_div(make_float2(m[j], m[j + 1]), d);
      const float2 n = adam_add(adam_product(h, make_float2(p[j], p[j + 1]), decay), adam_product(h, q, -h.step_size));
      root[j] = r.x;
      root[j + 1] = r.y;
      p[j] = n.x;
      p[j + 1] = n.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      root[j] = __fsqrt_rn(v[j]);
      const float q = __fdiv_rn(m[j], __fadd_rn(__fmul_rn(root[j], h.root_scale), h.eps));
      p[j] = __fsub_rn(__fmul_rn(p[j], decay), __fmul_rn(q, h.step_size));
    }
  }
  return plain;
}

struct AdamTensor {
  void* p;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  void* copy;
  long long n;
  float decay;
  int copy_dtype;
};

// 256 elements of a tensor as they come from memory, `n` of which exist.
template <int PD, int GD, int BITS, int VEC>
struct AdamChunk {
  AdamLoad<PD, VEC> p;
  AdamLoad<GD, VEC> g;
  AdamLoad<kGradF32, VEC> m, v;
  __device__ __forceinline__ void load(const AdamTensor& t, long long e0, int n, int lane) {
    g.load(t.g, e0, n, lane);
    p.load(t.p, e0, n, lane);
    m.load(t.m, e0, n, lane);
    v.load(t.v, e0, n, lane);
  }
};
template <int PD, int GD, int VEC>
struct AdamChunk<PD, GD, 8, VEC> {
  AdamLoad<PD, VEC> p;
  AdamLoad<GD, VEC> g;
  AdamCodes<VEC> m, v;
  float ms, vs;
  __device__ __forceinline__ void load(const AdamTensor& t, long long e0, int n, int lane) {
    g.load(t.g, e0, n, lane);
    p.load(t.p, e0, n, lane);
    m.load(t.m, e0, n, lane);
    v.load(t.v, e0, n, lane);
    ms = t.ms[e0 / kAdamBlock];
    vs = t.vs[e0 / kAdamBlock];
  }
};

// A chunk on its way to a warp's shared memory, 16 bytes a lane and copy.
template <int DT>
__device__ __forceinline__ void adam_fetch(uint32_t stage, const void* base, long long e0, int lane) {
  const char* p = static_cast<const char*>(base) + e0 * (DT == kGradF32 ? 4 : 2) + lane * 16;
  cp_async_16(stage + lane * 16, p, 16);
  if constexpr (DT == kGradF32) cp_async_16(stage + 512 + lane * 16, p + 512, 16);
}
constexpr int kAdamStageG = kAdamBlock * 4, kAdamStageM = kAdamBlock * 8, kAdamStageV = kAdamBlock * 9;
template <int PD, int GD>
__device__ __forceinline__ void adam_fetch_chunk(uint32_t stage, const AdamTensor& t, long long e0, int lane) {
  adam_fetch<GD>(stage + kAdamStageG, t.g, e0, lane);
  adam_fetch<PD>(stage, t.p, e0, lane);
  // codes: m by the lower lanes, v by the upper
  const char* c = static_cast<const char*>(lane < 16 ? t.m : t.v) + e0 + (lane & 15) * 16;
  cp_async_16(stage + kAdamStageM + lane * 16, c, 16);
}

// Its step, from e0 on.
template <int PD, int GD, int BITS, int VEC>
__device__ __forceinline__ void adam_chunk(const AdamTensor& t, const AdamHyper& h, const AdamChunk<PD, GD, BITS, VEC>& x,
                                           long long e0, int n, int lane) {
  float p[8], g[8], m[8], v[8], root[8], most_v;
  x.g.get(g);
  x.p.get(p);
  if constexpr (BITS == 32) {
    x.m.get(m);
    x.v.get(v);
    adam_update(h, t.decay, g, p, m, v, root, most_v);
    adam_store<kGradF32, VEC>(t.m, e0, n, lane, m);
    adam_store<kGradF32, VEC>(t.v, e0, n, lane, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 a = adam_m(x.m.w[j >> 2], j, x.ms), r = adam_root(x.v.w[j >> 2], j, x.vs), b = adam_mul(r, r);
      m[j] = a.x;
      m[j + 1] = a.y;
      v[j] = b.x;
      v[j + 1] = b.y;
    }
    const bool positive = adam_update(h, t.decay, g, p, m, v, root, most_v);
    float up = 0.0f, down = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      up = adam_max(up, m[j], m[j + 1]);
      down = adam_min(down, m[j], m[j + 1]);
    }
    // (elements that do not exist are zeros times the scale: NaN in a block that was not finite, as it stays.
    // The largest sqrt(v) is the largest v's.)
    const float most_m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(adam_max(up, -down, 0.0f))));
    const float2 most = make_float2(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most_v))), most_m);
    AdamScale sm, sv;
    if (positive && most_m >= 7.888609052210118e-31f && most_m <= 1.2676506002282294e30f) {
      // both at once, as adam_scale does
      const float root_v = adam_sqrt(adam_both(most.x)).x;
      const float2 f = make_float2(most_m, root_v), r = adam_reciprocal(f);
      const float2 scale = adam_mul(f, make_float2(1.0 / (127 * 127), 1.0 / (255 * 255)));
      const float2 inverse = adam_mul(r, make_float2(127 * 127, 255 * 255));
      sm = {scale.x, inverse.x};
      sv = {scale.y, inverse.y};
    } else {
      sm = adam_scale<127>(__float_as_uint(most_m));
      sv = adam_scale<255>(__float_as_uint(__fsqrt_rn(most.x)));
    }
    AdamCodes<VEC> cm, cv;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float2 c[2], k[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = 4 * w + 2 * i;
        c[i] = adam_code(make_float2(__fmul_rn(fabsf(m[j]), sm.inverse), __fmul_rn(fabsf(m[j + 1]), sm.inverse)));
        // with its sign, beside 1.5 2^23: in two's complement
        c[i] = adam_add(c[i], adam_both(-8388608.0f));
        c[i] = make_float2(copysignf(c[i].x, m[j]), copysignf(c[i].y, m[j + 1]));
        c[i] = adam_add(c[i], adam_both(12582912.0f));
        k[i] = adam_code(adam_mul(make_float2(root[j], root[j + 1]), adam_both(sv.inverse)));
        constexpr float kOne = 8388609.0f;
        if (positive)
          k[i] = make_float2(fmaxf(k[i].x, kOne), fmaxf(k[i].y, kOne));
        else
          k[i] = make_float2(root[j] > 0.0f ? fmaxf(k[i].x, kOne) : k[i].x, root[j + 1] > 0.0f ? fmaxf(k[i].y, kOne) : k[i].y);
      }
      cm.w[w] = adam_pack(c[0], c[1]);
      cv.w[w] = adam_pack(k[0], k[1]);
    }
    cm.store(t.m, e0, n, lane);
    cv.store(t.v, e0, n, lane);
    if (lane == 0) {
      t.ms[e0 / kAdamBlock] = sm.scale;
      t.vs[e0 / kAdamBlock] = sv.scale;
    }
  }
  adam_store<PD, VEC>(t.p, e0, n, lane, p);
  if (PD == kGradF32 && t.copy != nullptr) {
    if (t.copy_dtype == kGradF16) adam_store<kGradF16, VEC>(t.copy, e0, n, lane, p);
    else adam_store<kGradBf16, VEC>(t.copy, e0, n, lane, p);
  }
}

// A warp's chunks of one tensor: every kAdamWarps-th from c on, below end.  States
// in 8 bits take some sixty instructions an element, too many for loads and
// arithmetic of the warps that fit to take turns: the next two chunks are on their way to shared
// memory while one is worked on.
template <int PD, int GD, int BITS>
__device__ __forceinline__ void adam_run(const AdamTensor& t, const AdamHyper& h, bool vec, long long c, long long end,
                                         int lane, uint8_t* stages) {
  if (vec) {
    const long long whole = min(end, t.n / kAdamBlock);
    if constexpr (BITS == 8) {
      if (c < whole) {
        AdamChunk<PD, GD, BITS, kAdamEight> x;
        const uint32_t sa = smem_addr(stages);
        float ms[2], vs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const long long d = c + i * kAdamWarps;
          if (d < whole) {
            adam_fetch_chunk<PD, GD>(sa + i * kAdamStage, t, d * kAdamBlock, lane);
            ms[i] = t.ms[d];
            vs[i] = t.vs[d];
          }
          cp_async_commit();
        }
        int slot = 0;
        for (; c < whole; c += kAdamWarps) {
          cp_async_wait_group<1>();
          __syncwarp();
          const uint8_t* from = stages + slot * kAdamStage;
          x.g.load(from + kAdamStageG, 0, kAdamBlock, lane);
          x.p.load(from, 0, kAdamBlock, lane);
          x.m.load(from + kAdamStageM, 0, kAdamBlock, lane);
          x.v.load(from + kAdamStageV, 0, kAdamBlock, lane);
          x.ms = ms[0];
          x.vs = vs[0];
          ms[0] = ms[1];
          vs[0] = vs[1];
          __syncwarp();  // all lanes have read the slot
          const long long d = c + 2 * kAdamWarps;
          if (d < whole) {
            adam_fetch_chunk<PD, GD>(sa + slot * kAdamStage, t, d * kAdamBlock, lane);
            ms[1] = t.ms[d];
            vs[1] = t.vs[d];
          }
          cp_async_commit();
          slot ^= 1;
          adam_chunk<PD, GD, BITS, kAdamEight>(t, h, x, c * kAdamBlock, kAdamBlock, lane);
        }
        cp_async_wait_group<0>();
        __syncwarp();
      }
    } else {
      AdamChunk<PD, GD, BITS, kAdamFours> x;
      for (; c < whole; c += kAdamWarps) {
        x.load(t, c * kAdamBlock, kAdamBlock, lane);
        adam_chunk<PD, GD, BITS, kAdamFours>(t, h, x, c * kAdamBlock, kAdamBlock, lane);
      }
    }
  }
  for (; c < end; c += kAdamWarps) {
    const long long e0 = c * kAdamBlock;
    const int n = (int)min(t.n - e0, (long long)kAdamBlock);
    AdamChunk<PD, GD, BITS, kAdamEach> x;
    x.load(t, e0, n, lane);
    adam_chunk<PD, GD, BITS, kAdamEach>(t, h, x, e0, n, lane);
  }
}

template <int BITS>
__device__ __forceinline__ void adam_dispatch(int types, const AdamTensor& t, const AdamHyper& h, long long c, long long end,
                                              int lane, uint8_t* stages) {
  const bool vec = (types & kAdamVec) != 0;
  switch (types & 15) {
    case kGradF16 | kGradF16 << 2: return adam_run<kGradF16, kGradF16, BITS>(t, h, vec, c, end, lane, stages);
    case kGradF16 | kGradBf16 << 2: return adam_run<kGradF16, kGradBf16, BITS>(t, h, vec, c, end, lane, stages);
    case kGradF16 | kGradF32 << 2: return adam_run<kGradF16, kGradF32, BITS>(t, h, vec, c, end, lane, stages);
    case kGradBf16 | kGradF16 << 2: return adam_run<kGradBf16, kGradF16, BITS>(t, h, vec, c, end, lane, stages);
    case kGradBf16 | kGradBf16 << 2: return adam_run<kGradBf16, kGradBf16, BITS>(t, h, vec, c, end, lane, stages);
    case kGradBf16 | kGradF32 << 2: return adam_run<kGradBf16, kGradF32, BITS>(t, h, vec, c, end, lane, stages);
    case kGradF32 | kGradF16 << 2: return adam_run<kGradF32, kGradF16, BITS>(t, h, vec, c, end, lane, stages);
    case kGradF32 | kGradBf16 << 2: return adam_run<kGradF32, kGradBf16, BITS>(t, h, vec, c, end, lane, stages);
    default: return adam_run<kGradF32, kGradF32, BITS>(t, h, vec, c, end, lane, stages);
  }
}

// The factors of a step, in 64 bits: 1 - b^t = -expm1(t log b).
__host__ __device__ inline void adam_factors(double lr, double log_b1, double log_b2, double t, float* step_size,
                                             float* root_scale) {
  *step_size = (float)(lr / -expm1(t * log_b1));
  *root_scale = (float)(1.0 / sqrt(-expm1(t * log_b2)));
}

// The tensor of chunk c.
template <int T>
__device__ __forceinline__ int adam_find(const long long (&first)[T], int count, long long c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A block has consecutive chunks of all tensors', in equal shares, and its warps take them
// in turn.  GB300, 705M bfloat16 elements: states in FP32 2.24 ms (6.9 TB/s, four blocks of 64 registers
// an SM; 2.38 with one share for each resident block, as SMs differ in speed); in 8 bits 1.61 ms (4.4 TB/s, three
// blocks of 80 registers; 0.06 more with four, whose register pairs for packed constants spill), bound by the
// issue of about 65 instructions an element.
template <int T, int BITS>
__global__ void __launch_bounds__(kAdamThreads, BITS == 8 ? 3 : 4) adamw_kernel(const __grid_constant__ AdamTable<T> t, const AdamArgs a) {
  extern __shared__ __align__(16) uint8_t adam_smem[];
  __shared__ AdamHyper shared;
  grid_dep_wait();
  grid_dep_launch();
  AdamHyper h{a.b1, a.omb1, a.b2, a.omb2, a.eps, a.grad_scale, a.step_size, a.root_scale, 0.0f, a.minus_zero};
  if (a.lr_dev != nullptr || a.step_dev != nullptr || a.grad_scale_dev != nullptr) {
    if (threadIdx.x == 0) {
      const double lr = a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr;
      adam_factors(lr, a.log_b1, a.log_b2, (double)(a.step_dev != nullptr ? *a.step_dev : a.step), &h.step_size,
                   &h.root_scale);
      if (a.grad_scale_dev != nullptr) h.grad_scale = *a.grad_scale_dev;
      h.lr = (float)lr;
      shared = h;
    }
    __syncthreads();
    h = shared;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* const stages = adam_smem + warp * 2 * kAdamStage;
  const long long chunks = t.first[t.count];
  const long long c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
  int k = adam_find(t.first, t.count, c0);
  for (long long c = c0 + warp; c < c1;) {
    while (c >= t.first[k + 1]) ++k;
    AdamTensor x;
    x.p = t.p[k];
    x.g = t.g[k];
    x.m = t.m[k];
    x.v = t.v[k];
    x.ms = t.ms[k];
    x.vs = t.vs[k];
    x.copy = t.copy[k];
    x.n = t.n[k];
    x.decay = a.lr_dev != nullptr ? fmaf(-h.lr, t.decay[k], 1.0f) : t.decay[k];
    const int types = t.types[k];
    x.copy_dtype = (types >> 4) & 3;
    const long long first = t.first[k], end = min(c1, t.first[k + 1]);
    adam_dispatch<BITS>(types, x, h, c - first, end - first, lane, stages);
    c += (end - c + kAdamWarps - 1) / kAdamWarps * kAdamWarps;
  }
}

// ---- the values that 8-bit states stand for ----------------------------------------
// Bound by HBM: two bytes read, eight written an element (705M elements 1.05 ms, 6.7 TB/s).
template <int T>
struct AdamValueTable {
  const void* m[T];
  const void* v[T];
  const float* ms[T];
  const float* vs[T];
  float* mo[T];
  float* vo[T];
  long long n[T];
  long long first[T + 1];
  unsigned char vec[T];
  int count;
};

template <int VEC>
__device__ __forceinline__ void adam_expand(const void* m, const void* v, float ms, float vs, float* mo, float* vo,
                                            long long e0, int n, int lane) {
  AdamCodes<VEC> cm, cv;
  cm.load(m, e0, n, lane);
  cv.load(v, e0, n, lane);
  float fm[8], fv[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 a = adam_m(cm.w[j >> 2], j, ms), r = adam_root(cv.w[j >> 2], j, vs), b = adam_mul(r, r);
    fm[j] = a.x;
    fm[j + 1] = a.y;
    fv[j] = b.x;
    fv[j + 1] = b.y;
  }
  adam_store<kGradF32, VEC>(mo, e0, n, lane, fm);
  adam_store<kGradF32, VEC>(vo, e0, n, lane, fv);
}

template <int T>
__global__ void __launch_bounds__(kAdamThreads) adamw_values_kernel(const __grid_constant__ AdamValueTable<T> t) {
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long chunks = t.first[t.count];
  const long long c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
  int k = adam_find(t.first, t.count, c0);
  for (long long c = c0 + warp; c < c1; c += kAdamWarps) {
    while (c >= t.first[k + 1]) ++k;
    const long long block = c - t.first[k], e0 = block * kAdamBlock, left = t.n[k] - e0;
    const float ms = t.ms[k][block], vs = t.vs[k][block];
    if (t.vec[k] && left >= kAdamBlock)
      adam_expand<kAdamFours>(t.m[k], t.v[k], ms, vs, t.mo[k], t.vo[k], e0, kAdamBlock, lane);
    else
      adam_expand<kAdamEach>(t.m[k], t.v[k], ms, vs, t.mo[k], t.vo[k], e0, (int)min(left, (long long)kAdamBlock), lane);
  }
}

}  // namespace poot
